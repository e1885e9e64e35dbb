// mla_wait.h - the wait for threads that are certain to come (device code; the
// logic compiles for the host too, where it is tested).
#pragma once

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

// Polls ready() until it holds.  Gives up, and returns false, only after `cycles`
// of clock() and `polls` further polls: a block that was off its SM for longer
// finds the time gone at its next poll, while the threads it waits for have
// still to run.
template <class Ready, class Clock>
MLA_HD bool wait_for_all(Ready ready, Clock clock, long long cycles, unsigned polls) {
  if (ready()) return true;
  const long long since = clock();
  while (!ready())
    if (clock() - since > cycles && polls-- == 0) return false;
  return true;
}

}  // namespace mla
