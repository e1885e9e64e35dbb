// The wait of mla_wait.h against a made-up clock and peers, for test_waits.py:
// prints "<name> <returned> <polls made>".
#include <cstdio>

#include "mla_wait.h"

struct Case {
  const char* name;
  long long ready_at;  // the poll from which the phase is over (-1: never)
  long long jump_at;   // the poll at which the clock has jumped far ahead (-1: never)
};

int main() {
  const long long limit = 8000000000LL;
  const unsigned polls = 1u << 20;
  const Case cases[] = {{"at_once", 0, -1},        {"soon", 1000, -1},
                        {"off_the_sm", 500, 3},    {"off_the_sm_at_first", 5000, 1},
                        {"never", -1, -1},         {"never_and_off_the_sm", -1, 2}};
  for (const Case& c : cases) {
    long long made = 0, now = 0;
    auto ready = [&] { return c.ready_at >= 0 ? made++ >= c.ready_at : (made++, false); };
    auto clock = [&] {
      now += 4000;
      return c.jump_at >= 0 && made >= c.jump_at ? now + 100 * limit : now;
    };
    const bool ok = mla::wait_for_all(ready, clock, limit, polls);
    std::printf("%s %d %lld\n", c.name, ok ? 1 : 0, made);
  }
  return 0;
}
