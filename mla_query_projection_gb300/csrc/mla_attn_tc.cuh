// mla_attn_tc.cuh - what the tcgen05 attention kernels share: descriptors,
// MMA issue, TMEM access, the two-term weights and queries, bounded waits.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "mla_attn.cuh"
#include "mla_wait.h"

namespace mla {
namespace {

constexpr int kTcTile = kAttnTile;         // cache rows a tile: MMA M of S^T, K of O^T
constexpr int kPlane = kTcTile * 128;      // a 128-byte column plane of a tile
constexpr int kTcSoft = 256;               // softmax threads (warps 0-7)
constexpr int kTcThreads = kTcSoft + 64;   // + a TMA warp, an MMA warp
constexpr int kTcBar = 1;                  // named barrier of the softmax threads
constexpr long long kTcWait = 2000000000LL;  // ~1 s of SM clock
// Weights are kept times 2^5, and the reference moves when a logit (base 2)
// passes it by more than 3.75: 2^8.75 = 430 < 448, E4M3's largest.  (With 2^7
// and 1.75 a sixth of the tiles of normally distributed logits moved it, at
// 7,000 cycles each.)
constexpr float kPShift = 5.0f, kPRoom = 3.75f;

// Shared-memory matrix descriptors (tcgen05), version 1.  K-major, 128- or
// 64-byte swizzle: 8-row groups `sbo` bytes apart.  M/N-major with 128-byte
// swizzle: rows are K, 128 bytes of M or N each, groups of 8 K rows 1024 bytes
// apart (`sbo`); one atom covers M or N, so the leading offset is unused.
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr, uint32_t sbo, uint32_t swizzle) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(sbo >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)swizzle << 61;  // 2: 128 B, 4: 64 B
  return d;
}

// M-major over more than one atom: the atoms of 128 bytes of M `lbo` apart.
__device__ __forceinline__ uint64_t tc_desc_wide(uint32_t saddr, uint32_t sbo, uint32_t lbo) {
  return (tc_desc(saddr, sbo, 2) & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(lbo >> 4) << 16;
}

// Instruction descriptor, FP32 accumulators: operand types (0 E4M3, 1 E5M2; of
// kind::f16, 0 FP16, 1 BF16),
// and whether A and B are M/N-major.
__host__ __device__ constexpr uint32_t tc_idesc(int m, int n, int btype, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)btype << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One elected lane of a converged warp issues; the warp runs the code around it
// together, so that descriptors are computed in uniform registers (issued from
// a single lane's branch, an MMA cost about 100 cycles to issue against the
// 48 to 64 that it takes to run).
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Several MMAs into one accumulator by one elected lane: step k multiplies the
// operands at a + k * AS and b + k * BS (16-byte units); tc_mma4x2 follows each
// by the same A with B at BL more (its second term, idesc id1).
#define TC_MMA_ENTER                                                     \
  "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t" \
  "setp.eq.b32 t, %4, %4;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
#define TC_MMA_NEXT(da, db) "add.s64 x, x, " da ";\n\tadd.s64 y, y, " db ";\n\t"
#define TC_MMA_F8(id, pred) "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, " id ", " pred ";\n\t"
#define TC_MMA_F16(id, pred) "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, " id ", " pred ";\n\t"
template <int AS, int BS>
__device__ __forceinline__ void tc_mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                        uint32_t accumulate) {
  asm volatile(TC_MMA_ENTER "mov.b64 x, %1;\n\tmov.b64 y, %2;\n\t" TC_MMA_F8("%3", "p")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t") "}" ::"r"(d),
               "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(AS), "n"(BS)
               : "memory");
}
template <int AS, int BS>
__device__ __forceinline__ void tc_mma4_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                             uint32_t accumulate) {
  asm volatile(TC_MMA_ENTER "mov.b64 x, %1;\n\tmov.b64 y, %2;\n\t" TC_MMA_F16("%3", "p")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F16("%3", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F16("%3", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F16("%3", "t") "}" ::"r"(d),
               "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(AS), "n"(BS)
               : "memory");
}
template <int AS, int BS, int BL>
__device__ __forceinline__ void tc_mma4x2(uint32_t d, uint64_t a, uint64_t b, uint32_t id0,
                                          uint32_t id1, uint32_t accumulate) {
  asm volatile(TC_MMA_ENTER "mov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
               TC_MMA_F8("%3", "p") TC_MMA_NEXT("0", "%7") TC_MMA_F8("%8", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t") TC_MMA_NEXT("0", "%7") TC_MMA_F8("%8", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t") TC_MMA_NEXT("0", "%7") TC_MMA_F8("%8", "t")
               TC_MMA_NEXT("%5", "%6") TC_MMA_F8("%3", "t") TC_MMA_NEXT("0", "%7") TC_MMA_F8("%8", "t")
               "}" ::"r"(d),
               "l"(a), "l"(b), "r"(id0), "r"(accumulate), "n"(AS), "n"(BS - BL), "n"(BL), "r"(id1)
               : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// This warp's 32 lanes x 8, 16 or 32 columns.  A load's values may be used
// after tc_wait_ld and tc_landed (the compiler sees no other tie between the
// wait and the registers that the loads fill).
#define TC_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                    "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define TC_I8(v, i) "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), \
                    "r"(__float_as_uint(v[i + 2])), "r"(__float_as_uint(v[i + 3])), \
                    "r"(__float_as_uint(v[i + 4])), "r"(__float_as_uint(v[i + 5])), \
                    "r"(__float_as_uint(v[i + 6])), "r"(__float_as_uint(v[i + 7]))
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t addr, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : TC_R8(r, 0)
                 : "r"(addr));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : TC_R8(r, 0), TC_R8(r, 8)
        : "r"(addr));
  } else {
    static_assert(N == 32, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : TC_R8(r, 0), TC_R8(r, 8), TC_R8(r, 16), TC_R8(r, 24)
        : "r"(addr));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      TC_I8(v, 0), TC_I8(v, 8), TC_I8(v, 16), TC_I8(v, 24)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tc_landed(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// Packed FP32 sums (one instruction for two).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// 2^x by the hardware's approximation (2 ulp), subnormal results flushed.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four weights as the sum of two terms, E4M3 codes and E5M2 codes of the rest;
// they come as FP16 pairs (2^-11, below the terms' own errors; FP16 reaches down
// to 2^-24, further than E5M2).
//
// An E5M2 code is the upper byte of an FP16 value, so the rest is rounded by an
// addition to its bits: half a step (0x80) for weights of 2^-5 or more, which
// keeps 2^-8 of them.  E4M3's steps of 2^-9 hold smaller ones badly and from
// 2^-10 down not at all: a bare E5M2 value has three bits, and a context may
// have thousands of such weights, all alike, beside a large one.  Rounded to
// nearest they are off by the same 2^-3 of themselves, and their sum is too
// (65,535 of 2^-16 beside a weight of 1: 10 % of it; below 2^-22 nothing was
// left).  So these are rounded up or down by the place of their row: the 128
// rows of a tile have the 128 odd ones of a step's 256 thresholds, in
// bit-reversed order, and the sum of alike weights is off by a step in a tile.
// One weight is then off by up to a step of its rest: at most 2^-13, 2^-18 of
// the largest weight (which is 2^5 or more).  The choice costs two instructions
// a pair (8 tokens of 16,384 E4M3 rows, 128 heads: 43.4 us, so 43.9), and the
// rest's conversion is one less.
//
// weight_dither: the threshold of row `pos` of a token's tile n, for a pair.
// (Tiles differ in which rows have the low ones, so that values that alternate
// from row to row meet no rounding that does too.)
__device__ __forceinline__ uint32_t weight_dither(int pos, uint32_t n) {
  return 0x00010001u * (2u * ((__brev((uint32_t)pos) ^ (n * 0x9E3779B1u)) >> 25) + 1u);
}
// What a pair's rests are rounded by: the threshold for weights below `limit`.
// (A NaN is not below it, and half a step does not carry out of its half.)
__device__ __forceinline__ uint32_t weight_round(uint32_t w, uint32_t limit, uint32_t dither) {
  uint32_t small;
  asm("set.lt.u32.f16x2 %0, %1, %2;" : "=r"(small) : "r"(w), "r"(limit));
  return (small & dither) | (~small & 0x00800080u);
}
constexpr float kSmallWeight = 0.03125f;       // 2^-5
constexpr uint32_t kSmallWeight16 = 0x28002800u;  // the same as an FP16 pair
__device__ __forceinline__ void split_weights(uint32_t w0, uint32_t w1, uint32_t round0, uint32_t round1,
                                              uint32_t* hi, uint32_t* lo) {
  uint32_t d0, d1;
  asm("{\n\t.reg .b32 g;\n\t.reg .b16 c0, c1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c0, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c1, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 g, c0;\n\t"
      "sub.rn.f16x2 %1, %3, g;\n\t"
      "cvt.rn.f16x2.e4m3x2 g, c1;\n\t"
      "sub.rn.f16x2 %2, %4, g;\n\t"
      "mov.b32 %0, {c0, c1};\n\t}"
      : "=&r"(*hi), "=&r"(d0), "=&r"(d1)
      : "r"(w0), "r"(w1));
  *lo = __byte_perm(d0 + round0, d1 + round1, 0x7531);
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t p;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t p;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(b));
  return p;
}

struct OpMax {
  __device__ static float f(float a, float b) { return fmaxf(a, b); }
};
struct OpSum {
  __device__ static float f(float a, float b) { return a + b; }
};
// Reduces N values (8, 16 or 32) over the 32 lanes of a warp, halving what a
// lane carries at each step: lane l ends with the result of value l * N / 32.
template <int N, class Op>
__device__ __forceinline__ float lanes_reduce(const float (&in)[N]) {
  const int lane = threadIdx.x & 31;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in[i];
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
          v[i] = Op::f(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
        }
    } else {
      v[0] = Op::f(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
    }
  }
  return v[0];
}

__device__ __forceinline__ void tc_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(kTcBar), "r"(kTcSoft) : "memory");
}

// A value that every lane of the warp has, in a uniform register: what the MMA
// warp's loops and descriptors come from.  (From ordinary registers an MMA took
// 80 to 95 cycles to issue, from uniform ones no longer than it runs, 48 to 64.)
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }

// A bounded wait that gives up for good: once one has run out, the thread
// waits no more (its results do not count) and leaves.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (!dead && !mbar_wait_bounded(bar, parity, kTcWait)) dead = true;
}

// The same, and says so to the other softmax threads.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead, uint32_t* gave_up) {
  if (!dead && !mbar_wait_bounded(bar, parity, kTcWait)) {
    dead = true;
    *reinterpret_cast<volatile uint32_t*>(gave_up) = 1u;
  }
}

// The wait for the softmax warps' votes.  A warp's waits before its vote are
// bounded, and it votes whether they ran out or not, so every vote comes; what
// must not happen is that one thread gives this wait up and another, a poll
// later, does not: the threads that saw the vote alike go through barriers
// together.  Hence more time than the other waits have, and polls beyond it.
__device__ __forceinline__ void tc_wait_votes(uint64_t* bar, uint32_t parity, bool& dead, uint32_t* gave_up) {
  if (!dead && !wait_for_all([&] { return mbar_try_wait(bar, parity); }, [] { return clock64(); }, 4 * kTcWait,
                             1u << 20)) {
    dead = true;
    *reinterpret_cast<volatile uint32_t*>(gave_up) = 1u;
  }
}

// The first form by a converged warp: its lanes go on together.
__device__ __forceinline__ void tc_wait_warp(uint64_t* bar, uint32_t parity, bool& dead) {
  tc_wait(bar, parity, dead);
  dead = __any_sync(0xFFFFFFFFu, dead);
}

// Whether the phase is over, the same answer for the whole warp, at once (a
// try_wait may hold the thread for a while).
__device__ __forceinline__ bool tc_ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, ok != 0);
}

struct TcMaps {
  CUtensorMap latent;  // boxes of box_rows x 128 bytes, 128-byte swizzle
  CUtensorMap rope;    // boxes of box_rows x 64 bytes, 64-byte swizzle
  int box_rows;        // a power of two that divides the page, 8..128; 0: rows are copied
};

// Where plane p of a tile goes (0: rope, then the latent ones), the slot's
// barriers, and how often it was used before.
struct TcSlot {
  uint64_t *full, *empty;
  uint32_t use;
  uint8_t* dst;
};

// One plane of a tile by 16-byte copies, swizzled as TMA does it: 128 rows of
// WIDTH bytes, from byte `col` of the cache rows (lane l holds those of rows l,
// l + 32, ..; -1: zeros).
template <int WIDTH>
__device__ __forceinline__ void tc_copy_plane(const AttnArgs& a, int row_bytes, uint8_t* dst, int col,
                                              const int64_t (&rows)[4], int lane) {
  constexpr int kChunks = WIDTH / 16, kRows = 32 / kChunks;  // a row's chunks, rows an instruction
  const int c = lane % kChunks;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int it = 0; it < kChunks; ++it) {
      const int rl = it * kRows + lane / kChunks, r = 32 * g + rl;
      const int64_t row = __shfl_sync(0xFFFFFFFFu, rows[g], rl);
      const uint32_t d = smem_u32(dst) + r * WIDTH + ((WIDTH == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
      const uint8_t* s = a.cache + (row >= 0 ? row : 0) * row_bytes + col + 16 * c;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(s), "r"(row >= 0 ? 16 : 0)
                   : "memory");
    }
  }
}

// The producer warp where TMA boxes would be too low (8 does not divide the
// page: pages of one token would need 640 boxes a tile).  Up to three planes
// are under way while a fourth is asked for; a plane is told of when its copies
// have landed and are fenced for the tensor core.  32 requests of 4,096 E4M3
// rows, 64 heads: 73 us with pages of 1 (the mma.sync kernel: 183); with pages
// of 64 these copies take 64 us, TMA 45.
template <int ROW_BYTES, int ROPE_BYTES, int ROPE_COL, class Place>
__device__ __forceinline__ void tc_copy_tiles(const AttnArgs& a, const AttnPlan* plan, const AttnSeen* seen,
                                              uint32_t first, uint32_t end, int lane, bool& dead,
                                              Place place) {
  int i = 0, sent = 0, told = 0;  // tiles; planes
  auto tell = [&]() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(place(told / 5, told % 5).full);
    ++told;
  };
  uint32_t x = first;
  while (x < end && !dead) {
    const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
    x = max(x, k.start);
    const uint32_t seg_end = min(k.end, end);
    for (; x < seg_end && !dead; ++x, ++i) {
      int64_t rows[4], page;
#pragma unroll
      for (int g = 0; g < 4; ++g) rows[g] = attn_row(a, k, (x - k.start) * kTcTile + 32 * g + lane, &page);
#pragma unroll 1
      for (int p = 0; p < 5; ++p) {
        const TcSlot s = place(i, p);
        if (s.use >= 1) {
          if (!tc_ready(s.empty, (s.use - 1) & 1u)) {  // what frees it may need the planes under way
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            while (told < sent) tell();
          }
          tc_wait_warp(s.empty, (s.use - 1) & 1u, dead);
        }
        if (dead) break;
        if (p == 0)
          tc_copy_plane<ROPE_BYTES>(a, ROW_BYTES, s.dst, ROPE_COL, rows, lane);
        else
          tc_copy_plane<128>(a, ROW_BYTES, s.dst, 128 * (p - 1), rows, lane);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++sent - told > 3) {
          asm volatile("cp.async.wait_group 3;" ::: "memory");
          tell();
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  while (told < sent) tell();
}

// This thread's column of planes 2 half and 2 half + 1 of O^T (at `ot`, NH
// columns a plane), times factor[h] and the plane's f0 or f1: the output, or
// the worker's part.
template <int NH>
__device__ __forceinline__ void tc_store_out(const AttnArgs& a, const AttnToken& k, uint32_t ot,
                                             int half, int pos, int h0, int slot, bool whole,
                                             const float* factor, float f0, float f1) {
  const int lane = pos & 31;
#pragma unroll 1
  for (int c = 0; c < 2 * NH; c += 32) {
    float v[32];
    tc_ld(ot + 2 * half * NH + c, v);
    tc_wait_ld();
    tc_landed(v);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const int h = (c + e) % NH, j = 2 * half + (c + e) / NH;
      const float4 f = *reinterpret_cast<const float4*>(factor + h);
      const float fp = (c + e) / NH ? f1 : f0;
      const float v0 = v[e] * (f.x * fp), v1 = v[e + 1] * (f.y * fp), v2 = v[e + 2] * (f.z * fp),
                  v3 = v[e + 3] * (f.w * fp);
      if (whole) {
        // neighbouring lanes trade heads, so that each stores two columns
        const bool odd = lane & 1;
        const float g0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
        const float g1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v2 : v3, 1);
        const int h1 = h0 + h + odd;
        uint16_t* o = a.out + (int64_t)k.t * a.o_ts + (int64_t)h1 * a.o_hs + 128 * j + (pos & ~1);
        if (h1 < a.heads) *reinterpret_cast<uint32_t*>(o) = odd ? pack_bf16x2(g0, v1) : pack_bf16x2(v0, g0);
        if (h1 + 2 < a.heads)
          *reinterpret_cast<uint32_t*>(o + 2 * a.o_hs) = odd ? pack_bf16x2(g1, v3) : pack_bf16x2(v2, g1);
      } else {
        attn_part(a, slot, (h0 + h) >> 2, 128 * j + pos) = make_float4(v0, v1, v2, v3);
      }
    }
  }
}

// One token's queries of NH heads into shared memory as E4M3 terms (B of S^T):
// warp w takes heads w, w + 8, ..; a lane holds 16 latent columns of each, and
// lane 4 r + c the rope columns 16 c .. of the warp's r-th head.  Every load is
// issued before the first is used.  xs[h] turns head h's accumulators into
// logits in base 2 (`logit` times the inverse of its power of two).  Latent
// planes at sq, rope rows at sr: E4M3 terms in 64-byte rows, or with ROPE16
// BF16 times the same power of two in 128-byte rows.
template <int NH, bool FP8Q, bool ROPE16>
__device__ __forceinline__ void tc_queries(const AttnArgs& a, uint8_t* sq, uint8_t* sr, int t, int h0,
                                           int warp, int lane, float logit, float* xs) {
  constexpr int kQPlane = (FP8Q ? NH : 2 * NH) * 128;
  constexpr int kN = NH / 8;  // heads a warp
  constexpr int kV = FP8Q ? 1 : 2;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 lat[kN][kV], rope[kV];
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    const int h = h0 + warp + 8 * r;
    const int64_t e = (int64_t)t * a.ql_ts + (int64_t)h * a.ql_hs + 16 * lane;
    const uint4* p = reinterpret_cast<const uint4*>(a.q_latent + e * (FP8Q ? 1 : 2));
#pragma unroll
    for (int v = 0; v < kV; ++v) lat[r][v] = h < a.heads ? p[v] : zero;
  }
  {
    const int r = lane >> 2, h = h0 + warp + 8 * r;
    const int64_t e = (int64_t)t * a.qp_ts + (int64_t)h * a.qp_hs + 16 * (lane & 3);
    const uint4* p = reinterpret_cast<const uint4*>(a.q_pe + e * (FP8Q ? 1 : 2));
#pragma unroll
    for (int v = 0; v < kV; ++v) rope[v] = r < kN && h < a.heads ? p[v] : zero;
  }
  auto put = [&](int row, uint4 w) {  // latent chunk `lane` of a B row
    *reinterpret_cast<uint4*>(sq + (lane >> 3) * kQPlane + row * 128 +
                              (((lane ^ row) & 7) << 4)) = w;
  };
  auto put_rope = [&](int row, uint4 w) {  // rope chunk lane % 4
    *reinterpret_cast<uint4*>(sr + row * 64 + ((((lane & 3) ^ (row >> 1)) & 3) << 4)) = w;
  };
  auto put_rope16 = [&](int row, int c, uint4 w) {  // half c of rope columns 16 (lane % 4) ..
    *reinterpret_cast<uint4*>(sr + row * 128 + (((2 * (lane & 3) + c) ^ row) & 7) * 16) = w;
  };
  const int rr = lane >> 2, rh = warp + 8 * rr;  // the head whose rope this lane holds
  if constexpr (FP8Q) {
#pragma unroll
    for (int r = 0; r < kN; ++r) put(warp + 8 * r, lat[r][0]);
    if (rr < kN) {
      if constexpr (ROPE16) {
        const uint32_t w[4] = {rope[0].x, rope[0].y, rope[0].z, rope[0].w};
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v[4];
          e4m3x4_values(w[e], v);
          c[2 * e] = pack_bf16x2(v[0], v[1]);
          c[2 * e + 1] = pack_bf16x2(v[2], v[3]);
        }
        put_rope16(rh, 0, make_uint4(c[0], c[1], c[2], c[3]));
        put_rope16(rh, 1, make_uint4(c[4], c[5], c[6], c[7]));
      } else {
        put_rope(rh, rope[0]);
      }
    }
    if (lane < kN) xs[warp + 8 * lane] = logit;
  } else {
    // magnitudes as bits order like the values (NaN above infinity)
    auto magnitude = [](uint4 w) {
      const uint32_t s = 0x7FFF7FFFu;
      return __vmaxu2(__vmaxu2(w.x & s, w.y & s), __vmaxu2(w.z & s, w.w & s));
    };
    // A pair of columns times a power of two as two E4M3 terms: the first's
    // codes in the low half of the result, the rest's in the high half (FP16
    // holds the scaled values, at most 448, exactly down to 2^-17).
    auto split2 = [](uint32_t w, float up) {
      const float2 v = fmul2_rn(make_float2(bf16lo(w), bf16hi(w)), make_float2(up, up));
      uint32_t r;
      asm("{\n\t.reg .b32 p, g, d;\n\t.reg .b16 c, e;\n\t"
          "cvt.rn.f16x2.f32 p, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 c, p;\n\t"
          "cvt.rn.f16x2.e4m3x2 g, c;\n\t"
          "sub.rn.f16x2 d, p, g;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 e, d;\n\t"
          "mov.b32 %0, {c, e};\n\t}"
          : "=r"(r)
          : "f"(v.x), "f"(v.y));
      return r;
    };
    auto split = [&](const uint4* w, float up, uint4* hi, uint4* lo) {
      uint32_t c[4], d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 q = w[e >> 1];
        const uint32_t x = split2(e & 1 ? q.z : q.x, up), y = split2(e & 1 ? q.w : q.y, up);
        c[e] = __byte_perm(x, y, 0x5410);
        d[e] = __byte_perm(x, y, 0x7632);
      }
      *hi = make_uint4(c[0], c[1], c[2], c[3]);
      *lo = make_uint4(d[0], d[1], d[2], d[3]);
    };
    const uint32_t rope_mag = __vmaxu2(magnitude(rope[0]), magnitude(rope[kV - 1]));
    // BF16 rope values need no power of two: what they ask for is an exponent that
    // keeps their products in FP32's range where the latent part is far smaller
    // (or zero), 2^60 below their own.  An infinity or a NaN counts as it is.
    uint32_t rope_bits = rope_mag;
    if constexpr (ROPE16) {
      rope_bits = max(rope_mag & 0xFFFFu, rope_mag >> 16);
      if (rope_bits < 0x7F80u) rope_bits = max(rope_bits, 60u << 7) - (60u << 7);
    }
    float rope_up = 0.f;
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      uint32_t m = __vmaxu2(magnitude(lat[r][0]), magnitude(lat[r][kV - 1]));
      if (rr == r) m = __vmaxu2(m, rope_bits);
      m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
      // the power of two that brings the largest into (224, 448]: from its
      // exponent field, kept where both it and its inverse are normal
      int ex = (int)(m >> 7) - 127;
      ex = max(-100, min(ex, 126));
      if ((m & 0x7Fu) <= 0x60u) --ex;
      const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
      float x = logit * __uint_as_float((uint32_t)(127 - 7 + ex) << 23);
      // an infinite query: no finite logits (E4M3 has no infinity)
      if (m >= 0x7F80u) x = __int_as_float(0x7FC00000);
      uint4 hi, lo;
      split(lat[r], up, &hi, &lo);
      put(warp + 8 * r, hi);
      put(NH + warp + 8 * r, lo);
      if (lane == 0) xs[warp + 8 * r] = x;
      if (rr == r) rope_up = up;
    }
    if (rr < kN) {
      if constexpr (ROPE16) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w[4] = {rope[e].x, rope[e].y, rope[e].z, rope[e].w};
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = pack_bf16x2(bf16lo(w[k]) * rope_up, bf16hi(w[k]) * rope_up);
          put_rope16(rh, e, make_uint4(c[0], c[1], c[2], c[3]));
        }
      } else {
        uint4 hi, lo;
        split(rope, rope_up, &hi, &lo);
        put_rope(rh, hi);
        put_rope(NH + rh, lo);
      }
    }
  }
}

// A map of the cache's rows in boxes of box_rows x box_bytes (64 or 128, with the
// swizzle of that width).
// Rows a box has: the largest power of two that divides the page, up to a
// tile.  0, to copy the rows instead, for fewer than 8 (a box starts on a
// swizzle's 8 rows) and where a row's number passes a TMA coordinate.
inline int plane_box_rows(const AttnArgs& a) {
  const int r = a.page_size & -a.page_size;
  if (r < 8 || a.num_pages > (int64_t)0x7FFFFFFF / a.page_size) return 0;
  return r < kTcTile ? r : kTcTile;
}

inline bool encode_plane_map(CUtensorMap* map, const AttnArgs& a, int row_bytes, int box_bytes,
                      int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)(a.num_pages * a.page_size)};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.cache), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace mla
