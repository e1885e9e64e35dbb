// mla_attn_tc.cu - latent attention on the 5th-generation tensor cores
// (tcgen05, accumulators in TMEM), for the layouts whose rows are E4M3 codes
// under one FP32 scale (MLA_KV_FP8_E4M3, MLA_KV_FP8_E4M3_PAGE).
//
// The codes go from HBM to the tensor core as they are: TMA brings 128 cache
// rows a tile into shared memory in 128-byte column planes (four of the
// latent, one of 64 rope bytes), and both products read those planes.
//
//  * S^T = K Q^T (M = 128 rows, N = heads, K = 576 codes): A is K's plane,
//    K-major.  A BF16 query is the sum of two E4M3 terms, q = hi + lo, of its
//    row scaled by a power of two (8 significant bits split 4 + 4, exact but
//    for elements below 2^-11 of the row's largest): B holds the hi rows and
//    then the lo rows, one MMA forms both halves, and the softmax adds them.
//  * O^T += V^T P^T (M = 128 latent columns, N = heads, K = 128 rows): A is the
//    same plane read transposed (M-major), so no value is moved or converted.
//    P is the sum of an E4M3 and an E5M2 term (4 + 3 bits: 2^-7 of each
//    weight), two MMAs into one accumulator.  The second term in E5M2 keeps
//    weights down to 2^-21 of the largest: a context with one dominant key and
//    thousands of small ones needs their sum.
//
// Tokens lie on TMEM lanes in S^T: a softmax thread owns one cache row and
// half the heads, so a row's scale, mask and page are its scalars, and the
// denominators are sums that stay in its registers until the end.  The
// maximum is a reference, not the exact maximum: it moves (and O is rescaled)
// only when a weight would leave E4M3's range, so most tiles need no
// reduction across lanes at all.
//
// Two tiles' planes are in shared memory: while one tile's softmax runs, the
// tensor core works on the O of the tile before and the S of the one behind.
// Shared-memory reads of the tensor core bound a tile (64 heads: 18 MMAs of
// 8 KiB for S and 32 of 6 KiB for O at 128 B a cycle, 2700 cycles), next to
// HBM's share of 73.7 KiB a tile.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/mla_query.h"
#include "mla_attn.cuh"
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kTcTile = 128;               // cache rows a tile: MMA M of S^T, K of O^T
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

template <int NH, bool FP8Q>
struct TcSmem {
  static constexpr int kQRows = FP8Q ? NH : 2 * NH;  // MMA N of S^T
  static constexpr int kQPlane = kQRows * 128;
  static constexpr int oRing = 0;                      // [2 tiles][4 latent planes]
  static constexpr int oRope = oRing + 8 * kPlane;     // one rope plane, 64-byte rows
  static constexpr int oP = oRope + kPlane / 2;        // [row][hi | lo] 128 B
  static constexpr int oQ = oP + kPlane;               // 4 latent planes
  static constexpr int oQr = oQ + 4 * kQPlane;         // rope plane, 64-byte rows
  static constexpr int oRef = oQr + kQRows * 64;       // reference less kPShift, base 2 [NH]
  static constexpr int oXs = oRef + NH * 4;            // logit scale of a head's accumulators [NH]
  static constexpr int oRed = oXs + NH * 4;            // [4][NH] across the quadrants; [0][.] factors
  static constexpr int oVref = oRed + 4 * NH * 4;      // value scale: reference, its ratio, [4..7] warp maxima
  static constexpr int oBar = oVref + 32;
  // full[8] empty[8] rope_full rope_empty s_full[2] s_free[2] p_full pv_done q_full drain voted
  static constexpr int kBars = 27;
  static constexpr int oMoved = oBar + kBars * 8;      // [2] 1 + the last tile that moved the reference
  static constexpr int oPlan = oMoved + 8;
  static constexpr int oScan = oRed;                   // before the first tile
  static constexpr int oTmem = oPlan + (int)sizeof(AttnPlan);
  static constexpr int kBytes = oTmem + 8;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(oP % 1024 == 0 && oQ % 1024 == 0 && oRope % 1024 == 0 && oQr % 512 == 0 &&
                    kQPlane % 1024 == 0 && oRef % 16 == 0 && oXs % 16 == 0 && oRed % 16 == 0 &&
                    oBar % 8 == 0 && oPlan % 8 == 0 && oTmem % 4 == 0,
                "alignment");
};

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

// Instruction descriptor, FP32 accumulators: operand types (0 E4M3, 1 E5M2),
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

// S^T of one latent plane: four steps of 32 codes.
__device__ __forceinline__ void tc_qk_plane(uint32_t d, uint64_t a, uint64_t b, uint32_t id0, uint32_t id1,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %5, %5;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "add.u64 x, %1, 0;\n\tadd.u64 y, %2, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t"
      "add.u64 x, %1, 2;\n\tadd.u64 y, %2, 2;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 4;\n\tadd.u64 y, %2, 4;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 6;\n\tadd.u64 y, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(id0), "r"(id1), "r"(accumulate)
      : "memory");
}
// O^T of one plane: four steps of 32 rows (4096 bytes of V and of P), each with
// both terms of P (the second 64 bytes on).
__device__ __forceinline__ void tc_pv_plane(uint32_t d, uint64_t a, uint64_t b, uint32_t id0, uint32_t id1,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %5, %5;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "add.u64 x, %1, 0;\n\tadd.u64 y, %2, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t"
      "add.u64 x, %1, 0;\n\tadd.u64 y, %2, 4;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n\t"
      "add.u64 x, %1, 256;\n\tadd.u64 y, %2, 256;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 256;\n\tadd.u64 y, %2, 260;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n\t"
      "add.u64 x, %1, 512;\n\tadd.u64 y, %2, 512;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 512;\n\tadd.u64 y, %2, 516;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n\t"
      "add.u64 x, %1, 768;\n\tadd.u64 y, %2, 768;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 768;\n\tadd.u64 y, %2, 772;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(id0), "r"(id1), "r"(accumulate)
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

// Packed FP32 pairs (one instruction for two sums or products).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// 2^x by the hardware's approximation (2 ulp), subnormal results flushed.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A weight pair as the sum of two terms: E4M3 codes in the low half of the
// result, E5M2 codes of the rest in the high half.  The pair is rounded to
// FP16 first (2^-11, below the terms' 2^-7; FP16 reaches down to 2^-24, further
// than E5M2).
__device__ __forceinline__ uint32_t split_weights(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b32 p, g, d;\n\t.reg .b16 c, e;\n\t"
      "cvt.rn.f16x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c, p;\n\t"
      "cvt.rn.f16x2.e4m3x2 g, c;\n\t"
      "sub.rn.f16x2 d, p, g;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 e, d;\n\t"
      "mov.b32 %0, {c, e};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
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

// A bounded wait that gives up for good: once one has run out, the thread
// waits no more (its results do not count) and leaves.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (!dead && !mbar_wait_bounded(bar, parity, kTcWait)) dead = true;
}

// The same by a converged warp: its lanes go on together.
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
  int box_rows;        // a power of two that divides the page, 8..128
};

// One token's queries of NH heads into shared memory as E4M3 terms (B of S^T):
// warp w takes heads w, w + 8, ..; a lane holds 16 latent columns of each, and
// lane 4 r + c the rope columns 16 c .. of the warp's r-th head.  Every load is
// issued before the first is used.  xs[h] turns head h's accumulators into
// logits in base 2 (`logit` times the inverse of its power of two).
template <int NH, bool FP8Q>
__device__ __forceinline__ void tc_queries(const AttnArgs& a, uint8_t* smem, int t, int h0, int warp,
                                           int lane, float logit, float* xs) {
  using S = TcSmem<NH, FP8Q>;
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
    *reinterpret_cast<uint4*>(smem + S::oQ + (lane >> 3) * S::kQPlane + row * 128 +
                              (((lane ^ row) & 7) << 4)) = w;
  };
  auto put_rope = [&](int row, uint4 w) {  // rope chunk lane % 4
    *reinterpret_cast<uint4*>(smem + S::oQr + row * 64 + ((((lane & 3) ^ (row >> 1)) & 3) << 4)) = w;
  };
  const int rr = lane >> 2, rh = warp + 8 * rr;  // the head whose rope this lane holds
  if constexpr (FP8Q) {
#pragma unroll
    for (int r = 0; r < kN; ++r) put(warp + 8 * r, lat[r][0]);
    if (rr < kN) put_rope(rh, rope[0]);
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
    float rope_up = 0.f;
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      uint32_t m = __vmaxu2(magnitude(lat[r][0]), magnitude(lat[r][kV - 1]));
      if (rr == r) m = __vmaxu2(m, rope_mag);
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
      uint4 hi, lo;
      split(rope, rope_up, &hi, &lo);
      put_rope(rh, hi);
      put_rope(NH + rh, lo);
    }
  }
}

template <int NH, bool FP8Q, int LAYOUT>
__global__ void __launch_bounds__(kTcThreads, 1)
    mla_attn_tc_kernel(const AttnArgs a, const __grid_constant__ TcMaps maps) {
  using S = TcSmem<NH, FP8Q>;
  constexpr int kHalf = NH / 2;  // heads a softmax thread handles
  constexpr bool kPaged = LAYOUT == MLA_KV_FP8_E4M3_PAGE;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::oBar);  // [2][4]
  uint64_t* empty = full + 8;
  uint64_t* rope_full = empty + 8;
  uint64_t* rope_empty = rope_full + 1;
  uint64_t* s_full = rope_empty + 1;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_free + 2;
  uint64_t* pv_done = p_full + 1;
  uint64_t* q_full = pv_done + 1;
  uint64_t* drain = q_full + 1;
  uint64_t* voted = drain + 1;
  uint32_t* moved = reinterpret_cast<uint32_t*>(smem + S::oMoved);
  float* ref = reinterpret_cast<float*>(smem + S::oRef);
  float* xs = reinterpret_cast<float*>(smem + S::oXs);
  float* red = reinterpret_cast<float*>(smem + S::oRed);
  float* vref = reinterpret_cast<float*>(smem + S::oVref);
  AttnPlan* plan = reinterpret_cast<AttnPlan*>(smem + S::oPlan);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int group = blockIdx.x % a.groups, worker = blockIdx.x / a.groups;
  const int h0 = group * NH;
  if (tid == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(rope_full, 1);
    mbar_init(rope_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], kTcSoft / 32);
    }
    mbar_init(p_full, kTcSoft / 32);
    mbar_init(pv_done, 1);
    mbar_init(q_full, kTcSoft / 32);
    mbar_init(drain, 1);
    mbar_init(voted, kTcSoft / 32);
    moved[0] = moved[1] = 0;
    mbar_fence_init();
    // the swizzles go by address bits: the base is a multiple of 1 KiB
    if (smem_u32(smem) & 1023u) atomicOr(a.err, MLA_DEVERR_CHECK);
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tslot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == kTcSoft) {
    prefetch_tensormap(&maps.latent);
    prefetch_tensormap(&maps.rope);
  }
  pdl_launch_dependents();
  pdl_wait();
  tc_before();
  // (the plan's barriers order the set-up above)
  AttnSeen* seen = reinterpret_cast<AttnSeen*>(smem + S::oP);  // until the first weights
  attn_make_plan(a, plan, reinterpret_cast<uint32_t*>(smem + S::oScan), blockIdx.x == 0, seen);
  tc_after();
  const uint32_t tmem = __reduce_max_sync(0xFFFFFFFFu, *tslot);  // S^T buffers at columns 0 and 128, O^T planes from 256
  const uint32_t total = plan->end[a.batch - 1];
  const int workers = attn_workers(a, total);
  const uint32_t first = worker < workers ? attn_worker_start(total, workers, worker) : 0;
  const uint32_t end = worker < workers ? attn_worker_start(total, workers, worker + 1) : 0;
  bool dead = false;

  if (warp == 8) {
    // ================= TMA: a tile's planes in the order rope, 0, 1, 2, 3
    const int boxes = kTcTile / maps.box_rows;
    const int32_t no_row = (int32_t)(a.num_pages * a.page_size);  // past the end: zeros
    int i = 0, issued = 0;  // tiles, planes
    uint32_t x = first;
    while (x < end && !dead) {
      // (the first token's weights come after its queries and a tile of its
      // rows: this warp has read `seen` by then)
      const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
      const uint32_t seg_end = min(k.end, end);
      for (; x < seg_end && !dead; ++x, ++i) {
        int32_t y = no_row;
        if (lane < boxes) {
          int64_t page;
          const int64_t r = attn_row(a, k, (x - k.start) * kTcTile + lane * maps.box_rows, &page);
          if (r >= 0) y = (int32_t)r;
        }
        const int b = i & 1;
#pragma unroll 1
        for (int p = 0; p < 5; ++p) {
          uint64_t* f = p == 0 ? rope_full : &full[4 * b + p - 1];
          uint64_t* e = p == 0 ? rope_empty : &empty[4 * b + p - 1];
          if (p == 0 ? i >= 1 : i >= 2)
            tc_wait_warp(e, (uint32_t)((p == 0 ? i - 1 : i / 2 - 1) & 1), dead);
          if (dead) break;
          ++issued;
          if (lane == 0) mbar_arrive_expect_tx(f, p == 0 ? kPlane / 2 : kPlane);
          __syncwarp();
          if (lane < boxes) {
            if (p == 0)
              tma_g2s_2d(smem + S::oRope + lane * maps.box_rows * 64, &maps.rope, kKvLora, y, f);
            else
              tma_g2s_2d(smem + S::oRing + (4 * b + p - 1) * kPlane + lane * maps.box_rows * 128,
                         &maps.latent, 128 * (p - 1), y, f);
          }
        }
      }
    }
    // A wait ran out: the planes issued last land before the CTA leaves.
    // (Otherwise the MMAs have read them all.)
    if (dead && issued > 0) {
      (void)mbar_wait_bounded(rope_full, (uint32_t)(((issued - 1) / 5) & 1), kTcWait);
      for (int s = 0; s < 8; ++s) {
        const int b = s >> 2, n = issued - 2 - (s & 3);  // planes up to this one of some tile
        int last = n >= 0 ? n / 5 : -1;
        if (last >= 0 && (last & 1) != b) --last;
        if (last >= 0) (void)mbar_wait_bounded(&full[s], (uint32_t)((last >> 1) & 1), kTcWait);
      }
    }
  } else if (warp == 9) {
    // ================= MMA issuer (the warp together, one elected lane issues)
    constexpr uint32_t id_s = tc_idesc(128, S::kQRows, 0, false, false);
    constexpr uint32_t id_hi = tc_idesc(128, NH, 0, true, true);
    constexpr uint32_t id_lo = tc_idesc(128, NH, 1, true, true);
    const uint64_t dk = tc_desc(smem_u32(smem + S::oRing), 1024, 2);  // planes, K- or M-major
    const uint64_t dkr = tc_desc(smem_u32(smem + S::oRope), 512, 4);  // rope plane
    const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
    const uint64_t dqr = tc_desc(smem_u32(smem + S::oQr), 512, 4);
    const uint64_t dp = tc_desc(smem_u32(smem + S::oP), 1024, 2);
    constexpr uint64_t kPl = kPlane >> 4, kQPl = S::kQPlane >> 4;
    // O^T += V^T P^T of tile n (`add`: to what its stretch has so far)
    auto pv = [&](int n, uint32_t add) {
      tc_wait_warp(p_full, (uint32_t)(n & 1), dead);
      tc_after();
      const int b = n & 1;
      const uint64_t da = dk + (uint64_t)b * 4 * kPl;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tc_pv_plane(tmem + 256 + NH * j, da + j * kPl, dp, id_hi, id_lo, add);
        tc_commit(&empty[4 * b + j]);
      }
      tc_commit(pv_done);
    };
    // A wait that ran out ends no loop here (the loops are then the warp's, and
    // the descriptors stay in uniform registers): the MMAs go on over whatever
    // the planes hold, and the results do not count.
    const int tiles = (int)__reduce_max_sync(0xFFFFFFFFu, end - first);
    const uint32_t x0 = __reduce_max_sync(0xFFFFFFFFu, first);
    uint32_t seg_end = x0;
    int segs = 0;
    uint32_t add = 0;  // whether the tile before added to its O^T
    bool due = false;  // its PV is still to be issued
    for (int i = 0; i < tiles; ++i) {
      const int b = i & 1;
      const bool fresh = x0 + i == seg_end;
      if (fresh) {
        seg_end = __reduce_max_sync(0xFFFFFFFFu, plan->end[attn_token_of(plan, a.batch, x0 + i)]);
        if (due) pv(i - 1, add);  // its softmax must finish before the queries change
        due = false;
        tc_wait_warp(q_full, (uint32_t)(segs & 1), dead);
        ++segs;
      }
      if (i >= 2) tc_wait_warp(&s_free[b], (uint32_t)((i / 2 - 1) & 1), dead);
      tc_wait_warp(rope_full, (uint32_t)(i & 1), dead);
      tc_after();
      const uint32_t d = tmem + 128 * b;
      tc_mma_f8(d, dkr, dqr, id_s, 0u);
      tc_mma_f8(d, dkr + 2, dqr + 2, id_s, 1u);
      tc_commit(rope_empty);
      const uint64_t da = dk + (uint64_t)b * 4 * kPl;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // While a plane has not landed, weights may come: PV first then, which
        // is what frees the planes of the tile after this one.
        if (due) {
          const long long since = clock64();
          while (!tc_ready(&full[4 * b + j], (uint32_t)((i >> 1) & 1)) && clock64() - since < kTcWait)
            if (tc_ready(p_full, (uint32_t)((i - 1) & 1))) {
              pv(i - 1, add);
              due = false;
              break;
            }
        }
        tc_wait_warp(&full[4 * b + j], (uint32_t)((i >> 1) & 1), dead);
        tc_after();
        tc_qk_plane(d, da + j * kPl, dq + j * kQPl, id_s, id_s, 1u);
      }
      tc_commit(&s_full[b]);
      if (due) pv(i - 1, add);
      due = true;
      add = fresh ? 0u : 1u;
    }
    if (due) pv(tiles - 1, add);
    if (dead) {  // let what was issued finish before TMEM is freed
      tc_commit(drain);
      (void)mbar_wait_bounded(drain, 0u, kTcWait);
    }
  } else {
    // ================= softmax, rescaling, epilogue (warps 0-7)
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int pos = 32 * quad + lane;    // this thread's row of a tile
    const int hb = half * kHalf;         // its heads
    const float qinv = a.q_scale_inv != nullptr ? *a.q_scale_inv : 1.0f;
    const float tensor_scale = kPaged ? 1.0f : *a.k_scale;
    const float logit = a.scale / qinv * 1.4426950408889634f * tensor_scale;
    int i = 0;
    uint32_t x = first;
    // A thread whose wait has run out goes on without waiting: all of them
    // pass the same barriers to the end.
    while (x < end) {
      const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
      const uint32_t seg0 = x, seg_end = min(k.end, end);
      tc_queries<NH, FP8Q>(a, smem, k.t, h0, warp, lane, logit, xs);
      for (int h = tid; h < NH; h += kTcSoft) ref[h] = 0.f;
      if (tid == 0) vref[0] = kPaged ? 0.f : tensor_scale;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_barrier();
      if (lane == 0) mbar_arrive(q_full);
      int64_t page = 0;
      int64_t crow = attn_row(a, k, (x - k.start) * kTcTile + pos, &page);
      float rscale = crow >= 0 && kPaged ? a.k_scale[page] : 1.0f;
      bool started = false;  // a row that counts has been met
      float2 l[kHalf / 2];
#pragma unroll
      for (int h = 0; h < kHalf / 2; ++h) l[h] = make_float2(0.f, 0.f);

      for (; x < seg_end; ++x, ++i) {
        const int b = i & 1;
        const bool valid = crow >= 0;
        tc_wait(&s_full[b], (uint32_t)((i >> 1) & 1), dead);
        tc_after();
        float s[kHalf];
        // exponents: logits in base 2 less the reference, plus kPShift
        auto exponents = [&]() {
          tc_ld(tmem + lanes + 128 * b + hb, s);
          if constexpr (!FP8Q) {
            float lo[kHalf];
            tc_ld(tmem + lanes + 128 * b + NH + hb, lo);
            tc_wait_ld();
            tc_landed(s);
            tc_landed(lo);
#pragma unroll
            for (int h = 0; h < kHalf; h += 2) {
              const float2 v = add2(make_float2(s[h], s[h + 1]), make_float2(lo[h], lo[h + 1]));
              s[h] = v.x;
              s[h + 1] = v.y;
            }
          } else {
            tc_wait_ld();
            tc_landed(s);
          }
          const float rs = kPaged ? rscale : 1.0f;
#pragma unroll
          for (int h = 0; h < kHalf; h += 4) {
            const float4 sc = *reinterpret_cast<const float4*>(xs + hb + h);
            const float4 m = *reinterpret_cast<const float4*>(ref + hb + h);
            float2 c0 = make_float2(sc.x, sc.y), c1 = make_float2(sc.z, sc.w);
            if (kPaged) {
              c0 = fmul2_rn(c0, make_float2(rs, rs));
              c1 = fmul2_rn(c1, make_float2(rs, rs));
            }
            const float2 v0 = fma2(make_float2(s[h], s[h + 1]), c0, make_float2(-m.x, -m.y));
            const float2 v1 = fma2(make_float2(s[h + 2], s[h + 3]), c1, make_float2(-m.z, -m.w));
            s[h] = v0.x;
            s[h + 1] = v0.y;
            s[h + 2] = v1.x;
            s[h + 3] = v1.y;
          }
          if (!valid) {
#pragma unroll
            for (int h = 0; h < kHalf; ++h) s[h] = -INFINITY;
          }
        };
        // weights from the exponents, and their two terms
        uint32_t phi[kHalf / 4], plo[kHalf / 4];
        auto weights = [&]() {
          const float vs = kPaged ? (valid && vref[0] > 0.f ? rscale / vref[0] : 0.f) : 1.0f;
#pragma unroll
          for (int h = 0; h < kHalf; h += 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h + e] = ex2(s[h + e]);
            float2 p0 = make_float2(s[h], s[h + 1]), p1 = make_float2(s[h + 2], s[h + 3]);
            if (kPaged) {
              p0 = fmul2_rn(p0, make_float2(vs, vs));
              p1 = fmul2_rn(p1, make_float2(vs, vs));
            }
            const uint32_t w0 = split_weights(p0.x, p0.y), w1 = split_weights(p1.x, p1.y);
            phi[h / 4] = __byte_perm(w0, w1, 0x5410);
            plo[h / 4] = __byte_perm(w0, w1, 0x7632);
          }
        };
        exponents();
        float over = fmaxf(s[0], s[1]);
#pragma unroll
        for (int h = 2; h < kHalf; h += 2) over = fmaxf(over, fmaxf(s[h], s[h + 1]));
        // Does the reference have to move?  The warps' answers meet while the
        // weights are computed as if not.
        bool move = valid && (!started || over > kPShift + kPRoom);
        if (kPaged) move |= valid && fabsf(rscale) > vref[0];
        move = __any_sync(0xFFFFFFFFu, move);
        if (lane == 0) {
          if (move) *reinterpret_cast<volatile uint32_t*>(&moved[b]) = (uint32_t)i + 1;
          mbar_arrive(voted);
        }
        weights();
        tc_wait(voted, (uint32_t)(i & 1), dead);
        if (*reinterpret_cast<volatile uint32_t*>(&moved[b]) == (uint32_t)i + 1) {
          // the reference moves to the tile's maximum where that passes it by
          // too much (for the first rows that count, everywhere)
          exponents();
          const float mx = lanes_reduce<kHalf, OpMax>(s);
          if ((lane * kHalf) % 32 == 0) red[quad * NH + hb + lane * kHalf / 32] = mx;
          if (kPaged) {
            float v = valid ? fabsf(rscale) : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            if (lane == 0 && half == 0) vref[4 + quad] = v;
          }
          tc_barrier();
          if (tid < NH) {
            const float m = fmaxf(fmaxf(red[tid], red[NH + tid]), fmaxf(red[2 * NH + tid], red[3 * NH + tid]));
            const bool grow = started ? m > kPShift + kPRoom : m > -INFINITY;
            red[tid] = grow ? kPShift - m : 0.f;
            if (grow) ref[tid] += m - kPShift;
          }
          if (kPaged && tid == NH) {
            const float old = vref[0];
            const float v = fmaxf(fmaxf(vref[4], vref[5]), fmaxf(vref[6], vref[7]));
            vref[1] = v > old ? old / v : 1.0f;
            if (v > old) vref[0] = v;
          }
          tc_barrier();
          const float ratio = kPaged ? vref[1] : 1.0f;
#pragma unroll
          for (int h = 0; h < kHalf; ++h) {
            const float d = red[hb + h];
            s[h] += d;
            float& lh = h & 1 ? l[h / 2].y : l[h / 2].x;
            if (started) lh *= ex2(d);
          }
          if (started && x > seg0) {
            tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
            tc_after();
#pragma unroll 1
            for (int c = 0; c < 2 * NH; c += 32) {
              // planes 2 half and 2 half + 1 of O^T: columns are heads
              float v[32];
              const uint32_t at = tmem + lanes + 256 + 2 * half * NH + c;
              tc_ld(at, v);
              tc_wait_ld();
              tc_landed(v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= ex2(red[(c + e) % NH]) * ratio;
              tc_st32(at, v);
            }
            tc_wait_st();
          }
          started = true;
          weights();
          tc_barrier();  // red is read
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
#pragma unroll
        for (int h = 0; h < kHalf; h += 2) l[h / 2] = add2(l[h / 2], make_float2(s[h], s[h + 1]));
        // the previous tile's PV has read P
        if (i > 0) tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
        if (!valid && half == 0) {
          // a row that is loaded but does not count holds anything, NaN codes
          // too: no value of it may meet a weight of zero
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint4* d = reinterpret_cast<uint4*>(smem + S::oRing + (4 * b + j) * kPlane + pos * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = make_uint4(0, 0, 0, 0);
          }
        }
        uint8_t* prow = smem + S::oP + pos * 128;
        if constexpr (kHalf >= 16) {
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            const int ch = hb / 16 + c;
            *reinterpret_cast<uint4*>(prow + (((ch ^ pos) & 7) << 4)) =
                make_uint4(phi[4 * c], phi[4 * c + 1], phi[4 * c + 2], phi[4 * c + 3]);
            *reinterpret_cast<uint4*>(prow + ((((ch + 4) ^ pos) & 7) << 4)) =
                make_uint4(plo[4 * c], plo[4 * c + 1], plo[4 * c + 2], plo[4 * c + 3]);
          }
        } else {
          *reinterpret_cast<uint2*>(prow + ((pos & 7) << 4) + 8 * half) = make_uint2(phi[0], phi[1]);
          *reinterpret_cast<uint2*>(prow + (((4 ^ pos) & 7) << 4) + 8 * half) = make_uint2(plo[0], plo[1]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        // the next tile's row
        if (x + 1 < seg_end) {
          crow = attn_row(a, k, (x + 1 - k.start) * kTcTile + pos, &page);
          if (kPaged) rscale = crow >= 0 ? a.k_scale[page] : 1.0f;
        }
      }
      // ---- the stretch is done
      {
        float lv[kHalf];
#pragma unroll
        for (int h = 0; h < kHalf; ++h) lv[h] = h & 1 ? l[h / 2].y : l[h / 2].x;
        const float sum = lanes_reduce<kHalf, OpSum>(lv);
        if ((lane * kHalf) % 32 == 0) red[quad * NH + hb + lane * kHalf / 32] = sum;
      }
      tc_barrier();
      const bool whole = seg0 == k.start && seg_end == k.end;
      const int slot = 2 * worker + (seg0 == first ? 0 : 1);
      if (tid < NH) {
        const float sum = (red[tid] + red[NH + tid]) + (red[2 * NH + tid] + red[3 * NH + tid]);
        const float m = sum == 0.f ? -INFINITY : ref[tid];
        if (whole) {
          red[tid] = sum == 0.f ? 0.f : vref[0] / sum;
          if (a.lse != nullptr && h0 + tid < a.heads)
            a.lse[(int64_t)k.t * a.heads + h0 + tid] = attn_lse(m, sum);
        } else {
          red[tid] = sum == 0.f ? 0.f : vref[0];
          attn_part_ml(a, h0 + tid)[slot] = make_float2(m, sum);
        }
      }
      tc_barrier();
      tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
      tc_after();
#pragma unroll 1
      for (int c = 0; c < 2 * NH; c += 32) {
        float v[32];
        tc_ld(tmem + lanes + 256 + 2 * half * NH + c, v);
        tc_wait_ld();
        tc_landed(v);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const int h = (c + e) % NH, j = 2 * half + (c + e) / NH;
          const float4 f = *reinterpret_cast<const float4*>(red + h);
          const float v0 = v[e] * f.x, v1 = v[e + 1] * f.y, v2 = v[e + 2] * f.z, v3 = v[e + 3] * f.w;
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
      tc_before();
      tc_barrier();  // red is read
    }
  }
  if (dead) atomicOr(a.err, MLA_DEVERR_TIMEOUT);
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

template <int NH, bool FP8Q, int LAYOUT>
cudaError_t launch_tc(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.workers * a.groups));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = TcSmem<NH, FP8Q>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_attn_tc_kernel<NH, FP8Q, LAYOUT>, a, maps);
}

template <int NH>
cudaError_t launch_tc_heads(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
  const bool paged = a.layout == MLA_KV_FP8_E4M3_PAGE;
  if (a.q_scale_inv != nullptr)
    return paged ? launch_tc<NH, true, MLA_KV_FP8_E4M3_PAGE>(a, maps, stream)
                 : launch_tc<NH, true, MLA_KV_FP8_E4M3>(a, maps, stream);
  return paged ? launch_tc<NH, false, MLA_KV_FP8_E4M3_PAGE>(a, maps, stream)
               : launch_tc<NH, false, MLA_KV_FP8_E4M3>(a, maps, stream);
}

template <int NH, bool FP8Q, int LAYOUT>
cudaError_t prepare_tc() {
  return cudaFuncSetAttribute(mla_attn_tc_kernel<NH, FP8Q, LAYOUT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<NH, FP8Q>::kBytes);
}
template <int NH>
cudaError_t prepare_tc_heads() {
  cudaError_t e = prepare_tc<NH, false, MLA_KV_FP8_E4M3>();
  if (e == cudaSuccess) e = prepare_tc<NH, false, MLA_KV_FP8_E4M3_PAGE>();
  if (e == cudaSuccess) e = prepare_tc<NH, true, MLA_KV_FP8_E4M3>();
  if (e == cudaSuccess) e = prepare_tc<NH, true, MLA_KV_FP8_E4M3_PAGE>();
  return e;
}

bool encode_plane_map(CUtensorMap* map, const AttnArgs& a, int box_bytes, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kRowE4m3, (cuuint64_t)(a.num_pages * a.page_size)};
  cuuint64_t strides[1] = {(cuuint64_t)kRowE4m3};
  cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.cache), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int attn_tc_heads(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : 64; }
int attn_tc_tile() { return kTcTile; }

bool attn_tc_serves(const AttnArgs& a) {
  return row_scaled(a.layout) && a.page_size % 8 == 0 &&
         a.num_pages <= (int64_t)0x7FFFFFFF / a.page_size;
}

cudaError_t prepare_attn_tc() {
  cudaError_t e = prepare_tc_heads<16>();
  if (e == cudaSuccess) e = prepare_tc_heads<32>();
  if (e == cudaSuccess) e = prepare_tc_heads<64>();
  return e;
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream) {
  TcMaps maps;
  int r = a.page_size & -a.page_size;
  maps.box_rows = r < kTcTile ? r : kTcTile;
  if (!encode_plane_map(&maps.latent, a, 128, maps.box_rows) ||
      !encode_plane_map(&maps.rope, a, 64, maps.box_rows))
    return cudaErrorInvalidValue;
  switch (attn_tc_heads(a.heads)) {
    case 16: return launch_tc_heads<16>(a, maps, stream);
    case 32: return launch_tc_heads<32>(a, maps, stream);
    default: return launch_tc_heads<64>(a, maps, stream);
  }
}

}  // namespace mla
