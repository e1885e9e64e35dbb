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
//    weights down to 2^-23 of the largest: a context with one dominant key and
//    thousands of small ones needs their sum.
//
// Tokens lie on TMEM lanes in S^T: a softmax thread owns one cache row and
// half the heads, so a row's scale, mask and page are its scalars, and the
// denominators are sums that stay in its registers until the end.  The
// maximum is a reference, not the exact maximum: it moves (and O is rescaled)
// only when a weight would leave E4M3's range, so most tiles need no
// reduction across lanes at all.
//
// Shared-memory reads of the tensor core bound a tile (N = 64 heads: 18 MMAs of
// 8 KiB for S, 32 of 6 KiB for O, at 128 B a cycle), next to HBM's share of
// 73.7 KiB a tile.
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
// Weights are kept times 2^7, and the reference moves when a logit (base 2)
// passes it by more than 1.75: 2^8.75 = 430 < 448, E4M3's largest.
constexpr float kPShift = 7.0f, kPRoom = 1.75f;
constexpr float kNoMax = -1.0e30f;         // the reference before any key

template <int NH, bool FP8Q>
struct TcSmem {
  static constexpr int kQRows = FP8Q ? NH : 2 * NH;  // MMA N of S^T
  static constexpr int kQPlane = kQRows * 128;
  static constexpr int oQ = 0;                        // 4 latent planes
  static constexpr int oQr = oQ + 4 * kQPlane;        // rope plane, 64-byte rows
  static constexpr int oP = ((oQr + kQRows * 64 + 1023) / 1024) * 1024;  // [row][hi | lo] 128 B
  static constexpr int oRing = oP + kPlane;
  static constexpr int kSlots = (232448 - 1024 - 6144 - oRing) / kPlane > 11 ? 11 : (232448 - 1024 - 6144 - oRing) / kPlane;
  static constexpr int oBar = oRing + kSlots * kPlane;
  // full[slots] empty[slots] s_full[2] s_free[2] p_full pv_done q_full drain
  static constexpr int kBars = 2 * kSlots + 8;
  static constexpr int oMax = (oBar + kBars * 8 + 15) & ~15;  // reference [NH], read as float4
  static constexpr int oAlpha = oMax + NH * 4;        // its rescale factors [NH]
  static constexpr int oXs = oAlpha + NH * 4;         // logit scale of a head's accumulators [NH]
  static constexpr int oRed = oXs + NH * 4;           // [4][NH] across the quadrants
  static constexpr int oRef = oRed + 4 * NH * 4;      // value scale: [0] reference, [1] its ratio, [4..7] warp maxima
  static constexpr int oPlan = (oRef + 48 + 7) & ~7;
  static constexpr int oScan = oPlan + (int)sizeof(AttnPlan);
  static constexpr int oTmem = oScan + 64;
  static constexpr int kBytes = oTmem + 16;
  static constexpr int kAlloc = kBytes + 1024;        // the base is aligned up to 1 KiB
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(kSlots >= 8, "a tile's planes beside the previous tile's");
  static_assert(oP % 1024 == 0 && oRing % 1024 == 0 && oQr % 512 == 0 && kQPlane % 1024 == 0 &&
                    oBar % 8 == 0 && oMax % 16 == 0 && oAlpha % 16 == 0 && oXs % 16 == 0 &&
                    oRed % 16 == 0 && oPlan % 8 == 0 && oScan % 8 == 0 && oTmem % 4 == 0,
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

__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
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

// This warp's 32 lanes x 8 columns.  The loads need tc_wait_ld before use.
__device__ __forceinline__ void tc_ld8(uint32_t addr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
// After tc_wait_ld: the values may be used from here on (the compiler sees no
// other tie between the wait and the registers that the loads fill).
template <int N>
__device__ __forceinline__ void tc_landed(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t addr, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) tc_ld8(addr + i, v + i);
}

// Two FP32 -> two E5M2 codes, round to nearest even, saturating.
__device__ __forceinline__ uint16_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
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

// Whether any of the `count` threads on named barrier `id` says so.
__device__ __forceinline__ bool barrier_any(int id, int count, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tc_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(kTcBar), "r"(kTcSoft) : "memory");
}

// A bounded wait that gives up for good: once one has run out, the thread
// waits no more (its results do not count) and leaves.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (!dead && !mbar_wait_bounded(bar, parity, kTcWait)) dead = true;
}

struct TcMaps {
  CUtensorMap latent;  // boxes of box_rows x 128 bytes, 128-byte swizzle
  CUtensorMap rope;    // boxes of box_rows x 64 bytes, 64-byte swizzle
  int box_rows;        // a power of two that divides the page, 8..128
};

template <int NH, bool FP8Q, int LAYOUT>
__global__ void __launch_bounds__(kTcThreads, 1)
    mla_attn_tc_kernel(const AttnArgs a, const __grid_constant__ TcMaps maps) {
  using S = TcSmem<NH, FP8Q>;
  constexpr int kSlots = S::kSlots;
  constexpr int kHalf = NH / 2;  // heads a softmax thread handles
  constexpr bool kPaged = LAYOUT == MLA_KV_FP8_E4M3_PAGE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::oBar);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_free + 2;
  uint64_t* pv_done = p_full + 1;
  uint64_t* q_full = pv_done + 1;
  uint64_t* drain = q_full + 1;
  float* ref_max = reinterpret_cast<float*>(smem + S::oMax);
  float* alpha = reinterpret_cast<float*>(smem + S::oAlpha);
  float* xs = reinterpret_cast<float*>(smem + S::oXs);
  float* red = reinterpret_cast<float*>(smem + S::oRed);
  float* vref = reinterpret_cast<float*>(smem + S::oRef);
  AttnPlan* plan = reinterpret_cast<AttnPlan*>(smem + S::oPlan);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x % a.groups, worker = blockIdx.x / a.groups;
  const int h0 = group * NH;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], kTcSoft);
    }
    mbar_init(p_full, kTcSoft);
    mbar_init(pv_done, 1);
    mbar_init(q_full, kTcSoft);
    mbar_init(drain, 1);
    mbar_fence_init();
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
  attn_make_plan(a, plan, reinterpret_cast<int64_t*>(smem + S::oScan), blockIdx.x == 0);
  tc_after();
  const uint32_t tmem = *tslot;  // S^T buffers at columns 0 and 128, O^T planes from 256
  const int64_t total = plan->start[a.batch];
  const int workers = attn_workers(a, total);
  const int64_t first = worker < workers ? attn_worker_start(total, workers, worker) : 0;
  const int64_t end = worker < workers ? attn_worker_start(total, workers, worker + 1) : 0;
  bool dead = false;

  if (warp == 8) {
    // ================= TMA: a tile's planes in the order rope, 0, 1, 2, 3
    const int boxes = kTcTile / maps.box_rows;
    const int32_t no_row = (int32_t)(a.num_pages * a.page_size);  // past the end: zeros
    int n = 0;  // planes so far
    int64_t x = first;
    while (x < end && !dead) {
      const int t = attn_token_of(plan, a.batch, x);
      const int64_t t0 = plan->start[t], seg_end = min(plan->start[t + 1], end);
      const int row = a.token_row != nullptr ? a.token_row[t] : t;
      const int64_t len = a.lens[t], nv = attn_positions(a, t, false);
      for (int64_t tile = x; tile < seg_end && !dead; ++tile) {
        int32_t y = no_row;
        if (lane < boxes) {
          int64_t page;
          const int64_t r =
              attn_row(a, t, row, nv, len, (tile - t0) * kTcTile + lane * maps.box_rows, &page);
          if (r >= 0) y = (int32_t)r;
        }
        for (int p = 0; p < 5; ++p, ++n) {
          const int slot = n % kSlots;
          if (n >= kSlots) tc_wait(&empty[slot], (uint32_t)((n / kSlots - 1) & 1), dead);
          dead = __any_sync(0xFFFFFFFFu, dead);
          if (dead) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], p == 0 ? kPlane / 2 : kPlane);
          __syncwarp();
          uint8_t* dst = smem + S::oRing + slot * kPlane;
          if (lane < boxes) {
            if (p == 0)
              tma_g2s_2d(dst + lane * maps.box_rows * 64, &maps.rope, kKvLora, y, &full[slot]);
            else
              tma_g2s_2d(dst + lane * maps.box_rows * 128, &maps.latent, 128 * (p - 1), y, &full[slot]);
          }
        }
      }
      x = seg_end;
    }
    // every copy has landed before the CTA may leave
    for (int k = n > kSlots ? n - kSlots : 0; k < n; ++k)
      (void)mbar_wait_bounded(&full[k % kSlots], (uint32_t)((k / kSlots) & 1), kTcWait);
  } else if (warp == 9) {
    // ================= MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = tc_idesc(128, S::kQRows, 0, false, false);
      constexpr uint32_t id_hi = tc_idesc(128, NH, 0, true, true);
      constexpr uint32_t id_lo = tc_idesc(128, NH, 1, true, true);
      const uint64_t dk = tc_desc(smem_u32(smem + S::oRing), 1024, 2);   // planes, K- or M-major
      const uint64_t dkr = tc_desc(smem_u32(smem + S::oRing), 512, 4);   // rope planes
      const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
      const uint64_t dqr = tc_desc(smem_u32(smem + S::oQr), 512, 4);
      const uint64_t dp = tc_desc(smem_u32(smem + S::oP), 1024, 2);
      int i = 0;        // tiles so far
      int segs = 0;
      int prev_n = -1;  // first plane of the tile whose PV is still due
      bool prev_first = false;
      // S^T of a tile, planes [p0, p1) of rope, 0, 1, 2, 3
      auto qk = [&](int n, int b, int p0, int p1) {
        for (int p = p0; p < p1; ++p) {
          const int slot = (n + p) % kSlots;
          tc_wait(&full[slot], (uint32_t)(((n + p) / kSlots) & 1), dead);
          if (dead) return;
          tc_after();
          const uint32_t d = tmem + 128 * b;
          if (p == 0) {
            const uint64_t da = dkr + (uint64_t)(slot * (kPlane >> 4));
            tc_mma_f8(d, da, dqr, id_s, 0u);
            tc_mma_f8(d, da + 2, dqr + 2, id_s, 1u);
            tc_commit(&empty[slot]);
          } else {
            const uint64_t da = dk + (uint64_t)(slot * (kPlane >> 4));
            const uint64_t db = dq + (uint64_t)((p - 1) * (S::kQPlane >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) tc_mma_f8(d, da + 2 * k, db + 2 * k, id_s, 1u);
          }
        }
      };
      // O^T planes [j0, j1) of the previous tile
      auto pv = [&](int j0, int j1) {
        if (j0 == 0) {
          tc_wait(p_full, (uint32_t)((i - 1) & 1), dead);
          tc_after();
        }
        if (dead) return;
        for (int j = j0; j < j1; ++j) {
          const int slot = (prev_n + 1 + j) % kSlots;
          const uint64_t da = dk + (uint64_t)(slot * (kPlane >> 4));
          const uint32_t d = tmem + 256 + NH * j;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // 32 rows a step: 4096 bytes of V and of P; P's second term 64 bytes on
            tc_mma_f8(d, da + 256 * k, dp + 256 * k, id_hi, (k > 0 || !prev_first) ? 1u : 0u);
            tc_mma_f8(d, da + 256 * k, dp + 256 * k + 4, id_lo, 1u);
          }
          tc_commit(&empty[slot]);
        }
        if (j1 == 4) {
          tc_commit(pv_done);
          prev_n = -1;
        }
      };
      int64_t x = first;
      while (x < end && !dead) {
        const int t = attn_token_of(plan, a.batch, x);
        const int64_t seg_end = min(plan->start[t + 1], end);
        for (int64_t tile = x; tile < seg_end && !dead; ++tile, ++i) {
          const int n = 5 * i, b = i & 1;
          const bool first_tile = tile == x;
          if (first_tile) {
            if (prev_n >= 0) pv(0, 4);  // its softmax must finish before the queries change
            tc_wait(q_full, (uint32_t)(segs & 1), dead);
            tc_after();
          }
          if (i >= 2) {
            tc_wait(&s_free[b], (uint32_t)((i / 2 - 1) & 1), dead);
            tc_after();
          }
          if (dead) break;
          // With eight slots the previous tile's four latent planes leave room
          // for four of this tile's: its last comes once PV has freed one.
          if (prev_n >= 0 && kSlots < 9) {
            qk(n, b, 0, 4);
            pv(0, 1);
            qk(n, b, 4, 5);
            if (!dead) tc_commit(&s_full[b]);
            pv(1, 4);
          } else {
            qk(n, b, 0, 5);
            if (!dead) tc_commit(&s_full[b]);
            if (prev_n >= 0) pv(0, 4);
          }
          prev_n = n;
          prev_first = first_tile;
        }
        ++segs;
        x = seg_end;
      }
      if (prev_n >= 0 && !dead) pv(0, 4);
      if (dead) {  // let what was issued finish before TMEM is freed
        tc_commit(drain);
        (void)mbar_wait_bounded(drain, 0u, kTcWait);
      }
    }
  } else {
    // ================= softmax, rescaling, epilogue (warps 0-7)
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int pos = 32 * quad + lane;    // this thread's row of a tile
    const int hb = half * kHalf;         // its heads
    const float qinv = a.q_scale_inv != nullptr ? *a.q_scale_inv : 1.0f;
    const float logit = a.scale / qinv * 1.4426950408889634f;
    const float tensor_scale = kPaged ? 1.0f : *a.k_scale;
    int i = 0;
    int64_t x = first;
    // A thread whose wait has run out goes on without waiting: all of them
    // pass the same barriers to the end.
    while (x < end) {
      const int t = attn_token_of(plan, a.batch, x);
      const int64_t t0 = plan->start[t], t1 = plan->start[t + 1], seg_end = min(t1, end);
      const int row = a.token_row != nullptr ? a.token_row[t] : t;
      const int64_t len = a.lens[t], nv = attn_positions(a, t, false);
      int64_t page = 0;
      int64_t crow = attn_row(a, t, row, nv, len, (x - t0) * kTcTile + pos, &page);
      float rscale = crow >= 0 && kPaged ? a.k_scale[page] : 1.0f;
      // ---- queries: a warp a head, 16 latent columns a lane, 16 rope columns
      // for lanes 0-3 (every MMA on the previous queries has completed: its S
      // has been read)
      for (int h = warp; h < NH; h += 8) {
        uint4 hi = make_uint4(0, 0, 0, 0), hr = hi;
        float xscale = 0.f;
        if (h0 + h < a.heads) {
          const int64_t el = (int64_t)t * a.ql_ts + (int64_t)(h0 + h) * a.ql_hs + 16 * lane;
          const int64_t ep = (int64_t)t * a.qp_ts + (int64_t)(h0 + h) * a.qp_hs + 16 * lane;
          if constexpr (FP8Q) {
            hi = *reinterpret_cast<const uint4*>(a.q_latent + el);
            if (lane < 4) hr = *reinterpret_cast<const uint4*>(a.q_pe + ep);
            xscale = logit;
          } else {
            const uint4* l = reinterpret_cast<const uint4*>(a.q_latent + 2 * el);
            const uint4* r = reinterpret_cast<const uint4*>(a.q_pe + 2 * ep);
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 w[4] = {l[0], l[1], lane < 4 ? r[0] : z, lane < 4 ? r[1] : z};
            float v[32], mx = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t ww[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[8 * e + 2 * k] = bf16lo(ww[k]);
                v[8 * e + 2 * k + 1] = bf16hi(ww[k]);
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, fabsf(v[e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            // the power of two that brings the largest into (224, 448]: from
            // its exponent field, kept where both it and its inverse are normal
            int ex = (int)((__float_as_uint(mx) >> 23) & 255u) - 127;
            ex = max(-100, min(ex, 126));
            if ((__float_as_uint(mx) & 0x007FFFFFu) <= 0x00600000u) --ex;
            const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
            xscale = logit * __uint_as_float((uint32_t)(127 - 7 + ex) << 23);
            // an infinite query: no finite logits (E4M3 has no infinity)
            if (mx == INFINITY) xscale = __int_as_float(0x7FC00000);
            uint32_t c[8], d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float f0 = v[4 * e] * up, f1 = v[4 * e + 1] * up, f2 = v[4 * e + 2] * up,
                          f3 = v[4 * e + 3] * up;
              const uint16_t a0 = e4m3x2(f0, f1), a1 = e4m3x2(f2, f3);
              const float2 g0 = e4m3x2_value(a0), g1 = e4m3x2_value(a1);
              c[e] = (uint32_t)a0 | ((uint32_t)a1 << 16);
              d[e] = (uint32_t)e4m3x2(f0 - g0.x, f1 - g0.y) |
                     ((uint32_t)e4m3x2(f2 - g1.x, f3 - g1.y) << 16);
            }
            hi = make_uint4(c[0], c[1], c[2], c[3]);
            hr = make_uint4(c[4], c[5], c[6], c[7]);
            const int rl = NH + h;  // the second terms' row
            *reinterpret_cast<uint4*>(smem + S::oQ + (lane >> 3) * S::kQPlane + rl * 128 +
                                      (((lane ^ rl) & 7) << 4)) = make_uint4(d[0], d[1], d[2], d[3]);
            if (lane < 4)
              *reinterpret_cast<uint4*>(smem + S::oQr + rl * 64 + ((lane ^ ((rl >> 1) & 3)) << 4)) =
                  make_uint4(d[4], d[5], d[6], d[7]);
          }
        } else if constexpr (!FP8Q) {
          const int rl = NH + h;
          *reinterpret_cast<uint4*>(smem + S::oQ + (lane >> 3) * S::kQPlane + rl * 128 +
                                    (((lane ^ rl) & 7) << 4)) = hi;
          if (lane < 4)
            *reinterpret_cast<uint4*>(smem + S::oQr + rl * 64 + ((lane ^ ((rl >> 1) & 3)) << 4)) = hr;
        }
        *reinterpret_cast<uint4*>(smem + S::oQ + (lane >> 3) * S::kQPlane + h * 128 +
                                  (((lane ^ h) & 7) << 4)) = hi;
        if (lane < 4)
          *reinterpret_cast<uint4*>(smem + S::oQr + h * 64 + ((lane ^ ((h >> 1) & 3)) << 4)) = hr;
        if (lane == 0) {
          xs[h] = xscale;
          ref_max[h] = kNoMax;
        }
      }
      if (tid == 0) vref[0] = kPaged ? 0.f : tensor_scale;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
      tc_barrier();
      float l[kHalf];
#pragma unroll
      for (int h = 0; h < kHalf; ++h) l[h] = 0.f;

      for (int64_t tile = x; tile < seg_end; ++tile, ++i) {
        const int b = i & 1;
        const bool valid = crow >= 0;
        const float rs = kPaged ? rscale : tensor_scale;
        // a row that is loaded but does not count holds anything, NaN codes too
        const bool wipe = !valid;
        tc_wait(&s_full[b], (uint32_t)((i >> 1) & 1), dead);
        tc_after();
        float s[kHalf];
        tc_ld(tmem + lanes + 128 * b + hb, s);
        if constexpr (!FP8Q) {
          float lo[kHalf];
          tc_ld(tmem + lanes + 128 * b + NH + hb, lo);
          tc_wait_ld();
          tc_landed(s);
          tc_landed(lo);
#pragma unroll
          for (int h = 0; h < kHalf; ++h) s[h] += lo[h];
        } else {
          tc_wait_ld();
          tc_landed(s);
        }
        tc_before();
        mbar_arrive(&s_free[b]);
        // logits in base 2, and how far they pass the reference
        float over = -INFINITY;
#pragma unroll
        for (int h = 0; h < kHalf; h += 4) {
          const float4 sc = *reinterpret_cast<const float4*>(xs + hb + h);
          const float4 m = *reinterpret_cast<const float4*>(ref_max + hb + h);
          const float scv[4] = {sc.x, sc.y, sc.z, sc.w}, mv[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[h + e] = valid ? s[h + e] * (scv[e] * rs) : -INFINITY;
            over = fmaxf(over, s[h + e] - mv[e]);
          }
        }
        bool move = over > kPRoom;
        if (kPaged) move |= valid && fabsf(rscale) > vref[0];
        if (barrier_any(kTcBar, kTcSoft, move)) {
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
            const float old = ref_max[tid];
            const float m = fmaxf(fmaxf(red[tid], red[NH + tid]), fmaxf(red[2 * NH + tid], red[3 * NH + tid]));
            const bool grow = m - old > kPRoom;
            alpha[tid] = grow ? exp2f(old - m) : 1.0f;
            if (grow) ref_max[tid] = m;
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
          for (int h = 0; h < kHalf; ++h) l[h] *= alpha[hb + h];
          if (tile > x) {
            tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
            tc_after();
#pragma unroll 1
            for (int c = 0; c < 2 * NH; c += 8) {
              // planes 2 half and 2 half + 1 of O^T: columns are heads
              float v[8];
              const uint32_t at = tmem + lanes + 256 + 2 * half * NH + c;
              tc_ld8(at, v);
              tc_wait_ld();
              tc_landed(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= alpha[(c + e) % NH] * ratio;
              tc_st8(at, v);
            }
            tc_wait_st();
          }
        }
        // ---- weights
        const float vs = kPaged ? (valid && vref[0] > 0.f ? rscale / vref[0] : 0.f) : 1.0f;
        uint32_t phi[kHalf / 4], plo[kHalf / 4];
#pragma unroll
        for (int h = 0; h < kHalf; h += 4) {
          const float4 m = *reinterpret_cast<const float4*>(ref_max + hb + h);
          const float mv[4] = {m.x, m.y, m.z, m.w};
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = exp2f(s[h + e] - (mv[e] - kPShift));
            l[h + e] += p[e];
            if (kPaged) p[e] *= vs;
          }
          const uint16_t a0 = e4m3x2(p[0], p[1]), a1 = e4m3x2(p[2], p[3]);
          const float2 g0 = e4m3x2_value(a0), g1 = e4m3x2_value(a1);
          phi[h / 4] = (uint32_t)a0 | ((uint32_t)a1 << 16);
          plo[h / 4] = (uint32_t)e5m2x2(p[0] - g0.x, p[1] - g0.y) |
                       ((uint32_t)e5m2x2(p[2] - g1.x, p[3] - g1.y) << 16);
        }
        // the previous tile's PV has read P (and the planes that `wipe` touches
        // belong to this tile, whose S is done)
        if (i > 0) tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
        if (wipe && half == 0) {
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint4* d = reinterpret_cast<uint4*>(smem + S::oRing + ((5 * i + 1 + j) % kSlots) * kPlane + pos * 128);
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
        mbar_arrive(p_full);
        // the next tile's row
        if (tile + 1 < seg_end) {
          crow = attn_row(a, t, row, nv, len, (tile + 1 - t0) * kTcTile + pos, &page);
          if (kPaged) rscale = crow >= 0 ? a.k_scale[page] : 1.0f;
        }
      }
      // ---- the stretch is done
      {
        const float sum = lanes_reduce<kHalf, OpSum>(l);
        if ((lane * kHalf) % 32 == 0) red[quad * NH + hb + lane * kHalf / 32] = sum;
      }
      tc_barrier();
      const bool whole = x == t0 && seg_end == t1;
      const int slot = 2 * worker + (x == first ? 0 : 1);
      if (tid < NH) {
        const float sum = (red[tid] + red[NH + tid]) + (red[2 * NH + tid] + red[3 * NH + tid]);
        const float m = ref_max[tid];
        const bool none = m == kNoMax && sum == 0.f;
        const float mm = none ? -INFINITY : m - kPShift;
        if (whole) {
          alpha[tid] = none ? 0.f : vref[0] / sum;
          if (a.lse != nullptr && h0 + tid < a.heads)
            a.lse[(int64_t)t * a.heads + h0 + tid] = attn_lse(mm, sum);
        } else {
          alpha[tid] = none ? 0.f : vref[0];
          float* ml = a.part_ml + ((int64_t)slot * a.heads_pad + h0 + tid) * 2;
          ml[0] = mm;
          ml[1] = sum;
        }
      }
      tc_barrier();
      tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead);
      tc_after();
#pragma unroll 1
      for (int c = 0; c < 2 * NH; c += 8) {
        float v[8];
        tc_ld8(tmem + lanes + 256 + 2 * half * NH + c, v);
        tc_wait_ld();
        tc_landed(v);
        const int col = 128 * (2 * half + c / NH) + pos;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int h = (c + e) % NH;
          if (whole) {
            if (h0 + h < a.heads)
              a.out[(int64_t)t * a.o_ts + (int64_t)(h0 + h) * a.o_hs + col] = f2bf_bits(v[e] * alpha[h]);
          } else {
            a.part_o[((int64_t)slot * a.heads_pad + h0 + h) * kKvLora + col] = v[e] * alpha[h];
          }
        }
      }
      tc_before();
      tc_barrier();  // alpha and red are read
      x = seg_end;
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
  cfg.dynamicSmemBytes = TcSmem<NH, FP8Q>::kAlloc;
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
                              cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<NH, FP8Q>::kAlloc);
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
