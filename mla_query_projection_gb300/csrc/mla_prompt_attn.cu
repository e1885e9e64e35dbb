// mla_prompt_attn.cu - attention of a prompt on the 5th-generation tensor cores:
// packed documents, keys of 128 + 64 columns a head (the 64 shared by all
// heads), values of 128.
//
//   x_ij = cap(scale q_i . k_j) - slope |place_i - j|,  cap(x) = c tanh(x / c)
//   out_i = sum_j p_ij v_j,  p_i = softmax over the keys that row i sees
//
// A CTA takes 256 query rows of one head and document as two tiles of 128, and
// goes through the keys in tiles of 128 that both share.  S = Q K^T (M = 128
// rows, N = 128 keys, K = 192) and O += P V (K = 128 keys, N = 128 columns) are
// tcgen05 products with FP32 accumulators in TMEM; P goes back to TMEM as BF16
// in the place of its S, and is read from there.  While the softmax of one tile
// runs, the tensor core works for the other: O0 += P0 V, S0 of the next keys,
// O1 += P1 V, S1.
//
//  * A softmax thread owns one query row: its maximum, its sum and its mask need
//    no other lane.  The row's reference (what exponents are taken relative to)
//    moves only when a score passes it by more than 2^8, and only then is O
//    rescaled: P then reaches 256, as exact in BF16 as at 1.
//  * What a row sees are the first `bound` keys of its document: its own place
//    and all before it, or its document's two-way prefix, or all.  Tiles that no
//    row of theirs needs are not touched, and only those on an edge are masked.
//  * Keys and values come by TMA in units of 16 KiB through a ring of eight: 64
//    columns of 128 keys, or 64 keys of 128 values.
//  * A value that a row does not see may be an infinity or a NaN, and zero times
//    it is not zero.  So on the tiles with an edge the softmax threads look their
//    values over first: rows behind the document are zeroed; an infinity or a NaN
//    inside it is replaced by zero and noted for its column with its place, and
//    the rows that see it get it at the end.
//  * Few query rows: the keys are split over several CTAs, whose sums a second
//    kernel joins.
#include <stdlib.h>

#include "mla_attn_tc.cuh"
#include "mla_prompt.h"

struct mla_prompt {
  int device;
  int num_sms;
  int heads;
  uint32_t* err;
  float* part_o;    // sums of split rows
  float2* part_ml;  // their references and denominators
};

namespace mla {
namespace {

constexpr int kPrTile = 128;                  // query rows and keys of a tile
constexpr int kPrUnit = 16384;                // bytes of a ring unit
constexpr int kPrRing = 8;
constexpr int kPrThreads = 320;               // two softmax warpgroups, a TMA warp, an MMA warp
constexpr int kPrQ = 3 * kPrUnit;             // a query tile: planes of 64 columns
constexpr float kPrRoom = 8.0f;               // base 2

struct PrSmem {
  static constexpr int oQ = 0;
  static constexpr int oRing = 2 * kPrQ;
  static constexpr int oBar = oRing + kPrRing * kPrUnit;
  // full[8] empty[8] q_full[2] s_full[2] p_full[2] o_full[2] drain
  static constexpr int kBars = 25;
  static constexpr int oBad = oBar + kBars * 8;  // [3][128] first NaN, infinity, -infinity of a column
  static constexpr int oAny = oBad + 3 * 128 * 4;
  static constexpr int oPlan = oAny + 4;         // document, tile, total
  static constexpr int oScan = oPlan + 12;       // [10]
  static constexpr int oTmem = oScan + 40;
  static constexpr int kBytes = oTmem + 8;
  static_assert(kBytes <= 232448 && oBar % 8 == 0 && oBad % 4 == 0, "shared memory budget");
};

// O += P V, four steps of 16 keys: P in TMEM (8 columns a step), V's steps 2 KiB apart.
__device__ __forceinline__ void pr_mma4_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, %4, %4;\n\telect.sync _|q, 0xFFFFFFFF;\n\tmov.b32 x, %1;\n\tmov.b64 y, %2;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t"
      "add.s32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.s32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.s32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_g2s_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct PrDoc {
  int q0, nq, k0, nk, prefix, tile;
  // keys that query row i (of the document) sees
  __device__ __forceinline__ int bound(int i, bool causal) const {
    if (!causal) return nk;
    const int own = i + (nk - nq) + 1;
    return max(min(prefix, nk), max(0, min(own, nk)));
  }
};

// CAP: scores are capped; BIAS: they lose by distance.
template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kPrThreads, 1)
    mla_prompt_attn_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
  using S = PrSmem;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::oBar);
  uint64_t* empty = full + kPrRing;
  uint64_t* q_full = empty + kPrRing;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 2;
  int* bad = reinterpret_cast<int*>(smem + S::oBad);
  volatile uint32_t* any_bad = reinterpret_cast<uint32_t*>(smem + S::oAny);
  int* plan = reinterpret_cast<int*>(smem + S::oPlan);
  int* scan = reinterpret_cast<int*>(smem + S::oScan);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int head = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();

  // ---- which document and tile: the prefix sum of the documents' tiles, the
  // last tiles first (with causal masks they are the longest)
  const int each = (a.docs + kPrThreads - 1) / kPrThreads;
  const int d0 = min(a.docs, tid * each), d1 = min(a.docs, d0 + each);
  auto place = [&](const int32_t* cu, int d, int most, int* n) {
    const int lo = cu[d], hi = cu[d + 1];
    const int c0 = max(0, min(lo, most)), c1 = max(c0, min(hi, most));
    *n = c1 - c0;
    if ((c0 != lo || c1 != hi) && blockIdx.x == 0 && head == 0 && blockIdx.z == 0) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    return c0;
  };
  int mine = 0;
  for (int d = d0; d < d1; ++d) {
    int n;
    place(a.cu_q, d, a.q_tokens, &n);
    mine += (n + 2 * kPrTile - 1) / (2 * kPrTile);
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) scan[warp] = sum;
  if (tid == 0) plan[0] = -1;
  __syncthreads();
  int before = sum - mine, total = 0;
  for (int w = 0; w < kPrThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int x = total - 1 - (int)blockIdx.x;
  if (x >= before && x < before + mine) {
    int at = before;
    for (int d = d0; d < d1; ++d) {
      int n;
      place(a.cu_q, d, a.q_tokens, &n);
      const int t = (n + 2 * kPrTile - 1) / (2 * kPrTile);
      if (x < at + t) {
        plan[0] = d;
        plan[1] = x - at;
        break;
      }
      at += t;
    }
  }
  for (int c = tid; c < 3 * 128; c += kPrThreads) bad[c] = 0x7FFFFFFF;
  if (tid == 0) {
    *any_bad = 0;
    for (int s = 0; s < kPrRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&q_full[q], 1);
      mbar_init(&s_full[q], 1);
      mbar_init(&p_full[q], 4);
      mbar_init(&o_full[q], 1);
    }
    mbar_init(drain, 1);
    mbar_fence_init();
    if (smem_u32(smem) & 1023u) atomicOr(a.err, MLA_DEVERR_CHECK);
  }
  __syncthreads();
  const int d = plan[0];
  if (d < 0) return;  // (the grid is an upper bound of the tiles)
  PrDoc k;
  k.tile = plan[1];
  k.q0 = place(a.cu_q, d, a.q_tokens, &k.nq);
  k.k0 = place(a.cu_k, d, a.k_tokens, &k.nk);
  k.prefix = a.prefix != nullptr ? a.prefix[d] : 0;
  const bool causal = a.causal != 0;
  // query tile q: rows first[q] .. of the document, key tiles [j0, n[q])
  const int r0 = k.tile * 2 * kPrTile;
  int n[2], safe[2];  // key tiles below safe[q] are seen whole by every row
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int lo = r0 + q * kPrTile, hi = min(lo + kPrTile, k.nq);
    n[q] = hi > lo ? (k.bound(hi - 1, causal) + kPrTile - 1) / kPrTile : 0;
    safe[q] = hi > lo ? k.bound(lo, causal) / kPrTile : 0;
  }
  // this CTA's share of the key tiles
  const int all = max(n[0], n[1]);
  const int j0 = (int)((int64_t)all * blockIdx.z / a.splits), j1 = (int)((int64_t)all * (blockIdx.z + 1) / a.splits);
  n[0] = min(n[0], j1);
  n[1] = min(n[1], j1);
  const int end = max(n[0], n[1]);  // == j1, or none where j1 <= j0

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = uniform(*tslot);  // S at columns 0 and 128, O at 256 and 384
  bool dead = false;

  if (warp == 8) {
    // ================= TMA: queries, then units in the order K, V of tile after tile
    if (lane == 0 && j0 < end) {
      int use = 0;  // units so far
      auto next = [&]() -> int {
        const int s = use % kPrRing;
        if (use >= kPrRing) tc_wait(&empty[s], (uint32_t)((use / kPrRing - 1) & 1), dead);
        return s;
      };
      auto query = [&](int q) {
        if (n[q] <= j0) return;
        mbar_arrive_expect_tx(&q_full[q], kPrQ);
        const uint32_t dst = smem_u32(smem + S::oQ) + q * kPrQ;
        const int row = k.q0 + r0 + q * kPrTile;
        tma_g2s_3d(dst, &maps.q_nope, 0, head, row, &q_full[q]);
        tma_g2s_3d(dst + kPrUnit, &maps.q_nope, 64, head, row, &q_full[q]);
        tma_g2s_3d(dst + 2 * kPrUnit, &maps.q_pe, 0, head, row, &q_full[q]);
      };
      query(0);
      for (int j = j0; j < end && !dead; ++j) {
        const int row = k.k0 + j * kPrTile;
        for (int u = 0; u < 3 && !dead; ++u) {
          const int s = next();
          if (dead) break;
          const uint32_t dst = smem_u32(smem + S::oRing) + s * kPrUnit;
          mbar_arrive_expect_tx(&full[s], kPrUnit);
          if (u < 2)
            tma_g2s_3d(dst, &maps.k_nope, 64 * u, head, row, &full[s]);
          else
            tma_g2s_3d(dst, &maps.k_pe, 0, 0, row, &full[s]);
          ++use;
        }
        if (j == j0) query(1);
        for (int u = 0; u < 2 && !dead; ++u) {  // 64 keys, both halves of their columns
          const int s = next();
          if (dead) break;
          const uint32_t dst = smem_u32(smem + S::oRing) + s * kPrUnit;
          mbar_arrive_expect_tx(&full[s], kPrUnit);
          tma_g2s_3d(dst, &maps.v, 0, head, row + 64 * u, &full[s]);
          tma_g2s_3d(dst + kPrUnit / 2, &maps.v, 64, head, row + 64 * u, &full[s]);
          ++use;
        }
      }
      if (dead) {  // the copies under way land before the CTA leaves
        for (int q = 0; q < 2; ++q)
          if (n[q] > j0) (void)mbar_wait_bounded(&q_full[q], 0u, kTcWait);
        for (int s = 0; s < kPrRing; ++s)
          if (use > s) (void)mbar_wait_bounded(&full[s], (uint32_t)(((use - 1 - s) / kPrRing) & 1), kTcWait);
      }
    }
  } else if (warp == 9) {
    // ================= MMA issuer (the warp together, one elected lane issues)
    constexpr uint32_t kBf16 = 1u << 7;
    constexpr uint32_t id_s = tc_idesc(128, 128, 1, false, false) | kBf16;
    constexpr uint32_t id_o = tc_idesc(128, 128, 1, false, true) | kBf16;
    const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
    const uint64_t dk = tc_desc(smem_u32(smem + S::oRing), 1024, 2);
    const uint64_t dv = tc_desc_wide(smem_u32(smem + S::oRing), 1024, kPrUnit / 2);
    const int n0 = (int)uniform((uint32_t)n[0]), n1 = (int)uniform((uint32_t)n[1]);
    const int jb = (int)uniform((uint32_t)j0), je = max(n0, n1);
    // unit u of key tile j: 0..2 keys, 3, 4 values
    auto unit = [&](int j, int u) { return 5 * (j - jb) + u; };
    auto wait_unit = [&](int i) { tc_wait_warp(&full[i % kPrRing], (uint32_t)((i / kPrRing) & 1), dead); };
    auto scores = [&](int q, int j, bool last) {
      if (j == jb) tc_wait_warp(&q_full[q], 0u, dead);
#pragma unroll 1
      for (int u = 0; u < 3; ++u) {
        const int i = unit(j, u);
        wait_unit(i);
        tc_after();
        tc_mma4_f16<2, 2>(tmem + 128 * q, dq + (uint64_t)((q * kPrQ + u * kPrUnit) >> 4),
                          dk + (uint64_t)((i % kPrRing) * (kPrUnit >> 4)), id_s, u > 0);
        if (last) tc_commit(&empty[i % kPrRing]);
      }
      tc_commit(&s_full[q]);
    };
    auto values = [&](int q, int j, bool last) {
      tc_wait_warp(&p_full[q], (uint32_t)((j - jb) & 1), dead);
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        const int i = unit(j, 3 + u);
        wait_unit(i);
        tc_after();
        pr_mma4_pv(tmem + 256 + 128 * q, tmem + 128 * q + 32 * u, dv + (uint64_t)((i % kPrRing) * (kPrUnit >> 4)), id_o,
                   j > jb || u > 0);
        if (last) tc_commit(&empty[i % kPrRing]);
      }
    };
    if (jb < je) {
      if (jb < n0) scores(0, jb, jb >= n1);
      if (jb < n1) scores(1, jb, true);
      for (int j = jb; j < je; ++j) {
        if (j < n0) {
          values(0, j, j >= n1);
          if (j + 1 < n0) scores(0, j + 1, j + 1 >= n1);
          else tc_commit(&o_full[0]);
        }
        if (j < n1) {
          values(1, j, true);
          if (j + 1 < n1) scores(1, j + 1, true);
          else tc_commit(&o_full[1]);
        }
      }
      if (dead) {
        tc_commit(drain);
        (void)mbar_wait_bounded(drain, 0u, kTcWait);
      }
    }
  } else {
    // ================= softmax (warps 0-3: query tile 0, 4-7: tile 1)
    const int q = warp >> 2, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int i = r0 + q * kPrTile + 32 * quad + lane;  // this thread's row of the document
    const int bound = k.bound(min(i, k.nq - 1), causal);
    const int nq = n[q];
    const float scale2 = a.scale * 1.4426950408889634f;
    // capped: x = C - 2 C / (1 + 2^(s e)), e = 2 scale log2(e) / cap, in base 2
    const float capC = CAP ? a.cap * 1.4426950408889634f : 0.f, capE = CAP ? 2.0f * scale2 / a.cap : 0.f;
    const float slope = BIAS ? -a.slopes[head] * 1.4426950408889634f : 0.f;
    const float own = (float)(i + k.nk - k.nq);  // its place among the keys
    float ref = -INFINITY, l = 0.f;
    for (int j = j0; j < nq; ++j) {
      const uint32_t st = tmem + lanes + 128 * q;
      tc_wait(&s_full[q], (uint32_t)((j - j0) & 1), dead);
      tc_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc_ld(st + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
      tc_wait_ld();
      tc_landed(s);
      // Scores to base 2: at once where something is done to them, else with
      // the subtraction of the reference.
      if constexpr (CAP) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = fmaf(-2.0f * capC, rcp_approx(1.0f + ex2(s[c] * capE)), capC);
      }
      if constexpr (BIAS) {
        const float base = own - (float)(j * kPrTile);
#pragma unroll
        for (int c = 0; c < 128; ++c) {
          const float x2 = CAP ? s[c] : s[c] * scale2;
          s[c] = fmaf(slope, fabsf(base - (float)c), x2);
        }
      }
      const float unit2 = CAP || BIAS ? 1.0f : scale2;
      if (j >= safe[q]) {
        const int left = bound - j * kPrTile;  // keys of this tile that count
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < left ? s[c] : -INFINITY;
      }
      float m4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) m4[e] = fmaxf(s[e], s[e + 4]);
#pragma unroll
      for (int c = 8; c < 128; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], fmaxf(s[c + e], s[c + e + 4]));
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * unit2;
      // The reference: the first maximum; later only where it is passed by far.
      const bool grow = mx > ref + kPrRoom || (ref == -INFINITY && mx > -INFINITY);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        float f = 1.0f;
        if (grow) {
          f = ex2(ref - mx);  // 0 from -infinity
          ref = mx;
          l *= f;
        }
        if (j > j0) {
          // (S of this tile was issued after O of the one before: both are done)
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float v[32];
            const uint32_t at = tmem + lanes + 256 + 128 * q + c;
            tc_ld(at, v);
            tc_wait_ld();
            tc_landed(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= f;
            tc_st32(at, v);
          }
        }
      }
      const float minus = ref == -INFINITY ? 0.f : -ref;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 e = fma2(make_float2(s[64 * half + 2 * c], s[64 * half + 2 * c + 1]), make_float2(unit2, unit2),
                                make_float2(minus, minus));
          const float2 p = make_float2(ex2(e.x), ex2(e.y));
          sum[c & 1] = add2(sum[c & 1], p);
          pk[c] = __uint_as_float(pack_bf16x2(p.x, p.y));
        }
        tc_st32(st + 32 * half, pk);
      }
      const float2 both = add2(sum[0], sum[1]);
      l += both.x + both.y;
      // An edge in this tile (for either query tile): its values are looked over
      // by the first of the two that still has it.
      const bool edge = (j < n[0] && j >= safe[0]) || (j < n[1] && j >= safe[1]);
      if (edge && (q == 0 || j >= n[0])) {
        const int r = 32 * quad + lane, u = 5 * (j - j0) + 3 + (r >> 6), slot = u % kPrRing;
        tc_wait(&full[slot], (uint32_t)((u / kPrRing) & 1), dead);
        uint8_t* base = smem + S::oRing + slot * kPrUnit + (r & 63) * 128;
        const int key = j * kPrTile + r;
        if (key >= k.nk) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(base + (c >> 3) * (kPrUnit / 2) + (((c + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
        } else {
          uint32_t mag = 0;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(base + (c >> 3) * (kPrUnit / 2) + (((c + lane) & 7) << 4));
            const uint32_t g = 0x7FFF7FFFu;
            mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(w.x & g, w.y & g), __vmaxu2(w.z & g, w.w & g)));
          }
          if ((mag & 0xFFFFu) >= 0x7F80u || (mag >> 16) >= 0x7F80u) {
#pragma unroll 1
            for (int c = 0; c < 128; ++c) {
              // chunk c / 8 of the row lies where the 128-byte swizzle puts it
              uint16_t* e = reinterpret_cast<uint16_t*>(base + (c >> 6) * (kPrUnit / 2) +
                                                        ((((c >> 3) & 7) ^ (r & 7)) << 4)) + (c & 7);
              const uint32_t w = *e;
              if ((w & 0x7F80u) == 0x7F80u) {
                const int kind = (w & 0x7Fu) != 0 ? 0 : (w & 0x8000u) == 0 ? 1 : 2;
                atomicMin(&bad[kind * 128 + c], key);
                *e = 0;
              }
            }
            *any_bad = 1;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      tc_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[q]);
    }
    // ---- the sums
    if (nq > j0) {
      tc_wait(&o_full[q], 0u, dead);
      tc_after();
    }
    const bool have = i < k.nq;
    const int64_t row = k.q0 + i;
    const bool part = a.splits > 1;
    const float inv = part ? 1.0f : l == 0.f ? 0.f : 1.0f / l;
    const bool noted = nq > j0 && *any_bad != 0;
    if (have) {
      if (part)
        a.part_ml[((int64_t)blockIdx.z * a.heads + head) * a.q_tokens + row] = make_float2(ref, l);
      else if (a.lse != nullptr)
        a.lse[row * a.heads + head] = l == 0.f ? -INFINITY : ref * 0.6931471805599453f + logf(l);
    }
    float* po = a.part_o + (((int64_t)blockIdx.z * a.heads + head) * a.q_tokens + row) * 128;
    uint16_t* o = a.out + row * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      float v[32];
      if (nq > j0) {
        tc_ld(tmem + lanes + 256 + 128 * q + c, v);
        tc_wait_ld();
        tc_landed(v);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = nq > j0 && l != 0.f ? v[e] * inv : 0.f;
      if (noted && l != 0.f) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const bool nan = bad[c + e] < bound, up = bad[128 + c + e] < bound, down = bad[256 + c + e] < bound;
          if (nan || up || down) v[e] = nan || (up && down) ? __int_as_float(0x7FC00000) : v[e] + (up ? INFINITY : -INFINITY);
        }
      }
      if (have) {
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(po + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(o + c + e) =
                make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                           pack_bf16x2(v[e + 6], v[e + 7]));
        }
      }
    }
    tc_before();
  }
  if (dead) atomicOr(a.err, MLA_DEVERR_TIMEOUT);
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// --------------------------------------------------------------- joining
//
// A warp a (row, head): with M the largest reference of its parts,
// out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  A lane has four columns.
__global__ void __launch_bounds__(256) mla_prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = item / a.heads;
  const int head = (int)(item - row * a.heads);
  // rows of no document are left as they are
  if (row >= a.q_tokens || row < a.cu_q[0] || row >= a.cu_q[a.docs]) return;
  const int64_t step = (int64_t)a.heads * a.q_tokens, at = (int64_t)head * a.q_tokens + row;
  float M = -INFINITY;
  for (int s = 0; s < a.splits; ++s) M = fmaxf(M, a.part_ml[s * step + at].x);
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.part_ml[s * step + at];
    if (ml.y == 0.f) continue;  // saw nothing
    const float f = exp2f(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (s * step + at) * 128 + 4 * lane);
    l = fmaf(f, ml.y, l);
    o.x = fmaf(f, v.x, o.x);
    o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z);
    o.w = fmaf(f, v.w, o.w);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* out = a.out + row * a.o_ts + (int64_t)head * a.o_hs + 4 * lane;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (a.lse != nullptr && lane == 0)
    a.lse[row * a.heads + head] = l == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(l);
}

// A map of [tokens][heads][width] values in boxes of box_rows tokens x 64 columns.
bool encode_heads_map(CUtensorMap* map, const void* base, int64_t tokens, int heads, int width, int64_t ts, int64_t hs,
                      int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool CAP, bool BIAS>
cudaError_t launch_prompt_kernel(const PromptArgs& a, const PromptMaps& maps, int tiles, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)a.heads, (unsigned)a.splits);
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = PrSmem::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_prompt_attn_kernel<CAP, BIAS>, a, maps);
}

template <bool CAP, bool BIAS>
cudaError_t prepare_prompt_kernel() {
  return cudaFuncSetAttribute(mla_prompt_attn_kernel<CAP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrSmem::kBytes);
}

}  // namespace

cudaError_t prepare_prompt() {
  cudaError_t e = prepare_prompt_kernel<false, false>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<true, false>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<false, true>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<true, true>();
  return e;
}

cudaError_t launch_prompt(const PromptArgs& a, const PromptInputs& in, int tiles, cudaStream_t stream) {
  PromptMaps maps = {};
  const int keys = a.k_tokens > 0 ? a.k_tokens : 1;
  if (!encode_heads_map(&maps.q_nope, in.q_nope, a.q_tokens, a.heads, kNope, in.qn_ts, in.qn_hs, kPrTile) ||
      !encode_heads_map(&maps.q_pe, in.q_pe, a.q_tokens, a.heads, kRope, in.qp_ts, in.qp_hs, kPrTile) ||
      !encode_heads_map(&maps.k_nope, in.k_nope, keys, a.heads, kNope, in.kn_ts, in.kn_hs, kPrTile) ||
      !encode_heads_map(&maps.k_pe, in.k_pe, keys, 1, kRope, in.kp_ts, in.kp_ts, kPrTile) ||
      !encode_heads_map(&maps.v, in.v, keys, a.heads, kNope, in.v_ts, in.v_hs, kPrTile / 2))
    return cudaErrorInvalidValue;
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  cudaError_t e = cap ? (bias ? launch_prompt_kernel<true, true>(a, maps, tiles, stream)
                              : launch_prompt_kernel<true, false>(a, maps, tiles, stream))
                      : (bias ? launch_prompt_kernel<false, true>(a, maps, tiles, stream)
                              : launch_prompt_kernel<false, false>(a, maps, tiles, stream));
  if (e != cudaSuccess || a.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.q_tokens * a.heads + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_prompt_join_kernel, a);
}

namespace {

// Rows of partial sums a handle has room for: three CTAs' an SM.
int64_t part_rows(int num_sms) { return 3 * (int64_t)num_sms * 2 * kPrTile; }

// Over how many CTAs each tile's keys are split: as many as make the SMs' rounds
// shortest, counting three key tiles for what a CTA costs beside its own and four
// for the join; at least two key tiles each, as far as the lengths on average
// tell.
int prompt_splits(int64_t units, int64_t q_rows, int64_t key_tiles, int num_sms) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 64; ++s) {
    if (s > 1 && (s * 2 > key_tiles || s * q_rows > part_rows(num_sms))) break;
    const int64_t rounds = (units * s + num_sms - 1) / num_sms;
    const int64_t cost = rounds * ((key_tiles + s - 1) / s + 3) + (s > 1 ? 4 : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();
  return MLA_ECUDA;
}

// Strides of a [tokens][heads][width] operand; 0 means contiguous.
bool prompt_strides(int heads, int width, int64_t* ts, int64_t* hs) {
  if (*hs == 0) *hs = width;
  if (*ts == 0) *ts = heads * *hs;
  constexpr int64_t most = (int64_t)1 << 38;  // (a tensor map's strides: below 2^40 bytes)
  return *hs >= width && *ts >= width && *hs % 8 == 0 && *ts % 8 == 0 && *hs < most && *ts < most;
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_prompt_create(mla_prompt_t* out, int heads) {
  if (out == nullptr) return MLA_EINVAL;
  *out = nullptr;
  if (heads < 1 || heads > MLA_MAX_ROW_HEADS) return MLA_EINVAL;
  mla_prompt* h = static_cast<mla_prompt*>(calloc(1, sizeof(mla_prompt)));
  if (h == nullptr) return MLA_ENOMEM;
  h->heads = heads;
  int rc = MLA_ECUDA;
  size_t rows = 0;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
    goto fail;
  if (mla::prepare_prompt() != cudaSuccess || mla::tensor_map_encoder() == nullptr) goto fail;
  rows = (size_t)mla::part_rows(h->num_sms);
  rc = MLA_ENOMEM;
  if (cudaMalloc(&h->err, 256) != cudaSuccess ||
      cudaMalloc(&h->part_o, rows * mla::kNope * sizeof(float)) != cudaSuccess ||
      cudaMalloc(&h->part_ml, rows * sizeof(float2)) != cudaSuccess)
    goto fail;
  rc = MLA_ECUDA;
  if (cudaMemset(h->err, 0, 256) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) goto fail;
  *out = h;
  return MLA_OK;
fail:
  mla_prompt_destroy(h);
  cudaGetLastError();
  return rc;
}

int mla_prompt_attn(mla_prompt_t h, int docs, int64_t q_tokens, int64_t k_tokens, const void* q_nope,
                    int64_t qn_token_stride, int64_t qn_head_stride, const void* q_pe, int64_t qp_token_stride,
                    int64_t qp_head_stride, const void* k_nope, int64_t kn_token_stride, int64_t kn_head_stride,
                    const void* k_pe, int64_t kp_token_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, const int32_t* cu_q, const int32_t* cu_k, int causal,
                    const int32_t* prefix, float softmax_scale, float softcap, const float* slopes, void* out,
                    int64_t out_token_stride, int64_t out_head_stride, float* lse, void* stream) {
  if (h == nullptr || docs < 1 || docs > MLA_MAX_TABLE_ROWS || q_tokens < 0 || k_tokens < 0) return MLA_EINVAL;
  // (a tile's rows are counted in 32 bits, and so are the tiles)
  if (q_tokens > MLA_MAX_PROMPT_TOKENS || k_tokens > MLA_MAX_PROMPT_TOKENS) return MLA_EINVAL;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return mla::launched(cudaErrorInvalidDevice);
  if (dev != h->device) return MLA_EINVAL;  // its workspace lies elsewhere
  if (!(softmax_scale >= 0.0f) || softmax_scale > 3.0e38f || !(softcap >= 0.0f) || softcap > MLA_MAX_SOFTCAP)
    return MLA_EINVAL;
  if (q_tokens == 0) return MLA_OK;
  if (q_nope == nullptr || q_pe == nullptr || cu_q == nullptr || cu_k == nullptr || out == nullptr) return MLA_EINVAL;
  if (k_tokens > 0 && (k_nope == nullptr || k_pe == nullptr || v == nullptr)) return MLA_EINVAL;
  if (kp_token_stride == 0) kp_token_stride = mla::kRope;
  int64_t kp_heads = mla::kRope;
  if (!mla::prompt_strides(h->heads, mla::kNope, &qn_token_stride, &qn_head_stride) ||
      !mla::prompt_strides(h->heads, mla::kRope, &qp_token_stride, &qp_head_stride) ||
      !mla::prompt_strides(h->heads, mla::kNope, &kn_token_stride, &kn_head_stride) ||
      !mla::prompt_strides(1, mla::kRope, &kp_token_stride, &kp_heads) ||
      !mla::prompt_strides(h->heads, mla::kNope, &v_token_stride, &v_head_stride) ||
      !mla::prompt_strides(h->heads, mla::kNope, &out_token_stride, &out_head_stride))
    return MLA_EINVAL;
  if (!mla::aligned(q_nope, 16) || !mla::aligned(q_pe, 16) || !mla::aligned(k_nope, 16) || !mla::aligned(k_pe, 16) ||
      !mla::aligned(v, 16) || !mla::aligned(out, 16) || !mla::aligned(cu_q, 4) || !mla::aligned(cu_k, 4) ||
      !mla::aligned(prefix, 4) || !mla::aligned(slopes, 4) || !mla::aligned(lse, 4))
    return MLA_EINVAL;
  mla::PromptInputs in{q_nope,          q_pe,           k_nope,          k_pe,           v,
                       qn_token_stride, qn_head_stride, qp_token_stride, qp_head_stride, kn_token_stride,
                       kn_head_stride,  kp_token_stride, v_token_stride, v_head_stride};
  mla::PromptArgs a = {};
  a.k_tokens = (int)k_tokens;
  if (k_tokens == 0) {  // no key is read: the maps need some memory all the same
    in.k_nope = in.v = q_nope;
    in.k_pe = q_pe;
    in.kn_ts = in.v_ts = qn_token_stride;
    in.kn_hs = in.v_hs = qn_head_stride;
    in.kp_ts = qp_token_stride;
  }
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.prefix = prefix;
  a.slopes = slopes;
  a.docs = docs;
  a.heads = h->heads;
  a.q_tokens = (int)q_tokens;
  a.causal = causal != 0;
  // (a masked score is -infinity before it is scaled: not by zero)
  a.scale = softmax_scale < 1e-30f ? 1e-30f : softmax_scale;
  a.cap = softcap;
  a.out = static_cast<uint16_t*>(out);
  a.o_ts = out_token_stride;
  a.o_hs = out_head_stride;
  a.lse = lse;
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.err = h->err;
  const int64_t tiles = (q_tokens + (int64_t)(2 * mla::kPrTile - 1) * docs) / (2 * mla::kPrTile);
  a.splits = mla::prompt_splits(tiles * h->heads, q_tokens * h->heads,
                                (k_tokens / docs + mla::kPrTile - 1) / mla::kPrTile, h->num_sms);
  return mla::launched(mla::launch_prompt(a, in, (int)tiles, static_cast<cudaStream_t>(stream)));
}

int mla_prompt_get_error(mla_prompt_t h, unsigned* device_flags, void* stream) {
  if (h == nullptr || device_flags == nullptr) return MLA_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, h->err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess || cudaMemsetAsync(h->err, 0, sizeof(uint32_t), s) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ECUDA;
  }
  *device_flags = v;
  return MLA_OK;
}

void mla_prompt_destroy(mla_prompt_t h) {
  if (h == nullptr) return;
  if (h->err) cudaFree(h->err);
  if (h->part_o) cudaFree(h->part_o);
  if (h->part_ml) cudaFree(h->part_ml);
  free(h);
}

}  // extern "C"
