// mla_prompt_attn.cu - attention of a prompt on the 5th-generation tensor cores:
// packed documents, keys of 128 + 64 columns a head (the 64 shared by all
// heads), values of 128.
//
//   x_ij = cap(scale q_i . k_j) - slope |place_i - j|,  cap(x) = c tanh(x / c)
//   out_i = sum_j p_ij v_j,  p_i = softmax over the keys that row i sees
//
// A CTA takes an item of work after another: 256 query rows of a head and document,
// as two tiles of 128, through the keys in tiles of 128 that both share.  S = Q K^T
// (M = 128 rows, N = 128 keys, K = 192) and O += P V (K = 128 keys, N = 128 columns)
// are tcgen05 products with FP32 accumulators in TMEM; P goes back to TMEM as BF16
// in the place of its S, and is read from there.  While the softmax of one tile
// runs, the tensor core works for the other: O0 += P0 V, S0 of the next keys,
// O1 += P1 V, S1.  A warp for each tile issues its products.  (One for both spent
// 500 cycles a job on what comes next, against 1,280 of the tensor core, and far
// more where items are short: 24 documents of 100 to 1,000 rows took 325 us, then
// 304.)  The next item's queries and keys are loaded, and its first
// scores formed, while the last item's sums are written.
//
//  * A softmax thread owns one query row: its maximum, its sum and its mask need
//    no other lane.  The row's reference (what exponents are taken relative to)
//    is its first tile's maximum, and moves only when a score passes it by more
//    than 16 in base 2; only then is O rescaled.  All exponents are taken lower by as
//    much (`above`) as keeps the weights of all keys together below 1, so that no sum of
//    finite values leaves FP32's range; weights below 2^-80 of the largest are lost.
//    (Weights of up to 2^20 overflowed with values of 2^108.  Exponents stay within 32,
//    whose last bit is 2^-19, for 32,768 keys.  With a lower reference instead, by each
//    document's own keys, 24 documents of 100 to 1,000 rows took 292 us, so 287.)
//  * What a row sees are the first `bound` keys of its document: its own place
//    and all before it, or its document's two-way prefix, or all.  Tiles that no
//    row of theirs needs are not touched, and only those on an edge are masked.
//  * An item of 128 rows or fewer has one query tile: its key tiles go to the two
//    softmax warpgroups in turn, each with its own sums, which are added at the end.
//  * Keys and values come by TMA in units of 16 KiB through a ring of eight: 64
//    columns of 128 keys, or 64 keys of 128 values.
//  * A value that a row does not see may be an infinity or a NaN, and zero times
//    it is not zero.  So on the tiles with an edge the warp that hands out items looks
//    the values over first: rows behind the document are zeroed; an infinity or a NaN
//    inside it is replaced by zero and put at the end into the rows that see it.  So are
//    those of the other tiles, wherever the sums come out infinite or NaN.
//  * Items are handed out on the GPU as CTAs become free, of each group of heads the last
//    document's last query tile first and the first document's first one last (in a
//    causal document the longer tiles before the shorter): lengths are known there alone,
//    and documents are not ordered by theirs.
//  * Few query rows: the keys are split over several CTAs, whose sums a second
//    kernel joins.
//
// Long documents are bound by the tensor pipe: 8,192 causal rows of 16 heads take 218
// us back to back in a graph (1,576 TFLOP/s) and 232 called one by one; 4,096 rows of 64
// heads that see all 375 (1,833; up to 5 % more on a GPU that draws its power sooner).
// One row on 65,536 keys is bound by memory: 88 us, 6.2 TB/s.  Short documents are bound
// by the chain of scores, softmax and sums, of which TMEM holds two: 24 of 100 to 1,000
// rows, 64 heads, take 285 us, where their bytes take 144.
#include <math.h>
#include <stdlib.h>

#include "mla_attn_tc.cuh"
#include "mla_prompt.h"

struct mla_prompt {
  int device;
  int num_sms;
  int heads;
  uint32_t* err;    // flags, then (at 2 and 3) items handed out and CTAs done with them
  float* part_o;    // outputs of split rows' parts
  float2* part_ml;  // their references and denominators
};

namespace mla {
namespace {

constexpr int kPrTile = 128;     // query rows and keys of a tile
constexpr int kPrUnit = 16384;   // bytes of a ring slot
constexpr int kPrRing = 8;
constexpr int kPrThreads = 384;  // two softmax warpgroups; warps that load, multiply (two) and hand out work
constexpr int kPrQ = 3 * kPrUnit;  // a query tile: planes of 64 columns
constexpr int kPrRoom = 16;  // base 2
constexpr int kPrChunks = 96;    // sums of the documents' tiles
constexpr int kPrItems = 4;      // items of work in flight
constexpr int kPrReaders = 11;   // warps that read them

// One item of work: up to 256 query rows of a head and document, and the tiles
// of its keys that this CTA goes through.
struct PrItem {
  int valid;         // 0: there is no more
  int head, split;
  int q0, nq;        // the document's query rows
  int k0, nk;        // and keys
  int prefix;
  int r0;            // first row, in the document
  int j0, n[2];      // query tile q: key tiles j0 .. n[q] - 1
  int safe[2];       // tiles below are seen whole by every row of query tile q
  int solo;          // one query tile only: its keys are shared out, 1 + who begins
  uint32_t odd;      // values that are not finite were met
};

struct PrSmem {
  static constexpr int oQ = 0;
  static constexpr int oRing = 2 * kPrQ;
  static constexpr int oBar = oRing + kPrRing * kPrUnit;
  // k_full[2] v_full[2] k_free[2] v_free[2] q_full[2] q_free[2] s_full[2] p_full[4] o_full[2] o_free[2] ml_full[2]
  // item_full[4] item_free[4] drain[2] v_seen[2] turn[2]
  static constexpr int kBars = 38;
  static constexpr int oItem = oBar + kBars * 8;
  static constexpr int oMl = oItem + kPrItems * (int)sizeof(PrItem);  // [2][128] reference and sum of a shared row
  static constexpr int oScan = oMl + 2 * 128 * 8;                     // [96]
  static constexpr int oTmem = oScan + kPrChunks * 4;
  static constexpr int oLoads = oTmem + 4;  // key tiles whose loads have begun
  static constexpr int kBytes = oLoads + 4;
  static_assert(kBytes <= 232448 && oBar % 8 == 0 && oItem % 8 == 0 && oMl % 8 == 0, "shared memory budget");
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

// The same value, which the compiler does not know: a loop with a branch on it is
// not made into two loops.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// A bounded wait that gives up for good.
__device__ __forceinline__ bool pr_wait_long(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, kTcWait); }
__device__ __forceinline__ void pr_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (!dead && !pr_wait_long(bar, parity)) dead = true;
}
__device__ __forceinline__ void pr_wait_warp(uint64_t* bar, uint32_t parity, bool& dead) {
  pr_wait(bar, parity, dead);
  dead = __any_sync(0xFFFFFFFFu, dead);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The smaller, or NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Keys that query row i of a document sees: the first so many.
__device__ __forceinline__ int pr_bound(int i, int nq, int nk, int prefix, bool causal) {
  if (!causal) return nk;
  return max(min(prefix, nk), max(0, min(i + (nk - nq) + 1, nk)));
}
__device__ __forceinline__ bool pr_edge(const PrItem& k, int j) {
  return (j < k.n[0] && j >= k.safe[0]) || (j < k.n[1] && j >= k.safe[1]);
}

// A document's rows, cut to the tensor.
__device__ __forceinline__ int pr_place(const int32_t* cu, int d, int most, int* n, bool* cut) {
  const int lo = cu[d], hi = cu[d + 1];
  const int c0 = max(0, min(lo, most)), c1 = max(c0, min(hi, most));
  *n = c1 - c0;
  *cut = c0 != lo || c1 != hi;
  return c0;
}
__device__ __forceinline__ int pr_tiles(const PromptArgs& a, int d) {
  int n;
  bool cut;
  pr_place(a.cu_q, d, a.q_tokens, &n, &cut);
  return (n + 2 * kPrTile - 1) / (2 * kPrTile);
}

// A key's row of values in a ring unit (two halves of 128 bytes): zeros where the
// key lies behind its document; else what is not finite becomes zero.  Whether
// there was any.
__device__ __forceinline__ bool pr_look_over(uint8_t* base, int lane, bool behind) {
  auto piece = [&](int c) {
    return reinterpret_cast<uint4*>(base + (c >> 3) * (kPrUnit / 2) + (((c + lane) & 7) << 4));
  };
  uint32_t odd[2] = {0u, 0u};  // sums of zero times each value: NaN from what is not finite
  auto times_zero = [](uint32_t w, uint32_t& sum) { asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w), "r"(0u)); };
#pragma unroll
  for (int c0 = 0; c0 < 16; c0 += 8) {
    uint4 w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = *piece(c0 + c);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      times_zero(w[c].x, odd[0]);
      times_zero(w[c].y, odd[1]);
      times_zero(w[c].z, odd[0]);
      times_zero(w[c].w, odd[1]);
    }
  }
  if (behind) {
#pragma unroll 1
    for (int c = 0; c < 16; ++c) *piece(c) = make_uint4(0, 0, 0, 0);
    return false;
  }
  if (((odd[0] | odd[1]) & 0x7FFF7FFFu) == 0) return false;
#pragma unroll 1
  for (int c = 0; c < 128; ++c) {
    uint16_t* e = reinterpret_cast<uint16_t*>(base + (c >> 6) * (kPrUnit / 2)) + (c & 63);
    if ((*e & 0x7F80u) == 0x7F80u) *e = 0;
  }
  return true;
}

// Infinities and NaN among the values: a row's column that sees any is their sum, however
// small their weights (which are above zero, though FP32 may hold them as zero, and zero
// times an infinity is NaN; in the tiles that were looked over they count as zero in the
// products).  A warp for its 32 stored rows, `live` where a lane's counts: rows see
// ascending numbers of keys, so the item's keys are gone through once, four columns a
// lane, and each row takes the sums where its keys end.  Slow, and rare.
__device__ __noinline__ void pr_put_odd(const PromptArgs& a, const PrItem& k, int j0, int end, int bound, bool live, float* part,
                                        uint16_t* out) {
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31, last = min(end * kPrTile, k.nk);
  const unsigned rows = __ballot_sync(0xFFFFFFFFu, live);
  const uint16_t* v = a.v + (int64_t)k.k0 * a.v_ts + (int64_t)k.head * a.v_hs + 4 * lane;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int key = j0 * kPrTile;
#pragma unroll 1
  for (int r = 0; r < 32; ++r) {
    const int upto = min(__shfl_sync(0xFFFFFFFFu, bound, r), last);
#pragma unroll 1
    for (; key < upto; key += kAhead) {
      uint2 w[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
        w[n] = key + n < upto ? *reinterpret_cast<const uint2*>(v + (int64_t)(key + n) * a.v_ts) : make_uint2(0, 0);
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const uint32_t x[4] = {w[n].x << 16, w[n].x & 0xFFFF0000u, w[n].y << 16, w[n].y & 0xFFFF0000u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((x[i] & 0x7F800000u) == 0x7F800000u) sum[i] += __uint_as_float(x[i]);
      }
    }
    key = max(j0 * kPrTile, min(key, upto));
    if (!(rows >> r & 1u)) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sum[i] == 0.f) continue;
      if (part != nullptr)
        part[r * 128 + 4 * lane + i] = sum[i];
      else
        out[r * a.o_ts + 4 * lane + i] = f2bf_bits(sum[i]);
    }
  }
}

// CAP: scores are capped; BIAS: they lose by distance; LONG: capped scores in rounds of 64
// columns, not 32.
template <bool CAP, bool BIAS, bool LONG>
__global__ void __launch_bounds__(kPrThreads, 1)
    mla_prompt_attn_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
  using S = PrSmem;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::oBar);  // of a key tile, by its parity
  uint64_t* v_full = k_full + 2;
  uint64_t* k_free = v_full + 2;
  uint64_t* v_free = k_free + 2;
  uint64_t* q_full = v_free + 2;
  uint64_t* q_free = q_full + 2;
  uint64_t* s_full = q_free + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 4;  // (p_full: two halves a buffer)
  uint64_t* o_free = o_full + 2;
  uint64_t* ml_full = o_free + 2;
  uint64_t* item_full = ml_full + 2;
  uint64_t* item_free = item_full + kPrItems;
  uint64_t* drain = item_free + kPrItems;
  uint64_t* v_seen = drain + 2;
  uint64_t* turn = v_seen + 2;
  PrItem* items = reinterpret_cast<PrItem*>(smem + S::oItem);
  volatile float2* ml = reinterpret_cast<float2*>(smem + S::oMl);
  int* scan = reinterpret_cast<int*>(smem + S::oScan);
  volatile uint32_t* begun = reinterpret_cast<uint32_t*>(smem + S::oLoads);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const bool causal = a.causal != 0;
  const int each = (a.docs + kPrChunks - 1) / kPrChunks;  // documents a sum
  if (tid == 0) {
    for (int q = 0; q < 2; ++q) {
      mbar_init(&k_full[q], 1);
      mbar_init(&v_full[q], 1);
      mbar_init(&k_free[q], 2);
      mbar_init(&v_free[q], 2);
      mbar_init(&q_full[q], 1);
      mbar_init(&q_free[q], 2);
      mbar_init(&s_full[q], 1);
      mbar_init(&p_full[2 * q], 4);
      mbar_init(&p_full[2 * q + 1], 4);
      mbar_init(&o_full[q], 1);
      mbar_init(&o_free[q], 4);
      mbar_init(&ml_full[q], 4);
    }
    for (int i = 0; i < kPrItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_free[i], kPrReaders);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(&v_seen[0], 1);
    mbar_init(&v_seen[1], 1);
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);
    mbar_fence_init();
    *begun = 0;
    if (smem_u32(smem) & 1023u) atomicOr(a.err, MLA_DEVERR_CHECK);
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 8) {
    prefetch_tensormap(&maps.k_nope);
    prefetch_tensormap(&maps.k_pe);
    prefetch_tensormap(&maps.q_nope);
    prefetch_tensormap(&maps.q_pe);
    prefetch_tensormap(&maps.v);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (tid < kPrChunks) {
    int sum = 0;
#pragma unroll 1
    for (int d = tid * each, e = min(a.docs, d + each); d < e; ++d) sum += pr_tiles(a, d);
    scan[tid] = min(sum, a.tiles);  // (more only where the array descends)
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = uniform(*tslot);  // S at columns 0 and 128, O at 256 and 384
  bool dead = false;

  // What each reader of the items does: the next one, and that it is done with one.
  auto item_wait = [&](uint32_t i) -> const PrItem& {
    pr_wait_warp(&item_full[i % kPrItems], (i / kPrItems) & 1u, dead);
    return items[i % kPrItems];
  };
  auto item_done = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[i % kPrItems]);
  };

  // Registers: 168 a thread at the launch; the softmax takes 208, the others keep 88.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 10) {
    // ================= work: the items in order, each CTA the next one that is free; and the
    // values of every key tile as they come, looked over before they are used
    constexpr int kOwn = kPrChunks / 32;  // sums a lane
    int mine = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) mine += scan[lane * kOwn + e];
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += v;
    }
    const int tiles = min(__shfl_sync(0xFFFFFFFFu, before, 31), a.tiles);
    before -= mine;
    const uint32_t total = (uint32_t)tiles * (uint32_t)a.heads * (uint32_t)a.splits;
    int at = -1, doc = 0, tile = 0, last_q = 1;
    uint32_t u = blockIdx.x, ahead = 0;  // this item's number; the next one's (lane 0), asked for ahead
    uint32_t handed = 0, seen = 0;       // items handed out, gone through
    uint32_t t = 0;                      // key tiles gone through
    int j = 0, end = 0;                  // of item `seen`
    bool more = true, within = false;
    // The next item, or that there is none.
    auto hand_out = [&] {
      PrItem& k = items[handed % kPrItems];
      if (u >= total) {
        more = false;
        if (lane == 0) {
          k.valid = 0;
          mbar_arrive(&item_full[handed % kPrItems]);
        }
        return;
      }
      if (lane == 0) ahead = atomicAdd(a.next, 1u) + gridDim.x;
      // groups of heads; of a group the last tiles first (of a document the longest where
      // rows see what lies before them), head after head
      const uint32_t per_group = (uint32_t)a.group * (uint32_t)tiles * (uint32_t)a.splits;
      const uint32_t g = u / per_group, r = u - g * per_group;
      const int heads = min(a.group, a.heads - (int)g * a.group);
      const uint32_t row = (uint32_t)(heads * a.splits);
      const uint32_t nth = r / row;
      const int x = tiles - 1 - (int)nth, in = (int)(r - nth * row);
      if (x != at) {
        at = x;
        // the lane whose sums hold x, its sum, then the document
        const unsigned who = __ballot_sync(0xFFFFFFFFu, x >= before && x < before + mine);
        const int src = __ffs(who) - 1;
        int b = before, c = lane * kOwn;
#pragma unroll 1
        while (lane == src && x >= b + scan[c]) b += scan[c++];
        b = __shfl_sync(0xFFFFFFFFu, b, src);
        c = __shfl_sync(0xFFFFFFFFu, c, src);
#pragma unroll 1
        for (int d0 = c * each;; d0 += 32) {
          const int d = d0 + lane;
          int n = d < min(a.docs, (c + 1) * each) ? pr_tiles(a, d) : 0;
          const int own = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if (lane >= o) n += v;
          }
          const unsigned hit = __ballot_sync(0xFFFFFFFFu, x >= b + n - own && x < b + n);
          if (hit != 0) {
            const int w = __ffs(hit) - 1;
            doc = d0 + w;
            tile = x - (b + __shfl_sync(0xFFFFFFFFu, n - own, w));
            break;
          }
          b += __shfl_sync(0xFFFFFFFFu, n, 31);
          if (d0 >= a.docs) break;  // (documents that another program moves meanwhile)
        }
      }
      if (lane == 0) {
        bool cut_q, cut_k;
        k.q0 = pr_place(a.cu_q, doc, a.q_tokens, &k.nq, &cut_q);
        k.k0 = pr_place(a.cu_k, doc, a.k_tokens, &k.nk, &cut_k);
        k.prefix = a.prefix != nullptr ? a.prefix[doc] : 0;
        k.head = (int)(g * (uint32_t)a.group + (uint32_t)in / (uint32_t)a.splits);
        k.split = in - (k.head - (int)g * a.group) * a.splits;
        k.r0 = tile * 2 * kPrTile;
        int n[2], safe[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int lo = k.r0 + q * kPrTile, hi = min(lo + kPrTile, k.nq);
          n[q] = hi > lo ? (pr_bound(hi - 1, k.nq, k.nk, k.prefix, causal) + kPrTile - 1) / kPrTile : 0;
          safe[q] = hi > lo ? pr_bound(lo, k.nq, k.nk, k.prefix, causal) / kPrTile : 0;
        }
        // this item's share of the key tiles
        const int all = max(n[0], n[1]);
        const int j0 = (int)((uint32_t)(all * k.split) / (uint32_t)a.splits);  // (below 2^21 tiles, 64 parts)
        const int j1 = (int)((uint32_t)(all * (k.split + 1)) / (uint32_t)a.splits);
        k.j0 = j0;
        k.n[0] = min(n[0], j1);
        k.n[1] = min(n[1], j1);
        k.safe[0] = safe[0];
        k.safe[1] = safe[1];
        const int jobs = max(0, k.n[0] - j0);
        k.solo = 0;
        if (k.r0 + kPrTile >= k.nq) {
          k.solo = 2 - last_q;  // whoever did not end the item before begins
          if (jobs > 0) last_q = (k.solo - 1) ^ ((jobs - 1) & 1);
        } else if (k.n[1] > j0) {
          last_q = 1;
        }
        k.odd = 0;
        k.valid = 1;
        mbar_arrive(&item_full[handed % kPrItems]);
      }
      __syncwarp();
      ++handed;
    };
    long long since = clock64();
#pragma unroll 1
    while (!dead && (more || seen < handed)) {
      if (!within && seen < handed) {
        const PrItem& k = items[seen % kPrItems];
        j = k.j0;
        end = max(k.n[0], k.n[1]);
        within = j < end;
        if (!within) ++seen;
        continue;
      }
      if (within && __any_sync(0xFFFFFFFFu, tc_ready(&v_full[t & 1u], t >> 1 & 1u))) {
        // the values of key tile t, looked over where they have an edge
        PrItem& k = items[seen % kPrItems];
        pr_wait_warp(&v_full[t & 1u], t >> 1 & 1u, dead);
        if (pr_edge(k, j)) {
          bool odd = false;
#pragma unroll 1
          for (int r = lane; r < kPrTile; r += 32)
            odd = pr_look_over(smem + S::oRing + ((5 * t + 3 + (r >> 6)) % kPrRing) * kPrUnit + (r & 63) * 128, lane,
                               j * kPrTile + r >= k.nk) || odd;
          if (odd) *reinterpret_cast<volatile uint32_t*>(&k.odd) = 1u;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_seen[t & 1u]);
        ++t;
        within = ++j < end;
        if (!within) ++seen;
        since = clock64();
        continue;
      }
      if (more && (handed < kPrItems || (handed - seen < kPrItems &&
                                         __all_sync(0xFFFFFFFFu, tc_ready(&item_free[handed % kPrItems],
                                                                          (handed / kPrItems - 1) & 1u))))) {
        u = handed > 0 ? __shfl_sync(0xFFFFFFFFu, ahead, 0) : u;
        hand_out();
        since = clock64();
        continue;
      }
      dead = __any_sync(0xFFFFFFFFu, clock64() - since > kTcWait);
    }
    if (dead && more && lane == 0) {
      items[handed % kPrItems].valid = 0;
      mbar_arrive(&item_full[handed % kPrItems]);
    }
    // the last CTA to come here leaves the count of items as it was
    if (lane == 0) {
      __threadfence();
      if (atomicAdd(a.next + 1, 1u) == gridDim.x - 1) a.next[0] = a.next[1] = 0;
    }
    if (blockIdx.x == 0) {
      bool bad = false;
#pragma unroll 1
      for (int d = lane; d < a.docs; d += 32) {
        int n;
        bool cut_q, cut_k;
        pr_place(a.cu_q, d, a.q_tokens, &n, &cut_q);
        pr_place(a.cu_k, d, a.k_tokens, &n, &cut_k);
        bad = bad || cut_q || cut_k;
      }
      if (bad) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    }
  } else if (warp == 8) {
    // ================= TMA: K, V of key tile after key tile, the queries behind the first K
    //
    // Tile t of all that this CTA goes through has units 5 t .. of the ring: three of K,
    // two of V.  Its K comes in the place of K's last unit and V of tile t - 2, its V in
    // that of K's first two of tile t - 1.
    uint32_t tile = 0;               // key tiles so far
    uint32_t loads = 0, q_uses = 0;  // query buffers: used, parity of q_free; a bit a buffer
    for (uint32_t i = 0; !dead; ++i) {
      const PrItem& k = item_wait(i);
      if (dead || !k.valid) break;
      const int end = max(k.n[0], k.n[1]);
      if (lane == 0) {
        for (int j = k.j0; j < end && !dead; ++j, ++tile) {
          const int row = k.k0 + j * kPrTile;
          const uint32_t b = tile & 1u, ring = smem_u32(smem + S::oRing);
          auto unit = [&](uint32_t u) { return ring + ((5 * tile + u) % kPrRing) * kPrUnit; };
          mbar_arrive_expect_tx(&k_full[b], 3 * kPrUnit);
          __threadfence_block();
          *begun = tile + 1;
          tma_g2s_3d(unit(0), &maps.k_nope, 0, k.head, row, &k_full[b]);  // (K of tile t - 2 has been waited for)
          if (tile >= 2) pr_wait(&v_free[b], ((tile >> 1) - 1) & 1u, dead);
          if (dead) break;
          tma_g2s_3d(unit(1), &maps.k_nope, 64, k.head, row, &k_full[b]);
          tma_g2s_3d(unit(2), &maps.k_pe, 0, 0, row, &k_full[b]);
          if (j == k.j0) {
            // the queries (their buffers come free later than the ring's slots): tile
            // q into buffer `place`
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              if (k.n[q] <= j) continue;
              const int place = k.solo ? k.solo - 1 : q;
              if (loads >> place & 1u) {
                pr_wait(&q_free[place], q_uses >> place & 1u, dead);
                q_uses ^= 1u << place;
              }
              if (dead) break;
              loads |= 1u << place;
              mbar_arrive_expect_tx(&q_full[place], kPrQ);
              const uint32_t dst = smem_u32(smem + S::oQ) + place * kPrQ;
              const int at = k.q0 + k.r0 + q * kPrTile;
              tma_g2s_3d(dst, &maps.q_nope, 0, k.head, at, &q_full[place]);
              tma_g2s_3d(dst + kPrUnit, &maps.q_nope, 64, k.head, at, &q_full[place]);
              tma_g2s_3d(dst + 2 * kPrUnit, &maps.q_pe, 0, k.head, at, &q_full[place]);
            }
          }
          if (tile >= 1 && !dead) pr_wait(&k_free[b ^ 1u], ((tile - 1) >> 1) & 1u, dead);
          if (dead) break;
          mbar_arrive_expect_tx(&v_full[b], 2 * kPrUnit);
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // 64 keys, both halves of their columns
            tma_g2s_3d(unit(3 + u), &maps.v, 0, k.head, row + 64 * u, &v_full[b]);
            tma_g2s_3d(unit(3 + u) + kPrUnit / 2, &maps.v, 64, k.head, row + 64 * u, &v_full[b]);
          }
        }
      }
      dead = __any_sync(0xFFFFFFFFu, dead);
      item_done(i);
    }
    if (dead && lane == 0) {  // the copies under way land before the CTA leaves
      for (int q = 0; q < 2; ++q)  // (as often waited for as loaded, but for the last time)
        if (loads >> q & 1u) (void)pr_wait_long(&q_full[q], q_uses >> q & 1u);
      for (uint32_t t = tile > 1 ? tile - 1 : 0; t <= tile; ++t) {  // (a tile that was cut short runs the wait out)
        (void)pr_wait_long(&k_full[t & 1u], (t >> 1) & 1u);
        (void)pr_wait_long(&v_full[t & 1u], (t >> 1) & 1u);
      }
    }
  } else {
    // ================= products: warp 9 those of buffer 0, warp 11 of buffer 1 (a warp
    // together, one elected lane issues)
    //
    // A job is a key tile for a softmax warpgroup: key tile after key tile for both query
    // tiles, or shared out in turn.  S of a job follows O += P V of the job before in the
    // same buffer, whose P lies in its place: a buffer's jobs are a chain, and the two
    // chains need nothing of one another but that both give a slot back (what one of
    // them does not read, the other gives back twice).
    constexpr uint32_t kBf16 = 1u << 7;
    constexpr uint32_t id_s = tc_idesc(128, 128, 1, false, false) | kBf16;
    constexpr uint32_t id_o = tc_idesc(128, 128, 1, false, true) | kBf16;
    const uint32_t q = uniform(warp == 11 ? 1u : 0u);
    const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
    const uint64_t dk = tc_desc(smem_u32(smem + S::oRing), 1024, 2);
    const uint64_t dv = tc_desc_wide(smem_u32(smem + S::oRing), 1024, kPrUnit / 2);
    uint32_t tile = 0;                   // key tiles of the items before
    uint32_t q_uses = 0;                 // parities of q_full, a bit a buffer
    uint32_t p_uses = 0, o_uses = 0;     // jobs of this buffer, items
    uint32_t even = ~0u, odd = ~0u;      // the last such tiles whose keys were waited for
    auto give = [&](uint64_t* bar, bool alone) {
      tc_commit(bar);
      if (alone) tc_commit(bar);
    };
    // Where both chains read a key tile, they issue in turns, a job after the other's.
    // (Where their products mixed, their scores came at the same time, and the tensor core
    // idled while both took their softmax: 4,096 rows of 64 heads that see all took 520
    // us, in turns 379; 24 documents of 100 to 1,000 rows 298 and 304.)
    uint32_t turns = 0;
    auto turn_begins = [&] {
      if (q || turns > 0) pr_wait(&turn[q], (q ? turns : turns - 1) & 1u, dead);
    };
    auto turn_ends = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&turn[q ^ 1u]);
      ++turns;
    };
    // (A lane's wait that ran out is known to the others at the item's end: until
    // then products go on over whatever the slots hold, and do not count.)
#pragma unroll 1
    for (uint32_t i = 0; !dead; ++i) {
      const PrItem& k = item_wait(i);
      if (dead || !k.valid) break;
      const int j0 = k.j0, n0 = k.n[0], n1 = k.n[1];
      const uint32_t solo = uniform((uint32_t)k.solo);
      item_done(i);
      const int end = max(n0, n1);
      const uint32_t place = solo ? solo - 1 : q;  // of its queries
      const int first = j0 + (solo && place != q ? 1 : 0), step = solo ? 2 : 1;
      const int mine = solo || q == 0 ? n0 : n1;
      const int shared = solo ? 0 : min(n0, n1);  // key tiles below are read by both
      // O from P and the values of key tile j, t of all
      auto values = [&](int j, uint32_t t) {
        pr_wait(&v_seen[t & 1u], t >> 1 & 1u, dead);
        if (j + 1 < shared) turn_begins();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          pr_wait(&p_full[2 * q + u], p_uses & 1u, dead);
          tc_after();
          pr_mma4_pv(tmem + 256 + 128 * q, tmem + 128 * q + 32 * u,
                     dv + (uint64_t)(((5 * t + 3 + u) % kPrRing) * (kPrUnit >> 4)), id_o, u > 0 || j > first);
        }
        give(&v_free[t & 1u], j >= shared);
        ++p_uses;
      };
      auto scores = [&](int j, uint32_t t) {
        // A barrier tells this tile's loads from those two tiles before by a parity: those
        // have been waited for, or these have begun, which is after them.
        if ((t & 1u ? odd : even) != t - 2u) {
          const long long since = clock64();
          while (*begun <= t && !dead) dead = clock64() - since > kTcWait;
          __threadfence_block();
          dead = __any_sync(0xFFFFFFFFu, dead);
        }
        odd = t & 1u ? t : odd;
        even = t & 1u ? even : t;
        pr_wait(&k_full[t & 1u], t >> 1 & 1u, dead);
        if (j == first) pr_wait(&q_full[place], q_uses >> place & 1u, dead);
        tc_after();
#pragma unroll
        for (int u = 0; u < 3; ++u)
          tc_mma4_f16<2, 2>(tmem + 128 * q, dq + (uint64_t)((place * kPrQ + u * kPrUnit) >> 4),
                            dk + (uint64_t)(((5 * t + u) % kPrRing) * (kPrUnit >> 4)), id_s, u > 0);
        tc_commit(&s_full[q]);
        if (j < shared) turn_ends();
        give(&k_free[t & 1u], j >= shared);
      };
      if (first < mine) {
        uint32_t t = uniform(tile + (uint32_t)(first - j0));
        if (first < shared) turn_begins();
        scores(first, t);
        if (o_uses > 0) pr_wait(&o_free[q], o_uses - 1 & 1u, dead);  // (O of the item before has been read)
        ++o_uses;
#pragma unroll 1
        for (int j = first; j + step < mine; j += step) {
          values(j, t);
          t += step;
          scores(j + step, t);
        }
        give(&q_free[place], !solo || n0 - j0 < 2);
        values(mine - 1 - (solo ? (mine - 1 - first) & 1 : 0), t);
        tc_commit(&o_full[q]);
      }
      if (n0 > j0) q_uses ^= solo == 2 ? 2u : 1u;
      if (n1 > j0) q_uses ^= 2u;
      if (end > j0) tile += (uint32_t)(end - j0);
      dead = __any_sync(0xFFFFFFFFu, dead);
    }
    if (dead) {
      tc_commit(&drain[q]);
      (void)pr_wait_long(&drain[q], 0u);
    }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ================= softmax (warps 0-3: S and O of buffer 0, 4-7: of buffer 1)
    const int q = warp >> 2, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t st = tmem + lanes + 128 * q;
    const float scale2 = fminf(a.scale * 1.4426950408889634f, 3.4028234e38f);  // (finite: a score of zero stays zero)
    // capped: x = C - 2 C / (1 + 2^(s e)), e = 2 scale log2(e) / cap, in base 2
    const float capC = CAP ? a.cap * 1.4426950408889634f : 0.f, capE = CAP ? fminf(2.0f * scale2 / a.cap, 1e30f) : 0.f;
    const float unit2 = CAP || BIAS ? 1.0f : scale2;
    uint32_t uses = 0;     // jobs of this buffer so far
    uint32_t o_reads = 0;  // parities of o_full, a bit a buffer
    uint32_t shares = 0;   // items whose keys were shared out
    for (uint32_t it = 0; !dead; ++it) {
      const PrItem& k = item_wait(it);
      if (dead || !k.valid) break;
      const int solo = k.solo, qt = solo ? 0 : q;  // its query tile
      const int j0 = k.j0, nt = k.n[qt], step = solo ? 2 : 1, safe = k.safe[qt];
      const int jfirst = j0 + (solo && q != solo - 1 ? 1 : 0);
      const int base_row = k.r0 + qt * kPrTile + 32 * quad;
      const int i = base_row + lane;  // this thread's row of the document
      const int bound = pr_bound(min(i, k.nq - 1), k.nq, k.nk, k.prefix, causal);
      float slope = BIAS ? -a.slopes[k.head] * 1.4426950408889634f : 0.f;
      if (BIAS && fabsf(slope) == INFINITY) slope = copysignf(3.4028234e38f, slope);  // (none at no distance)
      float ref = -INFINITY, l = 0.f;
      for (int j = jfirst; j < nt; j += step) {
        pr_wait(&s_full[q], uses & 1u, dead);
        ++uses;
        tc_after();
        const uint32_t at_edge = j >= safe;
        const int left = bound - j * kPrTile;  // keys of this tile that count
        // What is done to the scores before their maximum where it takes many
        // instructions (caps, and keys on both sides of a biased row): some columns at a
        // time and back to TMEM, in a loop.  (Its code for all 128 at once drove the rest
        // out of the instruction cache: 24 documents of 100 to 1,000 rows took 579 us
        // capped, when 32 columns took 398.)
        const int near = base_row + (k.nk - k.nq) - j * kPrTile;  // the warp's first row among the tile's keys
        const bool apart = CAP || (BIAS && (at_edge || !(near >= kPrTile || near + 31 <= 0)));
        if (apart) {
          constexpr int kPre = LONG ? 64 : 32;
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += kPre) {
            const int count = left - c0;
            float s[kPre];
#pragma unroll
            for (int c = 0; c < kPre; c += 32) tc_ld(st + c0 + c, *reinterpret_cast<float(*)[32]>(s + c));
            tc_wait_ld();
            tc_landed(s);
            if constexpr (CAP) {
              if (opaque(at_edge)) {  // (neighbours share a reciprocal below)
#pragma unroll
                for (int c = 0; c < kPre; ++c) s[c] = c < count ? s[c] : 0.f;
              }
              // 1 / (1 + 2^y) for four at a time from one reciprocal of their product:
              // 2^30 as the largest power keeps that in range (and is 1 - 2^-29 as a tangent)
#pragma unroll
              for (int c = 0; c < kPre; c += 4) {
                const float2 e2 = make_float2(capE, capE), one = make_float2(1.0f, 1.0f);
                float2 x = fmul2_rn(make_float2(s[c], s[c + 1]), e2), y = fmul2_rn(make_float2(s[c + 2], s[c + 3]), e2);
                x = add2(make_float2(ex2(min_nan(x.x, 30.0f)), ex2(min_nan(x.y, 30.0f))), one);
                y = add2(make_float2(ex2(min_nan(y.x, 30.0f)), ex2(min_nan(y.y, 30.0f))), one);
                const float2 m = fmul2_rn(x, y);  // (x0 y0, x1 y1)
                const float r = rcp_approx(m.x * m.y);
                const float2 w = fmul2_rn(make_float2(m.y, m.x), make_float2(r, r));  // 1 / (x0 y0), 1 / (x1 y1)
                const float2 c2 = make_float2(capC, capC), d2 = make_float2(-2.0f * capC, -2.0f * capC);
                const float2 t0 = fma2(fmul2_rn(w, y), d2, c2), t1 = fma2(fmul2_rn(w, x), d2, c2);
                s[c] = t0.x;
                s[c + 1] = t0.y;
                s[c + 2] = t1.x;
                s[c + 3] = t1.y;
              }
            }
            if constexpr (BIAS) {  // by distance from this row's place
              const float own = (float)(near - c0 + lane);
#pragma unroll
              for (int c = 0; c < kPre; ++c) s[c] = fmaf(slope, fabsf(own - (float)c), CAP ? s[c] : s[c] * scale2);
            }
            if (opaque(at_edge)) {
#pragma unroll
              for (int c = 0; c < kPre; ++c) s[c] = c < count ? s[c] : -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < kPre; c += 32) tc_st32(st + c0 + c, *reinterpret_cast<float(*)[32]>(s + c));
          }
          tc_wait_st();
        }
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld(st + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
        tc_wait_ld();
        tc_landed(s);
        if constexpr (!CAP && !BIAS) {
          if (at_edge) {
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = c < left ? s[c] : -INFINITY;
          }
        }
        // What the scores below lack: the rounding of slope times place, the same for a
        // row's keys (2^-24 of it, which for a steep slope is more than a near key's own).
        // From 2^24 on that is more than an exponent has room for (slopes of 1e31 gave
        // infinite weights), and no two key tiles' keys that are so far weigh alike.
        float low = 0.f;
        if constexpr (BIAS && !CAP) {
          if (!apart) {  // keys on one side of the warp's rows: the distance is linear
            const float sg = near > 0 ? slope : -slope, own = (float)(near + lane);
            const float2 k0 = make_float2(sg * own, sg * own), k1 = make_float2(-sg, -sg), u2 = make_float2(scale2, scale2);
            low = fabsf(k0.x) < 0x1p24f ? fmaf(sg, own, -k0.x) : 0.f;
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              const float2 x = fma2(make_float2(s[c], s[c + 1]), u2, fma2(k1, make_float2((float)c, (float)(c + 1)), k0));
              s[c] = x.x;
              s[c + 1] = x.y;
            }
          }
        }
        float m4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(s[e], s[e + 4]);
#pragma unroll
        for (int c = 8; c < 128; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], s[c + e], s[c + e + 4]);
        const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * unit2 + low;
        // The reference: the first maximum; later only where it is passed by far.
        const bool grow = mx > ref + (float)kPrRoom || (ref == -INFINITY && mx > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          float f = 1.0f;
          if (grow) {
            f = ex2(ref - mx);  // 0 from -infinity
            ref = mx;
            l *= f;
          }
          if (j > jfirst) {
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
        const float minus = ref == -INFINITY ? 0.f : low - ref - a.above;
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
          tc_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * q + half]);
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
      }
      // ---- the sums: of a query tile whose keys were shared out, whoever began
      // takes both buffers
      const int end = max(k.n[0], k.n[1]), jobs = max(0, nt - j0);
      const int lead = solo - 1;  // (of a shared one)
      const bool shared = solo && jobs > 1;
      const bool mine = solo ? q == lead : true;
      const int other = q ^ 1;
      float f0 = 1.0f, f1 = 0.f;  // what this buffer's and the other's sums are taken times
      if (shared) {
        volatile float2* at = ml + 128 * (shares & 1u) + 32 * quad + lane;
        if (!mine) {
          at->x = ref;
          at->y = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ml_full[shares & 1u]);
        } else {
          pr_wait(&ml_full[shares & 1u], (shares >> 1) & 1u, dead);
          const float ref1 = at->x, l1 = at->y;
          const float m = fmaxf(ref, ref1);
          if (m > -INFINITY) {
            f0 = ex2(ref - m);
            f1 = ex2(ref1 - m);
            l = l * f0 + l1 * f1;
            ref = m;
          }
        }
        ++shares;
      }
      const bool used = solo ? jobs > (mine ? 0 : 1) : nt > j0;  // this buffer
      const bool used1 = solo ? jobs > (mine ? 1 : 0) : k.n[other] > j0;
      if (mine) {
        const bool have = i < k.nq, part = a.splits > 1;
        const uint32_t used_ = used, shared_ = shared, part_ = part;
        const int64_t row = k.q0 + i;
        const float inv = l == 0.f ? 0.f : rcp_approx(l);
        f0 *= inv;
        f1 *= inv;
        if (have) {
          const float sum = l * a.times;
          if (part)
            a.part_ml[((int64_t)k.split * a.heads + k.head) * a.q_tokens + row] = make_float2(ref, sum);
          else if (a.lse != nullptr)
            a.lse[row * a.heads + k.head] = l == 0.f ? -INFINITY : (ref + lg2_approx(sum)) * 0.6931471805599453f;
        }
        // Four neighbouring lanes trade 16-byte pieces, so that they store 64 bytes of
        // one row after another: 8 rows an instruction, not 32.
        const int sub = lane & 3;
        const int left = k.nq - (i - sub);  // rows from the first of the four on
        float* po = a.part_o + (((int64_t)k.split * a.heads + k.head) * a.q_tokens + row) * 128;
        uint16_t* o = a.out + (row - sub) * a.o_ts + (int64_t)k.head * a.o_hs + 8 * sub;
        if (used) pr_wait(&o_full[q], o_reads >> q & 1u, dead);
        if (shared) pr_wait(&o_full[other], o_reads >> other & 1u, dead);
        tc_after();
        // Sums of products of the row's values: not finite where one of them is not (or is
        // beyond 2^60: the look at the document's values is then in vain).  Only where a key
        // tile was not looked over.  (A product with zero for each value, in every item: 24
        // documents of 100 to 1,000 rows took 287 us, so 284, without any of it 282.)
        const uint32_t within_ = k.safe[0] > j0 || k.safe[1] > max(k.n[0], j0);
        float2 products = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          const bool used = opaque(used_), shared = opaque(shared_), part = opaque(part_);
          float v[32];
          if (used) {
            tc_ld(tmem + lanes + 256 + 128 * q + c, v);
            tc_wait_ld();
            tc_landed(v);
          }
          if (shared) {
            float w[32];
            tc_ld(tmem + lanes + 256 + 128 * other + c, w);
            tc_wait_ld();
            tc_landed(w);
            // (a buffer whose rows saw nothing holds zeros)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(w[e], f1, v[e] * f0);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= f0;
          }
          if (c == 96) {  // the sums are read: the buffers may be used again
            tc_before();
            __syncwarp();
            if (lane == 0) {
              if (used) mbar_arrive(&o_free[q]);
              if (shared) mbar_arrive(&o_free[other]);
            }
          }
          if (!used || l == 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.f;
          }
          if (opaque(within_)) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              products = fma2(make_float2(v[e], v[e + 1]), make_float2(v[e + 2], v[e + 3]), products);
          }
          if (part) {
            if (have) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(po + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          } else {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
#pragma unroll
            for (int x = 1; x <= 2; x *= 2) {
              const bool up = (sub & x) != 0;
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                if (p & x) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // piece p + x of the lower lane for piece p of the upper one
                  const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[4 * p + e] : w[4 * (p + x) + e], x);
                  w[4 * p + e] = up ? got : w[4 * p + e];
                  w[4 * (p + x) + e] = up ? w[4 * (p + x) + e] : got;
                }
              }
            }
#pragma unroll
            for (int p = 0; p < 4; ++p)
              if (p < left)
                *reinterpret_cast<uint4*>(o + p * a.o_ts + c) = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
          }
        }
        // (a row whose scores are NaN stays NaN)
        const bool live = have && l == l && l != 0.f, spoilt = live && !(fabsf(products.x + products.y) < INFINITY);
        const bool odd = *reinterpret_cast<volatile uint32_t*>(const_cast<uint32_t*>(&k.odd)) != 0u;
        if (__any_sync(0xFFFFFFFFu, odd || spoilt)) {
          __syncwarp();  // (the row's pieces are other lanes' stores)
          __threadfence_block();
          pr_put_odd(a, k, j0, end, bound, live, part ? po - 128 * lane : nullptr,
                     a.out + (row - lane) * a.o_ts + (int64_t)k.head * a.o_hs);
        }
      }
      if (used) o_reads ^= 1u << q;
      if (used1) o_reads ^= 1u << other;
      dead = __any_sync(0xFFFFFFFFu, dead);
      item_done(it);
    }
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
// A warp a (row, head): with M the largest reference of its parts and f_i = 2^(m_i - M) l_i,
// out = sum (f_i / sum f) o_i, o_i a part's output.  Lane i has the weights of parts i
// and i + 32, and four columns of every part, eight parts on their way at a time
// before their weights are known.  Bound by the trips to L2: 7 parts of 600 rows x
// 16 heads are 34 MB.
constexpr int kPrJoin = 8;
__global__ void __launch_bounds__(256) mla_prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = item / a.heads;
  const int head = (int)(item - row * a.heads);
  if (row >= a.q_tokens) return;
  const int64_t step = (int64_t)a.heads * a.q_tokens, at = (int64_t)head * a.q_tokens + row;
  const int begin = a.cu_q[0], end = a.cu_q[a.docs];
  float2 ml[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    ml[i] = s < a.splits ? a.part_ml[s * step + at] : make_float2(-INFINITY, 0.f);
  }
  const float4* part = reinterpret_cast<const float4*>(a.part_o + at * 128) + lane;
  float4 v[kPrJoin];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kPrJoin; ++i)
      if (s0 + i < a.splits) v[i] = part[(s0 + i) * step * 32];
  };
  fetch(0);
  if (row < begin || row >= end) return;  // rows of no document are left as they are
  float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float f[2];  // (what saw nothing may hold anything)
#pragma unroll
  for (int i = 0; i < 2; ++i) f[i] = ml[i].y == 0.f ? 0.f : exp2f(ml[i].x - M) * ml[i].y;
  const float l = warp_sum(f[0] + f[1]), inv = l == 0.f ? 0.f : 1.0f / l;
  f[0] *= inv;
  f[1] *= inv;
  // (an infinity counts whatever its weight)
  auto add = [](float w, float v, float o) { return fmaf(fabsf(v) < INFINITY ? w : 1.0f, v, o); };
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 0;; fetch(s0)) {
#pragma unroll
    for (int i = 0; i < kPrJoin; ++i) {
      const int s = s0 + i;
      if (s >= a.splits) break;
      const float w = __shfl_sync(0xFFFFFFFFu, s < 32 ? f[0] : f[1], s & 31);
      const float some = __shfl_sync(0xFFFFFFFFu, s < 32 ? ml[0].y : ml[1].y, s & 31);
      if (some == 0.f) continue;
      o.x = add(w, v[i].x, o.x);
      o.y = add(w, v[i].y, o.y);
      o.z = add(w, v[i].z, o.z);
      o.w = add(w, v[i].w, o.w);
    }
    s0 += kPrJoin;
    if (s0 >= a.splits) break;
  }
  uint16_t* out = a.out + row * a.o_ts + (int64_t)head * a.o_hs + 4 * lane;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
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

template <bool CAP, bool BIAS, bool LONG>
cudaError_t launch_prompt_kernel(const PromptArgs& a, const PromptMaps& maps, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = PrSmem::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_prompt_attn_kernel<CAP, BIAS, LONG>, a, maps);
}

// Documents of so many keys on average (over the parts that they are split into) take
// capped scores in rounds of 64 columns.  Us with 32 and with 64:
//   24 of 100 to 1,000 rows, 64 heads         382   421
//   1 of 1,000 rows, 64 heads                  45.1  44.7
//   1 of 2,000 rows, 64 heads                 112.7 110.1
//   2 of 300 rows on 16,000 keys, 16 heads    168   165   (7 parts)
//   1 of 4,000 rows, 32 heads                 196   191
//   1 of 8,192 rows, 16 heads                 357   345
// (More code drives other code out of the cache where items are short.)
constexpr int kLongKeys = 2000;

template <bool CAP, bool BIAS>
cudaError_t prepare_prompt_kernel() {
  const cudaError_t e = cudaFuncSetAttribute(mla_prompt_attn_kernel<CAP, BIAS, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, PrSmem::kBytes);
  return e != cudaSuccess || !CAP ? e
                                  : cudaFuncSetAttribute(mla_prompt_attn_kernel<CAP, BIAS, CAP>,
                                                         cudaFuncAttributeMaxDynamicSharedMemorySize, PrSmem::kBytes);
}
template <bool CAP, bool BIAS>
cudaError_t launch_prompt_long(const PromptArgs& a, const PromptMaps& maps, int ctas, cudaStream_t stream) {
  return CAP && a.k_tokens / a.docs / a.splits >= kLongKeys
             ? launch_prompt_kernel<CAP, BIAS, CAP>(a, maps, ctas, stream)
             : launch_prompt_kernel<CAP, BIAS, false>(a, maps, ctas, stream);
}

}  // namespace

cudaError_t prepare_prompt() {
  cudaError_t e = prepare_prompt_kernel<false, false>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<true, false>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<false, true>();
  if (e == cudaSuccess) e = prepare_prompt_kernel<true, true>();
  return e;
}

cudaError_t launch_prompt(const PromptArgs& a, const PromptInputs& in, int ctas, cudaStream_t stream) {
  PromptMaps maps = {};
  const int keys = a.k_tokens > 0 ? a.k_tokens : 1;
  if (!encode_heads_map(&maps.q_nope, in.q_nope, a.q_tokens, a.heads, kNope, in.qn_ts, in.qn_hs, kPrTile) ||
      !encode_heads_map(&maps.q_pe, in.q_pe, a.q_tokens, a.heads, kRope, in.qp_ts, in.qp_hs, kPrTile) ||
      !encode_heads_map(&maps.k_nope, in.k_nope, keys, a.heads, kNope, in.kn_ts, in.kn_hs, kPrTile) ||
      !encode_heads_map(&maps.k_pe, in.k_pe, keys, 1, kRope, in.kp_ts, in.kp_ts, kPrTile) ||
      !encode_heads_map(&maps.v, in.v, keys, a.heads, kNope, in.v_ts, in.v_hs, kPrTile / 2))
    return cudaErrorInvalidValue;
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  const cudaError_t e = cap ? (bias ? launch_prompt_long<true, true>(a, maps, ctas, stream)
                                    : launch_prompt_long<true, false>(a, maps, ctas, stream))
                            : (bias ? launch_prompt_long<false, true>(a, maps, ctas, stream)
                                    : launch_prompt_long<false, false>(a, maps, ctas, stream));
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
  if (!(softmax_scale >= 0.0f) || softmax_scale > 3.0e38f || !(softcap == 0.0f || softcap >= 1e-6f) || softcap > MLA_MAX_SOFTCAP)
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
  int above = mla::kPrRoom + 1;  // (1 for the reference's rounding)
  while (((int64_t)1 << (above - mla::kPrRoom - 1)) < k_tokens) ++above;
  a.above = (float)above;
  a.times = ldexpf(1.0f, above);
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.err = h->err;
  const int64_t tiles = (q_tokens + (int64_t)(2 * mla::kPrTile - 1) * docs) / (2 * mla::kPrTile);
  a.splits = mla::prompt_splits(tiles * h->heads, q_tokens * h->heads,
                                (k_tokens / docs + mla::kPrTile - 1) / mla::kPrTile, h->num_sms);
  const int64_t items = tiles * h->heads * a.splits;
  // Heads whose tiles are handed out together, the last tiles first, each for all of the
  // group's heads.  Where rows see what lies before them: enough for four items an SM, so
  // that short ones are left for the end; and as many as keep a document's keys and values
  // in half of L2, since rows of memory hold neighbouring heads.  Where all rows see all:
  // two items an SM, since only keys are shared.  Us with four items an SM throughout,
  // and as it is:
  //   24 of 100 to 1,000 rows, 64 heads, capped   380  358
  //   4 of 1,001 to 2,000 rows, 40 heads, biased  163  153
  //   20 of 600 rows, 128 heads                   515  448
  //   1 of 4,096 rows, 64 heads                   264  232
  //   1 of 4,096 rows, 64 heads, all to all       393  375
  //   4 of 2,000 rows, 64 heads, all to all       422  416
  //   16 of 500 rows, 64 heads, all to all        143  157
  // (The last loses: its keys are few, and the rule looks at no length where rows see all.)
  constexpr int64_t kKeys = (int64_t)64 << 20, row = 2 * mla::kNope * (int64_t)sizeof(uint16_t);
  const int64_t each = tiles * a.splits, keys = (k_tokens / docs + 1) * row;
  const int64_t even = ((causal ? 4 : 2) * (int64_t)h->num_sms + each - 1) / each;
  const int64_t group = causal && kKeys / keys > even ? kKeys / keys : even;
  a.group = (int)(group < h->heads ? group : h->heads);
  a.tiles = (int)tiles;
  a.next = h->err + 2;
  a.v = static_cast<const uint16_t*>(in.v);
  a.v_ts = in.v_ts;
  a.v_hs = in.v_hs;
  return mla::launched(mla::launch_prompt(a, in, (int)(items < h->num_sms ? items : h->num_sms),
                                          static_cast<cudaStream_t>(stream)));
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
