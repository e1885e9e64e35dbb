// mla_attn_nv.cu - latent attention on the 5th-generation tensor cores for
// nvfp4_ds_mla rows: 512 E2M1 codes, an E4M3 scale for each 16 of them, 64 E4M3
// rope values.
//
// A value is code times scale, 2 + 4 significant bits: FP16 holds every product
// exactly (largest 6 * 448, smallest step 2^-10), E4M3 does not, and the scale
// of 16 columns cannot leave a product over 512.  So the rows are widened to
// FP16 on their way to shared memory, and both products are FP16 MMAs:
//  * S^T = K Q^T (M = 128 rows, N = heads, K = 576): K's planes of 64 columns,
//    K-major.  A BF16 query times its row's power of two is exact in FP16 but
//    for elements below 2^-25 of the row's largest (half a step of 2^-24 there);
//    an E4M3 query is exact.
//  * O^T += V^T P^T (M = 128 columns, N = heads, K = 128 rows): two planes read
//    M-major.  P is rounded to FP16 (2^-11 of a weight; below 2^-24, or 2^-29 of
//    the largest, to steps of that size).
// Rows, masks, the reference that stands for the maximum: as for E4M3 rows.
//
// The eight warps that widen a tile are those of the softmax: a tile's planes
// are 147 KB, so there is room for one, and the steps of a tile follow one
// another but for the planes' turns: planes 2 j and 2 j + 1 are widened as soon
// as O has read those of the tile before, S reads them as soon as they are
// there.  The codes of the next tile (176 bytes a thread) are loaded before the
// softmax and wait in registers.  P takes the place of the rope plane, which S
// has read by then.
// What bounds a tile (64 heads) is that chain: 36 MMAs for S and 32 for O at 48
// cycles are 3264 cycles, the conversions (8 lanes a cycle) about 1000, the
// stores of the planes 1150, and they overlap in part.  32 tokens of 4,096 rows,
// 64 heads: 53 us (the rows' bytes at 6.77 TB/s: 7.5; an mma.sync kernel that
// widened to BF16 in the same way: 149).
#include "mla_attn_tc.cuh"

namespace mla {
namespace {

constexpr int kNvWarpMma = 8, kNvThreads = kTcSoft + 32;

template <int NH>
struct NvSmem {
  static constexpr int kQPlane = NH * 128;
  static constexpr int oK = 0;                     // [8 latent planes, rope] of 64 FP16 columns
  static constexpr int oP = oK + 8 * kPlane;       // [row][heads]: over the rope plane
  static constexpr int oSeen = oP;                 // until the first rope rows
  static constexpr int oQ = oK + 9 * kPlane;       // 9 planes
  static constexpr int oRef = oQ + 9 * kQPlane;    // reference less kPShift, base 2 [NH]
  static constexpr int oXs = oRef + NH * 4;        // logit scale of a head's accumulators [NH]
  static constexpr int oRed = oXs + NH * 4;        // [4][NH] across the quadrants; [0][.] factors
  static constexpr int oBar = oRed + 4 * NH * 4;
  // k_full[5] s_full p_full pv_done[4] q_full drain voted
  static constexpr int kBars = 14;
  static constexpr int oMoved = oBar + kBars * 8;  // [2] 1 + the last tile that moved the reference
  static constexpr int oPlan = oMoved + 8;
  static constexpr int oTmem = oPlan + (int)sizeof(AttnPlan);
  static constexpr int kBytes = oTmem + 8;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(sizeof(AttnSeen) <= kPlane, "seen lies over a plane");
  static_assert(oQ % 1024 == 0 && oRef % 16 == 0 && oXs % 16 == 0 && oRed % 16 == 0 && oBar % 8 == 0 &&
                    oPlan % 8 == 0 && oTmem % 4 == 0,
                "alignment");
};

// A thread's share of one cache row on its way from memory to the planes: row
// 16 warp + lane / 2 of a tile, its half `side` = lane % 2 of each 64 columns
// (so a warp's 16-byte stores of swizzled rows meet no bank twice, and a pair
// of lanes reads 32 bytes side by side).
struct NvRow {
  uint4 code[8], rope[2], scale;
  __device__ __forceinline__ void load(const AttnArgs& a, int64_t row, int side) {
    if (row < 0) {  // zeros
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < 8; ++p) code[p] = zero;
      rope[0] = rope[1] = scale = zero;
      return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(a.cache + row * kRowNvfp4);
#pragma unroll
    for (int j = 0; j < 8; ++j) code[j] = p[2 * j + side];
    scale = p[kNvScales / 16 + side];
    rope[0] = p[kNvRope / 16 + 2 * side];
    rope[1] = p[kNvRope / 16 + 2 * side + 1];
  }
  // plane j's half row (32 columns) at `row` of the plane
  __device__ __forceinline__ void put(uint8_t* row, int r, int side, int j) const {
    // blocks 4 j + 2 side and the next: byte j of the scales' 8-byte words 2 side, 2 side + 1
    const uint32_t s0 = j < 4 ? scale.x : scale.y, s1 = j < 4 ? scale.z : scale.w;
    const uint32_t f0 = e4m3x2_f16(__byte_perm(s0, 0, 0x11u * (j & 3)));
    const uint32_t f1 = e4m3x2_f16(__byte_perm(s1, 0, 0x11u * (j & 3)));
    const uint32_t w[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t h[4];
      e2m1x8_scaled(w[c], c < 2 ? f0 : f1, h);
      *reinterpret_cast<uint4*>(row + ((((4 * side + c) ^ r) & 7) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
  __device__ __forceinline__ void put_rope(uint8_t* row, int r, int side) const {
    const uint32_t w[8] = {rope[0].x, rope[0].y, rope[0].z, rope[0].w,
                           rope[1].x, rope[1].y, rope[1].z, rope[1].w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(row + ((((4 * side + c) ^ r) & 7) << 4)) =
          make_uint4(e4m3x2_f16(w[2 * c]), e4m3x2_f16(w[2 * c] >> 16), e4m3x2_f16(w[2 * c + 1]),
                     e4m3x2_f16(w[2 * c + 1] >> 16));
  }
};

// One token's queries of NH heads into shared memory as FP16 (B of S^T): warp w
// takes heads w, w + 8, ..; a lane holds 16 latent columns of each, and lane
// 4 r + c the rope columns 16 c .. of the warp's r-th head.
template <int NH, bool FP8Q>
__device__ __forceinline__ void nv_queries(const AttnArgs& a, uint8_t* sq, int t, int h0, int warp,
                                           int lane, float logit, float* xs) {
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
  const int rr = lane >> 2;  // the head whose rope this lane holds: warp + 8 rr
  {
    const int h = h0 + warp + 8 * rr;
    const int64_t e = (int64_t)t * a.qp_ts + (int64_t)h * a.qp_hs + 16 * (lane & 3);
    const uint4* p = reinterpret_cast<const uint4*>(a.q_pe + e * (FP8Q ? 1 : 2));
#pragma unroll
    for (int v = 0; v < kV; ++v) rope[v] = rr < kN && h < a.heads ? p[v] : zero;
  }
  // 16 columns, the (lane % 4)-th of plane p, of one head
  auto put = [&](int p, int row, const uint4* w, float up) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (FP8Q) {
        const uint32_t c = e < 4 ? (e < 2 ? w[0].x : w[0].y) : (e < 6 ? w[0].z : w[0].w);
        h[e] = e4m3x2_f16(e & 1 ? c >> 16 : c);
      } else {
        const uint4 q = w[e >> 2];
        const uint32_t c = (e & 3) < 2 ? (e & 1 ? q.y : q.x) : (e & 1 ? q.w : q.z);
        const float2 v = fmul2_rn(make_float2(bf16lo(c), bf16hi(c)), make_float2(up, up));
        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h[e]) : "f"(v.x), "f"(v.y));
      }
    }
    uint8_t* d = sq + p * (NH * 128) + row * 128;
    const int c = 2 * (lane & 3);
    *reinterpret_cast<uint4*>(d + (((c ^ row) & 7) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(d + ((((c + 1) ^ row) & 7) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
  };
  float rope_up = 1.0f;
  // magnitudes as bits order like the values (NaN above infinity)
  auto magnitude = [](uint4 w) {
    const uint32_t s = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(w.x & s, w.y & s), __vmaxu2(w.z & s, w.w & s));
  };
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    float up = 1.0f, x = logit;
    if constexpr (!FP8Q) {
      uint32_t m = __vmaxu2(magnitude(lat[r][0]), magnitude(lat[r][kV - 1]));
      if (rr == r) m = __vmaxu2(m, __vmaxu2(magnitude(rope[0]), magnitude(rope[kV - 1])));
      m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
      // the power of two that brings the largest into [256, 512): from its
      // exponent field, kept where both it and its inverse are normal
      int ex = (int)(m >> 7) - 127;
      ex = max(-100, min(ex, 126));
      up = __uint_as_float((uint32_t)(127 + 8 - ex) << 23);
      x = logit * __uint_as_float((uint32_t)(127 - 8 + ex) << 23);
      // an infinite query: no finite logits (the products alone would give -infinity
      // for rows of one sign, and a context of those would look empty)
      if (m >= 0x7F80u) x = __int_as_float(0x7FC00000);
    }
    put(lane >> 2, warp + 8 * r, lat[r], up);
    if (lane == 0) xs[warp + 8 * r] = x;
    if (rr == r) rope_up = up;
  }
  if (rr < kN) put(8, warp + 8 * rr, rope, rope_up);
}

template <int NH, bool FP8Q>
__global__ void __launch_bounds__(kNvThreads, 1) mla_attn_nv_kernel(const AttnArgs a) {
  using S = NvSmem<NH>;
  constexpr int kHalf = NH / 2;  // heads a softmax thread handles
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::oBar);
  uint64_t* s_full = k_full + 5;
  uint64_t* p_full = s_full + 1;
  uint64_t* pv_done = p_full + 1;
  uint64_t* q_full = pv_done + 4;
  uint64_t* drain = q_full + 1;
  uint64_t* voted = drain + 1;
  uint32_t* moved = reinterpret_cast<uint32_t*>(smem + S::oMoved);
  float* ref = reinterpret_cast<float*>(smem + S::oRef);
  float* xs = reinterpret_cast<float*>(smem + S::oXs);
  float* red = reinterpret_cast<float*>(smem + S::oRed);
  AttnPlan* plan = reinterpret_cast<AttnPlan*>(smem + S::oPlan);
  AttnSeen* seen = reinterpret_cast<AttnSeen*>(smem + S::oSeen);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);
  uint32_t* gave_up = tslot + 1;  // a softmax wait ran out

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int group = blockIdx.x % a.groups, worker = blockIdx.x / a.groups;
  const int h0 = group * NH;
  if (tid == 0) {
    for (int b = 0; b < 5; ++b) mbar_init(&k_full[b], kTcSoft / 32);
    mbar_init(s_full, 1);
    mbar_init(p_full, kTcSoft / 32);
    for (int b = 0; b < 4; ++b) mbar_init(&pv_done[b], 1);
    mbar_init(q_full, kTcSoft / 32);
    mbar_init(drain, 1);
    mbar_init(voted, kTcSoft / 32);
    moved[0] = moved[1] = 0;
    *gave_up = 0;
    mbar_fence_init();
    // the swizzles go by address bits: the base is a multiple of 1 KiB
    if (smem_u32(smem) & 1023u) atomicOr(a.err, MLA_DEVERR_CHECK);
  }
  if (warp == kNvWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tslot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();  // (after the wait: the join reads the lengths before its own)
  tc_before();
  // (the plan's barriers order the set-up above)
  attn_make_plan(a, plan, reinterpret_cast<uint32_t*>(red), blockIdx.x == 0, seen);
  tc_after();
  // S^T at column 0, O^T planes (128 columns of the latent each) from 256
  const uint32_t tmem = uniform(*tslot);
  uint32_t first, end;
  attn_range(a, plan, worker, &first, &end);
  bool dead = false;

  if (warp == kNvWarpMma) {
    // ================= MMA issuer (the warp together, one elected lane issues)
    constexpr uint32_t id_s = tc_idesc(128, NH, 0, false, false);
    constexpr uint32_t id_o = tc_idesc(128, NH, 0, true, true);
    const uint64_t dk = tc_desc(smem_u32(smem + S::oK), 1024, 2);
    const uint64_t dv = tc_desc_wide(smem_u32(smem + S::oK), 1024, kPlane);  // two planes, M-major
    const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
    const uint64_t dp = tc_desc(smem_u32(smem + S::oP), 1024, 2);
    constexpr uint64_t kPl = kPlane >> 4, kQPl = S::kQPlane >> 4;
    // (A wait that ran out ends no loop here: the loops are then the warp's, and
    // the descriptors stay in uniform registers.  The MMAs go on over whatever
    // the planes hold, and the results do not count.)
    const uint32_t x1 = uniform(end), lead = uniform(plan->lead);
    uint32_t x = uniform(first), seg_end = x;
    int segs = 0;
    for (int i = 0; x < x1; ++i, ++x) {
      const uint32_t par = (uint32_t)(i & 1);
      const bool fresh = x == seg_end;
      if (fresh) {
        const int t = attn_token_of(plan, a.batch, x);
        if (i > 0) x += lead;
        seg_end = uniform(plan->end[t]);
        tc_wait_warp(q_full, (uint32_t)(segs & 1), dead);
        ++segs;
      }
#pragma unroll
      for (int p = 0; p < 9; ++p) {
        if ((p & 1) == 0) {  // planes 2 j and 2 j + 1, then rope
          tc_wait_warp(&k_full[p >> 1], par, dead);
          tc_after();
        }
        tc_mma4_f16<2, 2>(tmem, dk + p * kPl, dq + p * kQPl, id_s, p > 0 ? 1u : 0u);
      }
      tc_commit(s_full);
      tc_wait_warp(p_full, par, dead);
      tc_after();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // 16 rows a step: 2048 bytes of V and of P
        const uint64_t da = dv + 2 * j * kPl;
        tc_mma4_f16<128, 128>(tmem + 256 + NH * j, da, dp, id_o, fresh ? 0u : 1u);
        tc_mma4_f16<128, 128>(tmem + 256 + NH * j, da + 512, dp + 512, id_o, 1u);
        tc_commit(&pv_done[j]);
      }
    }
    if (dead) {  // let what was issued finish before TMEM is freed
      tc_commit(drain);
      (void)mbar_wait_bounded(drain, 0u, kTcWait);
    }
  } else {
    // ================= widening, softmax, rescaling, epilogue (warps 0-7)
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int pos = 32 * quad + lane;    // this thread's row of a tile in the softmax
    const int hb = half * kHalf;         // its heads
    const int wrow = 16 * warp + (lane >> 1), side = lane & 1;  // its row to widen
    const float qinv = a.q_scale_inv != nullptr ? *a.q_scale_inv : 1.0f;
    const float logit = a.scale / qinv * 1.4426950408889634f;
    int i = 0;
    uint32_t x = first;
    // A thread whose wait has run out goes on without waiting: all of them
    // pass the same barriers to the end.  (It says so, and from then on none takes
    // the path that only some votes take.)
    while (x < end) {
      const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
      x = max(x, k.start);
      const uint32_t seg0 = x, seg_end = min(k.end, end);
      int64_t page;
      NvRow raw;
      bool valid_next = false;
      auto fetch = [&](uint32_t tile) {
        const uint32_t v = (tile - k.start) * kTcTile;
        raw.load(a, attn_row(a, k, v + wrow, &page), side);
        valid_next = attn_row(a, k, v + pos, &page) >= 0;
      };
      fetch(x);
      nv_queries<NH, FP8Q>(a, smem + S::oQ, k.t, h0, warp, lane, logit, xs);
      for (int h = tid; h < NH; h += kTcSoft) ref[h] = 0.f;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_barrier();
      if (lane == 0) mbar_arrive(q_full);
      bool started = false;  // a row that counts has been met
      float2 l[kHalf / 2];
#pragma unroll
      for (int h = 0; h < kHalf / 2; ++h) l[h] = make_float2(0.f, 0.f);

      for (; x < seg_end; ++x, ++i) {
        const int b = i & 1;
        // ---- the tile's planes
#pragma unroll
        for (int j = 0; j < 5; ++j) {
          if (i > 0 && j < 4) tc_wait(&pv_done[j], (uint32_t)((i - 1) & 1), dead, gave_up);
          uint8_t* row = smem + S::oK + 2 * j * kPlane + wrow * 128;
          if (j < 4) {
            raw.put(row, wrow, side, 2 * j);
            raw.put(row + kPlane, wrow, side, 2 * j + 1);
          } else {
            raw.put_rope(row, wrow, side);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_before();  // S of the tile before has been read
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[j]);
        }
        const bool valid = valid_next;
        if (x + 1 < seg_end) fetch(x + 1);
        // ---- S: exponents (logits in base 2 less the reference, plus kPShift)
        tc_wait(s_full, (uint32_t)b, dead, gave_up);
        tc_after();
        float p[kHalf];
        auto exponents = [&]() {
          tc_ld(tmem + lanes + hb, p);
          tc_wait_ld();
          tc_landed(p);
#pragma unroll
          for (int h = 0; h < kHalf; h += 4) {
            const float4 c = *reinterpret_cast<const float4*>(xs + hb + h);
            const float4 m = *reinterpret_cast<const float4*>(ref + hb + h);
            const float2 v0 = fma2(make_float2(p[h], p[h + 1]), make_float2(c.x, c.y), make_float2(-m.x, -m.y));
            const float2 v1 = fma2(make_float2(p[h + 2], p[h + 3]), make_float2(c.z, c.w), make_float2(-m.z, -m.w));
            p[h] = v0.x;
            p[h + 1] = v0.y;
            p[h + 2] = v1.x;
            p[h + 3] = v1.y;
          }
          if (!valid) {
#pragma unroll
            for (int h = 0; h < kHalf; ++h) p[h] = -INFINITY;
          }
        };
        exponents();
        float over = fmaxf(p[0], p[1]);
#pragma unroll
        for (int h = 2; h < kHalf; h += 2) over = fmaxf(over, fmaxf(p[h], p[h + 1]));
        bool move = valid && (!started || over > kPShift + kPRoom);
        move = __any_sync(0xFFFFFFFFu, move);
        __syncwarp();  // (what a lane has said by gave_up goes before the arrival)
        if (lane == 0) {
          if (move) *reinterpret_cast<volatile uint32_t*>(&moved[b]) = (uint32_t)i + 1;
          mbar_arrive(voted);
        }
        // (the weights as if nothing moved, while the warps' answers meet)
#pragma unroll
        for (int h = 0; h < kHalf; ++h) p[h] = ex2(p[h]);
        tc_wait_votes(voted, (uint32_t)(i & 1), dead, gave_up);
        if (*reinterpret_cast<volatile uint32_t*>(&moved[b]) == (uint32_t)i + 1 &&
            *reinterpret_cast<volatile uint32_t*>(gave_up) == 0u) {
          // the reference moves to the tile's maximum where that passes it by
          // too much (for the first rows that count, everywhere)
          exponents();
          const float mx = lanes_reduce<kHalf, OpMax>(p);
          if ((lane * kHalf) % 32 == 0) red[quad * NH + hb + lane * kHalf / 32] = mx;
          tc_barrier();
          if (tid < NH) {
            const float m = fmaxf(fmaxf(red[tid], red[NH + tid]), fmaxf(red[2 * NH + tid], red[3 * NH + tid]));
            const bool grow = started ? m > kPShift + kPRoom : m > -INFINITY;
            red[tid] = grow ? kPShift - m : 0.f;
            if (grow) ref[tid] += m - kPShift;
          }
          tc_barrier();
#pragma unroll
          for (int h = 0; h < kHalf; ++h) {
            const float d = red[hb + h];
            p[h] = ex2(p[h] + d);
            float& lh = h & 1 ? l[h / 2].y : l[h / 2].x;
            if (started) lh *= ex2(d);
          }
          if (started && x > seg0) {
            // (O of the tile before is complete: its planes have been written over)
#pragma unroll 1
            for (int c = 0; c < 2 * NH; c += 32) {
              // planes 2 half and 2 half + 1 of O^T: columns are heads
              float v[32];
              const uint32_t at = tmem + lanes + 256 + 2 * half * NH + c;
              tc_ld(at, v);
              tc_wait_ld();
              tc_landed(v);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                v[e] *= ex2(red[(c + e) % NH]);
              tc_st32(at, v);
            }
            tc_wait_st();
          }
          started = true;
          tc_barrier();  // red is read
        }
#pragma unroll
        for (int h = 0; h < kHalf; h += 2) l[h / 2] = add2(l[h / 2], make_float2(p[h], p[h + 1]));
        // ---- the weights, over the rope plane
        uint8_t* prow = smem + S::oP + pos * 128;
#pragma unroll
        for (int c = 0; c < kHalf / 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(w[e]) : "f"(p[8 * c + 2 * e]), "f"(p[8 * c + 2 * e + 1]));
          *reinterpret_cast<uint4*>(prow + ((((hb / 8 + c) ^ pos) & 7) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
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
        red[tid] = sum == 0.f ? 0.f : whole ? 1.0f / sum : 1.0f;
        if (!whole)
          attn_part_ml(a, h0 + tid)[slot] = make_float2(m, sum);
        else if (a.lse != nullptr && h0 + tid < a.heads)
          a.lse[(int64_t)k.t * a.heads + h0 + tid] = attn_lse(m, sum);
      }
      tc_barrier();
      for (int j = 0; j < 4; ++j) tc_wait(&pv_done[j], (uint32_t)((i - 1) & 1), dead, gave_up);
      tc_after();
      tc_store_out<NH>(a, k, tmem + lanes + 256, half, pos, h0, slot, whole, red, 1.0f, 1.0f);
      tc_before();
      tc_barrier();  // red is read
      x = seg_end;
    }
  }
  if (dead) atomicOr(a.err, MLA_DEVERR_TIMEOUT);
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == kNvWarpMma) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

template <int NH, bool FP8Q>
cudaError_t launch_nv(const AttnArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.workers * a.groups));
  cfg.blockDim = dim3(kNvThreads);
  cfg.dynamicSmemBytes = NvSmem<NH>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_attn_nv_kernel<NH, FP8Q>, a);
}

template <int NH>
cudaError_t launch_nv_heads(const AttnArgs& a, cudaStream_t stream) {
  return a.q_scale_inv != nullptr ? launch_nv<NH, true>(a, stream) : launch_nv<NH, false>(a, stream);
}

template <int NH>
cudaError_t prepare_nv_heads() {
  cudaError_t e = cudaFuncSetAttribute(mla_attn_nv_kernel<NH, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, NvSmem<NH>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(mla_attn_nv_kernel<NH, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             NvSmem<NH>::kBytes);
  return e;
}

}  // namespace

cudaError_t prepare_attn_nv() {
  cudaError_t e = prepare_nv_heads<16>();
  if (e == cudaSuccess) e = prepare_nv_heads<32>();
  if (e == cudaSuccess) e = prepare_nv_heads<64>();
  return e;
}

cudaError_t launch_attn_nv(const AttnArgs& a, cudaStream_t stream) {
  switch (a.cta_heads) {
    case 16: return launch_nv_heads<16>(a, stream);
    case 32: return launch_nv_heads<32>(a, stream);
    default: return launch_nv_heads<64>(a, stream);
  }
}

}  // namespace mla
