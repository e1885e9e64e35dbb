// mla_attn_ds.cu - latent attention on the 5th-generation tensor cores for
// fp8_ds_mla rows: 512 E4M3 codes under four FP32 scales (one for each 128
// columns of a token) and 64 BF16 rope values.
//
// As in mla_attn_tc.cu the codes stay codes.  A 128-column plane holds one
// scale tile, so the scales are factors outside the products:
//  * S^T: each plane's product has its own TMEM accumulator, D_j = C_j Q_j^T
//    (both terms of the queries into it), the rope product (BF16 x BF16,
//    queries times the same power of two as the codes' queries) another; the
//    softmax thread, which owns one row, adds R + sum_j scale_j D_j.
//  * O^T: plane j's weights are P times scale_j / ref_j, split into an E4M3 and
//    an E5M2 term each, ref_j the largest scale so far; O_j is multiplied by
//    ref_j at the end.  The factor and P go to FP16 first (2^-11 each, and the
//    factor exact where the scales are powers of two, as the decode step writes
//    them): half the conversions of FP32 pairs, small next to the terms' errors
//    (2^-7 of a weight down to 2^-10 of the largest weight times the largest
//    scale; below, 2^-17 of it, as for E4M3 rows).
// TMEM: four 64-column accumulators for the five products of a tile (the rope
// product and plane 3 share one, in turn), and O^T's four planes.
//
// Six latent planes, one rope plane and two weight tiles are in shared memory.
// The MMA warp issues in a fixed order, the first products of a tile's S before
// the O of the tile before it, the last ones behind: with loops and barriers
// known to the compiler the descriptors are uniform, and the planes with one
// copy are asked for last.  (Issuing whatever was ready, by test_wait, took
// 104 us at 62 tokens, 128 heads and up to 4,096 rows; this order 98 us.)
// What bounds a tile (64 heads): the chain of its steps, about 6,500 cycles.
// The tensor core's share, shared-memory reads (36 MMAs for S and 32 for O, 48
// cycles each), is 3264; the softmax warps' conversions (64 term pairs a
// thread) do not overlap it fully, since TMEM has room for one tile's S only.
// Sixteen softmax warps (97.7 us, with spills) or weights split once and
// shifted by exponent for each plane (109 us) gained nothing.
#include "mla_attn_tc.cuh"

namespace mla {
namespace {

// Latent planes in shared memory: two copies of planes 0 and 1 (slots 0-3, by
// the tile's parity), one of planes 2 and 3 (slots 4 and 5); a slot's n-th use.
constexpr int kDsSlots = 6;
__device__ __forceinline__ int ds_slot(int tile, int j) { return j < 2 ? 2 * (tile & 1) + j : 2 + j; }
__device__ __forceinline__ uint32_t ds_use(int tile, int j) { return j < 2 ? tile >> 1 : tile; }

template <int NH, bool FP8Q>
struct DsSmem {
  static constexpr int kQPlane = (FP8Q ? NH : 2 * NH) * 128;
  static constexpr int oRing = 0;
  static constexpr int oRope = oRing + kDsSlots * kPlane;  // [128 rows][128 B]
  static constexpr int oP = oRope + kPlane;                // [2][row][hi | lo]
  static constexpr int oQ = oP + 2 * kPlane;
  static constexpr int oQr = oQ + 4 * kQPlane;             // [NH][128 B] BF16
  static constexpr int oRef = oQr + NH * 128;
  static constexpr int oXs = oRef + NH * 4;
  static constexpr int oRed = oXs + NH * 4;                // [4][NH]
  static constexpr int oVref = oRed + 4 * NH * 4;          // [4] references, [4] ratios, [4][4] warp maxima
  static constexpr int oBar = oVref + 96;
  // full[6] empty[6] rope_full rope_empty d_full[4] d_free[4] p_full[2] pv_done[2] q_full drain voted
  static constexpr int kBars = 2 * kDsSlots + 2 + 8 + 4 + 3;
  static constexpr int oMoved = oBar + ((kBars + 1) & ~1) * 8;
  static constexpr int oPlan = oMoved + 8;
  static constexpr int oSeen = (oPlan + (int)sizeof(AttnPlan) + 15) & ~15;
  static constexpr int oTmem = oSeen + (int)sizeof(AttnSeen);
  static constexpr int kBytes = oTmem + 8;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(oP % 1024 == 0 && oQ % 1024 == 0 && oRope % 1024 == 0 && oQr % 1024 == 0 &&
                    oRef % 16 == 0 && oXs % 16 == 0 && oRed % 16 == 0 && oVref % 16 == 0 &&
                    oBar % 8 == 0 && oPlan % 8 == 0 && oTmem % 4 == 0,
                "alignment");
};

template <int NH, bool FP8Q, bool COPY>
__global__ void __launch_bounds__(kTcThreads, 1)
    mla_attn_ds_kernel(const AttnArgs a, const __grid_constant__ TcMaps maps) {
  using S = DsSmem<NH, FP8Q>;
  constexpr int kHalf = NH / 2;  // heads a softmax thread handles
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::oBar);
  uint64_t* empty = full + kDsSlots;
  uint64_t* rope_full = empty + kDsSlots;
  uint64_t* rope_empty = rope_full + 1;
  uint64_t* d_full = rope_empty + 1;
  uint64_t* d_free = d_full + 4;
  uint64_t* p_full = d_free + 4;
  uint64_t* pv_done = p_full + 2;
  uint64_t* q_full = pv_done + 2;
  uint64_t* drain = q_full + 1;
  uint64_t* voted = drain + 1;
  uint32_t* moved = reinterpret_cast<uint32_t*>(smem + S::oMoved);
  uint32_t* gave_up = reinterpret_cast<uint32_t*>(smem + S::oTmem + 4);  // a softmax wait ran out
  float* ref = reinterpret_cast<float*>(smem + S::oRef);
  float* xs = reinterpret_cast<float*>(smem + S::oXs);
  float* red = reinterpret_cast<float*>(smem + S::oRed);
  float* vref = reinterpret_cast<float*>(smem + S::oVref);
  AttnPlan* plan = reinterpret_cast<AttnPlan*>(smem + S::oPlan);
  AttnSeen* seen = reinterpret_cast<AttnSeen*>(smem + S::oSeen);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::oTmem);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int group = blockIdx.x % a.groups, worker = blockIdx.x / a.groups;
  const int h0 = group * NH;
  if (tid == 0) {
    for (int s = 0; s < kDsSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(rope_full, 1);
    mbar_init(rope_empty, 1);
    for (int b = 0; b < 4; ++b) {
      mbar_init(&d_full[b], 1);
      mbar_init(&d_free[b], kTcSoft / 32);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&p_full[b], kTcSoft / 32);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, kTcSoft / 32);
    mbar_init(drain, 1);
    mbar_init(voted, kTcSoft / 32);
    moved[0] = moved[1] = 0;
    *gave_up = 0;
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
  if (tid == kTcSoft) prefetch_tensormap(&maps.latent);
  pdl_wait();
  pdl_launch_dependents();  // (after the wait: the join reads the lengths before its own)
  tc_before();
  // (the plan's barriers order the set-up above)
  attn_make_plan(a, plan, reinterpret_cast<uint32_t*>(red), blockIdx.x == 0, seen);
  tc_after();
  // S^T accumulators at columns NH * b: rope and plane 3 in 0, planes 0-2 in
  // 1-3; O^T planes from 256
  const uint32_t tmem = uniform(*tslot);
  uint32_t first, end;
  attn_range(a, plan, worker, &first, &end);
  bool dead = false;

  if (warp == 8) {
    // ================= TMA: a tile's planes in the order rope, 0, 1, 2, 3
    if constexpr (COPY) {
      auto place = [&](int n, int p) {
        if (p == 0) return TcSlot{rope_full, rope_empty, (uint32_t)n, smem + S::oRope};
        const int s = ds_slot(n, p - 1);
        return TcSlot{&full[s], &empty[s], ds_use(n, p - 1), smem + S::oRing + s * kPlane};
      };
      tc_copy_tiles<kRowDs, 128, kDsRope>(a, plan, seen, first, end, lane, dead, place);
    } else {
      const int boxes = kTcTile / maps.box_rows;
      const int32_t no_row = (int32_t)(a.num_pages * a.page_size);  // past the end: zeros
      int i = 0, issued = 0;  // tiles, planes
      uint32_t x = first;
      while (x < end && !dead) {
        const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
        x = max(x, k.start);
        const uint32_t seg_end = min(k.end, end);
        for (; x < seg_end && !dead; ++x, ++i) {
          int32_t y = no_row;
          if (lane < boxes) {
            int64_t page;
            const int64_t r = attn_row(a, k, (x - k.start) * kTcTile + lane * maps.box_rows, &page);
            if (r >= 0) y = (int32_t)r;
          }
#pragma unroll 1
          for (int p = 0; p < 5; ++p) {
            const int slot = p == 0 ? 0 : ds_slot(i, p - 1);
            const uint32_t use = p == 0 ? i : ds_use(i, p - 1);
            uint64_t* f = p == 0 ? rope_full : &full[slot];
            if (use >= 1) tc_wait_warp(p == 0 ? rope_empty : &empty[slot], (use - 1) & 1u, dead);
            if (dead) break;
            ++issued;
            if (lane == 0) mbar_arrive_expect_tx(f, kPlane);
            __syncwarp();
            if (lane < boxes)
              tma_g2s_2d(smem + (p == 0 ? S::oRope : S::oRing + slot * kPlane) + lane * maps.box_rows * 128,
                         &maps.latent, p == 0 ? kDsRope : 128 * (p - 1), y, f);
          }
        }
      }
      // A wait ran out: the planes issued last land before the CTA leaves.
      // (Otherwise the MMAs have read them all.)
      if (dead && issued > 0) {
        (void)mbar_wait_bounded(rope_full, (uint32_t)(((issued - 1) / 5) & 1), kTcWait);
        for (int s = 0; s < kDsSlots; ++s) {
          const int j = s < 4 ? s & 1 : s - 2, n = issued - 2 - j;  // planes up to this one of some tile
          int last = n >= 0 ? n / 5 : -1;
          if (s < 4 && last >= 0 && (last & 1) != s >> 1) --last;
          if (last >= 0) (void)mbar_wait_bounded(&full[s], ds_use(last, j) & 1u, kTcWait);
        }
      }
    }
  } else if (warp == 9) {
    // ================= MMA issuer (the warp together, one elected lane issues)
    constexpr uint32_t id_s = tc_idesc(128, NH, 0, false, false);
    constexpr uint32_t id_r = tc_idesc(128, NH, 1, false, false) | (1u << 7);  // BF16 x BF16
    constexpr uint32_t id_hi = tc_idesc(128, NH, 0, true, true);
    constexpr uint32_t id_lo = tc_idesc(128, NH, 1, true, true);
    const uint64_t dk = tc_desc(smem_u32(smem + S::oRing), 1024, 2);  // planes, K- or M-major
    const uint64_t dkr = tc_desc(smem_u32(smem + S::oRope), 1024, 2);
    const uint64_t dq = tc_desc(smem_u32(smem + S::oQ), 1024, 2);
    const uint64_t dqr = tc_desc(smem_u32(smem + S::oQr), 1024, 2);
    const uint64_t dp = tc_desc(smem_u32(smem + S::oP), 1024, 2);
    constexpr uint64_t kPl = kPlane >> 4, kQPl = S::kQPlane >> 4;
    // (A wait that ran out ends no loop here: the loops are then the warp's, and
    // the descriptors stay in uniform registers.  The MMAs go on over whatever
    // the planes hold, and the results do not count.)
    const uint32_t x1 = uniform(end), lead = uniform(plan->lead);
    // O^T of plane j of tile n, the q-th in order (`add`: to what its stretch has)
    auto pv = [&](int n, int q, int j, uint32_t add) {
      tc_wait_warp(&p_full[q & 1], (uint32_t)(q >> 1), dead);
      tc_after();
      tc_mma4x2<256, 256, 4>(tmem + 256 + NH * j, dk + ds_slot(n, j) * kPl, dp + (q & 1) * kPl, id_hi,
                             id_lo, add);
      tc_commit(&empty[ds_slot(n, j)]);
      tc_commit(&pv_done[q & 1]);
    };
    // S^T: the rope product of tile n, and plane j's
    auto qk_rope = [&](int n) {
      if (n > 0) tc_wait_warp(&d_free[0], 1u, dead);  // plane 3 of the tile before has been read
      tc_wait_warp(rope_full, (uint32_t)(n & 1), dead);
      tc_after();
      tc_mma4_f16<2, 2>(tmem, dkr, dqr, id_r, 0u);
      tc_commit(rope_empty);
      tc_commit(&d_full[0]);
    };
    auto qk = [&](int n, int j) {
      const int d = (j + 1) & 3;
      if (d == 0)
        tc_wait_warp(&d_free[0], 0u, dead);  // the rope product has been read
      else if (n > 0)
        tc_wait_warp(&d_free[d], (uint32_t)((n - 1) & 1), dead);
      tc_wait_warp(&full[ds_slot(n, j)], ds_use(n, j) & 1u, dead);
      tc_after();
      const uint64_t da = dk + ds_slot(n, j) * kPl, db = dq + j * kQPl;
      if constexpr (FP8Q)
        tc_mma4<2, 2>(tmem + NH * d, da, db, id_s, 0u);
      else
        tc_mma4x2<2, 2, NH * 8>(tmem + NH * d, da, db, id_s, id_s, 0u);
      tc_commit(&d_full[d]);
    };
    uint32_t x = uniform(first), seg_end = x, add = 0;  // add: whether the tile before added to its O^T
    int segs = 0;
    for (int i = 0;; ++i, ++x) {
      // S of tile i around the O of tile i - 1: planes 2 and 3, of which there
      // is one copy, are freed first and asked for last
      const bool more = x < x1, fresh = more && x == seg_end, due = i > 0;
      if (more && !fresh) {
        qk_rope(i);
        qk(i, 0);
        qk(i, 1);
      }
      if (due) {
        pv(i - 1, 0, 2, add);
        pv(i - 1, 1, 3, add);
        pv(i - 1, 2, 0, add);
        pv(i - 1, 3, 1, add);
      }
      if (fresh) {  // new queries: they come when the stretch before is stored
        const int t = attn_token_of(plan, a.batch, x);
        if (due) x += lead;
        seg_end = uniform(plan->end[t]);
        tc_wait_warp(q_full, (uint32_t)(segs & 1), dead);
        ++segs;
        qk_rope(i);
        qk(i, 0);
        qk(i, 1);
      }
      if (more) {
        qk(i, 2);
        qk(i, 3);
      }
      if (!more) break;
      add = fresh ? 0u : 1u;
    }
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
    const float logit = a.scale / qinv * 1.4426950408889634f;
    auto row_scales = [&](int64_t r) {
      return r >= 0 ? *reinterpret_cast<const float4*>(a.cache + r * kRowDs + kDsScales)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    int i = 0;
    uint32_t x = first;
    // A thread whose wait has run out goes on without waiting: all of them
    // pass the same barriers to the end.  (It says so, and from then on none takes
    // the path that only some votes take.)
    while (x < end) {
      const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
      x = max(x, k.start);
      const uint32_t seg0 = x, seg_end = min(k.end, end);
      tc_queries<NH, FP8Q, true>(a, smem + S::oQ, smem + S::oQr, k.t, h0, warp, lane, logit, xs);
      for (int h = tid; h < NH; h += kTcSoft) ref[h] = 0.f;
      if (tid < 4) vref[tid] = 0.f;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_barrier();
      if (lane == 0) mbar_arrive(q_full);
      int64_t page = 0;
      int64_t crow = attn_row(a, k, (x - k.start) * kTcTile + pos, &page);
      float4 rscale = row_scales(crow);
      bool started = false;  // a row that counts has been met
      float2 l[kHalf / 2];
#pragma unroll
      for (int h = 0; h < kHalf / 2; ++h) l[h] = make_float2(0.f, 0.f);

      for (; x < seg_end; ++x, ++i) {
        const int b = i & 1;
        const bool valid = crow >= 0;
        const uint32_t dither = weight_dither(pos, x - k.start);
        const float sc[4] = {rscale.x, rscale.y, rscale.z, rscale.w};
        const bool more = x + 1 < seg_end;
        // ---- S: R + sum_j scale_j D_j
        float s[kHalf];
        auto read = [&](float (&v)[kHalf], int d, uint32_t parity) {
          tc_wait(&d_full[d], parity, dead, gave_up);
          tc_after();
          tc_ld(tmem + lanes + NH * d + hb, v);
        };
        auto scaled = [&](float (&v)[kHalf], float f) {
          tc_landed(v);
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int h = 0; h < kHalf; h += 2) {
            const float2 w = fma2(make_float2(v[h], v[h + 1]), f2, make_float2(s[h], s[h + 1]));
            s[h] = w.x;
            s[h + 1] = w.y;
          }
        };
        auto freed = [&](int d) {
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_free[d]);
        };
        {
          float v[kHalf], w[kHalf];
          read(s, 0, 0u);
          tc_wait_ld();
          tc_landed(s);
          freed(0);
          read(v, 1, (uint32_t)(i & 1));
          read(w, 2, (uint32_t)(i & 1));
          tc_wait_ld();
          scaled(v, sc[0]);
          scaled(w, sc[1]);
          freed(1);
          if (lane == 0) mbar_arrive(&d_free[2]);
          read(v, 3, (uint32_t)(i & 1));
          read(w, 0, 1u);
          tc_wait_ld();
          scaled(v, sc[2]);
          scaled(w, sc[3]);
          freed(3);
          if (lane == 0) mbar_arrive(&d_free[0]);
        }
        // exponents (logits in base 2 less the reference, plus kPShift), weights
        float p[kHalf];
        auto exponents = [&]() {
#pragma unroll
          for (int h = 0; h < kHalf; h += 4) {
            const float4 c = *reinterpret_cast<const float4*>(xs + hb + h);
            const float4 m = *reinterpret_cast<const float4*>(ref + hb + h);
            const float2 v0 = fma2(make_float2(s[h], s[h + 1]), make_float2(c.x, c.y), make_float2(-m.x, -m.y));
            const float2 v1 = fma2(make_float2(s[h + 2], s[h + 3]), make_float2(c.z, c.w), make_float2(-m.z, -m.w));
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
        const float4 vr = *reinterpret_cast<const float4*>(vref);
        bool move = valid && (!started || over > kPShift + kPRoom || sc[0] > vr.x || sc[1] > vr.y ||
                              sc[2] > vr.z || sc[3] > vr.w);
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
          // too much (for the first rows that count, everywhere), the planes'
          // references to the tile's largest scales
          exponents();
          const float mx = lanes_reduce<kHalf, OpMax>(p);
          if ((lane * kHalf) % 32 == 0) red[quad * NH + hb + lane * kHalf / 32] = mx;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v = valid ? sc[j] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            if (lane == 0 && half == 0) vref[8 + 4 * j + quad] = v;
          }
          tc_barrier();
          if (tid < NH) {
            const float m = fmaxf(fmaxf(red[tid], red[NH + tid]), fmaxf(red[2 * NH + tid], red[3 * NH + tid]));
            const bool grow = started ? m > kPShift + kPRoom : m > -INFINITY;
            red[tid] = grow ? kPShift - m : 0.f;
            if (grow) ref[tid] += m - kPShift;
          }
          if (tid >= NH && tid < NH + 4) {
            const int j = tid - NH;
            const float old = vref[j];
            const float v = fmaxf(fmaxf(vref[8 + 4 * j], vref[9 + 4 * j]), fmaxf(vref[10 + 4 * j], vref[11 + 4 * j]));
            vref[4 + j] = v > old ? old / v : 1.0f;
            if (v > old) vref[j] = v;
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
            tc_wait(&pv_done[0], 1u, dead, gave_up);  // both tiles of weights of the tile before
            tc_wait(&pv_done[1], 1u, dead, gave_up);
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
              for (int e = 0; e < 32; ++e)
                v[e] *= ex2(red[(c + e) % NH]) * vref[4 + 2 * half + (c + e) / NH];
              tc_st32(at, v);
            }
            tc_wait_st();
          }
          started = true;
          tc_barrier();  // red is read
        }
#pragma unroll
        for (int h = 0; h < kHalf; h += 2) l[h / 2] = add2(l[h / 2], make_float2(p[h], p[h + 1]));
        // ---- a plane's weights: P times the row's scale over the reference.
        // How their rests are rounded is settled once for the four planes, as
        // the smallest factor asks for it (where the factors differ, larger
        // weights go by the row's place too, and keep 2^-7; for each plane by
        // itself, 62 tokens of up to 4,096 rows at 128 heads took 85.5 us, not 81.8).
        float f[4], least = 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float vj = vref[j];
          f[j] = valid && vj > 0.f ? __fdividef(sc[j], vj) : 0.f;
          least = fminf(least, f[j]);
        }
        const float limit = fminf(__fdividef(kSmallWeight, least), 448.0f);  // (least 0: infinity, or a NaN)
        const uint32_t limit2 = f16x2_of(limit, limit);
        uint32_t p16[kHalf / 2], rests[kHalf / 2];
#pragma unroll
        for (int h = 0; h < kHalf; h += 2) {
          p16[h / 2] = f16x2_of(p[h], p[h + 1]);
          rests[h / 2] = weight_round(p16[h / 2], limit2, dither);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = (q + 2) & 3;  // planes 2, 3, 0, 1
          const uint32_t f2 = f16x2_of(f[j], f[j]);
          uint32_t phi[kHalf / 4], plo[kHalf / 4];
#pragma unroll
          for (int h = 0; h < kHalf; h += 4) {
            split_weights(mul_f16x2(p16[h / 2], f2), mul_f16x2(p16[h / 2 + 1], f2), rests[h / 2], rests[h / 2 + 1],
                          &phi[h / 4], &plo[h / 4]);
          }
          // use 2 i + q / 2 of this weight tile: the one before it has been read
          if (i > 0 || q >= 2) tc_wait(&pv_done[q & 1], (uint32_t)(q >= 2 ? 0 : 1), dead, gave_up);
          if (!valid && half == (j & 1)) {
            // a row that is loaded but does not count holds anything, NaN codes
            // too: no value of it may meet a weight of zero
            uint4* d = reinterpret_cast<uint4*>(smem + S::oRing + ds_slot(i, j) * kPlane + pos * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = make_uint4(0, 0, 0, 0);
          }
          uint8_t* prow = smem + S::oP + (q & 1) * kPlane + pos * 128;
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
          if (lane == 0) mbar_arrive(&p_full[q & 1]);
        }
        if (more) {  // the next tile's row
          crow = attn_row(a, k, (x + 1 - k.start) * kTcTile + pos, &page);
          rscale = row_scales(crow);
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
        red[tid] = sum == 0.f ? 0.f : whole ? 1.0f / sum : 1.0f;
        if (!whole)
          attn_part_ml(a, h0 + tid)[slot] = make_float2(m, sum);
        else if (a.lse != nullptr && h0 + tid < a.heads)
          a.lse[(int64_t)k.t * a.heads + h0 + tid] = attn_lse(m, sum);
      }
      tc_barrier();
      tc_wait(&pv_done[0], 1u, dead, gave_up);
      tc_wait(&pv_done[1], 1u, dead, gave_up);
      tc_after();
      tc_store_out<NH>(a, k, tmem + lanes + 256, half, pos, h0, slot, whole, red, vref[2 * half],
                       vref[2 * half + 1]);
      tc_before();
      tc_barrier();  // red and vref are read
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

template <int NH, bool FP8Q, bool COPY>
cudaError_t launch_ds(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.workers * a.groups));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = DsSmem<NH, FP8Q>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_attn_ds_kernel<NH, FP8Q, COPY>, a, maps);
}

template <int NH>
cudaError_t launch_ds_heads(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
  const bool copy = maps.box_rows == 0;
  if (a.q_scale_inv != nullptr)
    return copy ? launch_ds<NH, true, true>(a, maps, stream) : launch_ds<NH, true, false>(a, maps, stream);
  return copy ? launch_ds<NH, false, true>(a, maps, stream) : launch_ds<NH, false, false>(a, maps, stream);
}

template <int NH, bool FP8Q>
cudaError_t prepare_ds() {
  cudaError_t e = cudaFuncSetAttribute(mla_attn_ds_kernel<NH, FP8Q, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, DsSmem<NH, FP8Q>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(mla_attn_ds_kernel<NH, FP8Q, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, DsSmem<NH, FP8Q>::kBytes);
  return e;
}
template <int NH>
cudaError_t prepare_ds_heads() {
  cudaError_t e = prepare_ds<NH, false>();
  return e == cudaSuccess ? prepare_ds<NH, true>() : e;
}

}  // namespace

cudaError_t prepare_attn_ds() {
  cudaError_t e = prepare_ds_heads<16>();
  if (e == cudaSuccess) e = prepare_ds_heads<32>();
  if (e == cudaSuccess) e = prepare_ds_heads<64>();
  return e;
}

cudaError_t launch_attn_ds(const AttnArgs& a, cudaStream_t stream) {
  TcMaps maps = {};
  maps.box_rows = plane_box_rows(a);
  // one map: the four latent planes and the rope values are 128-byte boxes
  if (maps.box_rows > 0 && !encode_plane_map(&maps.latent, a, kRowDs, 128, maps.box_rows)) return cudaErrorInvalidValue;
  maps.rope = maps.latent;
  switch (a.cta_heads) {
    case 16: return launch_ds_heads<16>(a, maps, stream);
    case 32: return launch_ds_heads<32>(a, maps, stream);
    default: return launch_ds_heads<64>(a, maps, stream);
  }
}

}  // namespace mla
