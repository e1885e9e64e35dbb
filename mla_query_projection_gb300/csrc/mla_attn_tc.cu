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
//    P is the sum of an E4M3 and an E5M2 term, two MMAs into one accumulator:
//    4 + 3 bits, 2^-7 of a weight, down to 2^-10 of the largest; below, 2^-17 of
//    the largest, rounded so that thousands of alike small weights beside a
//    dominant one keep their sum (split_weights).
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
// HBM's share of 73.7 KiB a tile; measured, 3,650 cycles a tile, and 44 us for 8
// tokens of 16,384 rows at 128 heads (the tensor pipe 39 % active, plan, queries,
// first tiles, sums and their joining included).
#include "mla_attn_tc.cuh"

namespace mla {
namespace {

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

template <int NH, bool FP8Q, int LAYOUT, bool COPY>
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
  uint32_t* gave_up = reinterpret_cast<uint32_t*>(smem + S::oTmem + 4);  // a softmax wait ran out
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
  if (tid == kTcSoft) {
    prefetch_tensormap(&maps.latent);
    prefetch_tensormap(&maps.rope);
  }
  pdl_wait();
  pdl_launch_dependents();  // (after the wait: the join reads the lengths before its own)
  tc_before();
  // (the plan's barriers order the set-up above)
  AttnSeen* seen = reinterpret_cast<AttnSeen*>(smem + S::oP);  // until the first weights
  attn_make_plan(a, plan, reinterpret_cast<uint32_t*>(smem + S::oScan), blockIdx.x == 0, seen);
  tc_after();
  const uint32_t tmem = uniform(*tslot);  // S^T buffers at columns 0 and 128, O^T planes from 256
  uint32_t first, end;
  attn_range(a, plan, worker, &first, &end);
  bool dead = false;

  if (warp == 8) {
    // ================= TMA: a tile's planes in the order rope, 0, 1, 2, 3
    if constexpr (COPY) {
      auto place = [&](int n, int p) {
        const int s = 4 * (n & 1) + p - 1;
        return p == 0 ? TcSlot{rope_full, rope_empty, (uint32_t)n, smem + S::oRope}
                      : TcSlot{&full[s], &empty[s], (uint32_t)n >> 1, smem + S::oRing + s * kPlane};
      };
      tc_copy_tiles<kRowE4m3, 64, kKvLora>(a, plan, seen, first, end, lane, dead, place);
    } else {
      const int boxes = kTcTile / maps.box_rows;
      const int32_t no_row = (int32_t)(a.num_pages * a.page_size);  // past the end: zeros
      int i = 0, issued = 0;  // tiles, planes
      uint32_t x = first;
      while (x < end && !dead) {
        // (the first token's weights come after its queries and a tile of its
        // rows: this warp has read `seen` by then)
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
        // 32 rows a step: 4096 bytes of V and of P; P's second term 64 bytes on
        tc_mma4x2<256, 256, 4>(tmem + 256 + NH * j, da + j * kPl, dp, id_hi, id_lo, add);
        tc_commit(&empty[4 * b + j]);
      }
      tc_commit(pv_done);
    };
    // A wait that ran out ends no loop here (the loops are then the warp's, and
    // the descriptors stay in uniform registers): the MMAs go on over whatever
    // the planes hold, and the results do not count.
    const uint32_t x1 = uniform(end), lead = uniform(plan->lead);
    uint32_t x = uniform(first), seg_end = x;
    int segs = 0;
    uint32_t add = 0;  // whether the tile before added to its O^T
    bool due = false;  // its PV is still to be issued
    int i = 0;
    for (; x < x1; ++i, ++x) {
      const int b = i & 1;
      const bool fresh = x == seg_end;
      if (fresh) {
        const int t = attn_token_of(plan, a.batch, x);
        if (i > 0) x += lead;
        seg_end = uniform(plan->end[t]);
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
        tc_mma4<2, 2>(d, da + j * kPl, dq + j * kQPl, id_s, 1u);
      }
      tc_commit(&s_full[b]);
      if (due) pv(i - 1, add);
      due = true;
      add = fresh ? 0u : 1u;
    }
    if (due) pv(i - 1, add);
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
    // pass the same barriers to the end.  (It says so, and from then on none takes
    // the path that only some votes take.)
    while (x < end) {
      const AttnToken k = attn_token(a, plan, x, i == 0 ? seen : nullptr);
      x = max(x, k.start);
      const uint32_t seg0 = x, seg_end = min(k.end, end);
      tc_queries<NH, FP8Q, false>(a, smem + S::oQ, smem + S::oQr, k.t, h0, warp, lane, logit, xs);
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
        const uint32_t dither = weight_dither(pos, x - k.start);
        tc_wait(&s_full[b], (uint32_t)((i >> 1) & 1), dead, gave_up);
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
            const uint32_t w0 = f16x2_of(p0.x, p0.y), w1 = f16x2_of(p1.x, p1.y);
            split_weights(w0, w1, weight_round(w0, kSmallWeight16, dither), weight_round(w1, kSmallWeight16, dither),
                          &phi[h / 4], &plo[h / 4]);
          }
        };
        exponents();
        // A page's scale relative to the one that values are kept over, base 2:
        // a weight times it must stay in E4M3's range.  (That scale is the
        // first tile's largest, and stays.  While it grew with every larger page
        // scale, O was rescaled as often: 8 tokens, 128 heads, 32 pages of 64
        // selected, scales within a factor of 8 took 25.6 us, so 21.0.)
        const bool first_rows = !started || (kPaged && vref[0] == 0.f);
        // (At least -32: the denominators' terms stay far from FP32's limits.)
        const float up = kPaged && !first_rows ? fmaxf(__log2f(fabsf(rscale) / vref[0]), -32.0f) : 0.f;
        float over = fmaxf(s[0], s[1]);
#pragma unroll
        for (int h = 2; h < kHalf; h += 2) over = fmaxf(over, fmaxf(s[h], s[h + 1]));
        // Does the reference have to move?  The warps' answers meet while the
        // weights are computed as if not (unless there is no reference yet).
        const bool move = __any_sync(0xFFFFFFFFu, valid && (first_rows || over + up > kPShift + kPRoom));
        __syncwarp();  // (what a lane has said by gave_up goes before the arrival)
        if (lane == 0) {
          if (move) *reinterpret_cast<volatile uint32_t*>(&moved[b]) = (uint32_t)i + 1;
          mbar_arrive(voted);
        }
        if (started) weights();
        tc_wait_votes(voted, (uint32_t)(i & 1), dead, gave_up);
        if (*reinterpret_cast<volatile uint32_t*>(&moved[b]) == (uint32_t)i + 1 &&
            *reinterpret_cast<volatile uint32_t*>(gave_up) == 0u) {
          // the reference moves to the tile's maximum where that passes it by
          // too much (for the first rows that count, everywhere)
          if (started) exponents();
          if (kPaged && !first_rows) {
#pragma unroll
            for (int h = 0; h < kHalf; ++h) s[h] += up;
          }
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
          if (kPaged && tid == NH && first_rows)  // (O is zero so far)
            vref[0] = fmaxf(fmaxf(vref[4], vref[5]), fmaxf(vref[6], vref[7]));
          tc_barrier();
#pragma unroll
          for (int h = 0; h < kHalf; ++h) {
            const float d = red[hb + h];
            s[h] += d;
            float& lh = h & 1 ? l[h / 2].y : l[h / 2].x;
            if (started) lh *= ex2(d);
          }
          if (kPaged && !first_rows) exponents();  // s has `up` in it
          if (started && x > seg0) {
            tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead, gave_up);
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
              for (int e = 0; e < 32; ++e) v[e] *= ex2(red[(c + e) % NH]);
              tc_st32(at, v);
            }
            tc_wait_st();
          }
          started = true;
          weights();
          tc_barrier();  // red is read
        } else if (!started) {
          weights();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
#pragma unroll
        for (int h = 0; h < kHalf; h += 2) l[h / 2] = add2(l[h / 2], make_float2(s[h], s[h + 1]));
        // the previous tile's PV has read P
        if (i > 0) tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead, gave_up);
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
          red[tid] = sum == 0.f ? 0.f : 1.0f / sum;
          if (a.lse != nullptr && h0 + tid < a.heads)
            a.lse[(int64_t)k.t * a.heads + h0 + tid] = attn_lse(m, sum);
        } else {
          red[tid] = sum == 0.f ? 0.f : 1.0f;
          attn_part_ml(a, h0 + tid)[slot] = make_float2(m, sum);
        }
      }
      tc_barrier();
      tc_wait(pv_done, (uint32_t)((i - 1) & 1), dead, gave_up);
      tc_after();
      tc_store_out<NH>(a, k, tmem + lanes + 256, half, pos, h0, slot, whole, red, vref[0], vref[0]);
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

template <int NH, bool FP8Q, int LAYOUT, bool COPY>
cudaError_t launch_tc_kernel(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, mla_attn_tc_kernel<NH, FP8Q, LAYOUT, COPY>, a, maps);
}

template <int NH, bool FP8Q, int LAYOUT>
cudaError_t launch_tc(const AttnArgs& a, const TcMaps& maps, cudaStream_t stream) {
  return maps.box_rows == 0 ? launch_tc_kernel<NH, FP8Q, LAYOUT, true>(a, maps, stream)
                            : launch_tc_kernel<NH, FP8Q, LAYOUT, false>(a, maps, stream);
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
  cudaError_t e = cudaFuncSetAttribute(mla_attn_tc_kernel<NH, FP8Q, LAYOUT, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<NH, FP8Q>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(mla_attn_tc_kernel<NH, FP8Q, LAYOUT, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<NH, FP8Q>::kBytes);
  return e;
}
template <int NH>
cudaError_t prepare_tc_heads() {
  cudaError_t e = prepare_tc<NH, false, MLA_KV_FP8_E4M3>();
  if (e == cudaSuccess) e = prepare_tc<NH, false, MLA_KV_FP8_E4M3_PAGE>();
  if (e == cudaSuccess) e = prepare_tc<NH, true, MLA_KV_FP8_E4M3>();
  if (e == cudaSuccess) e = prepare_tc<NH, true, MLA_KV_FP8_E4M3_PAGE>();
  return e;
}

}  // namespace

cudaError_t prepare_attn_tc() {
  cudaError_t e = prepare_tc_heads<16>();
  if (e == cudaSuccess) e = prepare_tc_heads<32>();
  if (e == cudaSuccess) e = prepare_tc_heads<64>();
  return e;
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream) {
  TcMaps maps = {};
  maps.box_rows = plane_box_rows(a);
  if (maps.box_rows > 0 && (!encode_plane_map(&maps.latent, a, kRowE4m3, 128, maps.box_rows) ||
                            !encode_plane_map(&maps.rope, a, kRowE4m3, 64, maps.box_rows)))
    return cudaErrorInvalidValue;
  switch (a.cta_heads) {
    case 16: return launch_tc_heads<16>(a, maps, stream);
    case 32: return launch_tc_heads<32>(a, maps, stream);
    default: return launch_tc_heads<64>(a, maps, stream);
  }
}

}  // namespace mla
