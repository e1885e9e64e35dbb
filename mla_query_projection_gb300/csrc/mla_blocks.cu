// mla_blocks.cu - the selection of cache blocks (pages) for sparse attention:
// the mean key of a block (mla_blocks_mean), the score of every block for
// every query (mla_blocks_score) and the best-scored blocks of a query
// (mla_blocks_select).
#include <cuda_bf16.h>

#include "../../include/mla_query.h"
#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_rows.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------------- means
//
// mean[p][c] = bf16((sum over the page's filled rows of key[c]) / rows), the
// sum in FP32.  It reads each filled row once and writes 1152 bytes a page:
// bound by HBM.  One CTA a page: chunk c of the row (16 bytes) belongs to one
// thread of each of kGroups row groups, so a warp reads consecutive bytes of
// a row, and the groups' sums meet in shared memory in a fixed order.  FP16
// values (E4M3 codes, E2M1 times its scale) are added to the FP32 sums as they
// are (converted first, 8 prompts of 9,001 to 16,384 tokens took 17.6 us, not
// 16.6; with the present grid 15.5, where the rows' bytes are 8.9).

template <int LAYOUT>
struct MeanShape {
  static constexpr int kChunks = RowChunks<LAYOUT>::kChunks;
  static constexpr int kGroups = kChunks > 20 ? 8 : 14;
  static constexpr int kThreads = kChunks * kGroups;
  static constexpr int kDeep = kChunks > 20 ? 8 : 5;  // rows a thread has in flight (a 64-row page)
};

template <int LAYOUT>
__global__ void __launch_bounds__(MeanShape<LAYOUT>::kThreads)
    mla_blocks_mean_kernel(const MeanArgs m) {
  using R = RowChunks<LAYOUT>;
  using M = MeanShape<LAYOUT>;
  __shared__ float sums[M::kGroups][kRowElems];
  const int tid = threadIdx.x, chunk = tid % M::kChunks, group = tid / M::kChunks;
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.y;
  const int64_t ps = m.page_size;
  const int64_t cap = m.bt_cols * ps;
  const int64_t from = max(0, m.lens_from[r]), to = min((int64_t)m.lens_to[r], cap);
  for (int64_t j = from / ps + blockIdx.x; j * ps < to; j += gridDim.x) {
    const int64_t page = m.block_table[(int64_t)r * m.bt_stride + j];
    if (page < 0 || page >= m.num_pages) {
      if (tid == 0 && m.flags != nullptr) atomicOr(m.flags, MLA_DEVERR_BAD_SLOT);
      continue;  // the same for the whole CTA
    }
    const int filled = (int)min(ps, to - j * ps);
    const uint8_t* base = m.cache + page * ps * R::kBytes;
    float acc[R::kMax];
#pragma unroll
    for (int i = 0; i < R::kMax; ++i) acc[i] = 0.f;
    for (int t0 = group; t0 < filled; t0 += M::kGroups * M::kDeep) {
      uint4 w[M::kDeep];
#pragma unroll
      for (int d = 0; d < M::kDeep; ++d) {
        const int t = t0 + d * M::kGroups;
        if (t < filled)
          w[d] = *reinterpret_cast<const uint4*>(base + (int64_t)t * R::kBytes + R::offset(chunk));
      }
#pragma unroll
      for (int d = 0; d < M::kDeep; ++d) {
        const int t = t0 + d * M::kGroups;
        if (t < filled) R::add(base + (int64_t)t * R::kBytes, chunk, w[d], acc);
      }
    }
    const int col = R::col(chunk), width = R::width(chunk);
#pragma unroll
    for (int i = 0; i < R::kMax; ++i)
      if (i < width) sums[group][col + i] = acc[i];
    __syncthreads();
    const float mul = page_scale(m.k_scale, LAYOUT, page) / (float)filled;
    for (int c = 2 * tid; c < kRowElems; c += 2 * M::kThreads) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int g = 0; g < M::kGroups; ++g) {
        a += sums[g][c];
        b += sums[g][c + 1];
      }
      *reinterpret_cast<uint32_t*>(m.mean + page * kRowElems + c) = pack_bf16x2(a * mul, b * mul);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ scores
//
// score[t][j] = max over heads h of q[t][h] . mean[page of block j], FP32
// accumulation of exact BF16 products (FP8 queries are exact in BF16; their
// scale divides the result).  One CTA takes kTile blocks of one token: their
// means go to shared memory once, and its eight warps take 16 heads at a time
// straight from global memory (mma.sync m16n8k16).  The order of k inside a
// 32-column step is permuted the same way on both sides, so that each lane's
// share of a row is 16 contiguous bytes: two k16 steps a 16-byte load.

template <bool FP8Q>
struct ScoreWords {
  using type = uint4;
};
template <>
struct ScoreWords<true> {
  using type = uint2;
};

constexpr int kScorePitch = kRowElems * 2 + 64;  // 1216: 16-byte loads of 8 rows x 4 free of conflicts

// EARLY (one CTA an SM): a warp's first queries are loaded whole before the
// blocks' pages are looked up, and wait in registers (one query over 1,024
// blocks, 64 heads, call after call: 7.8 us, so 4.8).

template <int NT, bool FP8Q, bool EARLY>
__global__ void __launch_bounds__(256) mla_blocks_score_kernel(const ScoreArgs s) {
  constexpr int kTile = 8 * NT;
  extern __shared__ __align__(16) uint8_t keys[];  // [kTile][kScorePitch]
  __shared__ float best[8][kTile];
  __shared__ int64_t pages[kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.y;
  const int64_t ps = s.page_size;
  const int row = s.token_row != nullptr ? s.token_row[t] : t;
  int64_t nb = (max(0, s.lens[t]) + ps - 1) / ps;
  nb = min(nb, s.bt_stride);
  if (row < 0 || row >= s.table_rows) {
    if (nb > 0 && tid == 0 && s.flags != nullptr) atomicOr(s.flags, MLA_DEVERR_BAD_SLOT);
    nb = 0;
  }
  constexpr int kB = FP8Q ? 1 : 2;  // bytes per query element
  using Words = typename ScoreWords<FP8Q>::type;  // a lane's share of a row's 32 columns
  // heads h0 + g and h0 + g + 8, columns 32 k ..; heads past the last repeat the last
  auto query = [&](int h0, int k, Words* wa, Words* wb) {
    const int ha = min(h0 + g, s.heads - 1), hb = min(h0 + g + 8, s.heads - 1);
    const uint8_t* base = k < 16 ? s.q_latent : s.q_pe;
    const int64_t ts = k < 16 ? s.ql_ts : s.qp_ts, hs = k < 16 ? s.ql_hs : s.qp_hs;
    const int64_t at = (int64_t)t * ts + 32 * (k < 16 ? k : k - 16) + 8 * q4;
    *wa = *reinterpret_cast<const Words*>(base + (at + ha * hs) * kB);
    *wb = *reinterpret_cast<const Words*>(base + (at + hb * hs) * kB);
  };
  constexpr int kAll = kRowElems / 32;
  Words qa[EARLY ? kAll : 1], qb[EARLY ? kAll : 1];
  if constexpr (EARLY) {
#pragma unroll
    for (int k = 0; k < kAll; ++k) query(16 * warp, k, &qa[k], &qb[k]);
  }
  const int64_t j0 = (int64_t)blockIdx.x * kTile;
  float* out = s.scores + (int64_t)t * s.scores_stride;
  if (j0 >= nb) {
    for (int j = tid; j < kTile; j += 256)
      if (j0 + j < s.bt_stride) out[j0 + j] = -INFINITY;
    return;
  }
  if (tid < kTile) {
    int64_t page = -1;
    if (j0 + tid < nb) {
      page = s.block_table[(int64_t)row * s.bt_stride + j0 + tid];
      if (page < 0 || page >= s.num_pages) {
        page = -1;
        if (s.flags != nullptr) atomicOr(s.flags, MLA_DEVERR_BAD_SLOT);
      }
    }
    pages[tid] = page;
  }
  __syncthreads();
  // the means by 16-byte asynchronous copies, all in flight at once; with 16
  // blocks a CTA, where the call is a chain of latencies, the first third of
  // their columns is used while the others come (1,024 blocks, 64 heads: 5.6 us,
  // so 4.9; with 64 blocks a CTA 13.4 became 14.4)
  constexpr int kParts = NT == 2 ? 3 : 1;
  constexpr int kPart = kRowElems / 8 / kParts, kSteps = kRowElems / 32 / kParts;
#pragma unroll 1
  for (int part = 0; part < kParts; ++part) {
    for (int c = tid; c < kTile * kPart; c += 256) {
      const int b = c / kPart, k = part * kPart + c % kPart;
      uint8_t* d = keys + b * kScorePitch + 16 * k;
      if (pages[b] >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d)),
                     "l"(s.mean + pages[b] * kRowElems + 8 * k)
                     : "memory");
      else
        *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  float mx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
  if constexpr (kParts == 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
  }
  // (with parts, every warp passes the barriers of the first 16 heads, whether it has them or not)
  for (int h0 = 16 * warp; h0 < s.heads || (kParts > 1 && h0 < 128); h0 += 128) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll NT == 2 && !EARLY ? 6 : kAll
    for (int k = 0; k < kRowElems / 32; ++k) {
      if (kParts > 1 && h0 < 128 && k % kSteps == 0) {
        if (k == 0)
          asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (k == kSteps)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
      }
      Words wa, wb;
      if (EARLY && h0 < 128) {
        wa = qa[EARLY ? k : 0];
        wb = qb[EARLY ? k : 0];
      } else {
        query(h0, k, &wa, &wb);
      }
      uint4 va, vb;
      if constexpr (FP8Q) {
        float f[8], h[8];
        e4m3x4_values(wa.x, f);
        e4m3x4_values(wa.y, f + 4);
        e4m3x4_values(wb.x, h);
        e4m3x4_values(wb.y, h + 4);
        va = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
        vb = make_uint4(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]),
                        pack_bf16x2(h[6], h[7]));
      } else {
        va = wa;
        vb = wb;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 kv =
            *reinterpret_cast<const uint4*>(keys + (8 * n + g) * kScorePitch + 64 * k + 16 * q4);
        mma_bf16_16816(acc[n], va.x, vb.x, va.y, vb.y, kv.x, kv.y);
        mma_bf16_16816(acc[n], va.z, vb.z, va.w, vb.w, kv.z, kv.w);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // NaN wins, as it does in a maximum over the heads
      const float x = acc[n][0], y = acc[n][2], z = acc[n][1], w = acc[n][3];
      const float c0 = isnan(x) || isnan(y) ? NAN : fmaxf(x, y);
      const float c1 = isnan(z) || isnan(w) ? NAN : fmaxf(z, w);
      mx[n][0] = isnan(mx[n][0]) || isnan(c0) ? NAN : fmaxf(mx[n][0], c0);
      mx[n][1] = isnan(mx[n][1]) || isnan(c1) ? NAN : fmaxf(mx[n][1], c1);
    }
  }
  // the maximum over the 8 rows a column has in the warp, then over the warps
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = mx[n][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = isnan(u) || isnan(v) ? NAN : fmaxf(u, v);
      }
      if (g == 0) best[warp][8 * n + 2 * q4 + e] = v;
    }
  __syncthreads();
  const float inv = FP8Q ? *s.q_scale_inv : 1.0f;
  for (int j = tid; j < kTile; j += 256) {
    if (j0 + j >= s.bt_stride) continue;
    float v = best[0][j];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float u = best[w][j];
      v = isnan(u) || isnan(v) ? NAN : fmaxf(u, v);
    }
    if (FP8Q) v = v / inv;
    out[j0 + j] = pages[j] >= 0 ? v : -INFINITY;
  }
}

// --------------------------------------------------------------- selection
//
// The k blocks with the highest scores, ascending.  A score becomes a 32-bit
// key that orders like it; the k-th largest key is found by its leading 11,
// then 11, then 10 bits, each digit from a histogram of the keys that share
// the bits so far (2,048 bins: in the two later digits the keys of a warp seldom
// meet in one; the first is the sign, the exponent and two bits, of which alike
// scores fill few); then one pass in block order keeps every key above it and, of those
// equal, the first ones.  All sums are counts, so the result does not depend
// on the order of the atomics.  Keys stay in registers (up to 16 a thread;
// beyond 8,192 blocks they are formed again from the scores in each pass).
// Bound by latency: the barriers of the passes.

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16;  // a thread, in registers
constexpr int kSelBins = 2048;

__device__ __forceinline__ uint32_t score_key(float v, bool forced) {
  if (forced) v = INFINITY;
  if (isnan(v)) v = -INFINITY;
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0;  // -0 ties with +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <bool REGS>
__global__ void __launch_bounds__(kSelThreads, 2) mla_blocks_select_kernel(const SelectArgs s) {
  __shared__ __align__(16) uint32_t hist[kSelBins];
  __shared__ uint32_t counts[kSelWarps], pick_bin, pick_above, pick_all;
  __shared__ uint32_t place[kSelKeys * kSelWarps];  // (chunk, warp): above << 16 | equal
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  reinterpret_cast<uint4*>(hist)[tid] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  const int t = blockIdx.x;
  const float* sc = s.scores + (int64_t)t * s.scores_stride;
  int32_t* out = s.sel + (int64_t)t * s.sel_stride;
  const int64_t ps = s.page_size;
  const int n = (int)min((max((int64_t)s.lens[t], (int64_t)0) + ps - 1) / ps, (int64_t)s.max_blocks);
  const int k = min(s.k, n);
  const int last0 = n - s.keep_last;
  auto key_at = [&](int j) { return score_key(sc[j], j < s.keep_first || j >= last0); };
  uint32_t keys[REGS ? kSelKeys : 1];
  if (REGS) {
#pragma unroll
    for (int c = 0; c < kSelKeys; ++c) {
      const int j = c * kSelThreads + tid;
      keys[REGS ? c : 0] = j < n ? key_at(j) : 0u;
    }
  }
  for (int j = k + tid; j < s.k; j += kSelThreads) out[j] = -1;
  if (tid == 0) s.sel_count[t] = k;
  if (k == n) {
    for (int j = tid; j < n; j += kSelThreads) out[j] = j;
    return;
  }
  uint32_t kth = 0, need = (uint32_t)k;  // the bits found; keys needed among those that share them
  __syncthreads();                       // hist is clear
  int shift = 21, bits = 11;
  while (true) {
    const uint32_t mask = shift == 21 ? 0u : 0xFFFFFFFFu << (shift + bits);
    auto put = [&](uint32_t key) {
      if ((key & mask) == kth) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
    };
    if (REGS) {
#pragma unroll
      for (int c = 0; c < kSelKeys; ++c)
        if (c * kSelThreads + tid < n) put(keys[REGS ? c : 0]);
    } else {
      for (int j = tid; j < n; j += kSelThreads) put(key_at(j));
    }
    __syncthreads();
    // this thread's four bins, counted from the top, and cleared for the next pass
    uint4* mine = reinterpret_cast<uint4*>(hist) + (kSelThreads - 1 - tid);
    const uint4 h = *mine;
    *mine = make_uint4(0, 0, 0, 0);
    const uint32_t c[4] = {h.w, h.z, h.y, h.x};
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) counts[warp] = inc;
    __syncthreads();
    uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? counts[lane & (kSelWarps - 1)] : 0u);
    before += inc - sum;
    if (before < need && before + sum >= need) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < need && before + c[e] >= need) {
          pick_bin = (uint32_t)(kSelBins - 1 - 4 * tid - e);
          pick_above = before;
          pick_all = before + c[e] == need;  // the whole bin is in
        }
        before += c[e];
      }
    }
    __syncthreads();
    kth |= pick_bin << shift;
    need -= pick_above;
    if (pick_all || shift == 0) break;
    if (shift == 21) {
      shift = 10;
    } else {
      shift = 0;
      bits = 10;
    }
  }
  // Keys above the bits found (those that share them are `equal`, and where the
  // search stopped early all of them are in) ...
  const uint32_t low = shift == 0 ? 0u : (1u << shift) - 1u;
  const uint32_t top = kth | low;
  // ... and of those equal the first `need`.
  uint32_t base = 0, ties = 0;
  const uint32_t below = (1u << lane) - 1u;
  for (int j00 = 0; j00 < n; j00 += kSelKeys * kSelThreads) {
    uint32_t bg[kSelKeys], be[kSelKeys];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kSelKeys; ++c) {
      const int j = j00 + c * kSelThreads + tid;
      const uint32_t key = REGS ? keys[REGS ? c : 0] : j < n ? key_at(j) : 0u;
      bg[c] = __ballot_sync(0xFFFFFFFFu, j < n && key > top);
      be[c] = __ballot_sync(0xFFFFFFFFu, j < n && key >= kth && key <= top);
      if (lane == 0) place[c * kSelWarps + warp] = (uint32_t)__popc(bg[c]) << 16 | __popc(be[c]);
    }
    __syncthreads();
    // exclusive sums over (chunk, warp), by the first warp, eight entries a lane
    uint32_t sum_all = 0;
    if (warp == 0) {
      uint32_t v[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = place[8 * lane + e];
        sum += v[e];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      uint32_t ex = inc - sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        place[8 * lane + e] = ex;
        ex += v[e];
      }
      sum_all = __shfl_sync(0xFFFFFFFFu, inc, 31);
      if (lane == 0) pick_all = sum_all;
    }
    __syncthreads();
    sum_all = pick_all;
#pragma unroll
    for (int c = 0; c < kSelKeys; ++c) {
      const int j = j00 + c * kSelThreads + tid;
      const uint32_t at = place[c * kSelWarps + warp];
      const uint32_t g = base + (at >> 16) + __popc(bg[c] & below);
      const uint32_t e = ties + (at & 0xFFFFu) + __popc(be[c] & below);
      if (bg[c] >> lane & 1u) out[g + min(e, need)] = j;
      if ((be[c] >> lane & 1u) && e < need) out[g + e] = j;
    }
    base += sum_all >> 16;
    ties += sum_all & 0xFFFFu;
  }
}

}  // namespace

cudaError_t launch_blocks_mean(const MeanArgs& m, int num_sms, cudaStream_t stream) {
  // Four CTAs an SM in all, but no more a row than it can have blocks; six for
  // few rows, which then have many blocks each, in unequal numbers (8 prompts of
  // 9,001 to 16,384 tokens: 16.6 us with four, 15.5 with six or eight; 64 rows
  // of one new token: 4.0 and 4.2).
  const int64_t per_sm = m.rows <= 16 ? 6 : 4;
  int64_t gx = (per_sm * num_sms + m.rows - 1) / m.rows;
  if (gx > m.bt_cols) gx = m.bt_cols;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)gx, (unsigned)m.rows, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (m.layout) {
    case MLA_KV_FP8_E4M3:
      cfg.blockDim = dim3(MeanShape<MLA_KV_FP8_E4M3>::kThreads);
      return cudaLaunchKernelEx(&cfg, mla_blocks_mean_kernel<MLA_KV_FP8_E4M3>, m);
    case MLA_KV_FP8_E4M3_PAGE:
      cfg.blockDim = dim3(MeanShape<MLA_KV_FP8_E4M3_PAGE>::kThreads);
      return cudaLaunchKernelEx(&cfg, mla_blocks_mean_kernel<MLA_KV_FP8_E4M3_PAGE>, m);
    case MLA_KV_FP8_DS_MLA:
      cfg.blockDim = dim3(MeanShape<MLA_KV_FP8_DS_MLA>::kThreads);
      return cudaLaunchKernelEx(&cfg, mla_blocks_mean_kernel<MLA_KV_FP8_DS_MLA>, m);
    default:
      cfg.blockDim = dim3(MeanShape<MLA_KV_NVFP4_DS_MLA>::kThreads);
      return cudaLaunchKernelEx(&cfg, mla_blocks_mean_kernel<MLA_KV_NVFP4_DS_MLA>, m);
  }
}

namespace {
template <int NT, bool FP8Q, bool EARLY>
cudaError_t launch_score(const ScoreArgs& s, cudaStream_t stream) {
  constexpr int kBytes = 8 * NT * kScorePitch;
  auto kernel = mla_blocks_score_kernel<NT, FP8Q, EARLY>;
  if constexpr (kBytes > 40 * 1024) {  // beyond the default limit, on the device in use
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((s.bt_stride + 8 * NT - 1) / (8 * NT)), (unsigned)s.batch, 1);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, s);
}
}  // namespace

cudaError_t launch_blocks_score(const ScoreArgs& s, int num_sms, cudaStream_t stream) {
  // A CTA reads its token's queries once (128 heads: 147 KB), whatever its
  // tile: 64 blocks where that still fills the SMs, 16 blocks for few tokens.
  // (64 tokens of up to 256 blocks at 128 heads: 17.5 us with 16 blocks, 1,024
  // CTAs reading 150 MB of queries.)
  const bool large = (s.bt_stride + 63) / 64 * s.batch >= num_sms;
  const bool early = (s.bt_stride + 15) / 16 * s.batch <= num_sms;  // CTAs of 16 blocks
  if (s.q_scale_inv != nullptr)
    return large ? launch_score<8, true, false>(s, stream)
           : early ? launch_score<2, true, true>(s, stream)
                   : launch_score<2, true, false>(s, stream);
  return large ? launch_score<8, false, false>(s, stream)
         : early ? launch_score<2, false, true>(s, stream)
                 : launch_score<2, false, false>(s, stream);
}

cudaError_t launch_blocks_select(const SelectArgs& s, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)s.batch);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return s.max_blocks <= kSelKeys * kSelThreads
             ? cudaLaunchKernelEx(&cfg, mla_blocks_select_kernel<true>, s)
             : cudaLaunchKernelEx(&cfg, mla_blocks_select_kernel<false>, s);
}

}  // namespace mla
