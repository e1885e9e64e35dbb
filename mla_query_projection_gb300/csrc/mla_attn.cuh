// mla_attn.cuh - what the attention kernels share: the plan that spreads the
// batch's cache tiles over the workers, and the positions of a tile.
#pragma once

#include "mla_rows.cuh"

namespace mla {
namespace {

constexpr int kAttnMaxBatch = MLA_MAX_BATCH;

// Tiles of the batch, spread evenly.  Token t's context is a list of virtual
// positions 0 .. nv_t - 1 (its first len_t positions, or the positions of its
// selected blocks, block after block), cut into tiles; start[t] is the number
// of tiles before it.  Worker w of a head group takes tiles
// [w * total / workers, (w + 1) * total / workers), whatever requests they
// belong to.  A stretch of one token's tiles that is not all of them leaves
// the worker as a partial: its first stretch in slot 0, any other (then its
// last) in slot 1.
struct AttnPlan {
  int64_t start[kAttnMaxBatch + 1];
};

// Virtual positions of token t, 0 for a token that looks at nothing.
__device__ __forceinline__ int64_t attn_positions(const AttnArgs& a, int t, bool flag) {
  const int64_t len = a.lens[t];
  if (len <= 0) return 0;
  const int row = a.token_row != nullptr ? a.token_row[t] : t;
  if (row < 0 || row >= a.table_rows) {
    if (flag) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    return 0;
  }
  if (a.sel != nullptr) {
    const int64_t n = min((int64_t)max(a.sel_count[t], 0), a.sel_stride);
    return n * a.page_size;
  }
  const int64_t cap = a.bt_stride * a.page_size;
  if (len > cap && flag) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
  return min(len, cap);
}

// Fills the plan; all threads of the block call it (at least 256 of them, a
// multiple of 32), and may read it after the closing barrier.
__device__ __forceinline__ void attn_make_plan(const AttnArgs& a, AttnPlan* p, int64_t* red,
                                               bool flag) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t n = 0;
  if (tid < a.batch) n = (attn_positions(a, tid, flag) + a.tile - 1) / a.tile;
  int64_t inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31 && warp < kAttnMaxBatch / 32) red[warp] = inc;
  __syncthreads();
  if (tid < kAttnMaxBatch) {
    for (int w = 0; w < warp; ++w) inc += red[w];
    if (tid < a.batch) p->start[tid + 1] = inc;
    if (tid == 0) p->start[0] = 0;
  }
  __syncthreads();
}

// Workers with work: no more than there are tiles, so that every one of them
// has a tile, and every worker between the first and the last of a token
// leaves a part of it.
__device__ __forceinline__ int attn_workers(const AttnArgs& a, int64_t total) {
  return (int)min((int64_t)a.workers, total);
}
__device__ __forceinline__ int64_t attn_worker_start(int64_t total, int workers, int w) {
  return total * w / workers;
}
// The worker whose range holds tile x: the largest w with start(w) <= x.
__device__ __forceinline__ int attn_worker_of(int64_t total, int workers, int64_t x) {
  return (int)(((x + 1) * workers - 1) / total);
}

// The token of tile x: the last t with start[t] <= x (tokens without tiles
// are passed over).
__device__ __forceinline__ int attn_token_of(const AttnPlan* p, int batch, int64_t x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p->start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The cache row (page * page_size + offset) of virtual position v of token t,
// or -1 where the position does not count; *page receives the page.
__device__ __forceinline__ int64_t attn_row(const AttnArgs& a, int t, int row, int64_t nv, int64_t len,
                                            int64_t v, int64_t* page) {
  if (v >= nv) return -1;
  int64_t j = v / a.page_size;
  const int off = (int)(v - j * a.page_size);
  if (a.sel != nullptr) {
    j = a.sel[(int64_t)t * a.sel_stride + j];
    if (j < 0 || j >= a.bt_stride || j * a.page_size + off >= len) return -1;
  }
  const int64_t p = a.table[(int64_t)row * a.bt_stride + j];
  if (p < 0 || p >= a.num_pages) {
    atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    return -1;
  }
  *page = p;
  return p * a.page_size + off;
}

// Natural logarithm of the sum of exponentials, from the maximum in base 2 and
// the sum relative to it.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return m == -INFINITY && l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

}  // namespace
}  // namespace mla
