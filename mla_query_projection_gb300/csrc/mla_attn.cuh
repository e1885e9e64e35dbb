// mla_attn.cuh - what the attention kernels share: the plan that spreads the
// batch's cache tiles over the workers, and the positions of a tile.
#pragma once

#include "mla_rows.cuh"

namespace mla {
namespace {

constexpr int kAttnMaxBatch = MLA_MAX_BATCH;
constexpr uint32_t kAttnTile = 128;  // positions a tile

// Tiles of the batch, spread evenly.  Token t's context is a list of virtual
// positions 0 .. nv_t - 1 (its first len_t positions, or the positions of its
// selected blocks, block after block), cut into tiles; end[t] is the number of
// tiles up to and with its own.  Worker w of a head group takes tiles
// [w * total / workers, (w + 1) * total / workers), whatever requests they
// belong to.  A stretch of one token's tiles that is not all of them leaves
// the worker as a partial: its first stretch in slot 0, any other (then its
// last) in slot 1.
struct AttnPlan {
  uint32_t end[kAttnMaxBatch];
  __device__ uint32_t start(int t) const { return t > 0 ? end[t - 1] : 0u; }
};
// Positions of one token beyond this are left out (and flagged): 256 tokens'
// tiles stay within 31 bits.
constexpr int64_t kAttnMaxPositions = (int64_t)1 << 29;

// What a token looks at.
struct AttnToken {
  int t, row;
  uint32_t start, end;  // its tiles
  uint32_t nv;          // virtual positions
  int32_t len;
};

// Virtual positions of a token, 0 for one that looks at nothing.
__device__ __forceinline__ uint32_t attn_positions(const AttnArgs& a, int t, int32_t len, int row,
                                                   bool flag) {
  if (len <= 0) return 0;
  bool bad = row < 0 || row >= a.table_rows;
  int64_t n = 0;
  if (!bad) {
    const int64_t cap = a.bt_stride * a.page_size;
    if (a.sel != nullptr) {
      n = min((int64_t)max(a.sel_count[t], 0), a.sel_stride) * a.page_size;
    } else {
      n = min((int64_t)len, cap);
      bad = len > cap;
    }
    if (n > kAttnMaxPositions) {
      n = kAttnMaxPositions;
      bad = true;
    }
  }
  if (bad && flag) atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
  return (uint32_t)n;
}

// The tokens' lengths, rows and positions as the plan read them, kept where
// there is room until the first tile: a worker's first token needs no second
// trip to memory.
struct AttnSeen {
  int32_t len[kAttnMaxBatch], row[kAttnMaxBatch];
  uint32_t nv[kAttnMaxBatch];
};

// Fills the plan; all threads of the block call it (at least 256 of them, a
// multiple of 32), and may read it after the closing barrier.  red: 8 words.
__device__ __forceinline__ void attn_make_plan(const AttnArgs& a, AttnPlan* p, uint32_t* red,
                                               bool flag, AttnSeen* seen = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t n = 0;
  if (tid < a.batch) {
    const int32_t len = a.lens[tid];
    const int row = a.token_row != nullptr ? a.token_row[tid] : tid;
    const uint32_t nv = attn_positions(a, tid, len, row, flag);
    n = (nv + kAttnTile - 1) / kAttnTile;
    if (seen != nullptr) {
      seen->len[tid] = len;
      seen->row[tid] = row;
      seen->nv[tid] = nv;
    }
  }
  uint32_t inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31 && warp < kAttnMaxBatch / 32) red[warp] = inc;
  __syncthreads();
  if (tid < kAttnMaxBatch) {
    for (int w = 0; w < warp; ++w) inc += red[w];
    p->end[tid] = inc;
    // one CTA leaves the plan for the kernel that joins the parts
    if (flag) a.plan[tid] = inc;
  }
  __syncthreads();
}

// Workers with work: the fewest for which the busiest has no more tiles than
// it would have if all took part (every part less is one that need not be
// written and joined); so every one of them has a tile, and every worker
// between the first and the last of a token leaves a part of it.
__device__ __forceinline__ int attn_workers(const AttnArgs& a, uint32_t total) {
  if (total == 0) return 0;
  const uint32_t most = (total + a.workers - 1) / a.workers;
  return (int)((total + most - 1) / most);
}
__device__ __forceinline__ uint32_t attn_worker_start(uint32_t total, int workers, int w) {
  return (uint32_t)((uint64_t)total * w / workers);
}
// The worker whose range holds tile x: the largest w with start(w) <= x.
__device__ __forceinline__ int attn_worker_of(uint32_t total, int workers, uint32_t x) {
  return (int)((((uint64_t)x + 1) * workers - 1) / total);
}

// The token of tile x: the first t with end[t] > x.
__device__ __forceinline__ int attn_token_of(const AttnPlan* p, int batch, uint32_t x) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p->end[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}
__device__ __forceinline__ AttnToken attn_token(const AttnArgs& a, const AttnPlan* p, uint32_t x,
                                                const AttnSeen* seen = nullptr) {
  AttnToken k;
  k.t = attn_token_of(p, a.batch, x);
  k.start = p->start(k.t);
  k.end = p->end[k.t];
  if (seen != nullptr) {
    k.row = seen->row[k.t];
    k.len = seen->len[k.t];
    k.nv = seen->nv[k.t];
    return k;
  }
  k.row = a.token_row != nullptr ? a.token_row[k.t] : k.t;
  k.len = a.lens[k.t];
  k.nv = attn_positions(a, k.t, k.len, k.row, false);
  return k;
}

// The cache row (page * page_size + offset) of virtual position v, or -1 where
// the position does not count; *page receives the page.
__device__ __forceinline__ int64_t attn_row(const AttnArgs& a, const AttnToken& k, uint32_t v,
                                            int64_t* page) {
  if (v >= k.nv) return -1;
  const uint32_t b = v / (uint32_t)a.page_size;
  const int off = (int)(v - b * (uint32_t)a.page_size);
  int64_t j = b;
  if (a.sel != nullptr) {
    j = a.sel[(int64_t)k.t * a.sel_stride + b];
    if (j < 0 || j >= a.bt_stride || j * a.page_size + off >= k.len) return -1;
  }
  const int64_t p = a.table[(int64_t)k.row * a.bt_stride + j];
  if (p < 0 || p >= a.num_pages) {
    atomicOr(a.err, MLA_DEVERR_BAD_SLOT);
    return -1;
  }
  *page = p;
  return p * a.page_size + off;
}

// A part's sums: slot, then the head's group of four, then the column, four
// heads side by side, so that a thread that holds one column of several heads
// (a lane of O^T) writes 16 bytes, and a warp 512 bytes in a row.
__device__ __forceinline__ float4& attn_part(const AttnArgs& a, int slot, int quad, int col) {
  return a.part_o[((int64_t)slot * (a.heads_pad >> 2) + quad) * kKvLora + col];
}
// A head's (maximum in base 2, denominator), by slot.
__device__ __forceinline__ float2* attn_part_ml(const AttnArgs& a, int head) {
  return a.part_ml + (int64_t)head * 2 * a.workers;
}

// Natural logarithm of the sum of exponentials, from the maximum in base 2 and
// the sum relative to it.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return m == -INFINITY && l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

}  // namespace
}  // namespace mla
