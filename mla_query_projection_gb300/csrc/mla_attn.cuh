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
// selected blocks, block after block), cut into tiles.  On the axis that is
// shared out, a token with tiles has `lead` units without work and then a unit
// a tile; end[t] is the axis up to and with token t.  Worker w of a head group
// takes what lies in [w * total / workers, (w + 1) * total / workers), whatever
// requests it belongs to.  A stretch of one token's tiles that is not all of
// them leaves the worker as a partial: its first stretch in slot 0, any other
// (then its last) in slot 1.
//
// The lead stands for what a worker pays when it goes on from one token to the
// next: the sums are written, new queries come in and the reference is set
// anew, 5 to 8 us or a few tiles.  Without it a call waits for the few workers
// whose share spans two tokens (attn_lead has what it measured).
struct AttnPlan {
  uint32_t end[kAttnMaxBatch];
  uint32_t lead, pad;
  __device__ uint32_t start(int t) const { return t > 0 ? end[t - 1] : 0u; }
};
// Positions of one token beyond this are left out (and flagged): 256 tokens'
// tiles stay within 31 bits.
constexpr int64_t kAttnMaxPositions = (int64_t)1 << 29;

// What a token looks at.
struct AttnToken {
  int t, row;
  uint32_t start, end;  // its tiles on the axis
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
    const int64_t cap = a.bt_cols * a.page_size;
    bad = len > cap;
    if (a.sel != nullptr) {
      n = min((int64_t)max(__ldcg(a.sel_count + t), 0), a.sel_cols) * a.page_size;
    } else {
      n = min((int64_t)len, cap);
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

// Fills the plan; all threads of the block call it (at least 256 / TPT of them, a
// multiple of 32; TPT tokens a thread), and may read it after the closing
// barrier.  red: 16 words.
template <int TPT = 1>
__device__ __forceinline__ void attn_make_plan(const AttnArgs& a, AttnPlan* p, uint32_t* red,
                                               bool flag, AttnSeen* seen = nullptr) {
  constexpr int kWarps = kAttnMaxBatch / (32 * TPT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t n[TPT], sum = 0, below = 0, some = 0;  // tiles; tokens with tiles, in lower lanes and in the warp
#pragma unroll
  for (int i = 0; i < TPT; ++i) {
    const int t = TPT * tid + i;
    n[i] = 0;
    if (t < a.batch) {
      // (from L2: the join asks before its own wait, when only the kernel before
      // has waited for what wrote these)
      const int32_t len = __ldcg(a.lens + t);
      const int row = a.token_row != nullptr ? __ldcg(a.token_row + t) : t;
      const uint32_t nv = attn_positions(a, t, len, row, flag);
      n[i] = (nv + kAttnTile - 1) / kAttnTile;
      if (seen != nullptr) {
        seen->len[t] = len;
        seen->row[t] = row;
        seen->nv[t] = nv;
      }
    }
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, n[i] > 0);
    below += __popc(mask & ((1u << lane) - 1u));
    some += __popc(mask);
    sum += n[i];
  }
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31 && warp < kWarps) {
    red[warp] = inc;
    red[kWarps + warp] = some;
  }
  __syncthreads();
  if (warp < kWarps) {
    uint32_t at = inc - sum, count = below, tiles = 0, tokens = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        at += red[w];
        count += red[kWarps + w];
      }
      tiles += red[w];
      tokens += red[kWarps + w];
    }
    // (A share below a lead and a tile has nothing to even out.)
    const uint32_t lead = tokens > 1 && tiles >= (a.lead + 1) * a.workers ? a.lead : 0u;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
      at += n[i];
      count += n[i] > 0;
      p->end[TPT * tid + i] = at + lead * count;
    }
    if (tid == 0) p->lead = lead;
  }
  __syncthreads();
}

// Workers with work: the fewest for which the busiest has no more than it would
// have if all took part (every part less is one that need not be written and
// joined).  Every worker from the one that holds a token's first tile to the one
// that holds its last has a tile of it, and leaves a part.
__device__ __forceinline__ int attn_workers(const AttnArgs& a, uint32_t total) {
  if (total == 0) return 0;
  const uint32_t most = (total + a.workers - 1) / a.workers;
  return (int)((total + most - 1) / most);
}
__device__ __forceinline__ uint32_t attn_worker_start(uint32_t total, int workers, int w) {
  return (uint32_t)((uint64_t)total * w / workers);
}
// The worker whose range holds the tile at x: the largest w with start(w) <= x.
__device__ __forceinline__ int attn_worker_of(uint32_t total, int workers, uint32_t x) {
  return (int)((((uint64_t)x + 1) * workers - 1) / total);
}

// The token at x: the first t with end[t] > x.
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
  k.start = p->start(k.t) + p->lead;
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

// A worker's part of the axis, from a tile to behind a tile (nothing where
// first >= end).
__device__ __forceinline__ void attn_range(const AttnArgs& a, const AttnPlan* p, int worker, uint32_t* first,
                                           uint32_t* end) {
  const uint32_t total = p->end[a.batch - 1];
  const int workers = attn_workers(a, total);
  *first = *end = 0;
  if (worker >= workers) return;
  *first = attn_worker_start(total, workers, worker);
  *end = attn_worker_start(total, workers, worker + 1);
  if (p->lead == 0) return;
  *first = max(*first, p->start(attn_token_of(p, a.batch, *first)) + p->lead);
  if (*end < total) {  // not into the next token's lead
    const uint32_t s = p->start(attn_token_of(p, a.batch, *end));
    if (*end <= s + p->lead) *end = s;
  }
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
    if (j < 0 || j >= a.bt_cols || j * a.page_size + off >= k.len) return -1;
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
