// mla_prompt_rows.cu - the row operators of a prompt: rotary positions, cache
// rows of many tokens written, cached rows read back as BF16.
//
// All three move every byte once and are bound by HBM where there are many
// rows, by one trip to memory where there are few.
#include <math.h>
#include <stdlib.h>

#include "../../include/mla_query.h"
#include "mla_common.cuh"
#include "mla_prompt.h"
#include "mla_rows.cuh"

struct mla_rope {
  mla::RopeSpec spec;
};

namespace mla {
namespace {

// --------------------------------------------------------------- rotation
//
// Pair p of a 64-wide row turns by a = position * inv_freq[p]:
//   y0 = scale (x0 cos a - x1 sin a),  y1 = scale (x1 cos a + x0 sin a).
// A position of a million radians has no fraction left in FP32, and few bits
// in a product of two FP32 numbers.  So the frequency is kept as turns a
// position, a 64-bit fraction: the product with the position, modulo 2^64, is
// the angle's fraction of a turn, exact to position * 2^-64, in one integer
// multiplication.  Its upper 32 bits are half turns from -1 to 1 in FP32 (off
// by at most 2^-25 of a half turn).

// Lane p of a warp has pair p's frequency and axis for all its tokens.
struct RopeLane {
  uint64_t turns;
  const int32_t* positions;
  int64_t offset;
  float scale;
  __device__ __forceinline__ explicit RopeLane(const RopeArgs& r, int lane)
      : turns(r.spec.turns[lane]),
        positions(r.positions + (int64_t)r.spec.axis[lane] * r.pos_stride),
        offset(r.offset),
        scale(r.spec.scale) {}
  // (cos, sin) of this lane's pair at token t, times the scale
  __device__ __forceinline__ float2 at(int64_t t) const {
    const uint64_t turn = (uint64_t)((int64_t)positions[t] + offset) * turns;
    const int32_t half = (int32_t)((turn + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)half * 0x1p-31f, &s, &c);
    return make_float2(c * scale, s * scale);
  }
};

__device__ __forceinline__ float2 turned(float x0, float x1, float c, float s) {
  return make_float2(fmaf(x0, c, -(x1 * s)), fmaf(x1, c, x0 * s));
}

// Four lanes a head, eight heads a warp: lane j of four has pairs 8 j .. 8 j + 7,
// whose values are 32 bytes in a row (neighbours as pairs) or 16 bytes of each
// half (halves as pairs).  A warp stays with a token for `chunk` heads: one
// sine and cosine a lane, handed round by shuffles.  A lane reads all it turns
// before it writes, so the output may be the input.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(256) mla_rope_kernel(const __grid_constant__ RopeArgs r, int64_t tokens, int heads,
                                                       int chunk, const uint16_t* x, int64_t x_ts, int64_t x_hs,
                                                       uint16_t* out, int64_t o_ts, int64_t o_hs) {
  const int lane = threadIdx.x & 31, j = lane & 3;
  const int64_t warps = (int64_t)gridDim.x * 8;
  const RopeLane rope(r, lane);
  const int h0 = blockIdx.y * chunk + (lane >> 2), h1 = min(heads, (int)(blockIdx.y + 1) * chunk);
  // words 0..3 and 4..7 of a lane's share of a row, in values from its start
  const int a0 = INTERLEAVED ? 16 * j : 8 * j, a1 = INTERLEAVED ? 16 * j + 8 : 32 + 8 * j;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < tokens; t += warps) {
    const uint16_t* xt = x + t * x_ts;
    uint4 v0 = {}, v1 = {};
    if (h0 < h1) {
      v0 = *reinterpret_cast<const uint4*>(xt + (int64_t)h0 * x_hs + a0);
      v1 = *reinterpret_cast<const uint4*>(xt + (int64_t)h0 * x_hs + a1);
    }
    const float2 mine = rope.at(t);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = __shfl_sync(0xFFFFFFFFu, mine.x, 8 * j + i);
      s[i] = __shfl_sync(0xFFFFFFFFu, mine.y, 8 * j + i);
    }
    for (int h = h0; h < h1; h += 8) {
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      if (h + 8 < h1) {
        v0 = *reinterpret_cast<const uint4*>(xt + (int64_t)(h + 8) * x_hs + a0);
        v1 = *reinterpret_cast<const uint4*>(xt + (int64_t)(h + 8) * x_hs + a1);
      }
      uint32_t y[8];
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 p = turned(bf16lo(w[i]), bf16hi(w[i]), c[i], s[i]);
          y[i] = pack_bf16x2(p.x, p.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = turned(bf16lo(w[i]), bf16lo(w[i + 4]), c[2 * i], s[2 * i]);
          const float2 q = turned(bf16hi(w[i]), bf16hi(w[i + 4]), c[2 * i + 1], s[2 * i + 1]);
          y[i] = pack_bf16x2(p.x, q.x);
          y[i + 4] = pack_bf16x2(p.y, q.y);
        }
      }
      uint16_t* o = out + t * o_ts + (int64_t)h * o_hs;
      *reinterpret_cast<uint4*>(o + a0) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(o + a1) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// --------------------------------------------------------------- writing
//
// One warp a token: the decode step's insert (the same sums in the same order,
// so the same bytes), with the norm and the rotation optional, and the row
// handed on in BF16 where the caller wants it.  A lane has latent columns
// 8 lane .. and 256 + 8 lane ..; the first eight lanes have the rope part.
template <int LAYOUT>
__global__ void __launch_bounds__(256) mla_cache_write_kernel(const __grid_constant__ CacheWriteArgs w) {
  constexpr bool kDs = LAYOUT == MLA_KV_FP8_DS_MLA, kNv = LAYOUT == MLA_KV_NVFP4_DS_MLA;
  constexpr int kBytes = RowChunks<LAYOUT>::kBytes;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  const bool rope_on = w.rope.positions != nullptr;
  const RopeLane rope(w.rope, lane);
  const DecodeArgs none = {};
  pdl_wait();
  pdl_launch_dependents();
  uint4 gv[2] = {};
  if (w.gamma != nullptr) {
    gv[0] = *reinterpret_cast<const uint4*>(w.gamma + 8 * lane);
    gv[1] = *reinterpret_cast<const uint4*>(w.gamma + 256 + 8 * lane);
  }
  const float tensor_scale = LAYOUT == MLA_KV_FP8_E4M3 ? *w.k_scale : 1.0f;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < w.tokens; t += warps) {
    const uint16_t* kv = w.kv_c + t * w.kv_c_stride;
    const uint4 v[2] = {*reinterpret_cast<const uint4*>(kv + 8 * lane),
                        *reinterpret_cast<const uint4*>(kv + 256 + 8 * lane)};
    uint4 pe = {};
    if (lane < 8) pe = *reinterpret_cast<const uint4*>(w.k_pe + t * w.k_pe_stride + 8 * lane);
    int64_t slot = w.slots[t];
    if (slot >= w.capacity) {
      if (lane == 0 && w.flags != nullptr) atomicOr(w.flags, MLA_DEVERR_BAD_SLOT);
      slot = -1;
    }
    if (rope_on) {
      const float2 mine = rope.at(t);
      const uint32_t x[4] = {pe.x, pe.y, pe.z, pe.w};
      uint32_t y[4];
      if (w.rope.spec.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // pair 4 lane + i
          const float c = __shfl_sync(0xFFFFFFFFu, mine.x, (4 * lane + i) & 31);
          const float s = __shfl_sync(0xFFFFFFFFu, mine.y, (4 * lane + i) & 31);
          const float2 p = turned(bf16lo(x[i]), bf16hi(x[i]), c, s);
          y[i] = pack_bf16x2(p.x, p.y);
        }
      } else {
        const bool second = (lane & 4) != 0;  // of its pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, x[i], 4);
          const int p0 = 8 * (lane & 3) + 2 * i;
          const float c0 = __shfl_sync(0xFFFFFFFFu, mine.x, p0), s0 = __shfl_sync(0xFFFFFFFFu, mine.y, p0);
          const float c1 = __shfl_sync(0xFFFFFFFFu, mine.x, p0 + 1), s1 = __shfl_sync(0xFFFFFFFFu, mine.y, p0 + 1);
          const uint32_t x0 = second ? other : x[i], x1 = second ? x[i] : other;
          const float2 p = turned(bf16lo(x0), bf16lo(x1), c0, s0), q = turned(bf16hi(x0), bf16hi(x1), c1, s1);
          y[i] = second ? pack_bf16x2(p.y, q.y) : pack_bf16x2(p.x, q.x);
        }
      }
      pe = make_uint4(y[0], y[1], y[2], y[3]);
    }
    float n[2][8];
    const float s0 = kv_group_ss(v[0], n[0]), s1 = kv_group_ss(v[1], n[1]);
    if (w.gamma != nullptr) {
      const float total = warp_sum(s0) + warp_sum(s1);
      const float rr = __frsqrt_rn(__fadd_rn(__fmul_rn(total, 1.0f / 512.0f), w.eps));
      kv_group_norm(n[0], gv[0], rr, n[0]);
      kv_group_norm(n[1], gv[1], rr, n[1]);
    }
    if (w.rows != nullptr) {
      uint16_t* o = w.rows + t * w.rows_stride;
#pragma unroll
      for (int g = 0; g < 2; ++g)
        *reinterpret_cast<uint4*>(o + 256 * g + 8 * lane) =
            make_uint4(pack_bf16x2(n[g][0], n[g][1]), pack_bf16x2(n[g][2], n[g][3]), pack_bf16x2(n[g][4], n[g][5]),
                       pack_bf16x2(n[g][6], n[g][7]));
      if (lane < 8) *reinterpret_cast<uint4*>(o + kKvLora + 8 * lane) = pe;
    }
    if (slot < 0) continue;
    float ks = tensor_scale;
    if constexpr (LAYOUT == MLA_KV_FP8_E4M3_PAGE) ks = w.k_scale[slot / w.page_size];
    uint8_t* row = w.cache + slot * kBytes;
#pragma unroll
    for (int g = 0; g < 2; ++g)
      kv_store_group(none, row, n[g], g == 0 ? pe : make_uint4(0, 0, 0, 0), lane + 32 * g, kDs, kNv, ks);
  }
}

// --------------------------------------------------------------- reading
//
// A CTA takes R output rows in a row.  A thread each finds where they lie (the
// request by bisection, the page from the table); then all threads take 16-byte
// chunks of the rows, four under way at a time, and store their values.
constexpr int kReadThreads = 256, kReadMost = 64;

template <int LAYOUT>
__global__ void __launch_bounds__(kReadThreads) mla_cache_read_kernel(const __grid_constant__ CacheReadArgs a, int R) {
  using C = RowChunks<LAYOUT>;
  __shared__ int64_t source[kReadMost];  // byte offset of the cache row; -1: zeros, -2: left as it is
  __shared__ float scale[kReadMost];
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * R;
  pdl_wait();
  pdl_launch_dependents();
  if (tid < R) {
    const int64_t i = row0 + tid;
    int64_t src = -2;
    float sc = 1.0f;
    if (i < a.max_rows && i >= a.cu[0] && i < a.cu[a.requests]) {
      int lo = 0, hi = a.requests - 1;  // the last request with cu[r] <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int64_t pos = i - a.cu[lo] + (a.first != nullptr ? a.first[lo] : 0);
      int64_t page = -1, off = 0;
      if (pos >= 0 && pos <= 0xFFFFFFFFll) {
        const uint32_t b = (uint32_t)pos / (uint32_t)a.page_size;
        off = pos - (int64_t)b * a.page_size;
        if (b < a.bt_cols) page = a.table[(int64_t)lo * a.bt_stride + b];
      }
      if (page >= 0 && page < a.num_pages) {
        src = (page * a.page_size + off) * C::kBytes;
        sc = page_scale(a.k_scale, LAYOUT, page);
      } else {
        src = -1;
        if (a.flags != nullptr) atomicOr(a.flags, MLA_DEVERR_BAD_SLOT);
      }
    }
    source[tid] = src;
    scale[tid] = sc;
  }
  __syncthreads();
  constexpr int kAhead = 4;
  for (int base = tid; base < R * C::kChunks; base += kAhead * kReadThreads) {
    uint4 w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = base + u * kReadThreads, r = k / C::kChunks;
      w[u] = make_uint4(0, 0, 0, 0);
      if (k < R * C::kChunks && source[r] >= 0)
        w[u] = *reinterpret_cast<const uint4*>(a.cache + source[r] + C::offset(k - r * C::kChunks));
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = base + u * kReadThreads, r = k / C::kChunks, c = k - r * C::kChunks;
      if (k >= R * C::kChunks || source[r] == -2) continue;
      float v[C::kMax];
#pragma unroll
      for (int e = 0; e < C::kMax; ++e) v[e] = 0.f;
      if (source[r] >= 0) C::add(a.cache + source[r], c, w[u], v);
      const float sc = scale[r];
      uint16_t* o = a.rows + (row0 + r) * a.rows_stride + C::col(c);
#pragma unroll
      for (int e = 0; e < C::kMax; e += 8)
        if (e < C::width(c))
          *reinterpret_cast<uint4*>(o + e) =
              make_uint4(pack_bf16x2(v[e] * sc, v[e + 1] * sc), pack_bf16x2(v[e + 2] * sc, v[e + 3] * sc),
                         pack_bf16x2(v[e + 4] * sc, v[e + 5] * sc), pack_bf16x2(v[e + 6] * sc, v[e + 7] * sc));
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool known_layout(int layout) { return layout >= MLA_KV_FP8_E4M3 && layout <= MLA_KV_FP8_E4M3_PAGE; }
int launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();
  return MLA_ECUDA;
}
bool sm_count(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    return true;
  cudaGetLastError();
  return false;
}

// A launch that the kernel before may overlap (each kernel waits for it first).
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(dim3 grid, int threads, void* stream) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

// A cache's pages and rows that byte offsets of 64 bits reach.
bool cache_fits(int64_t num_pages, int page_size) {
  return num_pages >= 1 && page_size >= 1 && num_pages <= INT64_MAX / kRowDs / page_size;
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_rope_create(mla_rope_t* out, const double* inv_freq, const int32_t* axis, int interleaved, float scale) {
  if (out == nullptr) return MLA_EINVAL;
  *out = nullptr;
  if (inv_freq == nullptr || !(scale > -3.0e38f && scale < 3.0e38f)) return MLA_EINVAL;
  for (int p = 0; p < mla::kRopePairs; ++p) {
    if (!(fabs(inv_freq[p]) <= 1e6)) return MLA_EINVAL;
    if (axis != nullptr && (axis[p] < 0 || axis[p] >= MLA_MAX_ROPE_AXES)) return MLA_EINVAL;
  }
  mla_rope* h = static_cast<mla_rope*>(calloc(1, sizeof(mla_rope)));
  if (h == nullptr) return MLA_ENOMEM;
  // 1 / (2 pi) as the sum of two doubles: the turns a position to about 2^-64
  constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;
  for (int p = 0; p < mla::kRopePairs; ++p) {
    const double hi = inv_freq[p] * kTurn;
    const double lo = fma(inv_freq[p], kTurn, -hi) + inv_freq[p] * kTurnRest;
    double whole = hi - floor(hi);  // exact, in [0, 1]
    if (whole >= 1.0) whole = 0.0;
    h->spec.turns[p] = (uint64_t)ldexp(whole, 64) + (uint64_t)(int64_t)llrint(ldexp(lo, 64));
    h->spec.axis[p] = axis != nullptr ? (uint8_t)axis[p] : 0;
    if (h->spec.axis[p] >= h->spec.axes) h->spec.axes = h->spec.axis[p] + 1;
  }
  h->spec.interleaved = interleaved != 0;
  h->spec.scale = scale;
  *out = h;
  return MLA_OK;
}

int mla_rope_axes(mla_rope_t h) { return h == nullptr ? MLA_EINVAL : h->spec.axes; }

void mla_rope_destroy(mla_rope_t h) { free(h); }

int mla_rope_apply(mla_rope_t h, int64_t tokens, int heads, const void* x, int64_t x_token_stride,
                   int64_t x_head_stride, const int32_t* positions, int64_t pos_stride, int64_t pos_offset, void* out,
                   int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  if (h == nullptr || tokens < 0 || heads < 1 || heads > MLA_MAX_ROW_HEADS) return MLA_EINVAL;
  if (tokens == 0) return MLA_OK;
  if (x == nullptr || positions == nullptr || out == nullptr) return MLA_EINVAL;
  if (pos_stride == 0) pos_stride = tokens;
  if (pos_stride < tokens || pos_offset < INT32_MIN || pos_offset > INT32_MAX) return MLA_EINVAL;
  if (x_head_stride == 0) x_head_stride = mla::kRope;
  if (x_token_stride == 0) x_token_stride = heads * x_head_stride;
  if (out_head_stride == 0) out_head_stride = mla::kRope;
  if (out_token_stride == 0) out_token_stride = heads * out_head_stride;
  if (x_head_stride < mla::kRope || x_token_stride < mla::kRope || out_head_stride < mla::kRope ||
      out_token_stride < mla::kRope || (x_head_stride | x_token_stride | out_head_stride | out_token_stride) % 8)
    return MLA_EINVAL;
  if (!mla::aligned16(x) || !mla::aligned16(out) || !mla::aligned4(positions)) return MLA_EINVAL;
  int sms = 0;
  if (!mla::sm_count(&sms)) return MLA_ECUDA;
  // Heads a warp takes of a token: all of them (one sine and cosine for all)
  // while that makes eight warps an SM, down to one head a lane quad.
  int chunk = (heads + 7) / 8 * 8;
  while (chunk > 8 && tokens * ((heads + chunk - 1) / chunk) < 8 * (int64_t)sms) chunk = (chunk / 2 + 7) / 8 * 8;
  const int groups = (heads + chunk - 1) / chunk;
  int64_t ctas = (tokens + 7) / 8;
  const int64_t most = (8 * (int64_t)sms + groups - 1) / groups;  // eight CTAs an SM are resident
  if (ctas > most) ctas = most;
  mla::Launch l(dim3((unsigned)ctas, (unsigned)groups), 256, stream);
  const mla::RopeArgs r{h->spec, positions, pos_stride, pos_offset};
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint16_t* op = static_cast<uint16_t*>(out);
  return mla::launched(cudaLaunchKernelEx(&l.cfg, h->spec.interleaved ? mla::mla_rope_kernel<true> : mla::mla_rope_kernel<false>,
                                          r, tokens, heads, chunk, xp, x_token_stride, x_head_stride, op,
                                          out_token_stride, out_head_stride));
}

int mla_cache_write(int64_t tokens, const void* kv_c, int64_t kv_c_stride, const void* k_pe, int64_t k_pe_stride,
                    const void* gamma_kv, float eps, mla_rope_t rope, const int32_t* positions, int64_t pos_stride,
                    int64_t pos_offset, const int64_t* slot_mapping, void* kv_cache, int64_t num_pages, int page_size,
                    int layout, const float* k_scale, void* rows, int64_t rows_stride, unsigned* device_flags,
                    void* stream) {
  if (tokens < 0 || !mla::known_layout(layout) || (mla::row_scaled(layout) && k_scale == nullptr)) return MLA_EINVAL;
  if (!mla::cache_fits(num_pages, page_size) || !(eps >= 0.0f)) return MLA_EINVAL;
  if ((rope == nullptr) != (positions == nullptr)) return MLA_EINVAL;
  if (tokens == 0) return MLA_OK;
  if (kv_c == nullptr || k_pe == nullptr || slot_mapping == nullptr || kv_cache == nullptr) return MLA_EINVAL;
  if (kv_c_stride == 0) kv_c_stride = mla::kKvLora;
  if (k_pe_stride == 0) k_pe_stride = mla::kRope;
  if (rows_stride == 0) rows_stride = mla::kRowElems;
  if (pos_stride == 0) pos_stride = tokens;
  if (kv_c_stride < mla::kKvLora || k_pe_stride < mla::kRope || (kv_c_stride | k_pe_stride) % 8 ||
      (rows != nullptr && (rows_stride < mla::kRowElems || rows_stride % 8)))
    return MLA_EINVAL;
  if (rope != nullptr && (pos_stride < tokens || pos_offset < INT32_MIN || pos_offset > INT32_MAX)) return MLA_EINVAL;
  if (!mla::aligned16(kv_c) || !mla::aligned16(k_pe) || !mla::aligned16(gamma_kv) || !mla::aligned16(kv_cache) ||
      !mla::aligned16(rows) || !mla::aligned4(positions) || !mla::aligned4(k_scale) || !mla::aligned4(device_flags) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return MLA_EINVAL;
  int sms = 0;
  if (!mla::sm_count(&sms)) return MLA_ECUDA;
  mla::CacheWriteArgs w = {};
  w.tokens = tokens;
  w.kv_c = static_cast<const uint16_t*>(kv_c);
  w.k_pe = static_cast<const uint16_t*>(k_pe);
  w.kv_c_stride = kv_c_stride;
  w.k_pe_stride = k_pe_stride;
  w.gamma = static_cast<const uint16_t*>(gamma_kv);
  w.eps = eps;
  if (rope != nullptr) w.rope = mla::RopeArgs{rope->spec, positions, pos_stride, pos_offset};
  w.slots = slot_mapping;
  w.cache = static_cast<uint8_t*>(kv_cache);
  w.capacity = num_pages * page_size;
  w.page_size = page_size;
  w.k_scale = k_scale;
  w.rows = static_cast<uint16_t*>(rows);
  w.rows_stride = rows_stride;
  w.flags = device_flags;
  int64_t ctas = (tokens + 7) / 8;
  if (ctas > 8 * (int64_t)sms) ctas = 8 * (int64_t)sms;
  mla::Launch l(dim3((unsigned)ctas), 256, stream);
  cudaError_t e;
  switch (layout) {
    case MLA_KV_FP8_DS_MLA: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_write_kernel<MLA_KV_FP8_DS_MLA>, w); break;
    case MLA_KV_NVFP4_DS_MLA: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_write_kernel<MLA_KV_NVFP4_DS_MLA>, w); break;
    case MLA_KV_FP8_E4M3_PAGE: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_write_kernel<MLA_KV_FP8_E4M3_PAGE>, w); break;
    default: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_write_kernel<MLA_KV_FP8_E4M3>, w);
  }
  return mla::launched(e);
}

int mla_cache_read(const void* kv_cache, int64_t num_pages, int page_size, int layout, const float* k_scale,
                   const int32_t* block_table, int64_t bt_stride, int64_t bt_cols, int requests, const int32_t* cu_rows,
                   const int32_t* first, int64_t max_rows, void* rows, int64_t rows_stride, unsigned* device_flags,
                   void* stream) {
  if (kv_cache == nullptr || block_table == nullptr || cu_rows == nullptr) return MLA_EINVAL;
  if (!mla::known_layout(layout) || (mla::row_scaled(layout) && k_scale == nullptr)) return MLA_EINVAL;
  if (!mla::cache_fits(num_pages, page_size) || bt_cols < 1 || bt_stride < bt_cols || requests < 1 ||
      requests > MLA_MAX_TABLE_ROWS || max_rows < 0 || max_rows > INT32_MAX)
    return MLA_EINVAL;
  if (rows_stride == 0) rows_stride = mla::kRowElems;
  if (rows_stride < mla::kRowElems || rows_stride % 8) return MLA_EINVAL;
  if (!mla::aligned16(kv_cache) || !mla::aligned16(rows) || !mla::aligned4(k_scale) || !mla::aligned4(block_table) ||
      !mla::aligned4(cu_rows) || !mla::aligned4(first) || !mla::aligned4(device_flags))
    return MLA_EINVAL;
  if (max_rows == 0) return MLA_OK;
  if (rows == nullptr) return MLA_EINVAL;
  int sms = 0;
  if (!mla::sm_count(&sms)) return MLA_ECUDA;
  mla::CacheReadArgs a = {};
  a.cache = static_cast<const uint8_t*>(kv_cache);
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.k_scale = k_scale;
  a.table = block_table;
  a.bt_stride = bt_stride;
  a.bt_cols = bt_cols;
  a.requests = requests;
  a.cu = cu_rows;
  a.first = first;
  a.max_rows = max_rows;
  a.rows = static_cast<uint16_t*>(rows);
  a.rows_stride = rows_stride;
  a.flags = device_flags;
  // Rows a CTA: 8 while all CTAs are resident at once, 32 beyond.
  const int R = max_rows <= 8 * 8 * (int64_t)sms ? 8 : 32;
  mla::Launch l(dim3((unsigned)((max_rows + R - 1) / R)), mla::kReadThreads, stream);
  cudaError_t e;
  switch (layout) {
    case MLA_KV_FP8_DS_MLA: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_read_kernel<MLA_KV_FP8_DS_MLA>, a, R); break;
    case MLA_KV_NVFP4_DS_MLA: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_read_kernel<MLA_KV_NVFP4_DS_MLA>, a, R); break;
    case MLA_KV_FP8_E4M3_PAGE: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_read_kernel<MLA_KV_FP8_E4M3_PAGE>, a, R); break;
    default: e = cudaLaunchKernelEx(&l.cfg, mla::mla_cache_read_kernel<MLA_KV_FP8_E4M3>, a, R);
  }
  return mla::launched(e);
}

}  // extern "C"
