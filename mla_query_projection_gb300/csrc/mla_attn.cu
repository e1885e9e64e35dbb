// mla_attn.cu - latent attention over the paged cache: the C entry points and
// the kernel that joins the parts of a context that several workers read.
// (What reads the cache is in mla_attn_tc.cu, mla_attn_ds.cu and mla_attn_nv.cu,
// by layout.)
//
//   o[t][h] = sum_i p_i c_i[0..511],  p = softmax_i(scale * q[t][h] . c_i),
//   lse[t][h] = log sum_i exp(scale * q[t][h] . c_i)
//
// over the cache rows c_i (512 latent and 64 rope values) of the token's
// context.  The sums run once over the data: with m the running maximum (in
// base 2), l = sum 2^(x_i - m) and o = sum 2^(x_i - m) c_i are rescaled by
// 2^(m_old - m_new) whenever m grows.
#include <stdlib.h>

#include "../../include/mla_query.h"
#include "mla_attn.cuh"
#include "mla_device.cuh"
#include "mla_internal.h"

struct mla_attn {
  int device;
  int num_sms;
  int heads;
  int max_batch;
  uint32_t* err;
  float4* part_o;   // partial sums of the workers (mla_attn.cuh, attn_part)
  float2* part_ml;  // their maxima and denominators
};

namespace mla {
namespace {

// --------------------------------------------------------------- joining
//
// With M the largest maximum of a (token, head)'s parts,
// o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  Tokens whose context one
// worker read whole are done already; those that look at nothing get zeros
// and an lse of -infinity.  Bound by the parts' bytes (L2), and by latency
// where there are few.  Before it waits for the parts a CTA works out the plan
// for itself (the kernel before has waited for what wrote the lengths by the
// time this one may start), so that the first trip to memory is for the parts.
// It then takes four heads of a token at a time, which lie side by side in the
// parts (attn_part), in one of three shapes by the parts a token has on average
// (attn_join_cols), COLS columns a lane:
//  1: 32 columns a CTA, the eight warps every eighth part each, their shares
//     summed in order;
//  2: all columns, 64 a warp, the parts in order;
//  4: the same, 128 a warp, so that more CTAs fit.

template <int COLS>
__global__ void __launch_bounds__(COLS == 4 ? 128 : 256) mla_attn_join_kernel(const AttnArgs a) {
  __shared__ AttnPlan plan;
  __shared__ uint32_t red[16];
  __shared__ float4 weight[kMaxCtas];  // a part's factors for the four heads
  constexpr bool WIDE = COLS == 1;
  __shared__ float4 scale4, sums[WIDE ? 8 : 1][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  attn_make_plan<COLS == 4 ? 2 : 1>(a, &plan, red, false);
  const uint32_t total = plan.end[a.batch - 1];
  const int workers = attn_workers(a, total);
  const int quads = (a.heads + 3) / 4;
  pdl_wait();
  for (int item = blockIdx.x; item < a.batch * quads * (WIDE ? 16 : 1); item += gridDim.x) {
    const int tq = WIDE ? item >> 4 : item, t = tq / quads, quad = tq - t * quads, h0 = 4 * quad;
    const uint32_t t0 = plan.start(t), t1 = plan.end[t];
    int w0 = 0, n = 0;
    if (t1 > t0) {
      w0 = attn_worker_of(total, workers, t0 + plan.lead);  // its first tile
      n = attn_worker_of(total, workers, t1 - 1) - w0 + 1;  // parts, at most kMaxCtas
      if (n == 1) continue;
    }
    // part i is worker w0 + i's; the first lies in slot 1 where that worker
    // began with another token
    const int slot0 = 2 * w0 + (n > 0 && attn_worker_start(total, workers, w0) < t0 ? 1 : 0);
    auto slot_of = [&](int i) { return i == 0 ? slot0 : 2 * (w0 + i); };
    // The first parts are on their way while the factors are worked out: warp w's
    // parts w, w + 8, .. of one column, or the first parts of two or four.
    constexpr int kPre = COLS == 4 ? 2 : 4;
    const int c0 = WIDE ? 32 * (item & 15) + lane : 32 * COLS * warp + lane;
    float4 pre[COLS * kPre];
#pragma unroll
    for (int u = 0; u < kPre; ++u) {
      const int i = WIDE ? warp + 8 * u : u;
      if (i < n) {
        if constexpr (WIDE) {
          pre[u] = attn_part(a, slot_of(i), quad, c0);
        } else {
#pragma unroll
          for (int e = 0; e < COLS; ++e) pre[COLS * u + e] = attn_part(a, slot_of(i), quad, c0 + 32 * e);
        }
      }
    }
    if (warp < 4) {  // warp e: the factors of head h0 + e
      const float2* ml = attn_part_ml(a, h0 + warp);
      float M = -INFINITY, l = 0.f;
      for (int i = lane; i < n; i += 32) M = fmaxf(M, ml[slot_of(i)].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
      const float m_use = M == -INFINITY ? 0.f : M;
      for (int i = lane; i < n; i += 32) {
        const float2 v = ml[slot_of(i)];
        const float f = v.x == -INFINITY ? 0.f : exp2f(v.x - m_use);
        l += f * v.y;
        reinterpret_cast<float*>(&weight[i])[warp] = f;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (lane == 0) {
        reinterpret_cast<float*>(&scale4)[warp] = l == 0.f ? 0.f : 1.0f / l;
        if (a.lse != nullptr && h0 + warp < a.heads && (!WIDE || (item & 15) == 0))
          a.lse[(int64_t)t * a.heads + h0 + warp] = attn_lse(M, l);
      }
    }
    __syncthreads();
    const float4 r = scale4;
    auto add = [](float4& acc, float4 f, float4 v) {
      // (a part that saw nothing holds zeros, so its factor of zero needs no test)
      acc.x = fmaf(f.x, v.x, acc.x);
      acc.y = fmaf(f.y, v.y, acc.y);
      acc.z = fmaf(f.z, v.z, acc.z);
      acc.w = fmaf(f.w, v.w, acc.w);
    };
    auto put = [&](int col, float4 v) {
      uint16_t* o = a.out + (int64_t)t * a.o_ts + (int64_t)h0 * a.o_hs + col;
      const float w[4] = {v.x * r.x, v.y * r.y, v.z * r.z, v.w * r.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (h0 + e < a.heads) o[e * a.o_hs] = f2bf_bits(w[e]);
    };
    if constexpr (WIDE) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kPre; ++u)
        if (warp + 8 * u < n) add(acc, weight[warp + 8 * u], pre[u]);
#pragma unroll 8
      for (int i = warp + 8 * kPre; i < n; i += 8) add(acc, weight[i], attn_part(a, slot_of(i), quad, c0));
      sums[warp][lane] = acc;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int g = 1; g < 8; ++g) {
          const float4 b = sums[g][lane];
          acc.x += b.x;
          acc.y += b.y;
          acc.z += b.z;
          acc.w += b.w;
        }
        put(c0, acc);
      }
    } else {
      float4 acc[COLS];
#pragma unroll
      for (int e = 0; e < COLS; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kPre; ++u) {
        if (u >= n) continue;
#pragma unroll
        for (int e = 0; e < COLS; ++e) add(acc[e], weight[u], pre[COLS * u + e]);
      }
#pragma unroll COLS == 4 ? 2 : 4
      for (int i = kPre; i < n; ++i) {
        const int slot = slot_of(i);
#pragma unroll
        for (int e = 0; e < COLS; ++e) add(acc[e], weight[i], attn_part(a, slot, quad, c0 + 32 * e));
      }
#pragma unroll
      for (int e = 0; e < COLS; ++e) put(c0 + 32 * e, acc[e]);
    }
    __syncthreads();  // weight, scale4 and sums are read
  }
}

// The shape by the parts a token has on average, workers / batch; with few parts
// and many fours of heads the smallest CTAs.  Us a call with 1, 2 and 4 columns:
//   1 token of 65,536 E4M3 rows, 64 heads         25.3   51.6  77.4
//   8 tokens of 16,384 rows, 128 heads            59.4   43.4  45.6
//   60 tokens of 300 to 2,000 rows, 16 heads      37.9   21.0  22.0
//   32 tokens of 4,096 rows, 64 heads             69.8   35.9  34.0
//   62 tokens, 128 heads, fp8_ds_mla             210     84.7  83.1
int attn_join_cols(const AttnArgs& a, int num_sms) {
  const int items = (a.heads + 3) / 4 * a.batch;
  if (a.workers >= 16 * a.batch && 16 * items <= 8 * num_sms) return 1;
  return a.workers >= 6 * a.batch || items <= 3 * num_sms ? 2 : 4;
}

template <int COLS>
cudaError_t launch_join_cols(const AttnArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t items = (int64_t)a.batch * ((a.heads + 3) / 4) * (COLS == 1 ? 16 : 1);
  const int64_t most = (COLS == 4 ? 6 : 3) * (int64_t)num_sms;  // about what fits at once
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < most ? items : most));
  cfg.blockDim = dim3(COLS == 4 ? 128 : 256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_attn_join_kernel<COLS>, a);
}

cudaError_t launch_join(const AttnArgs& a, int num_sms, cudaStream_t stream) {
  switch (attn_join_cols(a, num_sms)) {
    case 1: return launch_join_cols<1>(a, num_sms, stream);
    case 2: return launch_join_cols<2>(a, num_sms, stream);
    default: return launch_join_cols<4>(a, num_sms, stream);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool known_layout(int layout) { return layout >= MLA_KV_FP8_E4M3 && layout <= MLA_KV_FP8_E4M3_PAGE; }

int sm_count(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ECUDA;
  }
  return MLA_OK;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();
  return MLA_ECUDA;
}

// Heads a CTA takes at most: 16 or 32 where that covers all of them (less
// padding, and more workers of the same tiles), 64 otherwise.
int attn_most_heads(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : 64; }

// Heads a CTA takes, by the most tiles that the columns of the call's tables or
// selections can hold (the lengths are known on the GPU only).  With half the heads a CTA has
// half the queries to load, half the softmax, half the sums to write and join;
// it has twice the tiles, and each costs more than half (the rows' bytes and,
// with nvfp4_ds_mla rows, the widening stay).  So: while every CTA still has one
// tile at most; and for 8-bit rows from 64 to 32 between three and seven tiles
// (at one to three the tiles are too coarse to share out).  Us with 64, 32 and 16
// heads a CTA, and tiles a CTA at 32:
//   1 x 64 heads, 512 E4M3 rows       0.05   13.8  10.7   9.5
//   1 x 128, 2,048 E4M3 rows          0.4    16.3  13.7  12.5
//   4 x 64, 2,000 fp8_ds_mla rows     0.8    21.7  18.5  17.2
//   2 x 64, 2,048 nvfp4_ds_mla rows   0.4    17.5  14.8  13.5
//   16 x 128, 500 E4M3 rows           1.7    18.1  20.0  19.9
//   6 x 96, 4,096 E4M3 rows           3.8    29.6  18.7
//   1 x 64, 65,536 E4M3 rows          6.7    25.4  23.9  30.3
//   2 x 128, 16,384 E4M3 rows         6.7    28.8  26.0  30.6
//   2 x 128, 16,384 fp8_ds_mla rows   6.7    33.5  32.1
//   1 x 128, 32,768 nvfp4_ds_mla rows 6.7    31.7  34.3  50.2
//   4 x 128, 16,384 E4M3 rows         13     34.5  35.2  50.8
//   32 x 64, 4,096 E4M3 rows          13     33.8  37.5  54.2
// Between 7 and 13 tiles neither is better throughout (64 and 32 heads a CTA):
//   2 x 128, 20,480 E4M3 rows         8.4    26.4  27.9
//   20 x 64, 4,096 E4M3 rows          8.4    31.7  25.3
//   20 x 64, 4,096 fp8_ds_mla rows    8.4    30.5  34.0
//   8 x 64, 12,288 E4M3 rows          10     28.6  28.1
//   2 x 128, 24,576 fp8_ds_mla rows   10     36.9  39.8
//   2 x 128, 28,672 E4M3 rows         12     35.3  32.1
// Columns that no request reaches count too: 1 x 64 heads over 512 E4M3 rows
// take 9.4 us with a table of 8 or 32 blocks, 10.6 with 128 and 10.8 with 1,024;
// 4 x 64 over 2,000 fp8_ds_mla rows 17.8 with 32 blocks, 21.2 with 512 (and 17.8
// with the first 32 columns of those 512: mla_attn_decode_cols).
int attn_cta_heads(const AttnArgs& a, int num_sms) {
  const int64_t blocks = a.sel != nullptr ? (a.sel_cols < a.bt_cols ? a.sel_cols : a.bt_cols) : a.bt_cols;
  const int64_t most = blocks * a.page_size;
  const int64_t tiles = a.batch * (((most < kAttnMaxPositions ? most : kAttnMaxPositions) + kAttnTile - 1) / kAttnTile);
  int n = attn_most_heads(a.heads);
  for (; n > 16; n /= 2) {
    const int64_t all = tiles * ((a.heads + n / 2 - 1) / (n / 2));
    const bool few = n == 64 && a.layout != MLA_KV_NVFP4_DS_MLA && all >= 3 * num_sms && all <= 7 * num_sms;
    if (all > num_sms && !few) break;
  }
  return n;
}

// What a worker's going on from one token to the next costs, in tiles: 5 where
// a tile is quick against it (E4M3 rows, 64 heads a CTA), else 3.  Us without a
// lead and with leads of 2, 3 and 5:
//   E4M3, 8 tokens of 16,384 rows, 128 heads      54.5  52.1  49.4  47.8
//   E4M3, 32 tokens of 4,096 rows, 64 heads       41.7  39.3  37.2  35.5
//   E4M3, 60 tokens of 300 to 2,000, 16 heads     25.1  22.3  22.5  23.5
//   fp8_ds_mla, 62 tokens of 700 to 4,096, 128    92.7  85.4  81.1  83.6
//   nvfp4_ds_mla, 32 tokens of 4,096 rows, 64     57.3  54.6  54.3  54.6
uint32_t attn_lead(const AttnArgs& a) { return row_scaled(a.layout) && a.cta_heads == 64 ? 5u : 3u; }

// Columns that a length or a count of 32 bits can reach: their product with the
// page size fits 64 bits (a single row's stride may be any number).
int64_t counted_cols(int64_t cols) { return cols < 0x7FFFFFFF ? cols : 0x7FFFFFFF; }

// Strides of a [batch][heads][width] operand; 0 means contiguous.
bool fill_strides(int heads, int width, int unit, int64_t* ts, int64_t* hs) {
  if (*hs == 0) *hs = width;
  if (*ts == 0) *ts = (int64_t)heads * *hs;
  return *hs >= width && *ts >= width && *hs % unit == 0 && *ts % unit == 0;
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_attn_create(mla_attn_t* out, int max_batch, int heads) {
  if (out == nullptr) return MLA_EINVAL;
  *out = nullptr;
  if (max_batch < 1 || max_batch > MLA_MAX_BATCH || heads < 1 || heads > MLA_MAX_ROW_HEADS)
    return MLA_EINVAL;
  mla_attn* h = static_cast<mla_attn*>(calloc(1, sizeof(mla_attn)));
  if (h == nullptr) return MLA_ENOMEM;
  h->heads = heads;
  h->max_batch = max_batch;
  int rc = MLA_ECUDA;
  const int gh = mla::attn_most_heads(heads);
  const int groups = (heads + gh - 1) / gh;
  size_t slots = 0;
  if (cudaGetDevice(&h->device) != cudaSuccess) goto fail;
  if (cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
    goto fail;
  if (h->num_sms > mla::kMaxCtas || groups > h->num_sms) {
    rc = MLA_EUNSUPPORTED;
    goto fail;
  }
  if (mla::prepare_attn_tc() != cudaSuccess || mla::prepare_attn_ds() != cudaSuccess ||
      mla::prepare_attn_nv() != cudaSuccess)
    goto fail;
  slots = (size_t)(h->num_sms / groups) * 2 * groups * gh;
  rc = MLA_ENOMEM;
  if (cudaMalloc(&h->err, 256) != cudaSuccess ||
      cudaMalloc(&h->part_o, slots * mla::kKvLora * sizeof(float)) != cudaSuccess ||
      cudaMalloc(&h->part_ml, slots * sizeof(float2)) != cudaSuccess)
    goto fail;
  rc = MLA_ECUDA;
  if (cudaMemset(h->err, 0, 256) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) goto fail;
  *out = h;
  return MLA_OK;
fail:
  mla_attn_destroy(h);
  cudaGetLastError();
  return rc;
}

int mla_attn_decode(mla_attn_t h, int batch, const void* q_latent, int64_t ql_token_stride,
                    int64_t ql_head_stride, const void* q_pe, int64_t qp_token_stride,
                    int64_t qp_head_stride, const float* q_scale_inv, const void* kv_cache,
                    int64_t num_pages, int page_size, int layout, const float* k_scale,
                    const int32_t* block_table, int64_t bt_stride, int table_rows,
                    const int32_t* token_row, const int32_t* lens, const int32_t* sel,
                    int64_t sel_stride, const int32_t* sel_count, float softmax_scale, void* out,
                    int64_t out_token_stride, int64_t out_head_stride, float* lse, void* stream) {
  return mla_attn_decode_cols(h, batch, q_latent, ql_token_stride, ql_head_stride, q_pe, qp_token_stride,
                              qp_head_stride, q_scale_inv, kv_cache, num_pages, page_size, layout, k_scale,
                              block_table, bt_stride, bt_stride, table_rows, token_row, lens, sel, sel_stride,
                              sel_stride, sel_count, softmax_scale, out, out_token_stride, out_head_stride, lse,
                              stream);
}

int mla_attn_decode_cols(mla_attn_t h, int batch, const void* q_latent, int64_t ql_token_stride,
                         int64_t ql_head_stride, const void* q_pe, int64_t qp_token_stride,
                         int64_t qp_head_stride, const float* q_scale_inv, const void* kv_cache,
                         int64_t num_pages, int page_size, int layout, const float* k_scale,
                         const int32_t* block_table, int64_t bt_stride, int64_t bt_cols, int table_rows,
                         const int32_t* token_row, const int32_t* lens, const int32_t* sel,
                         int64_t sel_stride, int64_t sel_cols, const int32_t* sel_count,
                         float softmax_scale, void* out, int64_t out_token_stride,
                         int64_t out_head_stride, float* lse, void* stream) {
  if (h == nullptr || batch < 1 || batch > h->max_batch) return MLA_EINVAL;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return mla::launched(cudaErrorInvalidDevice);
  if (dev != h->device) return MLA_EINVAL;  // its workspace lies elsewhere
  if (q_latent == nullptr || q_pe == nullptr || kv_cache == nullptr || block_table == nullptr ||
      lens == nullptr || out == nullptr)
    return MLA_EINVAL;
  if (!mla::known_layout(layout) || (mla::row_scaled(layout) && k_scale == nullptr)) return MLA_EINVAL;
  if (num_pages < 1 || page_size < 1 || bt_cols < 1 || bt_stride < bt_cols || table_rows < 1) return MLA_EINVAL;
  if (token_row == nullptr && table_rows < batch) return MLA_EINVAL;
  if ((sel == nullptr) != (sel_count == nullptr)) return MLA_EINVAL;
  if (sel != nullptr && (sel_cols < 1 || sel_stride < sel_cols)) return MLA_EINVAL;
  if (!(softmax_scale >= 0.0f) || softmax_scale > 3.0e38f) return MLA_EINVAL;
  const int unit = q_scale_inv != nullptr ? 16 : 8;
  if (!mla::fill_strides(h->heads, mla::kKvLora, unit, &ql_token_stride, &ql_head_stride) ||
      !mla::fill_strides(h->heads, mla::kRope, unit, &qp_token_stride, &qp_head_stride) ||
      !mla::fill_strides(h->heads, mla::kKvLora, 8, &out_token_stride, &out_head_stride))
    return MLA_EINVAL;
  if (!mla::aligned16(q_latent) || !mla::aligned16(q_pe) || !mla::aligned16(kv_cache) ||
      !mla::aligned16(out) || !mla::aligned4(q_scale_inv) || !mla::aligned4(k_scale) ||
      !mla::aligned4(block_table) || !mla::aligned4(token_row) || !mla::aligned4(lens) ||
      !mla::aligned4(sel) || !mla::aligned4(sel_count) || !mla::aligned4(lse))
    return MLA_EINVAL;

  mla::AttnArgs a = {};
  a.q_latent = static_cast<const uint8_t*>(q_latent);
  a.q_pe = static_cast<const uint8_t*>(q_pe);
  a.ql_ts = ql_token_stride;
  a.ql_hs = ql_head_stride;
  a.qp_ts = qp_token_stride;
  a.qp_hs = qp_head_stride;
  a.q_scale_inv = q_scale_inv;
  a.cache = static_cast<const uint8_t*>(kv_cache);
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.layout = layout;
  a.k_scale = k_scale;
  a.table = block_table;
  a.bt_stride = bt_stride;
  a.bt_cols = mla::counted_cols(bt_cols);
  a.table_rows = table_rows;
  a.token_row = token_row;
  a.lens = lens;
  a.sel = sel;
  a.sel_stride = sel_stride;
  a.sel_cols = mla::counted_cols(sel_cols);
  a.sel_count = sel_count;
  a.scale = softmax_scale;
  a.out = static_cast<uint16_t*>(out);
  a.o_ts = out_token_stride;
  a.o_hs = out_head_stride;
  a.lse = lse;
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.err = h->err;
  a.heads = h->heads;
  a.batch = batch;
  const int gh = a.cta_heads = mla::attn_cta_heads(a, h->num_sms);
  a.groups = (h->heads + gh - 1) / gh;
  a.heads_pad = a.groups * gh;
  a.workers = h->num_sms / a.groups;
  a.lead = mla::attn_lead(a);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (layout) {
    case MLA_KV_FP8_DS_MLA: e = mla::launch_attn_ds(a, st); break;
    case MLA_KV_NVFP4_DS_MLA: e = mla::launch_attn_nv(a, st); break;
    default: e = mla::launch_attn_tc(a, st);
  }
  int rc = mla::launched(e);
  if (rc != MLA_OK) return rc;
  return mla::launched(mla::launch_join(a, h->num_sms, st));
}

int mla_attn_get_error(mla_attn_t h, unsigned* device_flags, void* stream) {
  if (h == nullptr || device_flags == nullptr) return MLA_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, h->err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemsetAsync(h->err, 0, sizeof(uint32_t), s) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ECUDA;
  }
  *device_flags = v;
  return MLA_OK;
}

void mla_attn_destroy(mla_attn_t h) {
  if (h == nullptr) return;
  if (h->err) cudaFree(h->err);
  if (h->part_o) cudaFree(h->part_o);
  if (h->part_ml) cudaFree(h->part_ml);
  free(h);
}

int mla_tables_step(int rows, const int32_t* new_tokens, const int32_t* lens, int32_t* lens_out,
                    int32_t* block_table, int64_t bt_stride, int32_t* free_pages,
                    const int32_t* free_count, int32_t* free_count_out, int64_t num_pages,
                    int page_size, int max_tokens, int64_t* slot_mapping, int32_t* token_row,
                    int32_t* token_len, int32_t* cu_tokens, unsigned* device_flags, void* stream) {
  if (rows < 1 || rows > MLA_MAX_TABLE_ROWS || bt_stride < 1 || num_pages < 1 ||
      num_pages > 0x7FFFFFFF || page_size < 1 || max_tokens < 1)
    return MLA_EINVAL;
  if (new_tokens == nullptr || lens == nullptr || lens_out == nullptr || block_table == nullptr ||
      free_pages == nullptr || free_count == nullptr || free_count_out == nullptr ||
      slot_mapping == nullptr || token_row == nullptr || token_len == nullptr || cu_tokens == nullptr)
    return MLA_EINVAL;
  if (!mla::aligned4(new_tokens) || !mla::aligned4(lens) || !mla::aligned4(lens_out) ||
      !mla::aligned4(block_table) || !mla::aligned4(free_pages) || !mla::aligned4(free_count) ||
      !mla::aligned4(free_count_out) || !mla::aligned4(token_row) || !mla::aligned4(token_len) ||
      !mla::aligned4(cu_tokens) || !mla::aligned4(device_flags) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return MLA_EINVAL;
  const mla::TableArgs t{rows,          new_tokens, lens,           lens_out,  block_table,
                         bt_stride,     free_pages, free_count,     free_count_out, num_pages,
                         page_size,     max_tokens, slot_mapping,   token_row, token_len,
                         cu_tokens,     device_flags};
  return mla::launched(mla::launch_tables(t, static_cast<cudaStream_t>(stream)));
}

int mla_blocks_mean(const void* kv_cache, int64_t num_pages, int page_size, int layout,
                    const float* k_scale, const int32_t* block_table, int64_t bt_stride, int rows,
                    const int32_t* lens_from, const int32_t* lens_to, void* mean,
                    unsigned* device_flags, void* stream) {
  return mla_blocks_mean_cols(kv_cache, num_pages, page_size, layout, k_scale, block_table, bt_stride, bt_stride,
                              rows, lens_from, lens_to, mean, device_flags, stream);
}

int mla_blocks_mean_cols(const void* kv_cache, int64_t num_pages, int page_size, int layout,
                         const float* k_scale, const int32_t* block_table, int64_t bt_stride,
                         int64_t bt_cols, int rows, const int32_t* lens_from, const int32_t* lens_to,
                         void* mean, unsigned* device_flags, void* stream) {
  if (kv_cache == nullptr || block_table == nullptr || lens_from == nullptr || lens_to == nullptr ||
      mean == nullptr)
    return MLA_EINVAL;
  if (!mla::known_layout(layout) || (mla::row_scaled(layout) && k_scale == nullptr)) return MLA_EINVAL;
  if (num_pages < 1 || page_size < 1 || bt_cols < 1 || bt_stride < bt_cols || rows < 1 ||
      rows > MLA_MAX_TABLE_ROWS)
    return MLA_EINVAL;
  if (!mla::aligned16(kv_cache) || !mla::aligned16(mean) || !mla::aligned4(k_scale) ||
      !mla::aligned4(block_table) || !mla::aligned4(lens_from) || !mla::aligned4(lens_to) ||
      !mla::aligned4(device_flags))
    return MLA_EINVAL;
  int sms = 0;
  if (mla::sm_count(&sms) != MLA_OK) return MLA_ECUDA;
  const mla::MeanArgs m{static_cast<const uint8_t*>(kv_cache), num_pages, page_size, layout, k_scale,
                        block_table, bt_stride, mla::counted_cols(bt_cols), rows, lens_from, lens_to,
                        static_cast<uint16_t*>(mean), device_flags};
  return mla::launched(mla::launch_blocks_mean(m, sms, static_cast<cudaStream_t>(stream)));
}

int mla_blocks_score(int batch, int heads, const void* q_latent, int64_t ql_token_stride,
                     int64_t ql_head_stride, const void* q_pe, int64_t qp_token_stride,
                     int64_t qp_head_stride, const float* q_scale_inv, const void* mean,
                     int64_t num_pages, int page_size, const int32_t* block_table,
                     int64_t bt_stride, int table_rows, const int32_t* token_row,
                     const int32_t* lens, float* scores, int64_t scores_stride,
                     unsigned* device_flags, void* stream) {
  if (batch < 1 || batch > MLA_MAX_BATCH || heads < 1 || heads > MLA_MAX_ROW_HEADS) return MLA_EINVAL;
  if (q_latent == nullptr || q_pe == nullptr || mean == nullptr || block_table == nullptr ||
      lens == nullptr || scores == nullptr)
    return MLA_EINVAL;
  if (num_pages < 1 || page_size < 1 || bt_stride < 1 || bt_stride > 0x7FFFFFFF || table_rows < 1 ||
      (token_row == nullptr && table_rows < batch) || scores_stride < bt_stride)
    return MLA_EINVAL;
  const int unit = q_scale_inv != nullptr ? 16 : 8;
  if (!mla::fill_strides(heads, mla::kKvLora, unit, &ql_token_stride, &ql_head_stride) ||
      !mla::fill_strides(heads, mla::kRope, unit, &qp_token_stride, &qp_head_stride))
    return MLA_EINVAL;
  if (!mla::aligned16(q_latent) || !mla::aligned16(q_pe) || !mla::aligned16(mean) ||
      !mla::aligned4(q_scale_inv) || !mla::aligned4(block_table) || !mla::aligned4(token_row) ||
      !mla::aligned4(lens) || !mla::aligned4(scores) || !mla::aligned4(device_flags))
    return MLA_EINVAL;
  int sms = 0;
  if (mla::sm_count(&sms) != MLA_OK) return MLA_ECUDA;
  const mla::ScoreArgs s{batch, heads, static_cast<const uint8_t*>(q_latent),
                         static_cast<const uint8_t*>(q_pe), ql_token_stride, ql_head_stride,
                         qp_token_stride, qp_head_stride, q_scale_inv,
                         static_cast<const uint16_t*>(mean), num_pages, page_size, block_table,
                         bt_stride, table_rows, token_row, lens, scores, scores_stride, device_flags};
  return mla::launched(mla::launch_blocks_score(s, sms, static_cast<cudaStream_t>(stream)));
}

int mla_blocks_select(int batch, const float* scores, int64_t scores_stride, int max_blocks,
                      const int32_t* lens, int page_size, int keep_first, int keep_last, int k,
                      int32_t* sel, int64_t sel_stride, int32_t* sel_count, void* stream) {
  if (batch < 1 || batch > MLA_MAX_BATCH || scores == nullptr || lens == nullptr || sel == nullptr ||
      sel_count == nullptr)
    return MLA_EINVAL;
  if (max_blocks < 1 || scores_stride < max_blocks || page_size < 1 || keep_first < 0 ||
      keep_last < 0 || k < 1 || sel_stride < k)
    return MLA_EINVAL;
  if (!mla::aligned4(scores) || !mla::aligned4(lens) || !mla::aligned4(sel) || !mla::aligned4(sel_count))
    return MLA_EINVAL;
  const mla::SelectArgs s{batch, scores, scores_stride, max_blocks, lens, page_size, keep_first,
                          keep_last, k, sel, sel_stride, sel_count};
  return mla::launched(mla::launch_blocks_select(s, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
