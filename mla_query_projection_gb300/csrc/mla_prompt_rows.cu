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

// A CTA takes 64 rows (tokens' heads, one after another) after another, four threads
// for two neighbours: thread j of four has pairs 8 j .. 8 j + 7, whose values are 32
// bytes in a row (neighbours as pairs) or 16 bytes of each half (halves as pairs), and
// reads their sines and cosines once where both rows are one token's.  (A row a thread
// took 9.9 us for 8,191 tokens of 16 heads, so 8.6: what bounds it is shared memory.)
// The next rows' values are on their way, and their tokens' sines and cosines worked
// out once, into shared memory, while these are turned.  (Without that, 4,096 tokens of
// 128 heads took 35 us, so 27: 5.0 TB/s.)  A thread reads all it turns before it
// writes, so the output may be the input.
constexpr int kRopeRows = 64, kRopeThreads = 2 * kRopeRows;

// MANY: a CTA has more than one round.
template <bool INTERLEAVED, bool MANY>
__global__ void __launch_bounds__(kRopeThreads, 6) mla_rope_kernel(const __grid_constant__ RopeArgs r, int64_t tokens, int heads,
                                                          const uint16_t* x, int64_t x_ts, int64_t x_hs, uint16_t* out,
                                                          int64_t o_ts, int64_t o_hs) {
  __shared__ float2 turns[MANY ? 2 : 1][(kRopeRows + 1) * kRopePairs];
  const int tid = threadIdx.x, j = tid & 3;
  const int64_t rows = tokens * heads, step = (int64_t)gridDim.x * kRopeRows;
  // words 0..3 and 4..7 of a thread's share of a row, in values from its start
  const int a0 = INTERLEAVED ? 16 * j : 8 * j, a1 = INTERLEAVED ? 16 * j + 8 : 32 + 8 * j;
  const RopeLane rope(r, tid & 31);
  const bool narrow = rows <= 0xFFFFFFFFll;
  auto token_of = [&](int64_t row) -> int64_t { return narrow ? (uint32_t)row / (uint32_t)heads : row / heads; };
  pdl_wait();
  pdl_launch_dependents();
  struct Part {
    uint4 v[2][2];
    int64_t t;   // the first row's token
    int h, n;    // its head, its token's place among the CTA's
  };
  // a thread's values of the rows from row0 on, and the turns of their tokens
  auto fetch = [&](int64_t row0, float2* turn) -> Part {
    Part p = {};
    const int64_t row = row0 + 2 * (tid >> 2), t0 = token_of(row0);
    if (row < rows) {
      p.t = token_of(row);
      p.h = (int)(row - p.t * heads);
      p.n = (int)(p.t - t0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool over = p.h + e >= heads;  // the next token's first head
        const uint16_t* at = x + (p.t + over) * x_ts + (int64_t)(over ? 0 : p.h + e) * x_hs;
        if (e == 0 || row + 1 < rows) {
          p.v[e][0] = *reinterpret_cast<const uint4*>(at + a0);
          p.v[e][1] = *reinterpret_cast<const uint4*>(at + a1);
        }
      }
    }
    const int count = (int)(token_of((row0 + kRopeRows < rows ? row0 + kRopeRows : rows) - 1) - t0);
    for (int n = tid >> 5; n <= count; n += kRopeThreads / 32) turn[n * kRopePairs + (tid & 31)] = rope.at(t0 + n);
    return p;
  };
  int64_t row0 = (int64_t)blockIdx.x * kRopeRows;
  Part p = fetch(row0, turns[0]);
  for (int b = 0; row0 < rows; b ^= 1, row0 += step) {
    __syncthreads();
    Part next = {};
    if (MANY && row0 + step < rows) next = fetch(row0 + step, turns[b ^ 1]);
    const int64_t row = row0 + 2 * (tid >> 2);
    if (row < rows) {
      float4 f[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (e == 1 && row + 1 >= rows) break;
        const bool over = p.h + e >= heads;
        if (e == 0 || over) {
          const float4* cs = reinterpret_cast<const float4*>(turns[b] + (p.n + over) * kRopePairs + 8 * j);  // two pairs each
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = cs[i];
        }
        const uint4 v0 = p.v[e][0], v1 = p.v[e][1];
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (INTERLEAVED) {
            const float2 u = turned(bf16lo(w[2 * i]), bf16hi(w[2 * i]), f[i].x, f[i].y);
            const float2 v = turned(bf16lo(w[2 * i + 1]), bf16hi(w[2 * i + 1]), f[i].z, f[i].w);
            y[2 * i] = pack_bf16x2(u.x, u.y);
            y[2 * i + 1] = pack_bf16x2(v.x, v.y);
          } else {
            const float2 u = turned(bf16lo(w[i]), bf16lo(w[i + 4]), f[i].x, f[i].y);
            const float2 v = turned(bf16hi(w[i]), bf16hi(w[i + 4]), f[i].z, f[i].w);
            y[i] = pack_bf16x2(u.x, v.x);
            y[i + 4] = pack_bf16x2(u.y, v.y);
          }
        }
        uint16_t* o = out + (p.t + over) * o_ts + (int64_t)(over ? 0 : p.h + e) * o_hs;
        *reinterpret_cast<uint4*>(o + a0) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(o + a1) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    if (!MANY) break;
    p = next;
  }
}

// --------------------------------------------------------------- writing
//
// One warp a token: the decode step's insert (the same sums in the same order,
// so the same bytes), with the norm and the rotation optional, and the row
// handed on in BF16 where the caller wants it.  A lane has latent columns
// 8 lane .. and 256 + 8 lane .., and two values of the rope part.  The next token's row is on its way while this one is worked on.

// a b + c of two, each rounded once, down: a sum of zeros of both signs is -0.
__device__ __forceinline__ float2 fma2_rm(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rm.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Quotients of a token by one divisor, each correctly rounded, as a division gives
// them: by P. Markstein's theorem (IBM Journal of Research and Development 34, 1990),
// with y the rounded reciprocal of b and q = a y rounded, q + (a - b q) y rounded once
// is the rounded a / b.  What is in brackets is exact, so that its rounding decides
// the sign of a zero alone: -0 leaves q its own.  Where the quotient is far beyond
// E4M3's range the product is as good (and may be infinite); divisors near the ends of
// FP32's range, and negative ones, are divided by.
struct Divisor {
  float b, y;
  bool plain;
  __device__ __forceinline__ explicit Divisor(float divisor) {
    b = divisor;
    y = __frcp_rn(divisor);
    plain = !(divisor >= 0x1p-60f && divisor <= 0x1p60f);
  }
  // two, in packed arithmetic
  __device__ __forceinline__ float2 quotients(float2 a) const {
    const float2 y2 = make_float2(y, y), q = fmul2_rn(a, y2);
    const float2 r = fma2(fma2_rm(make_float2(-q.x, -q.y), make_float2(b, b), a), y2, q);
    return make_float2(fabsf(q.x) < 0x1p20f ? r.x : q.x, fabsf(q.y) < 0x1p20f ? r.y : q.y);
  }
  // the E4M3 codes of a pair of BF16 values, of two pairs
  __device__ __forceinline__ uint16_t codes(uint32_t w) const {
    const float2 a = make_float2(bf16lo(w), bf16hi(w));
    const float2 p = plain ? make_float2(__fdiv_rn(a.x, b), __fdiv_rn(a.y, b)) : quotients(a);
    return e4m3x2(p.x, p.y);
  }
  __device__ __forceinline__ uint32_t codes(uint32_t w0, uint32_t w1) const {
    float2 p = make_float2(bf16lo(w0), bf16hi(w0)), q = make_float2(bf16lo(w1), bf16hi(w1));
    if (plain) {
      p = make_float2(__fdiv_rn(p.x, b), __fdiv_rn(p.y, b));
      q = make_float2(__fdiv_rn(q.x, b), __fdiv_rn(q.y, b));
    } else {
      p = quotients(p);
      q = quotients(q);
    }
    return (uint32_t)e4m3x2(p.x, p.y) | ((uint32_t)e4m3x2(q.x, q.y) << 16);
  }
};

template <int LAYOUT>
__global__ void __launch_bounds__(256, 4) mla_cache_write_kernel(const __grid_constant__ CacheWriteArgs w) {
  constexpr bool kDs = LAYOUT == MLA_KV_FP8_DS_MLA, kNv = LAYOUT == MLA_KV_NVFP4_DS_MLA;
  constexpr int kBytes = RowChunks<LAYOUT>::kBytes;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  const bool rope_on = w.rope.positions != nullptr;
  const RopeLane rope(w.rope, lane);
  const DecodeArgs none = {};
  pdl_wait();
  pdl_launch_dependents();
  const float tensor_scale = LAYOUT == MLA_KV_FP8_E4M3 ? *w.k_scale : 1.0f;
  struct Token {
    uint4 v[2];
    uint32_t pe;
    int64_t slot;
    float2 turn;
    float scale;
  };
  auto fetch = [&](int64_t t) -> Token {
    Token k;
    const uint16_t* kv = w.kv_c + t * w.kv_c_stride;
    k.v[0] = *reinterpret_cast<const uint4*>(kv + 8 * lane);
    k.v[1] = *reinterpret_cast<const uint4*>(kv + 256 + 8 * lane);
    k.pe = *reinterpret_cast<const uint32_t*>(w.k_pe + t * w.k_pe_stride + 2 * lane);
    k.slot = w.slots[t];
    if (k.slot >= w.capacity) {
      if (lane == 0 && w.flags != nullptr) atomicOr(w.flags, MLA_DEVERR_BAD_SLOT);
      k.slot = -1;
    }
    k.scale = tensor_scale;
    if (LAYOUT == MLA_KV_FP8_E4M3_PAGE && k.slot >= 0)
      k.scale = w.k_scale[k.slot <= 0xFFFFFFFFll ? (uint32_t)k.slot / (uint32_t)w.page_size : k.slot / w.page_size];
    k.turn = rope_on ? rope.at(t) : make_float2(1.f, 0.f);
    return k;
  };
  int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= w.tokens) return;
  Token k = fetch(t);
  for (;;) {
    const int64_t after = t + warps;
    Token next;
    if (after < w.tokens) next = fetch(after);
    uint32_t pe = k.pe;
    if (rope_on) {
      if (w.rope.spec.interleaved) {  // the lane's pair
        const float2 p = turned(bf16lo(pe), bf16hi(pe), k.turn.x, k.turn.y);
        pe = pack_bf16x2(p.x, p.y);
      } else {  // one value each of two pairs
        const int p0 = 2 * (lane & 15);
        const float c0 = __shfl_sync(0xFFFFFFFFu, k.turn.x, p0), c1 = __shfl_sync(0xFFFFFFFFu, k.turn.x, p0 + 1);
        float s0 = __shfl_sync(0xFFFFFFFFu, k.turn.y, p0), s1 = __shfl_sync(0xFFFFFFFFu, k.turn.y, p0 + 1);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, pe, 16);
        if (lane < 16) {
          s0 = -s0;
          s1 = -s1;
        }
        pe = pack_bf16x2(fmaf(bf16lo(pe), c0, bf16lo(other) * s0), fmaf(bf16hi(pe), c1, bf16hi(other) * s1));
      }
    }
    uint32_t n[2][4] = {{k.v[0].x, k.v[0].y, k.v[0].z, k.v[0].w}, {k.v[1].x, k.v[1].y, k.v[1].z, k.v[1].w}};
    if (w.gamma != nullptr) {
      float x[8];
      const float s0 = kv_group_ss(k.v[0], x), s1 = kv_group_ss(k.v[1], x);
      const float total = warp_sum(s0) + warp_sum(s1);
      const float rr = __frsqrt_rn(__fadd_rn(__fmul_rn(total, 1.0f / 512.0f), w.eps));
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4 gv = *reinterpret_cast<const uint4*>(w.gamma + 256 * g + 8 * lane);
        const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) n[g][i] = rms_scale_bf16x2(n[g][i], rr, gw[i]);
      }
    }
    if (w.rows != nullptr) {
      uint16_t* o = w.rows + t * w.rows_stride;
#pragma unroll
      for (int g = 0; g < 2; ++g)
        *reinterpret_cast<uint4*>(o + 256 * g + 8 * lane) = make_uint4(n[g][0], n[g][1], n[g][2], n[g][3]);
      *reinterpret_cast<uint32_t*>(o + kKvLora + 2 * lane) = pe;
    }
    if (k.slot >= 0) {
      uint8_t* row = w.cache + k.slot * kBytes;
      if constexpr (kDs || kNv) {
        uint32_t p[4];  // (as the step stores it: eight values for each of the first eight lanes)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xFFFFFFFFu, pe, (4 * lane + i) & 31);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16lo(n[g][i]);
            x[2 * i + 1] = bf16hi(n[g][i]);
          }
          kv_store_group(none, row, x, g == 0 ? make_uint4(p[0], p[1], p[2], p[3]) : make_uint4(0, 0, 0, 0), lane + 32 * g, kDs, kNv, 1.0f);
        }
      } else {
        const Divisor d(k.scale);
#pragma unroll
        for (int g = 0; g < 2; ++g)
          *reinterpret_cast<uint2*>(row + 256 * g + 8 * lane) = make_uint2(d.codes(n[g][0], n[g][1]), d.codes(n[g][2], n[g][3]));
        *reinterpret_cast<uint16_t*>(row + kKvLora + 2 * lane) = d.codes(pe);
      }
    }
    if (after >= w.tokens) break;
    t = after;
    k = next;
  }
}

// --------------------------------------------------------------- reading
//
// A row's 576 values are 72 groups of eight, whatever the layout: a thread turns the 4, 8
// or 16 bytes of a group into 16 bytes of output, so that a warp's loads and stores
// both are rows of bytes without gaps.  (16 bytes a load and two stores of 16 took 28 us
// for 65,536 rows.)  A CTA takes a batch of R rows after another.  Where rows lie is
// found two batches ahead (the request by bisection, the page from the table, a thread
// each: three trips to memory), their groups are loaded one batch ahead.
constexpr int kReadThreads = 256, kReadGroups = kRowElems / 8;

template <int LAYOUT>
struct ReadGroup;

template <>
struct ReadGroup<MLA_KV_FP8_E4M3> {
  static constexpr int kBytes = kRowE4m3, kAhead = 8;
  using Raw = uint2;
  __device__ static Raw load(const uint8_t* row, int g) { return *reinterpret_cast<const uint2*>(row + 8 * g); }
  __device__ static void values(Raw w, int, float scale, float (&v)[8]) {
    e4m3x4_values(w.x, v);
    e4m3x4_values(w.y, v + 4);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 p = fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(scale, scale));
      v[i] = p.x;
      v[i + 1] = p.y;
    }
  }
};
template <>
struct ReadGroup<MLA_KV_FP8_E4M3_PAGE> : ReadGroup<MLA_KV_FP8_E4M3> {};
template <>
struct ReadGroup<MLA_KV_FP8_DS_MLA> {
  static constexpr int kBytes = kRowDs, kAhead = 4;
  using Raw = uint4;  // codes, scale; or eight BF16
  __device__ static Raw load(const uint8_t* row, int g) {
    if (g >= 64) return *reinterpret_cast<const uint4*>(row + kDsRope + 16 * (g - 64));
    const uint2 c = *reinterpret_cast<const uint2*>(row + 8 * g);
    return make_uint4(c.x, c.y, *reinterpret_cast<const uint32_t*>(row + kDsScales + 4 * (g >> 4)), 0);
  }
  __device__ static void values(Raw w, int g, float, float (&v)[8]) {
    if (g < 64) {
      ReadGroup<MLA_KV_FP8_E4M3>::values(make_uint2(w.x, w.y), g, __uint_as_float(w.z), v);
    } else {
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(x[i]);
        v[2 * i + 1] = bf16hi(x[i]);
      }
    }
  }
};
template <>
struct ReadGroup<MLA_KV_NVFP4_DS_MLA> {
  static constexpr int kBytes = kRowNvfp4, kAhead = 8;
  using Raw = uint2;  // codes, scale; or eight E4M3
  __device__ static Raw load(const uint8_t* row, int g) {
    if (g >= 64) return *reinterpret_cast<const uint2*>(row + kNvRope + 8 * (g - 64));
    const int s = g >> 1;
    return make_uint2(*reinterpret_cast<const uint32_t*>(row + 4 * g), row[kNvScales + 8 * (s & 3) + (s >> 2)]);
  }
  __device__ static void values(Raw w, int g, float, float (&v)[8]) {
    if (g >= 64) {
      e4m3x4_values(w.x, v);
      e4m3x4_values(w.y, v + 4);
      return;
    }
    uint32_t h[4];
    e2m1x8_scaled(w.x, e4m3x2_f16(0x0101u * w.y), h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = v[2 * i + 1] = 0.f;
      add_f16x2(h[i], v + 2 * i);
    }
  }
};

template <int LAYOUT>
__global__ void __launch_bounds__(kReadThreads, 4) mla_cache_read_kernel(const __grid_constant__ CacheReadArgs a, int R) {
  using G = ReadGroup<LAYOUT>;
  using Raw = typename G::Raw;
  constexpr int kAhead = G::kAhead, kMost = kAhead * kReadThreads / kReadGroups;
  __shared__ int64_t source[3][kMost];  // byte offset of the cache row; -1: zeros, -2: left as it is
  __shared__ float scale[3][kMost];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t first = a.cu[0], last = min((int64_t)a.cu[a.requests], a.max_rows), step = (int64_t)gridDim.x * R;
  auto look_up = [&](int64_t row0, int buffer) {
    if (tid >= R) return;
    const int64_t i = row0 + tid;
    int64_t src = -2;
    float sc = 1.0f;
    if (i < last && i >= first) {
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
        src = (page * a.page_size + off) * G::kBytes;
        sc = page_scale(a.k_scale, LAYOUT, page);
      } else {
        src = -1;
        if (a.flags != nullptr) atomicOr(a.flags, MLA_DEVERR_BAD_SLOT);
      }
    }
    source[buffer][tid] = src;
    scale[buffer][tid] = sc;
  };
  const int groups = R * kReadGroups;
  auto load = [&](Raw (&to)[kAhead], int b) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = tid + u * kReadThreads, r = k / kReadGroups;
      to[u] = Raw{};
      if (k < groups && source[b][r] >= 0) to[u] = G::load(a.cache + source[b][r], k - r * kReadGroups);
    }
  };
  int64_t row0 = (int64_t)blockIdx.x * R;
  if (row0 >= last) return;
  Raw w[kAhead];
  look_up(row0, 0);
  const bool many = row0 + step < last;
  if (many) look_up(row0 + step, 1);
  __syncthreads();
  load(w, 0);
  for (int b = 0; row0 < last; row0 += step) {
    const int b1 = b == 2 ? 0 : b + 1, b2 = b1 == 2 ? 0 : b1 + 1;
    Raw next[kAhead];
    if (row0 + step < last) {
      if (row0 + 2 * step < last) look_up(row0 + 2 * step, b2);
      load(next, b1);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = tid + u * kReadThreads, r = k / kReadGroups, g = k - r * kReadGroups;
      if (k >= groups || source[b][r] == -2) continue;
      float v[8];
      G::values(w[u], g, scale[b][r], v);
      *reinterpret_cast<uint4*>(a.rows + (row0 + r) * a.rows_stride + 8 * g) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    if (!many) break;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) w[u] = next[u];
    b = b1;
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

// Rows a batch: as many as the threads take with all their loads, or fewer where that
// gives every SM four CTAs (a row alone at the least).
template <int LAYOUT>
cudaError_t launch_read(const CacheReadArgs& a, int sms, void* stream) {
  constexpr int kMost = ReadGroup<LAYOUT>::kAhead * kReadThreads / kReadGroups;
  const int64_t even = (a.max_rows + 4 * sms - 1) / (4 * sms);
  const int R = (int)(even < kMost ? even : kMost);
  int64_t ctas = (a.max_rows + R - 1) / R;
  if (ctas > 4 * (int64_t)sms) ctas = 4 * (int64_t)sms;
  Launch l(dim3((unsigned)ctas), kReadThreads, stream);
  return cudaLaunchKernelEx(&l.cfg, mla_cache_read_kernel<LAYOUT>, a, R);
}

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
    const double f = fabs(inv_freq[p]), hi = f * kTurn;
    const double lo = fma(f, kTurn, -hi) + f * kTurnRest;
    const double part = hi - floor(hi);  // exact, in [0, 1)
    const uint64_t turns = (uint64_t)ldexp(part, 64) + (uint64_t)(int64_t)llrint(ldexp(lo, 64));
    h->spec.turns[p] = inv_freq[p] < 0.0 ? 0 - turns : turns;  // (1 less a small one would not be exact)
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
  constexpr int64_t most = (int64_t)1 << 38;
  if (x_head_stride >= most || x_token_stride >= most || out_head_stride >= most || out_token_stride >= most)
    return MLA_EINVAL;
  if (x_head_stride == 0) x_head_stride = mla::kRope;
  if (x_token_stride == 0) x_token_stride = heads * x_head_stride;
  if (out_head_stride == 0) out_head_stride = mla::kRope;
  if (out_token_stride == 0) out_token_stride = heads * out_head_stride;
  if (x_head_stride < mla::kRope || x_token_stride < mla::kRope || out_head_stride < mla::kRope ||
      out_token_stride < mla::kRope || (x_head_stride | x_token_stride | out_head_stride | out_token_stride) % 8)
    return MLA_EINVAL;
  if (!mla::aligned16(x) || !mla::aligned16(out) || !mla::aligned4(positions)) return MLA_EINVAL;
  if (tokens > INT64_MAX / 2048) return MLA_EINVAL;
  int sms = 0;
  if (!mla::sm_count(&sms)) return MLA_ECUDA;
  int64_t ctas = (tokens * heads + mla::kRopeRows - 1) / mla::kRopeRows;
  const bool many = ctas > 6 * (int64_t)sms;  // (six CTAs an SM are resident)
  if (many) ctas = 6 * (int64_t)sms;
  mla::Launch l(dim3((unsigned)ctas), mla::kRopeThreads, stream);
  const mla::RopeArgs r{h->spec, positions, pos_stride, pos_offset};
  auto kernel = h->spec.interleaved ? (many ? mla::mla_rope_kernel<true, true> : mla::mla_rope_kernel<true, false>)
                                    : (many ? mla::mla_rope_kernel<false, true> : mla::mla_rope_kernel<false, false>);
  return mla::launched(cudaLaunchKernelEx(&l.cfg, kernel, r, tokens, heads, static_cast<const uint16_t*>(x),
                                          x_token_stride, x_head_stride, static_cast<uint16_t*>(out), out_token_stride,
                                          out_head_stride));
}

int mla_cache_write(int64_t tokens, const void* kv_c, int64_t kv_c_stride, const void* k_pe, int64_t k_pe_stride,
                    const void* gamma_kv, float eps, mla_rope_t rope, const int32_t* positions, int64_t pos_stride,
                    int64_t pos_offset, const int64_t* slot_mapping, void* kv_cache, int64_t num_pages, int page_size,
                    int layout, const float* k_scale, void* rows, int64_t rows_stride, unsigned* device_flags,
                    void* stream) {
  if (tokens < 0 || tokens > INT64_MAX / 2048 || !mla::known_layout(layout) || (mla::row_scaled(layout) && k_scale == nullptr)) return MLA_EINVAL;
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
  if (ctas > 4 * (int64_t)sms) ctas = 4 * (int64_t)sms;
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
  cudaError_t e;
  switch (layout) {
    case MLA_KV_FP8_DS_MLA: e = mla::launch_read<MLA_KV_FP8_DS_MLA>(a, sms, stream); break;
    case MLA_KV_NVFP4_DS_MLA: e = mla::launch_read<MLA_KV_NVFP4_DS_MLA>(a, sms, stream); break;
    case MLA_KV_FP8_E4M3_PAGE: e = mla::launch_read<MLA_KV_FP8_E4M3_PAGE>(a, sms, stream); break;
    default: e = mla::launch_read<MLA_KV_FP8_E4M3>(a, sms, stream);
  }
  return mla::launched(e);
}

}  // extern "C"
