// mla_rows.cuh - reading the paged latent cache: where a token's row lies and
// what its bytes stand for, in each of the layouts the decode step writes.
#pragma once

#include "../../include/mla_query.h"
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

// Two E4M3 codes (low byte first) as their exact FP16 values, widened.
__device__ __forceinline__ float2 e4m3x2_value(uint16_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float* v) {
  const float2 a = e4m3x2_value((uint16_t)(w & 0xFFFFu)), b = e4m3x2_value((uint16_t)(w >> 16));
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

// Eight E2M1 codes times a scale (twice in `sc`) as four FP16 pairs: exact, at
// most 2 + 4 significant bits.
__device__ __forceinline__ void e2m1x8_scaled(uint32_t w, uint32_t sc, uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 v;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 v, b0;\n\tmul.rn.f16x2 %0, v, %2;\n\t}"
        : "=r"(h[i])
        : "r"(w >> (8 * i)), "r"(sc));
}
// Two E4M3 codes (the low ones of w) as an FP16 pair.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return h;
}

// acc[0..1] += an FP16 pair, in FP32 (one instruction each: no conversion).
__device__ __forceinline__ void add_f16x2(uint32_t h, float* acc) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tadd.f32.f16 %0, l, %0;\n\t"
      "add.f32.f16 %1, u, %1;\n\t}"
      : "+f"(acc[0]), "+f"(acc[1])
      : "r"(h));
}
__device__ __forceinline__ void add_e4m3x4(uint32_t w, float* acc) {
  add_f16x2(e4m3x2_f16(w), acc);
  add_f16x2(e4m3x2_f16(w >> 16), acc + 2);
}

// A row as 16-byte chunks (chunk c at byte offset(c)), each with its columns
// [col(c), col(c) + width(c)).  add() adds their values to FP32 sums: the codes
// themselves for the layouts whose scale is one FP32 for the row (the caller
// applies it), code times scale for the two ds layouts.
template <int LAYOUT>
struct RowChunks;

template <>
struct RowChunks<MLA_KV_FP8_E4M3> {
  static constexpr int kBytes = kRowE4m3, kChunks = 36, kMax = 16;
  __device__ static int offset(int c) { return 16 * c; }
  __device__ static int col(int c) { return 16 * c; }
  __device__ static int width(int) { return 16; }
  __device__ static void add(const uint8_t*, int, uint4 w, float (&acc)[kMax]) {
    add_e4m3x4(w.x, acc);
    add_e4m3x4(w.y, acc + 4);
    add_e4m3x4(w.z, acc + 8);
    add_e4m3x4(w.w, acc + 12);
  }
};

template <>
struct RowChunks<MLA_KV_FP8_DS_MLA> {
  static constexpr int kBytes = kRowDs, kChunks = 40, kMax = 16;
  __device__ static int offset(int c) { return c < 32 ? 16 * c : kDsRope + 16 * (c - 32); }
  __device__ static int col(int c) { return c < 32 ? 16 * c : kKvLora + 8 * (c - 32); }
  __device__ static int width(int c) { return c < 32 ? 16 : 8; }
  __device__ static void add(const uint8_t* row, int c, uint4 w, float (&acc)[kMax]) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    if (c < 32) {
      const float s = *reinterpret_cast<const float*>(row + kDsScales + 4 * (c >> 3));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
        e4m3x4_values(ww[i], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[4 * i + e] = fmaf(v[e], s, acc[4 * i + e]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += bf16lo(ww[i]);
        acc[2 * i + 1] += bf16hi(ww[i]);
      }
    }
  }
};

template <>
struct RowChunks<MLA_KV_NVFP4_DS_MLA> {
  static constexpr int kBytes = kRowNvfp4, kChunks = 20, kMax = 32;
  __device__ static int offset(int c) { return c < 16 ? 16 * c : kNvRope + 16 * (c - 16); }
  __device__ static int col(int c) { return c < 16 ? 32 * c : kKvLora + 16 * (c - 16); }
  __device__ static int width(int c) { return c < 16 ? 32 : 16; }
  __device__ static void add(const uint8_t* row, int c, uint4 w, float (&acc)[kMax]) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    if (c < 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // words 0, 1 are block 2c, words 2, 3 block 2c + 1
        const int s = 2 * c + (i >> 1);
        uint32_t h[4];
        e2m1x8_scaled(ww[i], e4m3x2_f16(0x0101u * row[kNvScales + 8 * (s & 3) + (s >> 2)]), h);
#pragma unroll
        for (int e = 0; e < 4; ++e) add_f16x2(h[e], acc + 8 * i + 2 * e);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) add_e4m3x4(ww[i], acc + 4 * i);
    }
  }
};

template <>
struct RowChunks<MLA_KV_FP8_E4M3_PAGE> : RowChunks<MLA_KV_FP8_E4M3> {};

// Whether a layout's values carry a scale outside the row, and a row's scale.
__host__ __device__ constexpr bool row_scaled(int layout) {
  return layout == MLA_KV_FP8_E4M3 || layout == MLA_KV_FP8_E4M3_PAGE;
}
__device__ __forceinline__ float page_scale(const float* k_scale, int layout, int64_t page) {
  return layout == MLA_KV_FP8_E4M3 ? *k_scale : layout == MLA_KV_FP8_E4M3_PAGE ? k_scale[page] : 1.0f;
}

}  // namespace
}  // namespace mla
