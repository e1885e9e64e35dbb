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

// Eight E2M1 codes, value 2k in the low half of byte k.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h)
        : "r"(w >> (8 * i)));
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h));
  }
}

// A row as 16-byte chunks (chunk c at byte kFirst(c)), each with its columns
// [col(c), col(c) + width(c)).  decode() gives their values: the codes
// themselves for the layouts whose scale is one FP32 for the row (the caller
// applies it), the exact products of code and scale for the two ds layouts
// (at most 4 + 4 significant bits: exact in BF16 too).
template <int LAYOUT>
struct RowChunks;

template <>
struct RowChunks<MLA_KV_FP8_E4M3> {
  static constexpr int kBytes = kRowE4m3, kChunks = 36, kMax = 16;
  __device__ static int offset(int c) { return 16 * c; }
  __device__ static int col(int c) { return 16 * c; }
  __device__ static int width(int) { return 16; }
  __device__ static void decode(const uint8_t*, int, uint4 w, float (&v)[kMax]) {
    e4m3x4_values(w.x, v);
    e4m3x4_values(w.y, v + 4);
    e4m3x4_values(w.z, v + 8);
    e4m3x4_values(w.w, v + 12);
  }
};

template <>
struct RowChunks<MLA_KV_FP8_DS_MLA> {
  static constexpr int kBytes = kRowDs, kChunks = 40, kMax = 16;
  __device__ static int offset(int c) { return c < 32 ? 16 * c : kDsRope + 16 * (c - 32); }
  __device__ static int col(int c) { return c < 32 ? 16 * c : kKvLora + 8 * (c - 32); }
  __device__ static int width(int c) { return c < 32 ? 16 : 8; }
  __device__ static void decode(const uint8_t* row, int c, uint4 w, float (&v)[kMax]) {
    if (c < 32) {
      RowChunks<MLA_KV_FP8_E4M3>::decode(row, c, w, v);
      const float s = *reinterpret_cast<const float*>(row + kDsScales + 4 * (c >> 3));
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= s;
    } else {
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(ww[i]);
        v[2 * i + 1] = bf16hi(ww[i]);
        v[8 + 2 * i] = 0.f;
        v[9 + 2 * i] = 0.f;
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
  __device__ static void decode(const uint8_t* row, int c, uint4 w, float (&v)[kMax]) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    if (c < 16) {
      // blocks 2c and 2c + 1 of 16 values
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int s = 2 * c + b;
        const float sc = e4m3x2_value(row[kNvScales + 8 * (s & 3) + (s >> 2)]).x;
        e2m1x8_values(ww[2 * b], v + 16 * b);
        e2m1x8_values(ww[2 * b + 1], v + 16 * b + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[16 * b + i] *= sc;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) e4m3x4_values(ww[i], v + 4 * i);
#pragma unroll
      for (int i = 16; i < 32; ++i) v[i] = 0.f;
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
