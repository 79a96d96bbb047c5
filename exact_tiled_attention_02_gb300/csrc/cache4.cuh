// cache4.cuh -- device helpers of the 4-bit key/value cache: where a block of
// 16 tokens lies, and its codes and scales to and from numbers.
//
// A block holds 16 consecutive tokens of one head in 18 d bytes:
//   key codes    [d/16][16 tokens][8]   16 channels of a token in 8 bytes
//   key scales   [16 tokens][d/16]
//   value codes  [d][8]                 16 tokens of a channel in 8 bytes
//   value scales [d/16][16 tokens]
// Keys are laid out for a thread a token, values for a thread a channel: a
// product over tokens wants neighbouring tokens of a channel side by side.
// Two codes a byte, the first in the low half.  A code is e2m1 and a scale
// e4m3; code * scale has at most 6 significant bits between 2^-10 and 2688, so
// it is exact in fp16, and in bf16.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "seq_kernels.h"

namespace fa {
namespace cache4 {

constexpr int kBlock = 16;  // tokens of a block, and entries that share a scale

__device__ __forceinline__ int block_bytes(int d) { return 18 * d; }
__device__ __forceinline__ int off_k_scale(int d) { return 8 * d; }
__device__ __forceinline__ int off_v(int d) { return 9 * d; }
__device__ __forceinline__ int off_v_scale(int d) { return 17 * d; }

// Tokens that a sequence can hold; its length, held to that.
__host__ __device__ __forceinline__ int capacity(const Cache4& c) { return c.page_size * c.max_pages; }
__device__ __forceinline__ int length(const Cache4& c, int b, bool report) {
  const int n = c.lens[b];
  const int nk = min(max(n, 0), capacity(c));
  if (report && n != nk) atomicOr(c.status, kStatusInput);
  return nk;
}
// The page of block i of sequence b, or -1 (reported) where the table has none.
__device__ __forceinline__ int page_of(const Cache4& c, int b, int i) {
  const int at = i / (c.page_size / kBlock);
  const int page = c.table != nullptr ? c.table[static_cast<long long>(b) * c.max_pages + at] : b;
  if (page >= 0 && page < c.n_pages) return page;
  atomicOr(c.status, kStatusInput);
  return -1;
}
// Byte offset of block i of a sequence, head h, in its page.
__device__ __forceinline__ long long block_at(const Cache4& c, int page, int h, int i) {
  const int blocks = c.page_size / kBlock;
  return ((static_cast<long long>(page) * c.Hkv + h) * blocks + i % blocks) * block_bytes(c.d);
}

// Eight codes of a word, the first in the lowest bits, as four fp16 pairs (exact).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t* o) {
  asm("{\n.reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Four scales of a word as two fp16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ void scales_f16(uint32_t w, uint32_t* o) {
  asm("{\n.reg .b16 a, b;\n"
      "mov.b32 {a, b}, %2;\n"
      "cvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(o[0]), "=r"(o[1])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 floats(uint32_t h2) { return __half22float2(*reinterpret_cast<const __half2*>(&h2)); }
__device__ __forceinline__ float scale_f32(uint8_t s) {
  uint32_t o[2];
  scales_f16(s, o);
  return floats(o[0]).x;
}

// Eight numbers as codes of a word, the first in the lowest bits: nearest, ties
// to even, saturating.
__device__ __forceinline__ uint32_t to_codes(const float* q) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}
// max |.| of all, NaN if any is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

// How y = x / (the tensor's scale) and y / s are taken.  kDivide: two divisions
// an entry, each the nearest float32 number.  That of y / s lies on a border b
// between codes only where the quotient does: b s has at most 7 bits, so the next
// y differs by more than half a step of y / s.  kMultiply: the tensor's scale is a
// power of two, and a product with its reciprocal the same number.  kShort: so it
// is, and entries have 8 significant bits (bf16).  Where y / s is not a border it
// is at least 2^-9 away from one, so y (1 / s), within 2^-22, rounded to 13 bits
// falls on the border where the quotient does, and to its side of it elsewhere.
// Prompts of 290,920 tokens and heads, d = 128 (replayed graphs): bf16, kShort 42
// us, kDivide 90; float32, kMultiply 68, kDivide 96.
enum Quotient { kDivide, kMultiply, kShort };

// Sixteen entries to codes and a scale (the definition is in fa.h); `scale` is the
// tensor's, or its reciprocal unless kDivide.
template <Quotient Q>
__device__ __forceinline__ uint8_t quantise16(float (&x)[16], float scale, uint2& codes) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (Q == kDivide) x[i] = x[i] / scale;
    if (Q == kMultiply) x[i] = x[i] * scale;
    amax = max_nan(amax, x[i]);
  }
  if (Q == kShort) amax *= scale;
  uint32_t s;  // a NaN gives e4m3's NaN
  asm("{\n.reg .b16 t;\ncvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\ncvt.u32.u16 %0, t;\n}\n"
      : "=r"(s)
      : "f"(0.f), "f"(amax / 6.f));
  s &= 0xffu;
  const float sf = scale_f32(static_cast<uint8_t>(s));
  if (Q == kShort) {
    const float f = 1.f / sf * scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float((__float_as_uint(x[i] * f) + 0x200u) & 0xfffffc00u);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] / sf;
  }
  codes = s == 0 ? make_uint2(0, 0) : make_uint2(to_codes(x), to_codes(x + 8));  // 0: every entry rounds to zero
  return static_cast<uint8_t>(s);
}

// Eight rows of eight codes become eight columns of them.
__device__ __forceinline__ void transpose_codes(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // nibbles within bytes
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0f0f0f0fu) | ((b & 0x0f0f0f0fu) << 4);
    w[i + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4) {  // bytes within halves
#pragma unroll
    for (int j = i; j < i + 2; ++j) {
      const uint32_t a = w[j], b = w[j + 2];
      w[j] = __byte_perm(a, b, 0x6240);
      w[j + 2] = __byte_perm(a, b, 0x7351);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // halves
    const uint32_t a = w[j], b = w[j + 4];
    w[j] = __byte_perm(a, b, 0x5410);
    w[j + 4] = __byte_perm(a, b, 0x7632);
  }
}

}  // namespace cache4
}  // namespace fa
