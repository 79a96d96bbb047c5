// seq_simt.cuh -- tiles of the fp32 CUDA-core kernels of the language-model
// operators: 64 x 64 chunks, row-major in shared memory, filled from registers
// that were loaded while the previous chunk was being used.
#pragma once

#include <cuda_runtime.h>

namespace fa {
namespace simt {

constexpr int T64 = 64;       // rows of a tile, and columns of a chunk
constexpr int LD = 68;        // row stride of a chunk in floats: rows 16-byte aligned, 8 rows apart in 32 banks
constexpr int kThreads = 256;
constexpr int CHUNK = T64 * LD;

// Entries d .. d + 3 of a row, zeros at and past n.
__device__ __forceinline__ float4 load4(const float* row, int d, int n, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row == nullptr || d >= n) return v;
  if (vec) return *reinterpret_cast<const float4*>(row + d);
  v.x = row[d];
  if (d + 1 < n) v.y = row[d + 1];
  if (d + 2 < n) v.z = row[d + 2];
  if (d + 3 < n) v.w = row[d + 3];
  return v;
}
// The same of a row in two parts, n1 and n2 entries; no row (zeros) where r1 is null.
__device__ __forceinline__ float4 load4(const float* r1, int n1, const float* r2, int n2, int d, bool vec) {
  if (r1 == nullptr) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec || d + 4 <= n1 || d >= n1) return d < n1 ? load4(r1, d, n1, vec) : load4(r2, d - n1, n2, vec);
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = d + e;
    x[e] = c < n1 ? r1[c] : c - n1 < n2 ? r2[c - n1] : 0.f;
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Thread tid's share of a chunk: rows tid / 16 + 16 i, columns 4 (tid % 16) ..
template <int N>
__device__ __forceinline__ void put(float* chunk, const float4 (&v)[N]) {
  const int row = threadIdx.x >> 4, c = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<float4*>(chunk + (row + 16 * i) * LD + c) = v[i];
}

// acc[i][j] += row R ty + i of A . row tx + 16 j of B, over the first n4 groups of four columns
template <int R>
__device__ __forceinline__ void dot(float (&acc)[R][4], const float* a, const float* b, int n4, int ty, int tx) {
#pragma unroll 4
  for (int c = 0; c < 4 * n4; c += 4) {
    float4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LD + c);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(a + (R * ty + i) * LD + c);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(x.w, y[j].w, fmaf(x.z, y[j].z, fmaf(x.y, y[j].y, fmaf(x.x, y[j].x, acc[i][j]))));
    }
  }
}

// acc[i][e] += sum over the 64 rows r of w[R ty + i][r] b[r][4 tx + e]
template <int R>
__device__ __forceinline__ void accumulate(float (&acc)[R][4], const float* w, const float* b, int ty, int tx) {
#pragma unroll 4
  for (int r = 0; r < T64; r += 4) {
    float4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(w + (R * ty + i) * LD + r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 y = *reinterpret_cast<const float4*>(b + (r + k) * LD + 4 * tx);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float xv = k == 0 ? x[i].x : k == 1 ? x[i].y : k == 2 ? x[i].z : x[i].w;
        acc[i][0] = fmaf(xv, y.x, acc[i][0]);
        acc[i][1] = fmaf(xv, y.y, acc[i][1]);
        acc[i][2] = fmaf(xv, y.z, acc[i][2]);
        acc[i][3] = fmaf(xv, y.w, acc[i][3]);
      }
    }
  }
}

}  // namespace simt
}  // namespace fa
