// seq_simt.cuh -- tiles of the fp32 CUDA-core kernels of the language-model
// operators: 64 x 64 chunks, row-major in shared memory, copied there
// asynchronously several chunks ahead of their use.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {
namespace simt {

constexpr int T64 = 64;       // rows of a streamed tile, and columns of a chunk
constexpr int LD = 68;        // row stride of a chunk in floats: rows 16-byte aligned, 8 rows apart in 32 banks
constexpr int kThreads = 256;
constexpr int CHUNK = T64 * LD;

// Asynchronous copy of 16 or 4 bytes to shared memory; zeros where !on (then
// src is any valid address).
__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(float* dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's committed groups are still on their way.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Entries d .. d + 3 of a row of n to dst, zeros past n and where there is no
// row (on false; row is then any valid address).  vec: rows are 16-byte
// aligned and n a multiple of 4.
__device__ __forceinline__ void copy_row4(float* dst, const float* row, bool on, int d, int n, bool vec) {
  if (vec) {
    copy16(dst, on && d < n ? row + d : row, on && d < n);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) copy4(dst + e, on && d + e < n ? row + d + e : row, on && d + e < n);
  }
}
// The same of a row in two parts, n1 and n2 entries.
__device__ __forceinline__ void copy_row4(float* dst, const float* r1, int n1, const float* r2, int n2, bool on, int d,
                                          bool vec) {
  if (vec) {
    if (d < n1)
      copy_row4(dst, r1, on, d, n1, true);
    else
      copy_row4(dst, r2, on, d - n1, n2, true);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = d + e;
      const bool in = on && c < n1 + n2;
      copy4(dst + e, !in ? r1 : c < n1 ? r1 + c : r2 + c - n1, in);
    }
  }
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
