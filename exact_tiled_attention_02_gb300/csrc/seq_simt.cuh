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

// A CTA's TR own rows (64, 32 or 16) meet the 64 rows or columns of a chunk in
// 4 x 4 blocks a thread, whatever TR: at 32 and 16 rows the threads form G = 2
// or 4 groups, which share out the columns of a dot product (their partial
// sums are added once a tile) and the rows of an accumulation (added once, at
// the end).  A 4 x 4 block reads 12 wavefronts of shared memory for 64
// multiply-add instructions; one row a thread would read 9 for 16.
template <int TR>
struct Block {
  static constexpr int G = 64 / TR;           // groups of threads
  static constexpr int THREADS = 256 / G;     // of a group
  int grp, ty, tx;                            // own rows 4 ty .., 16 lanes tx
  __device__ Block() {
    grp = threadIdx.x / THREADS;
    ty = threadIdx.x % THREADS / 16;
    tx = threadIdx.x & 15;
  }
  // acc[i][j] += own row 4 ty + i of A . row tx + 16 j of B, over this group's
  // share of the first n4 groups of four columns
  __device__ __forceinline__ void dot(float (&acc)[4][4], const float* a, const float* b, int n4) const {
    const float* ar = a + 4 * ty * LD;
    const float* br = b + tx * LD;
#pragma unroll 2
    for (int g = grp; g < n4; g += G) {
      float4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(br + 16 * j * LD + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(ar + i * LD + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, acc[i][j]))));
    }
  }
  // acc[i][e] += sum over this group's rows r of w[4 ty + i][r] b[r][4 tx + e]
  __device__ __forceinline__ void accumulate(float (&acc)[4][4], const float* w, const float* b) const {
    const float* wr = w + 4 * ty * LD + grp * (T64 / G);
    const float* bc = b + grp * (T64 / G) * LD + 4 * tx;
#pragma unroll 2
    for (int r = 0; r < T64 / G; r += 4) {
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(wr + i * LD + r);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(bc + (r + k) * LD);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xv = k == 0 ? x[i].x : k == 1 ? x[i].y : k == 2 ? x[i].z : x[i].w;
          acc[i][0] = fmaf(xv, y.x, acc[i][0]);
          acc[i][1] = fmaf(xv, y.y, acc[i][1]);
          acc[i][2] = fmaf(xv, y.z, acc[i][2]);
          acc[i][3] = fmaf(xv, y.w, acc[i][3]);
        }
      }
    }
  }
  // The groups' dot products to red ([G][TR][LD]); entry (row, col) is then the sum of the G.
  __device__ __forceinline__ void put_dot(float* red, const float (&acc)[4][4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[(grp * TR + 4 * ty + i) * LD + tx + 16 * j] = acc[i][j];
  }
  __device__ static __forceinline__ float get(const float* red, int row, int col) {
    float x = red[row * LD + col];
#pragma unroll
    for (int g = 1; g < G; ++g) x += red[(g * TR + row) * LD + col];
    return x;
  }
  // Adds the groups' accumulators up in group 0 (whole CTA; red: [G][TR][LD]).
  __device__ __forceinline__ void add_up(float* red, float (&acc)[4][4]) const {
    if constexpr (G > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(red + (grp * TR + 4 * ty + i) * LD + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 1; g < G; ++g) {
            const float4 y = *reinterpret_cast<const float4*>(red + (g * TR + 4 * ty + i) * LD + 4 * tx);
            acc[i][0] += y.x;
            acc[i][1] += y.y;
            acc[i][2] += y.z;
            acc[i][3] += y.w;
          }
      }
    }
  }
};

}  // namespace simt
}  // namespace fa
