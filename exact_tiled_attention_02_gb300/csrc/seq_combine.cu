// seq_combine.cu -- merges partial attention results of one query row over
// disjoint sets of keys.
//
// Partial result s of a row is (O_s, lse_s), normalised over its own keys.
// With M = max_s lse_s and w_s = exp(lse_s - M):  O = sum_s w_s O_s / sum_s w_s,
// lse = M + ln sum_s w_s: the merge of "Flash attention and efficient
// attention -- Hinglish notes", "Derivation: Incremental Softmax", Steps 2-3,
// for normalised parts.  A part with lse -inf (no key) has weight 0 and its O
// is not read; a row without keys gives O = 0 and lse = -inf.
//
// One warp per row; reads every part once, fp32.
#include <cmath>

#include <cuda_bf16.h>

#include "seq_kernels.h"

namespace fa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    fa_seq_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse, int splits,
                          long long total, int dv, T* __restrict__ o, float* __restrict__ lse) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (row >= total) return;
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, part_lse[s * total + row]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float n = 0.f;
  for (int s = lane; s < splits; s += 32) n += expf(part_lse[s * total + row] - ref);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) n += __shfl_xor_sync(0xffffffffu, n, x);
  const float inv = n == 0.f ? 0.f : 1.f / n;
  for (int c0 = 0; c0 < dv; c0 += 128) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) {
      const float ls = part_lse[s * total + row];
      if (ls == -INFINITY) continue;
      const float w = expf(ls - ref) * inv;
      const float* src = part_o + (s * total + row) * dv;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = c0 + e * 32 + lane;
        if (c < dv) acc[e] = fmaf(w, src[c], acc[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + e * 32 + lane;
      if (c < dv) store(o + row * dv + c, acc[e]);
    }
  }
  if (lane == 0 && lse != nullptr) lse[row] = m + logf(n);
}

}  // namespace

cudaError_t launch_seq_combine(const float* part_o, const float* part_lse, int splits, long long total, int dv,
                               void* o, float* lse, fa_dtype dt, cudaStream_t s) {
  const long long blocks = (total + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dt == FA_DTYPE_F32)
    fa_seq_combine_kernel<float><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(
        part_o, part_lse, splits, total, dv, static_cast<float*>(o), lse);
  else
    fa_seq_combine_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(
        part_o, part_lse, splits, total, dv, static_cast<__nv_bfloat16*>(o), lse);
  return cudaGetLastError();
}

}  // namespace fa
