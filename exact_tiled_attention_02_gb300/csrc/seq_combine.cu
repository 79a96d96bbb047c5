// seq_combine.cu -- merges partial attention results of one query row over
// disjoint sets of keys (float32 outputs).
//
// Partial result s of a row is (O_s, lse_s), normalised over its own keys.
// With M = max_s lse_s and w_s = exp(lse_s - M):  O = sum_s w_s O_s / sum_s w_s,
// lse = M + ln sum_s w_s: the merge of "Flash attention and efficient
// attention -- Hinglish notes", "Derivation: Incremental Softmax", Steps 2-3,
// for normalised parts.  A part with lse -inf (no key) has weight 0 and its O
// is not read; a row without keys gives O = 0 and lse = -inf.
//
// One warp per row and 32 of its columns; lane i holds the weight of part i,
// so that the parts' loads do not wait for one another.  Bound by latency: two
// dependent rounds of loads, a few microseconds for a decoding batch.
#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32)
    fa_seq_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse, int splits,
                          long long total, int dv, float* __restrict__ o, float* __restrict__ lse) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = (dv + 31) / 32;
  const long long idx = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long row = idx / slices;
  const int slice = static_cast<int>(idx % slices);
  seq::pdl_wait();
  if (row >= total) return;
  const float mine = lane < splits ? part_lse[lane * total + row] : -INFINITY;
  float m = mine;
  for (int s = lane + 32; s < splits; s += 32) m = fmaxf(m, part_lse[s * total + row]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float n = lane < splits ? expf(mine - ref) : 0.f;
  for (int s = lane + 32; s < splits; s += 32) n += expf(part_lse[s * total + row] - ref);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) n += __shfl_xor_sync(0xffffffffu, n, x);
  const float inv = n == 0.f ? 0.f : 1.f / n;
  const int c = slice * 32 + lane;
  float acc = 0.f;
  for (int s0 = 0; s0 < splits; s0 += 32) {
    const float ls = s0 == 0 ? mine : (s0 + lane < splits ? part_lse[(s0 + lane) * total + row] : -INFINITY);
    const float w = expf(ls - ref) * inv;
    const int k = min(32, splits - s0);
#pragma unroll 8
    for (int i = 0; i < k; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (wi != 0.f && c < dv) acc = fmaf(wi, part_o[((s0 + i) * total + row) * dv + c], acc);
    }
  }
  if (c < dv) o[row * dv + c] = acc;
  if (slice == 0 && lane == 0 && lse != nullptr) lse[row] = m + logf(n);
}

}  // namespace

cudaError_t launch_seq_combine(const float* part_o, const float* part_lse, int splits, long long total, int dv,
                               float* o, float* lse, cudaStream_t s) {
  const long long blocks = (total * ((dv + 31) / 32) + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return seq::launch_after(fa_seq_combine_kernel, static_cast<unsigned>(blocks), kWarps * 32, 0, s, part_o, part_lse,
                           splits, total, dv, o, lse);
}

}  // namespace fa
