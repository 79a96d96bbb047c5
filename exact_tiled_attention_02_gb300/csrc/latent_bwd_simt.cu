// latent_bwd_simt.cu -- the expanded latent attention's backward in fp32 on
// CUDA cores, and the small kernels around every type's backward.
//
// Recomputation as in "Flash attention and efficient attention -- Hinglish
// notes", "Backward Pass: Recomputation".  With k_j = [kn_j | kr_j] (kr
// shared by the heads) and row i seeing keys j <= i + Nk - Nq when causal:
//   P_ij = exp(scale q_i.k_j - lse_i),  dS_ij = P_ij (dO_i.v_j - D_i),
//   D_i = dO_i.O_i,  dV_j = sum_i P_ij dO_i,  dQ_i = scale sum_j dS_ij k_j,
//   dk_j = scale sum_i dS_ij q_i,  dkn_j = dk_j[:dn],  dkr_j = sum_heads dk_j[dn:].
//
//   prep   -lse_i log2 e and -D_i of every row (padded to 128 rows a head);
//   dkdv   one CTA per 64 keys of a head over the 64-row query tiles that see
//          them; the rotary part of dk goes to an fp32 array per head;
//   dq     one CTA per 64 queries over the key tiles they see;
//   dkr    sums the rotary parts over the heads, in head order.
// No atomics: every sum has one fixed order.  A row that sees no key has
// P = 0 throughout.  Head dimensions stream through shared memory 64 at a
// time, transposed ([d][64]); a thread holds a 4 x 4 block of S and dP and,
// of its 4 rows, columns tx + 16 m of the accumulated gradients.
#include <cmath>

#include "seq_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int T64 = 64;
constexpr int LD = 68;
constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__global__ void __launch_bounds__(128) fa_latent_bwd_prep_f32_kernel(const float* __restrict__ o,
                                                                     const float* __restrict__ dO,
                                                                     const float* __restrict__ lse,
                                                                     float* __restrict__ lse2, float* __restrict__ dsum,
                                                                     long long rows, int Nq, int npad, int dv) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long prow = static_cast<long long>(blockIdx.x) * 4 + warp;
  if (prow >= rows) return;
  const long long bh = prow / npad;
  const int i = static_cast<int>(prow % npad);
  float acc = 0.f, l2 = -INFINITY;
  if (i < Nq) {
    const long long src = (bh * Nq + i) * dv;
    for (int c = lane; c < dv; c += 32) acc = fmaf(o[src + c], dO[src + c], acc);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
    const float l = lse[bh * Nq + i];
    l2 = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;  // no key seen: P = 2^(x - inf) = 0
  }
  if (lane == 0) {
    lse2[prow] = l2;
    dsum[prow] = i < Nq ? -acc : 0.f;
  }
}

// bf16, dv = 128: sixteen lanes a row (16 bytes of O and dO each), two rows a
// pass, four passes a warp with all their loads in flight; a warp's eight rows
// lie in one padded head (128 divides npad).
__global__ void __launch_bounds__(256)
    fa_latent_bwd_prep_bf16_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dO,
                                   const float* __restrict__ lse, float* __restrict__ lse2, float* __restrict__ dsum,
                                   long long rows, int Nq, int npad) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long base = (static_cast<long long>(blockIdx.x) * 8 + warp) * 8;
  if (base >= rows) return;
  const long long bh = base / npad;
  const int i0 = static_cast<int>(base % npad), c = lane & 15, sub = lane >> 4;
  uint4 ov[4], gv[4];
  float lv[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = i0 + 2 * u + sub;
    ov[u] = gv[u] = make_uint4(0u, 0u, 0u, 0u);
    lv[u] = -INFINITY;
    if (i < Nq) {
      const long long src = (bh * Nq + i) * 128 + 8 * c;
      ov[u] = __ldg(reinterpret_cast<const uint4*>(o + src));
      gv[u] = __ldg(reinterpret_cast<const uint4*>(dO + src));
      lv[u] = __ldg(lse + bh * Nq + i);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const __nv_bfloat162* op = reinterpret_cast<const __nv_bfloat162*>(&ov[u]);
    const __nv_bfloat162* gp = reinterpret_cast<const __nv_bfloat162*>(&gv[u]);
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = __bfloat1622float2(op[e]), b = __bfloat1622float2(gp[e]);
      acc = fmaf(a.x, b.x, acc);
      acc = fmaf(a.y, b.y, acc);
    }
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
    if (c == 0) {
      const long long prow = base + 2 * u + sub;
      lse2[prow] = lv[u] == -INFINITY ? -INFINITY : -lv[u] * 1.4426950408889634f;  // no key seen: P = 2^(x - inf) = 0
      dsum[prow] = -acc;
    }
  }
}

// rows [r0, r0 + 64) of columns [c0, c0 + 64) of a matrix, transposed:
// dst[c * LD + row]; zero outside
template <typename T>
__device__ __forceinline__ void load_t(float* dst, const T* __restrict__ src, int r0, int n, int stride, int c0, int d) {
  for (int idx = threadIdx.x; idx < T64 * T64; idx += kThreads) {
    const int c = idx & 63, row = idx >> 6;
    dst[c * LD + row] =
        (r0 + row < n && c0 + c < d) ? to_f32(src[static_cast<long long>(r0 + row) * stride + c0 + c]) : 0.f;
  }
}
// the same of [kn | kr] rows
template <typename T>
__device__ __forceinline__ void load_k(float* dst, const T* __restrict__ kn, const T* __restrict__ kr, int r0, int n,
                                       int dn, int dr, int c0) {
  for (int idx = threadIdx.x; idx < T64 * T64; idx += kThreads) {
    const int c = idx & 63, row = idx >> 6, d = c0 + c;
    float x = 0.f;
    if (r0 + row < n && d < dn + dr)
      x = d < dn ? to_f32(kn[static_cast<long long>(r0 + row) * dn + d])
                 : to_f32(kr[static_cast<long long>(r0 + row) * dr + d - dn]);
    dst[c * LD + row] = x;
  }
}

// acc += A B^T over a chunk: rows 4ty.. of A, 4tx.. of B, both transposed
__device__ __forceinline__ void block_abt(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
#pragma unroll 4
  for (int c = 0; c < T64; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(a + c * LD + 4 * ty);
    const float4 y = *reinterpret_cast<const float4*>(b + c * LD + 4 * tx);
    const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], yv[j], acc[i][j]);
  }
}

// acc[i][m] += sum_r w[4ty + i][r] b[tx + 16 m][r] over the 64 rows of a tile
__device__ __forceinline__ void accum_wb(float (&acc)[4][4], const float* w, const float* b, int ty, int tx) {
#pragma unroll 2
  for (int r4 = 0; r4 < T64; r4 += 4) {
    float wv[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(w + (4 * ty + i) * LD + r4);
      wv[i][0] = t.x;
      wv[i][1] = t.y;
      wv[i][2] = t.z;
      wv[i][3] = t.w;
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float4 t = *reinterpret_cast<const float4*>(b + (tx + 16 * m) * LD + r4);
      const float bv[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int rr = 0; rr < 4; ++rr)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][m] = fmaf(wv[i][rr], bv[rr], acc[i][m]);
    }
  }
}

constexpr int kSmem = 4 * T64 * LD * 4;

// NK, NV: 64-column chunks of dn + dr and of dv
template <typename T, int NK, int NV>
__global__ void __launch_bounds__(kThreads) fa_latent_bwd_dkdv_kernel(const LatentBwd p) {
  extern __shared__ float4 smem4[];
  float* A = reinterpret_cast<float*>(smem4);
  float* Bt = A + T64 * LD;
  float* P = Bt + T64 * LD;   // [key][query]
  float* dS = P + T64 * LD;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int ktiles = (p.Nk + T64 - 1) / T64;
  const long long bh = blockIdx.x / ktiles;
  const int j0 = (blockIdx.x % ktiles) * T64;
  const int dk = p.dn + p.dr, npad = (p.Nq + 127) / 128 * 128;
  const T* q = static_cast<const T*>(p.q) + bh * p.Nq * dk;
  const T* kn = static_cast<const T*>(p.kn) + bh * p.Nk * p.dn;
  const T* kr = static_cast<const T*>(p.kr) + (bh / p.H) * p.Nk * p.dr;
  const T* v = static_cast<const T*>(p.v) + bh * p.Nk * p.dv;
  const T* dO = static_cast<const T*>(p.dO) + bh * p.Nq * p.dv;
  const float* lse2 = p.lse2 + bh * npad;
  const float* dsum = p.dsum + bh * npad;
  const float sl = p.scale * 1.4426950408889634f;
  const int off = p.Nk - p.Nq;
  float ak[NK][4][4], av[NV][4][4];
#pragma unroll
  for (int c = 0; c < NK; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) ak[c][i][m] = 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) av[c][i][m] = 0.f;
  const int first = p.causal ? max(0, j0 - off) / T64 : 0;  // the first query tile with a row that sees key j0
  for (int i0 = first * T64; i0 < p.Nq; i0 += T64) {
    float s[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
    for (int c = 0; c < NK; ++c) {
      __syncthreads();
      load_k(A, kn, kr, j0, p.Nk, p.dn, p.dr, c * T64);
      load_t(Bt, q, i0, p.Nq, dk, c * T64, dk);
      __syncthreads();
      block_abt(s, A, Bt, ty, tx);
    }
    for (int c = 0; c < NV; ++c) {
      __syncthreads();
      load_t(A, v, j0, p.Nk, p.dv, c * T64, p.dv);
      load_t(Bt, dO, i0, p.Nq, p.dv, c * T64, p.dv);
      __syncthreads();
      block_abt(dp, A, Bt, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = j0 + 4 * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = i0 + 4 * tx + j;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        const float pr = in ? exp2f(fmaf(s[i][j], sl, lse2[row])) : 0.f;
        P[(4 * ty + i) * LD + 4 * tx + j] = pr;
        dS[(4 * ty + i) * LD + 4 * tx + j] = in ? pr * (dp[i][j] + dsum[row]) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      __syncthreads();
      load_t(Bt, dO, i0, p.Nq, p.dv, c * T64, p.dv);
      __syncthreads();
      accum_wb(av[c], P, Bt, ty, tx);
    }
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      __syncthreads();
      load_t(Bt, q, i0, p.Nq, dk, c * T64, dk);
      __syncthreads();
      accum_wb(ak[c], dS, Bt, ty, tx);
    }
  }
  T* dkn = static_cast<T*>(p.dkn) + bh * p.Nk * p.dn;
  T* dv = static_cast<T*>(p.dv_out) + bh * p.Nk * p.dv;
  float* dkr = p.dkr_part + bh * p.Nk * p.dr;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long key = j0 + 4 * ty + i;
    if (key >= p.Nk) continue;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + tx + 16 * m;
        const float x = ak[c][i][m] * p.scale;
        if (d < p.dn)
          store(dkn + key * p.dn + d, x);
        else if (d < dk)
          dkr[key * p.dr + d - p.dn] = x;
      }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + tx + 16 * m;
        if (d < p.dv) store(dv + key * p.dv + d, av[c][i][m]);
      }
  }
}

template <typename T, int NK, int NV>
__global__ void __launch_bounds__(kThreads) fa_latent_bwd_dq_kernel(const LatentBwd p) {
  extern __shared__ float4 smem4[];
  float* A = reinterpret_cast<float*>(smem4);
  float* Bt = A + T64 * LD;
  float* dS = Bt + T64 * LD;  // [query][key]
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int qtiles = (p.Nq + T64 - 1) / T64;
  const long long bh = blockIdx.x / qtiles;
  const int i0 = (blockIdx.x % qtiles) * T64;
  const int dk = p.dn + p.dr, npad = (p.Nq + 127) / 128 * 128;
  const T* q = static_cast<const T*>(p.q) + bh * p.Nq * dk;
  const T* kn = static_cast<const T*>(p.kn) + bh * p.Nk * p.dn;
  const T* kr = static_cast<const T*>(p.kr) + (bh / p.H) * p.Nk * p.dr;
  const T* v = static_cast<const T*>(p.v) + bh * p.Nk * p.dv;
  const T* dO = static_cast<const T*>(p.dO) + bh * p.Nq * p.dv;
  const float* lse2 = p.lse2 + bh * npad;
  const float* dsum = p.dsum + bh * npad;
  const float sl = p.scale * 1.4426950408889634f;
  const int off = p.Nk - p.Nq;
  float aq[NK][4][4];
#pragma unroll
  for (int c = 0; c < NK; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) aq[c][i][m] = 0.f;
  const int end = p.causal ? min(p.Nk, min(p.Nq, i0 + T64) + off) : p.Nk;  // keys that some row of the tile sees
  for (int j0 = 0; j0 < end; j0 += T64) {
    float s[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
    for (int c = 0; c < NK; ++c) {
      __syncthreads();
      load_t(A, q, i0, p.Nq, dk, c * T64, dk);
      load_k(Bt, kn, kr, j0, p.Nk, p.dn, p.dr, c * T64);
      __syncthreads();
      block_abt(s, A, Bt, ty, tx);
    }
    for (int c = 0; c < NV; ++c) {
      __syncthreads();
      load_t(A, dO, i0, p.Nq, p.dv, c * T64, p.dv);
      load_t(Bt, v, j0, p.Nk, p.dv, c * T64, p.dv);
      __syncthreads();
      block_abt(dp, A, Bt, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + 4 * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + 4 * tx + j;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        const float pr = in ? exp2f(fmaf(s[i][j], sl, lse2[row])) : 0.f;
        dS[(4 * ty + i) * LD + 4 * tx + j] = in ? pr * (dp[i][j] + dsum[row]) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      __syncthreads();
      load_k(Bt, kn, kr, j0, p.Nk, p.dn, p.dr, c * T64);
      __syncthreads();
      accum_wb(aq[c], dS, Bt, ty, tx);
    }
  }
  T* dq = static_cast<T*>(p.dq) + bh * p.Nq * dk;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = i0 + 4 * ty + i;
    if (row >= p.Nq) continue;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + tx + 16 * m;
        if (d < dk) store(dq + row * dk + d, aq[c][i][m] * p.scale);
      }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) fa_latent_bwd_dkr_kernel(const float* __restrict__ part, T* __restrict__ dkr,
                                                                int H, long long per_head, long long total) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const float* src = part + (i / per_head) * H * per_head + i % per_head;
  float x = 0.f;
  for (int h = 0; h < H; ++h) x += src[h * per_head];
  store(dkr + i, x);
}

template <typename T, int NK, int NV>
cudaError_t launch_nkv(const LatentBwd& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(fa_latent_bwd_dkdv_kernel<T, NK, NV>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fa_latent_bwd_dq_kernel<T, NK, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const long long bh = static_cast<long long>(p.B) * p.H;
  const long long kb = bh * ((p.Nk + T64 - 1) / T64), qb = bh * ((p.Nq + T64 - 1) / T64);
  if (kb > 0x7fffffffLL || qb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  fa_latent_bwd_dkdv_kernel<T, NK, NV><<<static_cast<unsigned>(kb), kThreads, kSmem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fa_latent_bwd_dq_kernel<T, NK, NV><<<static_cast<unsigned>(qb), kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const LatentBwd& p, cudaStream_t s) {
  const int dk = p.dn + p.dr;
  if (dk > 256 || p.dv > 128) return cudaErrorInvalidValue;
  if (p.dv <= 64) {
    if (dk <= 64) return launch_nkv<T, 1, 1>(p, s);
    if (dk <= 128) return launch_nkv<T, 2, 1>(p, s);
    return dk <= 192 ? launch_nkv<T, 3, 1>(p, s) : launch_nkv<T, 4, 1>(p, s);
  }
  if (dk <= 128) return launch_nkv<T, 2, 2>(p, s);
  return dk <= 192 ? launch_nkv<T, 3, 2>(p, s) : launch_nkv<T, 4, 2>(p, s);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t latent_bwd_workspace_layout(int B, int H, int Nq, int Nk, int dr, size_t* off_dsum, size_t* off_part) {
  const size_t bh = static_cast<size_t>(B) * H;
  const size_t rows = up256(bh * ((static_cast<size_t>(Nq) + 127) / 128 * 128) * 4);
  if (off_dsum) *off_dsum = rows;
  if (off_part) *off_part = 2 * rows;
  return 2 * rows + up256(bh * Nk * dr * 4);
}

cudaError_t launch_latent_bwd_prep(const LatentBwd& p, fa_dtype dt, cudaStream_t s) {
  const int npad = (p.Nq + 127) / 128 * 128;
  const long long rows = static_cast<long long>(p.B) * p.H * npad;
  if (rows / 4 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dt == FA_DTYPE_F32)
    fa_latent_bwd_prep_f32_kernel<<<static_cast<unsigned>(rows / 4), 128, 0, s>>>(
        static_cast<const float*>(p.o), static_cast<const float*>(p.dO), p.lse, p.lse2, p.dsum, rows, p.Nq, npad, p.dv);
  else
    fa_latent_bwd_prep_bf16_kernel<<<static_cast<unsigned>(rows / 64), 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(p.o), static_cast<const __nv_bfloat16*>(p.dO), p.lse, p.lse2, p.dsum, rows,
        p.Nq, npad);
  return cudaGetLastError();
}

cudaError_t launch_latent_bwd_simt(const LatentBwd& p, fa_dtype dt, cudaStream_t s) {
  return dt == FA_DTYPE_F32 ? launch_t<float>(p, s) : launch_t<__nv_bfloat16>(p, s);
}

cudaError_t launch_latent_bwd_dkr(const LatentBwd& p, fa_dtype dt, cudaStream_t s) {
  const long long per_head = static_cast<long long>(p.Nk) * p.dr, total = per_head * p.B;
  const long long blocks = (total + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dt == FA_DTYPE_F32)
    fa_latent_bwd_dkr_kernel<float><<<static_cast<unsigned>(blocks), 256, 0, s>>>(
        p.dkr_part, static_cast<float*>(p.dkr), p.H, per_head, total);
  else
    fa_latent_bwd_dkr_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), 256, 0, s>>>(
        p.dkr_part, static_cast<__nv_bfloat16*>(p.dkr), p.H, per_head, total);
  return cudaGetLastError();
}

}  // namespace fa
