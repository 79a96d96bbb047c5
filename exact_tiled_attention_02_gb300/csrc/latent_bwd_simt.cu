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
// P = 0 throughout.  The CTA's own tile stays in shared memory; the other
// side streams through one 64 x 64 chunk, loaded into registers while the
// chunk before it is used: q (S), dO (dP), then dO (dV) and q (dK) again for
// dkdv; k (S), v (dP), k (dQ) for dq.  Thread (ty, tx): rows 4 ty .., columns
// tx + 16 j of S and dP, columns 4 tx .. of every chunk of a gradient.
// Bound by the latency of the chunks at small sizes, else by shared memory.
#include <cmath>

#include "seq_kernels.h"
#include "seq_simt.cuh"
#include "sm103.cuh"

namespace fa {
namespace {

using namespace simt;

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

// NK, NV: 64-column chunks of dn + dr and of dv
template <int NK, int NV>
constexpr int bwd_smem() {
  return (NK + NV + 3) * CHUNK * 4;  // own tile, the streamed chunk, P and dS
}

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads) fa_latent_bwd_dkdv_kernel(const LatentBwd p, int vec) {
  extern __shared__ float4 smem4[];
  float* C = reinterpret_cast<float*>(smem4);  // the streamed chunk
  float* P = C + CHUNK;                        // [key][query]
  float* dS = P + CHUNK;
  float* K = dS + CHUNK;                       // [NK] chunks of the CTA's keys
  float* V = K + NK * CHUNK;                   // [NV]
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int ktiles = (p.Nk + T64 - 1) / T64;
  const long long bh = blockIdx.x / ktiles;
  const int j0 = (blockIdx.x % ktiles) * T64;
  const int dk = p.dn + p.dr, npad = (p.Nq + 127) / 128 * 128;
  const float* q = static_cast<const float*>(p.q) + bh * p.Nq * dk;
  const float* kn = static_cast<const float*>(p.kn) + bh * p.Nk * p.dn;
  const float* kr = static_cast<const float*>(p.kr) + (bh / p.H) * p.Nk * p.dr;
  const float* v = static_cast<const float*>(p.v) + bh * p.Nk * p.dv;
  const float* dO = static_cast<const float*>(p.dO) + bh * p.Nq * p.dv;
  const float* lse2 = p.lse2 + bh * npad;
  const float* dsum = p.dsum + bh * npad;
  const float sl = p.scale * 1.4426950408889634f;
  const int off = p.Nk - p.Nq;
  const int first = p.causal ? max(0, j0 - off) / T64 : 0;  // the first query tile with a row that sees key j0
  const int tiles = (p.Nq + T64 - 1) / T64;
  float4 buf[4];
  // chunk of the stream: NK of q, NV of dO, NV of dO, NK of q per query tile
  auto fetch = [&](int tile, int stage) {
    const bool of_q = stage < NK || stage >= NK + 2 * NV;
    const int c = stage < NK ? stage : stage < NK + NV ? stage - NK : stage < NK + 2 * NV ? stage - NK - NV : stage - NK - 2 * NV;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tile * T64 + ty + 16 * i;
      const float* row = r >= p.Nq ? nullptr : of_q ? q + static_cast<long long>(r) * dk : dO + static_cast<long long>(r) * p.dv;
      buf[i] = load4(row, c * T64 + 4 * tx, of_q ? dk : p.dv, vec);
    }
  };
  auto next = [&](int tile, int stage) {  // the chunk in C; the one after it is under way
    __syncthreads();
    put(C, buf);
    __syncthreads();
    if (stage + 1 < 2 * (NK + NV))
      fetch(tile, stage + 1);
    else if (tile + 1 < tiles)
      fetch(tile + 1, 0);
  };
  if (first < tiles) fetch(first, 0);
#pragma unroll
  for (int c = 0; c < NK + NV; ++c) {
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = j0 + ty + 16 * i;
      const bool in = r < p.Nk;
      x[i] = c < NK ? load4(in ? kn + r * p.dn : nullptr, p.dn, kr + r * p.dr, p.dr, c * T64 + 4 * tx, vec)
                    : load4(in ? v + r * p.dv : nullptr, (c - NK) * T64 + 4 * tx, p.dv, vec);
    }
    put(K + c * CHUNK, x);
  }
  float ak[NK][4][4], av[NV][4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int c = 0; c < NK; ++c) ak[c][i][m] = 0.f;
#pragma unroll
      for (int c = 0; c < NV; ++c) av[c][i][m] = 0.f;
    }
  for (int t = first; t < tiles; ++t) {
    const int i0 = t * T64;
    float s[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      next(t, c);
      dot<4>(s, K + c * CHUNK, C, 16, ty, tx);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      next(t, NK + c);
      dot<4>(dp, V + c * CHUNK, C, 16, ty, tx);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = i0 + tx + 16 * j;
      const float l2 = row < p.Nq ? lse2[row] : 0.f, dd = row < p.Nq ? dsum[row] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = j0 + 4 * ty + i;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        const float pr = in ? exp2f(fmaf(s[i][j], sl, l2)) : 0.f;
        P[(4 * ty + i) * LD + tx + 16 * j] = pr;
        dS[(4 * ty + i) * LD + tx + 16 * j] = in ? pr * (dp[i][j] + dd) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      next(t, NK + NV + c);
      accumulate<4>(av[c], P, C, ty, tx);
    }
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      next(t, NK + 2 * NV + c);
      accumulate<4>(ak[c], dS, C, ty, tx);
    }
  }
  float* dkn = static_cast<float*>(p.dkn) + bh * p.Nk * p.dn;
  float* dv = static_cast<float*>(p.dv_out) + bh * p.Nk * p.dv;
  float* dkr = p.dkr_part + bh * p.Nk * p.dr;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long key = j0 + 4 * ty + i;
    if (key >= p.Nk) continue;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + 4 * tx + m;
        const float x = ak[c][i][m] * p.scale;
        if (d < p.dn)
          dkn[key * p.dn + d] = x;
        else if (d < dk)
          dkr[key * p.dr + d - p.dn] = x;
      }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + 4 * tx + m;
        if (d < p.dv) dv[key * p.dv + d] = av[c][i][m];
      }
  }
}

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads) fa_latent_bwd_dq_kernel(const LatentBwd p, int vec) {
  extern __shared__ float4 smem4[];
  float* C = reinterpret_cast<float*>(smem4);
  float* dS = C + CHUNK;      // [query][key]
  float* Q = dS + CHUNK;      // [NK] chunks of the CTA's queries
  float* G = Q + NK * CHUNK;  // [NV] of their dO
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int qtiles = (p.Nq + T64 - 1) / T64;
  const long long bh = blockIdx.x / qtiles;
  const int i0 = (blockIdx.x % qtiles) * T64;
  const int dk = p.dn + p.dr, npad = (p.Nq + 127) / 128 * 128;
  const float* q = static_cast<const float*>(p.q) + bh * p.Nq * dk;
  const float* kn = static_cast<const float*>(p.kn) + bh * p.Nk * p.dn;
  const float* kr = static_cast<const float*>(p.kr) + (bh / p.H) * p.Nk * p.dr;
  const float* v = static_cast<const float*>(p.v) + bh * p.Nk * p.dv;
  const float* dO = static_cast<const float*>(p.dO) + bh * p.Nq * p.dv;
  const float sl = p.scale * 1.4426950408889634f;
  const int off = p.Nk - p.Nq;
  const int end = p.causal ? min(p.Nk, min(p.Nq, i0 + T64) + off) : p.Nk;  // keys that some row of the tile sees
  const int tiles = end > 0 ? (end + T64 - 1) / T64 : 0;
  float4 buf[4];
  auto fetch = [&](int tile, int stage) {  // NK chunks of k, NV of v, NK of k per key tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = tile * T64 + ty + 16 * i;
      const bool in = r < p.Nk;
      const int c = stage < NK ? stage : stage - NK - NV;
      buf[i] = stage >= NK && stage < NK + NV
                   ? load4(in ? v + r * p.dv : nullptr, (stage - NK) * T64 + 4 * tx, p.dv, vec)
                   : load4(in ? kn + r * p.dn : nullptr, p.dn, kr + r * p.dr, p.dr, c * T64 + 4 * tx, vec);
    }
  };
  auto next = [&](int tile, int stage) {
    __syncthreads();
    put(C, buf);
    __syncthreads();
    if (stage + 1 < 2 * NK + NV)
      fetch(tile, stage + 1);
    else if (tile + 1 < tiles)
      fetch(tile + 1, 0);
  };
  if (tiles > 0) fetch(0, 0);
#pragma unroll
  for (int c = 0; c < NK + NV; ++c) {
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = i0 + ty + 16 * i;
      const bool in = r < p.Nq;
      x[i] = c < NK ? load4(in ? q + r * dk : nullptr, c * T64 + 4 * tx, dk, vec)
                    : load4(in ? dO + r * p.dv : nullptr, (c - NK) * T64 + 4 * tx, p.dv, vec);
    }
    put(Q + c * CHUNK, x);
  }
  float l2[4], dd[4], aq[NK][4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i0 + 4 * ty + i;  // padded to whole tiles
    l2[i] = p.lse2[bh * npad + row];
    dd[i] = p.dsum[bh * npad + row];
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) aq[c][i][m] = 0.f;
  }
  for (int t = 0; t < tiles; ++t) {
    const int j0 = t * T64;
    float s[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      next(t, c);
      dot<4>(s, Q + c * CHUNK, C, 16, ty, tx);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      next(t, NK + c);
      dot<4>(dp, G + c * CHUNK, C, 16, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + 4 * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        const float pr = in ? exp2f(fmaf(s[i][j], sl, l2[i])) : 0.f;
        dS[(4 * ty + i) * LD + tx + 16 * j] = in ? pr * (dp[i][j] + dd[i]) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      next(t, NK + NV + c);
      accumulate<4>(aq[c], dS, C, ty, tx);
    }
  }
  float* dq = static_cast<float*>(p.dq) + bh * p.Nq * dk;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = i0 + 4 * ty + i;
    if (row >= p.Nq) continue;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + 4 * tx + m;
        if (d < dk) dq[row * dk + d] = aq[c][i][m] * p.scale;
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

template <int NK, int NV>
cudaError_t launch_nkv(const LatentBwd& p, cudaStream_t s) {
  constexpr int SMEM = bwd_smem<NK, NV>();
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  cudaError_t e =
      cudaFuncSetAttribute(fa_latent_bwd_dkdv_kernel<NK, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fa_latent_bwd_dq_kernel<NK, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long bh = static_cast<long long>(p.B) * p.H;
  const long long kb = bh * ((p.Nk + T64 - 1) / T64), qb = bh * ((p.Nq + T64 - 1) / T64);
  if (kb > 0x7fffffffLL || qb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int vec = p.dn % 4 == 0 && p.dr % 4 == 0 && p.dv % 4 == 0;  // 16-byte rows
  fa_latent_bwd_dkdv_kernel<NK, NV><<<static_cast<unsigned>(kb), kThreads, SMEM, s>>>(p, vec);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fa_latent_bwd_dq_kernel<NK, NV><<<static_cast<unsigned>(qb), kThreads, SMEM, s>>>(p, vec);
  return cudaGetLastError();
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

cudaError_t launch_latent_bwd_simt(const LatentBwd& p, cudaStream_t s) {
  const int dk = p.dn + p.dr;
  if (dk > 256 || p.dv > 128) return cudaErrorInvalidValue;
  if (p.dv <= 64) {
    if (dk <= 64) return launch_nkv<1, 1>(p, s);
    if (dk <= 128) return launch_nkv<2, 1>(p, s);
    return dk <= 192 ? launch_nkv<3, 1>(p, s) : launch_nkv<4, 1>(p, s);
  }
  if (dk <= 128) return launch_nkv<2, 2>(p, s);
  return dk <= 192 ? launch_nkv<3, 2>(p, s) : launch_nkv<4, 2>(p, s);
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
