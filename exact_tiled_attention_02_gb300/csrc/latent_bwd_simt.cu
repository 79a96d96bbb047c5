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
//   dkdv   one CTA per 64 (32, 16) keys of a head over the 64-row query tiles that see
//          them; the rotary part of dk goes to an fp32 array per head;
//   dq     one CTA per 64 (32, 16) queries over the key tiles they see, beside dkdv
//          on the room that leaves (6 heads of 333 tokens: 124 us so 101);
//   dkr    sums the rotary parts over the heads, in head order.
// No atomics: every sum has one fixed order.  A row that sees no key has
// P = 0 throughout.  The CTA's own tile stays in shared memory; the other
// side streams through a ring of 64 x 64 chunks, copied asynchronously two
// ahead: q (S), dO (dP), then dO (dV) and q (dK) again for dkdv; k (S), v (dP),
// k (dQ) for dq.  Products go in 4 x 4 blocks a thread (seq_simt.cuh).
// Bound by the latency of the chunks at small sizes, else by shared memory.
#include <cmath>

#include "seq_kernels.h"
#include "seq_simt.cuh"
#include "seq_sm103.cuh"

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
  seq::pdl_launch();
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

constexpr int DEPTH = 3;  // chunks of the ring

// NK, NV: 64-column chunks of dn + dr and of dv; BR rows a CTA
template <int NK, int NV, int BR>
constexpr int bwd_smem() {
  return (DEPTH * CHUNK + CHUNK + (NK + NV + 2) * BR * LD) * 4;  // ring, partial sums, own rows, P and dS
}

// CTAs of dkdv an SM, or of dkdv and dq: two where shared memory holds them and
// 128 registers a thread do
template <int NK, int NV, int BR>
constexpr int bwd_ctas() {
  return NK <= 2 && bwd_smem<NK, NV, BR>() <= 113 * 1024 ? 2 : 1;
}

// The ring: chunk after chunk of a stream, copied DEPTH - 1 ahead of its use.
// F: f(n, dst) copies this thread's share of the n-th chunk to dst.
template <typename F>
struct Ring {
  float* base;
  int total, asked, slot, f_slot;
  F f;
  __device__ Ring(float* b, int n, F fn) : base(b), total(n), asked(0), slot(0), f_slot(0), f(fn) {}
  __device__ void ask() {
    if (asked < total) f(asked, base + f_slot * CHUNK);
    ++asked;
    copies_commit();  // a group a call, empty or not, so that the wait below counts chunks
    f_slot = f_slot + 1 == DEPTH ? 0 : f_slot + 1;
  }
  // the next chunk, complete, and what threads wrote to shared memory before;
  // asks for a later one into the slot that every thread has left
  __device__ const float* next() {
    copies_wait<DEPTH - 2>();
    __syncthreads();
    const float* chunk = base + slot * CHUNK;
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    ask();
    return chunk;
  }
};

template <int NK, int NV, int BR>
__global__ void __launch_bounds__(kThreads, bwd_ctas<NK, NV, BR>()) fa_latent_bwd_dkdv_kernel(const LatentBwd p, int vec) {
  constexpr int R = BR / 16, OWN = BR * LD;
  seq::pdl_launch();  // dq reads nothing of this kernel's: it starts on the SMs that are left
  const Block<BR> blk;
  extern __shared__ float4 smem4[];
  float* base = reinterpret_cast<float*>(smem4);
  float* red = base + DEPTH * CHUNK;  // the groups' partial sums
  float* P = red + CHUNK;           // [key][query]
  float* dS = P + OWN;
  float* K = dS + OWN;              // [NK] chunks of the CTA's keys
  float* V = K + NK * OWN;          // [NV]
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int ktiles = (p.Nk + BR - 1) / BR;
  const long long bh = blockIdx.x / ktiles;
  const int j0 = (blockIdx.x % ktiles) * BR;
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
  constexpr int PER = 2 * (NK + NV);  // chunks a query tile: NK of q, NV of dO, NV of dO, NK of q
  auto fetch = [&](int n, float* dst) {
    const int tile = first + n / PER, stage = n % PER;
    const bool of_q = stage < NK || stage >= NK + 2 * NV;
    const int c = stage < NK ? stage : stage < NK + NV ? stage - NK : stage < NK + 2 * NV ? stage - NK - NV : stage - NK - 2 * NV;
    dst += ty * LD + 4 * tx;
#pragma unroll
    for (int i = 0; i < 4; ++i, dst += 16 * LD) {
      const long long r = tile * T64 + ty + 16 * i;
      const bool on = r < p.Nq;
      if (of_q)
        copy_row4(dst, q + (on ? r * dk : 0), on, c * T64 + 4 * tx, dk, vec);
      else
        copy_row4(dst, dO + (on ? r * p.dv : 0), on, c * T64 + 4 * tx, p.dv, vec);
    }
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = ty + 16 * i;
    const long long r = j0 + row;
    const bool on = r < p.Nk;
#pragma unroll
    for (int c = 0; c < NK; ++c)
      copy_row4(K + c * OWN + row * LD + 4 * tx, kn + (on ? r * p.dn : 0), p.dn, kr + (on ? r * p.dr : 0), p.dr, on,
                c * T64 + 4 * tx, vec);
#pragma unroll
    for (int c = 0; c < NV; ++c)
      copy_row4(V + c * OWN + row * LD + 4 * tx, v + (on ? r * p.dv : 0), on, c * T64 + 4 * tx, p.dv, vec);
  }
  Ring ring(base, max(0, tiles - first) * PER, fetch);  // (the own rows travel in the first chunk's group)
#pragma unroll
  for (int c = 0; c < DEPTH - 1; ++c) ring.ask();
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
    for (int c = 0; c < NK; ++c) blk.dot(s, K + c * OWN, ring.next(), 16);
#pragma unroll
    for (int c = 0; c < NV; ++c) blk.dot(dp, V + c * OWN, ring.next(), 16);
    // the groups' sums, S then dP through the same array; thread: keys R ty .., queries tx + 16 j
    float pr[R][4];
    blk.put_dot(red, s);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = i0 + tx + 16 * j;
      const float l2 = row < p.Nq ? lse2[row] : 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int key = j0 + R * ty + i;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        pr[i][j] = in ? exp2f(fmaf(Block<BR>::get(red, R * ty + i, tx + 16 * j), sl, l2)) : 0.f;
        P[(R * ty + i) * LD + tx + 16 * j] = pr[i][j];
      }
    }
    __syncthreads();
    blk.put_dot(red, dp);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = i0 + tx + 16 * j;
      const float dd = row < p.Nq ? dsum[row] : 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float g = Block<BR>::get(red, R * ty + i, tx + 16 * j);
        dS[(R * ty + i) * LD + tx + 16 * j] = pr[i][j] == 0.f ? 0.f : pr[i][j] * (g + dd);
      }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) blk.accumulate(av[c], P, ring.next());
#pragma unroll
    for (int c = 0; c < NK; ++c) blk.accumulate(ak[c], dS, ring.next());
  }
  copies_wait<0>();
#pragma unroll
  for (int c = 0; c < NK; ++c) blk.add_up(red, ak[c]);
#pragma unroll
  for (int c = 0; c < NV; ++c) blk.add_up(red, av[c]);
  if (blk.grp != 0) return;
  float* dkn = static_cast<float*>(p.dkn) + bh * p.Nk * p.dn;
  float* dv = static_cast<float*>(p.dv_out) + bh * p.Nk * p.dv;
  float* dkr = p.dkr_part + bh * p.Nk * p.dr;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long key = j0 + 4 * blk.ty + i;
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

template <int NK, int NV, int BR>
__global__ void __launch_bounds__(kThreads) fa_latent_bwd_dq_kernel(const LatentBwd p, int vec) {
  constexpr int R = BR / 16, OWN = BR * LD;
  const Block<BR> blk;
  extern __shared__ float4 smem4[];
  float* base = reinterpret_cast<float*>(smem4);
  float* red = base + DEPTH * CHUNK;  // the groups' partial sums
  float* dS = red + CHUNK;           // [query][key]
  float* Q = dS + OWN;               // [NK] chunks of the CTA's queries
  float* G = Q + NK * OWN;           // [NV] of their dO
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int qtiles = (p.Nq + BR - 1) / BR;
  const long long bh = blockIdx.x / qtiles;
  const int i0 = (blockIdx.x % qtiles) * BR;
  const int dk = p.dn + p.dr, npad = (p.Nq + 127) / 128 * 128;
  const float* q = static_cast<const float*>(p.q) + bh * p.Nq * dk;
  const float* kn = static_cast<const float*>(p.kn) + bh * p.Nk * p.dn;
  const float* kr = static_cast<const float*>(p.kr) + (bh / p.H) * p.Nk * p.dr;
  const float* v = static_cast<const float*>(p.v) + bh * p.Nk * p.dv;
  const float* dO = static_cast<const float*>(p.dO) + bh * p.Nq * p.dv;
  const float sl = p.scale * 1.4426950408889634f;
  const int off = p.Nk - p.Nq;
  const int end = p.causal ? min(p.Nk, min(p.Nq, i0 + BR) + off) : p.Nk;  // keys that some row of the tile sees
  const int tiles = end > 0 ? (end + T64 - 1) / T64 : 0;
  constexpr int PER = 2 * NK + NV;  // chunks a key tile: NK of k, NV of v, NK of k
  auto fetch = [&](int n, float* dst) {
    const int tile = n / PER, stage = n % PER;
    const bool of_v = stage >= NK && stage < NK + NV;
    const int c = stage < NK ? stage : of_v ? stage - NK : stage - NK - NV;
    dst += ty * LD + 4 * tx;
#pragma unroll
    for (int i = 0; i < 4; ++i, dst += 16 * LD) {
      const long long r = tile * T64 + ty + 16 * i;
      const bool on = r < p.Nk;
      if (of_v)
        copy_row4(dst, v + (on ? r * p.dv : 0), on, c * T64 + 4 * tx, p.dv, vec);
      else
        copy_row4(dst, kn + (on ? r * p.dn : 0), p.dn, kr + (on ? r * p.dr : 0), p.dr, on, c * T64 + 4 * tx, vec);
    }
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = ty + 16 * i;
    const long long r = i0 + row;
    const bool on = r < p.Nq;
#pragma unroll
    for (int c = 0; c < NK; ++c)
      copy_row4(Q + c * OWN + row * LD + 4 * tx, q + (on ? r * dk : 0), on, c * T64 + 4 * tx, dk, vec);
#pragma unroll
    for (int c = 0; c < NV; ++c)
      copy_row4(G + c * OWN + row * LD + 4 * tx, dO + (on ? r * p.dv : 0), on, c * T64 + 4 * tx, p.dv, vec);
  }
  Ring ring(base, tiles * PER, fetch);
#pragma unroll
  for (int c = 0; c < DEPTH - 1; ++c) ring.ask();
  float l2[R], dd[R], aq[NK][4][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = i0 + R * ty + i;  // padded to whole tiles
    l2[i] = p.lse2[bh * npad + row];
    dd[i] = p.dsum[bh * npad + row];
  }
#pragma unroll
  for (int c = 0; c < NK; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) aq[c][i][m] = 0.f;
  for (int t = 0; t < tiles; ++t) {
    const int j0 = t * T64;
    float s[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c) blk.dot(s, Q + c * OWN, ring.next(), 16);
#pragma unroll
    for (int c = 0; c < NV; ++c) blk.dot(dp, G + c * OWN, ring.next(), 16);
    float pr[R][4];  // thread: queries R ty .., keys tx + 16 j
    blk.put_dot(red, s);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = i0 + R * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        const bool in = row < p.Nq && key < p.Nk && (!p.causal || key <= row + off);
        pr[i][j] = in ? exp2f(fmaf(Block<BR>::get(red, R * ty + i, tx + 16 * j), sl, l2[i])) : 0.f;
      }
    }
    __syncthreads();
    blk.put_dot(red, dp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = Block<BR>::get(red, R * ty + i, tx + 16 * j);
        dS[(R * ty + i) * LD + tx + 16 * j] = pr[i][j] == 0.f ? 0.f : pr[i][j] * (g + dd[i]);
      }
#pragma unroll
    for (int c = 0; c < NK; ++c) blk.accumulate(aq[c], dS, ring.next());
  }
  copies_wait<0>();
#pragma unroll
  for (int c = 0; c < NK; ++c) blk.add_up(red, aq[c]);
  if (blk.grp != 0) return;
  float* dq = static_cast<float*>(p.dq) + bh * p.Nq * dk;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = i0 + 4 * blk.ty + i;
    if (row >= p.Nq) continue;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int d = c * T64 + 4 * tx + m;
        if (d < dk) dq[row * dk + d] = aq[c][i][m] * p.scale;
      }
  }
  seq::pdl_wait();  // dkr, which waits for this kernel, reads what dkdv wrote
}

template <typename T>
__global__ void __launch_bounds__(256) fa_latent_bwd_dkr_kernel(const float* __restrict__ part, T* __restrict__ dkr,
                                                                int H, long long per_head, long long total) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  seq::pdl_wait();
  if (i >= total) return;
  const float* src = part + (i / per_head) * H * per_head + i % per_head;
  float x = 0.f;
  for (int h = 0; h < H; ++h) x += src[h * per_head];
  store(dkr + i, x);
}

template <int NK, int NV, int BR>
cudaError_t launch_rows(const LatentBwd& p, cudaStream_t s) {
  constexpr int SMEM = bwd_smem<NK, NV, BR>();
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static seq::SmemOnce once_kv, once_q;
  cudaError_t e = once_kv(fa_latent_bwd_dkdv_kernel<NK, NV, BR>, SMEM);
  if (e != cudaSuccess) return e;
  e = once_q(fa_latent_bwd_dq_kernel<NK, NV, BR>, SMEM);
  if (e != cudaSuccess) return e;
  const long long bh = static_cast<long long>(p.B) * p.H;
  const long long kb = bh * ((p.Nk + BR - 1) / BR), qb = bh * ((p.Nq + BR - 1) / BR);
  if (kb > 0x7fffffffLL || qb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int vec = p.dn % 4 == 0 && p.dr % 4 == 0 && p.dv % 4 == 0;  // 16-byte rows
  fa_latent_bwd_dkdv_kernel<NK, NV, BR><<<static_cast<unsigned>(kb), kThreads, SMEM, s>>>(p, vec);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return seq::launch_after(fa_latent_bwd_dq_kernel<NK, NV, BR>, static_cast<unsigned>(qb), kThreads, SMEM, s, p, vec);
}
// Rows a CTA: 32 where that fills the SMs, else 16, which take less time each;
// 64 where that fills them and two CTAs of 32 do not fit an SM.  Forward and
// backward with 64, 32, 16 rows, 68 + 40 wide: 6 heads of 333 tokens 148, 114,
// 101 us, of 1500 tokens 925, 739, 749; 96 + 64 wide: 64 heads of 1000 tokens
// 2424, 2267, 2692; 192 + 128 wide (one CTA an SM): 16 heads of 1000 tokens
// 1445, 1548, 1823.
template <int NK, int NV>
cudaError_t launch_nkv(const LatentBwd& p, cudaStream_t s) {
  const long long n = p.Nk < p.Nq ? p.Nk : p.Nq, bh = static_cast<long long>(p.B) * p.H;
  if constexpr (bwd_ctas<NK, NV, 32>() == 1)
    if (bh * ((n + 63) / 64) >= 152) return launch_rows<NK, NV, 64>(p, s);
  return bh * ((n + 31) / 32) >= 152 ? launch_rows<NK, NV, 32>(p, s) : launch_rows<NK, NV, 16>(p, s);
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
    return seq::launch_after(fa_latent_bwd_dkr_kernel<float>, static_cast<unsigned>(blocks), 256, 0, s, p.dkr_part,
                             static_cast<float*>(p.dkr), p.H, per_head, total);
  return seq::launch_after(fa_latent_bwd_dkr_kernel<__nv_bfloat16>, static_cast<unsigned>(blocks), 256, 0, s,
                           p.dkr_part, static_cast<__nv_bfloat16*>(p.dkr), p.H, per_head, total);
}

}  // namespace fa
