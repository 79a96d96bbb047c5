// seq_fwd_simt.cu -- exact attention of groups of query rows over their own
// keys, fp32 on CUDA cores: latent attention (expanded and absorbed) and
// shared-prefix attention, in every shape the entry points accept.
//
// Per query row i of a group:  S_ij = scale (q_i . k_j) over the keys j the
// row sees, O_i = sum_j softmax_j(S_i) v_j, lse_i = ln sum_j exp(S_ij), by
// one pass over the keys with the row's running maximum and sum (all fp32,
// accurate expf / logf).  A row that sees no key gives O = 0, lse = -inf.
//
// One CTA of 256 threads per TR query rows (64, or 16 for small groups) and
// split of the keys; tiles of 64 keys.  The head dimensions stream through
// shared memory 64 at a time, so any width fits: per tile, S accumulates over
// the chunks of q and k (thread (ty, tx): rows TR/16 ty.., keys 4tx..), P
// goes through shared memory, and O accumulates chunk by chunk in registers
// (the thread's rows, columns 4tx.. of every chunk).  Where a key's row is
// (a page, a shared rotary part) is worked out once per tile and key.
#include <cmath>

#include "seq_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int BK = 64;        // keys per tile
constexpr int CH = 64;        // head dimensions per chunk
constexpr int LD = 68;        // row stride (floats) of the shared-memory tiles: 16-byte aligned rows
constexpr int kThreads = 256;

__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <int TR>
constexpr int smem_bytes() {
  return (CH * LD + CH * LD + TR * LD) * 4 + TR * 8 + 2 * BK * 8 + TR * 4;
}

// NCV: 64-column chunks of O a thread holds (dv <= 64 NCV)
template <typename T, int TR, int NCV>
__global__ void __launch_bounds__(kThreads) fa_seq_fwd_simt_kernel(const SeqAttn p) {
  constexpr int RPT = TR / 16;
  extern __shared__ float4 smem4[];
  float* Qs = reinterpret_cast<float*>(smem4);  // [CH][LD]: chunk column c of row r at c * LD + r
  float* Ks = Qs + CH * LD;                     // [CH][LD]: chunk column c of key j; V: [BK][LD]
  float* Ps = Ks + CH * LD;                     // [TR][LD]
  long long* q_row = reinterpret_cast<long long*>(Ps + TR * LD);  // [TR], -1 past the last row
  long long* k_row = q_row + TR;                                  // [BK], -1: no such key (reads as zero)
  long long* k2_row = k_row + BK;                                 // [BK]
  int* limit = reinterpret_cast<int*>(k2_row + BK);               // [TR] keys the row sees

  const int row_tiles = (p.rows + TR - 1) / TR;
  const int g = blockIdx.x / row_tiles;
  const int r0 = (blockIdx.x % row_tiles) * TR;
  const int split = blockIdx.y;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int dk = p.d1 + p.d2;

  int nk = p.n_keys;
  if (p.lens != nullptr) {
    const int n = p.lens[g / p.lens_div];
    nk = min(max(n, 0), p.n_keys);
    if (n != nk && tid == 0) atomicOr(p.status, sm103::kStatusInput);
  }
  if (tid < TR) {
    const int r = r0 + tid;
    q_row[tid] = r < p.rows ? (g / p.group_div) * p.q_s1 + (g % p.group_div) * p.q_s2 +
                                  (r / p.row_block) * p.q_s3 + r % p.row_block
                            : -1;
    limit[tid] = r < p.rows ? (p.causal ? nk - (p.n_new - 1 - r % p.n_new) : nk) : 0;
  }
  // keys that some row of this CTA sees
  int seen = nk;
  if (p.causal && r0 % p.n_new + TR <= p.n_new) seen = min(nk, nk - (p.n_new - 1 - min(r0 + TR - 1, p.rows - 1) % p.n_new));
  const int tiles = seen > 0 ? (seen + BK - 1) / BK : 0;
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / p.splits);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / p.splits);

  const T* q = static_cast<const T*>(p.q);
  const T* k1 = static_cast<const T*>(p.k1);
  const T* k2 = static_cast<const T*>(p.k2);
  const T* v = static_cast<const T*>(p.v);
  float m[RPT], l[RPT], acc[RPT][NCV][4];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NCV; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.f;
  }

  for (int kt = t0; kt < t1; ++kt) {
    const int k0 = kt * BK;
    __syncthreads();  // the previous tile is no longer read
    if (tid < BK) {
      const int j = k0 + tid;
      long long row = -1, row2 = -1;
      if (j < nk) {
        row = static_cast<long long>(g) * p.n_keys + j;
        row2 = static_cast<long long>(g / p.k2_div) * p.n_keys + j;
        if (p.page_size > 0) {
          const int page = p.table != nullptr ? p.table[static_cast<long long>(g) * p.max_pages + j / p.page_size] : g;
          const bool bad = page < 0 || page >= p.n_pages;
          if (bad) atomicOr(p.status, sm103::kStatusInput);
          row = bad ? -1 : static_cast<long long>(page) * p.page_size + j % p.page_size;
        }
      }
      k_row[tid] = row;
      k2_row[tid] = row2;
    }
    float s[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int c0 = 0; c0 < dk; c0 += CH) {
      const int cc = min(CH, dk - c0);
      __syncthreads();
      for (int idx = tid; idx < TR * CH; idx += kThreads) {
        const int c = idx & (CH - 1), r = idx / CH;
        if (c < cc) Qs[c * LD + r] = q_row[r] >= 0 ? to_f32(q[q_row[r] * dk + c0 + c]) : 0.f;
      }
      for (int idx = tid; idx < BK * CH; idx += kThreads) {
        const int c = idx & (CH - 1), j = idx / CH;
        if (c < cc) {
          const int d = c0 + c;
          float x = 0.f;
          if (k_row[j] >= 0) x = d < p.d1 ? to_f32(k1[k_row[j] * p.d1 + d]) : to_f32(k2[k2_row[j] * p.d2 + d - p.d1]);
          Ks[c * LD + j] = x;
        }
      }
      __syncthreads();
#pragma unroll 4
      for (int c = 0; c < cc; ++c) {
        const float4 b = *reinterpret_cast<const float4*>(Ks + c * LD + 4 * tx);
        const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float a = Qs[c * LD + RPT * ty + i];
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a, bv[j], s[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int lim = limit[RPT * ty + i];
      float tmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = k0 + 4 * tx + j < lim ? s[i][j] * p.scale : -INFINITY;
        tmax = fmaxf(tmax, s[i][j]);
      }
      const float m_new = fmaxf(m[i], half_warp_max(tmax));
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = expf(m[i] - ref);  // 0 while the row has seen no key
      float pv[4], rs = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pv[j] = expf(s[i][j] - ref);
        rs += pv[j];
      }
      l[i] = l[i] * alpha + half_warp_sum(rs);
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < NCV; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] *= alpha;
      *reinterpret_cast<float4*>(Ps + (RPT * ty + i) * LD + 4 * tx) = make_float4(pv[0], pv[1], pv[2], pv[3]);
    }
#pragma unroll
    for (int cv = 0; cv < NCV; ++cv) {
      if (cv * CH >= p.dv) break;
      __syncthreads();
      for (int idx = tid; idx < BK * CH; idx += kThreads) {
        const int c = idx & (CH - 1), j = idx / CH, d = cv * CH + c;
        Ks[j * LD + c] = (k_row[j] >= 0 && d < p.dv) ? to_f32(v[k_row[j] * p.v_stride + d]) : 0.f;
      }
      __syncthreads();
#pragma unroll 2
      for (int j4 = 0; j4 < BK; j4 += 4) {
        float pr[RPT][4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float4 t = *reinterpret_cast<const float4*>(Ps + (RPT * ty + i) * LD + j4);
          pr[i][0] = t.x;
          pr[i][1] = t.y;
          pr[i][2] = t.z;
          pr[i][3] = t.w;
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float4 b = *reinterpret_cast<const float4*>(Ks + (j4 + jj) * LD + 4 * tx);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][cv][e] = fmaf(pr[i][jj], bv[e], acc[i][cv][e]);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int rt = RPT * ty + i;
    const long long row = r0 + rt < p.rows ? (g / p.group_div) * p.q_s1 + (g % p.group_div) * p.q_s2 +
                                                 ((r0 + rt) / p.row_block) * p.q_s3 + (r0 + rt) % p.row_block
                                           : -1;
    if (row < 0) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // no key: 0; NaN stays NaN
    const float lse = m[i] + logf(l[i]);                                     // no key: -inf
    const long long prow = (p.part0 + split) * p.total + row;
#pragma unroll
    for (int c = 0; c < NCV; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = c * CH + 4 * tx + e;
        if (d < p.dv) {
          if (p.part_o != nullptr)
            p.part_o[prow * p.dv + d] = acc[i][c][e] * inv;
          else
            store(static_cast<T*>(p.o) + row * p.dv + d, acc[i][c][e] * inv);
        }
      }
    if (tx == 0) {
      if (p.part_o != nullptr)
        p.part_lse[prow] = lse;
      else if (p.lse != nullptr)
        p.lse[row] = lse;
    }
  }
}

template <typename T, int TR, int NCV>
cudaError_t launch_one(const SeqAttn& p, cudaStream_t s) {
  constexpr int SMEM = smem_bytes<TR>();
  const cudaError_t e = cudaFuncSetAttribute(fa_seq_fwd_simt_kernel<T, TR, NCV>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.groups) * ((p.rows + TR - 1) / TR);
  if (blocks > 0x7fffffffLL || p.splits > 65535) return cudaErrorInvalidConfiguration;
  fa_seq_fwd_simt_kernel<T, TR, NCV><<<dim3(static_cast<unsigned>(blocks), p.splits), kThreads, SMEM, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int TR>
cudaError_t launch_tr(const SeqAttn& p, cudaStream_t s) {
  if (p.dv <= 64) return launch_one<T, TR, 1>(p, s);
  if (p.dv <= 128) return launch_one<T, TR, 2>(p, s);
  if (p.dv <= 256) return launch_one<T, TR, 4>(p, s);
  if (p.dv <= 512) return launch_one<T, TR, 8>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace

int seq_simt_splits(long long groups, int rows, int max_keys) {
  const long long blocks = groups * (rows <= 16 ? 1 : (rows + 63) / 64);
  const int tiles = (max_keys + BK - 1) / BK;
  long long n = (4 * 152 + blocks - 1) / blocks;
  if (n > tiles) n = tiles;
  if (n > 64) n = 64;
  return n < 1 ? 1 : static_cast<int>(n);
}

cudaError_t launch_seq_simt(const SeqAttn& p, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_DTYPE_F32) return p.rows <= 16 ? launch_tr<float, 16>(p, s) : launch_tr<float, 64>(p, s);
  return p.rows <= 16 ? launch_tr<__nv_bfloat16, 16>(p, s) : launch_tr<__nv_bfloat16, 64>(p, s);
}

}  // namespace fa
