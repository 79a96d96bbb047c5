// seq_fwd_simt.cu -- exact attention of groups of query rows over their own
// keys, fp32 on CUDA cores: latent attention (expanded and absorbed) and
// shared-prefix attention on float32 tensors, any head width.
//
// Per query row i of a group:  S_ij = scale (q_i . k_j) over the keys j the
// row sees, O_i = sum_j softmax_j(S_i) v_j, lse_i = ln sum_j exp(S_ij), by
// one pass over the keys with the row's running maximum and sum (all fp32,
// accurate expf / logf).  A row that sees no key gives O = 0, lse = -inf.
//
// One CTA of 256 threads per TR query rows (32 or 16, by the launch's size) and
// split of the keys; tiles of 64 keys.  The queries stay in shared memory; keys
// and values stream through a ring of 64 x 64 chunks, copied asynchronously up
// to three chunks ahead.  Products go in 4 x 4 blocks a
// thread (seq_simt.cuh); the scores pass through shared memory, where the
// softmax takes them a half-warp a row.
// Calls with few rows are bound by the latency of one tile's chunks (the keys
// are split until every CTA has about one tile), many rows by the multiply-adds
// (16 heads of 2500 tokens, q and k 96 wide, v 64, causal: 809 us, 20 TFLOP/s).
#include <cmath>

#include "seq_kernels.h"
#include "seq_simt.cuh"
#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace simt;

constexpr int BK = T64;  // keys per tile
constexpr int DEPTH = 4;  // chunks of the ring

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

__device__ __forceinline__ long long out_row(const SeqAttn& p, int g, int r) {
  return (g / p.group_div) * p.q_s1 + (g % p.group_div) * p.q_s2 + (r / p.row_block) * p.q_s3 + r % p.row_block;
}

// NCV: 64-column chunks of O a thread holds (dv <= 64 NCV)
// VEC: every row and part begins on a 16-byte boundary
template <int TR, int NCV, bool VEC>
__global__ void __launch_bounds__(kThreads, NCV <= 2 ? 2 : 1) fa_seq_fwd_simt_kernel(const __grid_constant__ SeqAttn p) {
  constexpr bool vec = VEC;
  constexpr int RPT = TR / 16;  // rows of the softmax a half-warp
  extern __shared__ float4 smem4[];
  seq::pdl_launch();  // the merge waits for this kernel's end before it reads
  float* ring = reinterpret_cast<float*>(smem4);  // [DEPTH] chunks of keys or values
  float* red = ring + DEPTH * CHUNK;              // [G][TR][LD] the groups' scores, or sums
  float* Ps = red;                                // [TR][LD] P: an entry replaces group 0's score of the same thread
  float* row_alpha = red + T64 * LD;           // [TR] factor of a row's O, then 1 / its sum
  float* Qs = row_alpha + TR;                     // [chunks of dk][TR][LD]
  const int row_tiles = (p.rows + TR - 1) / TR;
  const int g = blockIdx.x / row_tiles;
  const int r0 = (blockIdx.x % row_tiles) * TR;
  const int split = blockIdx.y;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const Block<TR> blk;
  const int dk = p.d1 + p.d2, nck = (dk + T64 - 1) / T64, ncv = (p.dv + T64 - 1) / T64;
  const float* q = static_cast<const float*>(p.q);
  const float* k1 = static_cast<const float*>(p.k1);
  const float* k2 = static_cast<const float*>(p.k2);
  const float* v = static_cast<const float*>(p.v);

  int nk = p.n_keys;
  if (p.lens != nullptr) {
    const int n = p.lens[g / p.lens_div];
    nk = min(max(n, 0), p.n_keys);
    if (n != nk && tid == 0) atomicOr(p.status, kStatusInput);
  }
  // keys that some row of this CTA sees
  int seen = nk;
  if (p.causal && r0 % p.n_new + TR <= p.n_new)
    seen = min(nk, nk - (p.n_new - 1 - min(r0 + TR - 1, p.rows - 1) % p.n_new));
  const int tiles = seen > 0 ? (seen + BK - 1) / BK : 0;
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / p.splits);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / p.splits);

  // this thread's four rows of a tile of keys (null: no such key, reads as zero)
  const float *kp[4], *k2p[4], *vp[4];
  auto place = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = tile * BK + ty + 16 * i;
      kp[i] = nullptr;
      if (j >= nk) continue;
      long long row = static_cast<long long>(g) * p.n_keys + j;
      k2p[i] = k2 + (static_cast<long long>(g / p.k2_div) * p.n_keys + j) * p.d2;
      if (p.page_size > 0) {
        const int at = j / p.page_size;
        const int page = p.table != nullptr ? p.table[static_cast<long long>(g) * p.max_pages + at] : g;
        if (page < 0 || page >= p.n_pages) {
          atomicOr(p.status, kStatusInput);
          continue;
        }
        row = static_cast<long long>(page) * p.page_size + (j - at * p.page_size);
      }
      kp[i] = k1 + row * p.d1;
      vp[i] = v + row * p.v_stride;
    }
  };
  // chunk `stage` of the tile that was placed (keys first, then values) to ring slot `slot`
  auto fetch = [&](int stage, int slot) {
    float* dst = ring + slot * CHUNK + ty * LD + 4 * tx;
#pragma unroll
    for (int i = 0; i < 4; ++i, dst += 16 * LD) {
      const bool on = kp[i] != nullptr;
      if (stage < nck)
        copy_row4(dst, on ? kp[i] : k1, p.d1, on ? k2p[i] : k2, p.d2, on, stage * T64 + 4 * tx, vec);
      else
        copy_row4(dst, on ? vp[i] : v, on, (stage - nck) * T64 + 4 * tx, p.dv, vec);
    }
  };
  // the stream: nck + ncv chunks a tile; (f_tile, f_stage) is the next one to ask for, into slot f_slot
  int f_tile = t0, f_stage = 0, f_slot = 0, slot = 0;
  auto ask = [&]() {
    if (f_tile < t1) {
      if (f_stage == 0) place(f_tile);
      fetch(f_stage, f_slot);
      if (++f_stage == nck + ncv) {
        f_stage = 0;
        ++f_tile;
      }
    }
    copies_commit();  // a group a call, empty or not, so that the wait below counts chunks
    f_slot = f_slot + 1 == DEPTH ? 0 : f_slot + 1;
  };
  // the next chunk of the stream, complete; asks for the one DEPTH - 1 later,
  // whose slot every thread has left
  auto next = [&]() -> const float* {
    copies_wait<DEPTH - 2>();
    __syncthreads();
    const float* chunk = ring + slot * CHUNK;
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    ask();
    return chunk;
  };
#pragma unroll 1
  for (int i = 0; i < RPT; ++i) {
    const int r = r0 + ty + 16 * i;
    const bool on = r < p.rows;
    const float* row = q + (on ? out_row(p, g, r) * dk : 0);
#pragma unroll 1
    for (int c = 0; c < nck; ++c)
      copy_row4(Qs + (c * TR + ty + 16 * i) * LD + 4 * tx, row, on, c * T64 + 4 * tx, dk, vec);
  }
  // (the queries travel in the first chunk's group)
#pragma unroll 1
  for (int c = 0; c < DEPTH - 1; ++c) ask();
  int limit[RPT];  // keys that the thread's rows see
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = r0 + RPT * ty + i;
    limit[i] = r < p.rows ? (p.causal ? nk - (p.n_new - 1 - r % p.n_new) : nk) : 0;
  }
  float m[RPT], l[RPT], acc[NCV][4][4];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll
  for (int c = 0; c < NCV; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[c][i][e] = 0.f;

#pragma unroll 1
  for (int kt = t0; kt < t1; ++kt) {
    const int k0 = kt * BK;
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 1
    for (int c = 0; c < nck + ncv; ++c) {
      const float* chunk = next();  // (also makes P and the rows' factors visible)
      if (c < nck) blk.dot(s, Qs + c * TR * LD, chunk, (min(T64, dk - c * T64) + 3) >> 2);
      if (c == nck) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = row_alpha[4 * blk.ty + i];
#pragma unroll
          for (int e = 0; e < NCV; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[e][i][x] *= a;
        }
      }
#pragma unroll
      for (int e = 0; e < NCV; ++e)
        if (c == nck + e) blk.accumulate(acc[e], Ps, chunk);
      if (c != nck - 1) continue;
      blk.put_dot(red, s);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = RPT * ty + i;
        float tmax = -INFINITY, x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sc = Block<TR>::get(red, r, tx + 16 * j);
          x[j] = k0 + tx + 16 * j < limit[i] ? sc * p.scale : -INFINITY;
          tmax = fmaxf(tmax, x[j]);
        }
        const float m_new = fmaxf(m[i], half_warp_max(tmax));
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = expf(m[i] - ref);  // 0 while the row has seen no key
        float rs = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pv = expf(x[j] - ref);
          rs += pv;
          Ps[r * LD + tx + 16 * j] = pv;
        }
        l[i] = l[i] * alpha + half_warp_sum(rs);
        m[i] = m_new;
        if (tx == 0) row_alpha[r] = alpha;
      }
    }
  }
  copies_wait<0>();
#pragma unroll
  for (int c = 0; c < NCV; ++c)
    if (c < ncv) blk.add_up(red, acc[c]);
  __syncthreads();  // row_alpha is no longer read
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = RPT * ty + i;
    if (tx == 0) {
      row_alpha[r] = l[i] == 0.f ? 0.f : 1.f / l[i];  // no key: 0
      if (r0 + r < p.rows) {
        const long long row = out_row(p, g, r0 + r);
        const float lse = m[i] + logf(l[i]);  // no key: -inf
        if (p.part_o != nullptr)
          p.part_lse[(p.part0 + split) * p.total + row] = lse;
        else if (p.lse != nullptr)
          p.lse[row] = lse;
      }
    }
  }
  __syncthreads();
  if (blk.grp == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * blk.ty + i;
      if (r0 + r >= p.rows) continue;
      const long long row = out_row(p, g, r0 + r);
      const float inv = row_alpha[r];
      float* dst = p.part_o != nullptr ? p.part_o + ((p.part0 + split) * p.total + row) * p.dv
                                       : static_cast<float*>(p.o) + row * p.dv;
#pragma unroll
      for (int c = 0; c < NCV; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = c * T64 + 4 * tx + e;
          if (d < p.dv) dst[d] = acc[c][i][e] * inv;
        }
    }
  }
  seq::pdl_wait();  // a kernel of the same call may run beside this one: the merge waits for both
}

template <int TR, int NCV, bool VEC>
cudaError_t launch_vec(const SeqAttn& p, bool beside, cudaStream_t s) {
  const int nck = (p.d1 + p.d2 + T64 - 1) / T64;
  const int smem = (DEPTH * CHUNK + TR * LD * nck + 64 * LD + TR) * 4;
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  static seq::SmemOnce once;
  const cudaError_t e = once(fa_seq_fwd_simt_kernel<TR, NCV, VEC>, 227 * 1024);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.groups) * ((p.rows + TR - 1) / TR);
  if (blocks > 0x7fffffffLL || p.splits > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), p.splits);
  if (beside) return seq::launch_after(fa_seq_fwd_simt_kernel<TR, NCV, VEC>, grid, kThreads, smem, s, p);
  fa_seq_fwd_simt_kernel<TR, NCV, VEC><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int TR, int NCV>
cudaError_t launch_one(const SeqAttn& p, bool beside, cudaStream_t s) {
  const bool vec = p.d1 % 4 == 0 && p.d2 % 4 == 0 && p.dv % 4 == 0 && p.v_stride % 4 == 0;
  return vec ? launch_vec<TR, NCV, true>(p, beside, s) : launch_vec<TR, NCV, false>(p, beside, s);
}

template <int TR>
cudaError_t launch_tr(const SeqAttn& p, bool beside, cudaStream_t s) {
  if (p.dv <= 64) return launch_one<TR, 1>(p, beside, s);
  if (p.dv <= 128) return launch_one<TR, 2>(p, beside, s);
  if (p.dv <= 256) return launch_one<TR, 4>(p, beside, s);
  if (p.dv <= 512) return launch_one<TR, 8>(p, beside, s);
  return cudaErrorInvalidValue;
}

// Rows of a CTA: 32, or 16 where that leaves SMs idle (a chunk costs such a CTA
// less, though more for each row).  Causal, 68 + 40 wide, 6 heads: 333 tokens
// 33 us with 32 rows, 27 with 16; 1500 tokens 168 and 181.  (64 rows: 48 and
// 169; 16 heads of 2500 tokens, 96 and 64 wide: 804 us with 32 rows, 875 with 64.)
int rows_per_cta(long long groups, int rows, int splits) {
  return rows > 16 && groups * ((rows + 31) / 32) * splits >= 152 ? 32 : 16;
}

}  // namespace

// Splits of the keys: `ctas` CTAs an SM of 152, or a tile a split.  Where as many
// fit an SM at once this is one round (a second one costs more than a second
// tile); past 128 value columns only one does (absorbed_layout has both sides).
int seq_simt_splits(long long groups, int rows, int max_keys, int ctas) {
  const int tr = rows <= 16 ? 16 : 32;
  const long long blocks = groups * ((rows + tr - 1) / tr);
  const int tiles = (max_keys + BK - 1) / BK;
  long long n = ctas * 152LL / blocks;
  if (n > tiles) n = tiles;
  if (n > 64) n = 64;
  return n < 1 ? 1 : static_cast<int>(n);
}

cudaError_t launch_seq_simt(const SeqAttn& args, bool beside, cudaStream_t s) {
  SeqAttn p = args;
  if (p.k2 == nullptr) p.k2 = p.k1;  // never read: copies of nothing still name an address
  return rows_per_cta(p.groups, p.rows, p.splits) == 32 ? launch_tr<32>(p, beside, s) : launch_tr<16>(p, beside, s);
}

}  // namespace fa
