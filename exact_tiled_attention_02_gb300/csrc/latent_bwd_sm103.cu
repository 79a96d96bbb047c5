// latent_bwd_sm103.cu -- the expanded latent attention's backward, bf16 in /
// fp32 accumulate, on the tensor cores of GB300 (sm_103a).
//
// Recomputation as in "Flash attention and efficient attention -- Hinglish
// notes", "Backward Pass: Recomputation".  With k_j = [kn_j | kr_j] (128 + 64
// wide, kr shared by the heads), v and dO 128 wide:
//   P_ij = exp(scale q_i.k_j - lse_i),  dS_ij = P_ij (dO_i.v_j - D_i),
//   dV_j = sum_i P_ij dO_i,  dk_j = scale sum_i dS_ij q_i,
//   dQ_i = scale sum_j dS_ij k_j.
//
// One kernel in two forms, each rebuilding S and dP on chip; every gradient
// row is summed by one CTA in one order, so there are no atomics and results
// repeat bit for bit:
//   keys form     CTA = 128 keys of a head, streams the query tiles that see
//                 them:  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   queries form  CTA = 128 queries, streams the key tiles they see:
//                 S = Q K^T, dP = dO V^T, dQ += dS K
// (A fused kernel would spend 5 products instead of the 4 + 3 here, but needs
// the 128 x 192 fp32 dQ tiles added up in device memory by every key tile's
// CTA, and beside dK (192 columns) and dV (128) tensor memory has no room for
// them.)
//
// Each form keeps its stationary 128 rows (A1 192 wide, A2 128 wide) in shared
// memory and streams tiles of 64 rows (B1, B2) through three stages:
//   S = A1 B1^T and dP = A2 B2^T (128 x 64), then element-wise P and dS, then
//   acc2 += dS B1 and, in the keys form, acc1 += P B2.
// Tensor memory: acc2 [0,192), acc1 [192,320), S in two buffers [320,384) and
// [384,448), dP [448,512); P and dS (packed bf16, the A operands of the
// accumulating products) overwrite their S, each warpgroup's in the 32
// columns that it alone reads.  Issue order per step i: S_{i+1}, then once the
// element-wise work of step i is published dP_{i+1}, acc1, acc2: the tensor
// core has acc_i and S_{i+2} to run while step i + 1's element-wise work goes on.
// 384 threads: warps 0-7 element-wise (thread = row, warpgroup = half of the
// 64 columns), warp 8 MMA issuer and TMEM owner, warp 9 TMA producer.
//
// Bound by the tensor core's shared-memory reads: a 128 x 64 product reads
// (128 + 64) x 32 bytes of operands a K step (48 cycles at 128 bytes a cycle)
// for 32 cycles of multiplying.
#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BR = 128;   // stationary rows
constexpr int BC = 64;    // streamed rows per step
constexpr int DQK = 192, DN = 128, DR = 64, DV = 128;
constexpr int kThreads = 384;
constexpr int STAGES = 3;
constexpr int A_CHUNK = BR * 128, B_CHUNK = BC * 128;  // bytes of 64 columns
constexpr int OFF_A1 = 0;
constexpr int OFF_A2 = OFF_A1 + 3 * A_CHUNK;
constexpr int OFF_B = OFF_A2 + 2 * A_CHUNK;
constexpr int STAGE_BYTES = 5 * B_CHUNK;                // B1 (three chunks), B2 (two)
constexpr int OFF_VEC = OFF_B + STAGES * STAGE_BYTES;   // keys form: per stage 64 lse terms, 64 D terms
constexpr int VEC_BYTES = 2 * BC * 4;
constexpr int OFF_BAR = OFF_VEC + STAGES * VEC_BYTES;
// a_full, st_full[3], st_free[3], s_full[2], dp_full, e_full, fin
constexpr int NBAR = 1 + 2 * STAGES + 5;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM_USED = OFF_MISC + 16;
constexpr int SMEM_BYTES = SMEM_USED + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(OFF_VEC % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
constexpr uint32_t TM_ACC2 = 0, TM_ACC1 = 192, TM_S = 320, TM_DP = 448;

struct Bars {
  uint32_t base;
  __device__ uint32_t a_full() const { return base; }
  __device__ uint32_t st_full(int s) const { return base + 8 * (1 + s); }
  __device__ uint32_t st_free(int s) const { return base + 8 * (1 + STAGES + s); }
  __device__ uint32_t s_full(int b) const { return base + 8 * (1 + 2 * STAGES + b); }
  __device__ uint32_t dp_full() const { return base + 8 * (3 + 2 * STAGES); }
  __device__ uint32_t e_full() const { return base + 8 * (4 + 2 * STAGES); }
  __device__ uint32_t fin() const { return base + 8 * (5 + 2 * STAGES); }
};

// keys form: a1 = kn, a1r = kr, a2 = v (128-row boxes); b1 = q, b2 = dO (64-row boxes).
// queries form: a1 = q, a2 = dO; b1 = kn, b1r = kr, b2 = v.
struct BwdMapsL {
  CUtensorMap a1, a1r, a2, b1, b1r, b2;
};

template <bool KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    fa_latent_bwd_sm103_kernel(const __grid_constant__ BwdMapsL m, const __grid_constant__ LatentBwd p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  if (pad + SMEM_USED > static_cast<uint32_t>(SMEM_BYTES)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusLayout);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const Bars bar{sb + OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  const WaitCtl wc{p.status, abort_flag, p.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // heads vary fastest, the longest tiles come first
  const int heads = p.B * p.H;
  const int bh = blockIdx.x % heads, b = bh / p.H;
  const int off = p.Nk - p.Nq;  // row i sees keys j <= i + off when causal
  const int n_rows = KEYS ? p.Nk : p.Nq, n_cols = KEYS ? p.Nq : p.Nk;
  const int tiles = (n_rows + BR - 1) / BR;
  const int tile = KEYS ? blockIdx.x / heads : tiles - 1 - blockIdx.x / heads;
  const int r0 = tile * BR;
  int c_lo = 0, c_hi = (n_cols + BC - 1) / BC;  // streamed tiles
  if (p.causal) {
    if (KEYS)
      c_lo = min(c_hi, max(0, r0 - off) / BC);
    else
      c_hi = max(0, min(n_cols, min(n_rows, r0 + BR) + off) + BC - 1) / BC;
  }
  const int nsteps = max(0, c_hi - c_lo);

  if (threadIdx.x == 0) {
    mbar_init(bar.a_full(), 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar.st_full(s), 1);
      mbar_init(bar.st_free(s), 1);
    }
    mbar_init(bar.s_full(0), 1);
    mbar_init(bar.s_full(1), 1);
    mbar_init(bar.dp_full(), 1);
    mbar_init(bar.e_full(), 8);  // one arrive per element-wise warp
    mbar_init(bar.fin(), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The keys form waits for the row terms and only then lets the queries form
  // start, which fills its last round and, as the last of the two to end,
  // waits for it (they share no output).
  if (KEYS) {
    pdl_wait();
    pdl_launch();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 9) {
    // ------------------------------------------------------------------ TMA
    if (lane == 0 && nsteps > 0) {
      mbar_arrive_expect_tx(bar.a_full(), 5 * A_CHUNK);
      for (int c = 0; c < 3; ++c) {
        if (KEYS && c == 2)
          tma_load_3d(sb + OFF_A1 + c * A_CHUNK, &m.a1r, bar.a_full(), 0, r0, b);
        else
          tma_load_3d(sb + OFF_A1 + c * A_CHUNK, &m.a1, bar.a_full(), c * 64, r0, bh);
      }
      for (int c = 0; c < 2; ++c) tma_load_3d(sb + OFF_A2 + c * A_CHUNK, &m.a2, bar.a_full(), c * 64, r0, bh);
      const size_t npad = static_cast<size_t>((p.Nq + 127) / 128) * 128;
      int it = 0;
      for (; it < nsteps; ++it) {
        const int st = it % STAGES;
        if (it >= STAGES && !mbar_wait_backoff(bar.st_free(st), ((it / STAGES) - 1) & 1, wc)) break;
        const int c0 = (c_lo + it) * BC;
        const uint32_t dst = sb + OFF_B + st * STAGE_BYTES;
        mbar_arrive_expect_tx(bar.st_full(st), STAGE_BYTES + (KEYS ? VEC_BYTES : 0));
        for (int c = 0; c < 3; ++c) {
          if (!KEYS && c == 2)
            tma_load_3d(dst + c * B_CHUNK, &m.b1r, bar.st_full(st), 0, c0, b);
          else
            tma_load_3d(dst + c * B_CHUNK, &m.b1, bar.st_full(st), c * 64, c0, bh);
        }
        if (KEYS) {
          const uint32_t vec = sb + OFF_VEC + st * VEC_BYTES;
          bulk_load(vec, p.lse2 + bh * npad + c0, BC * 4, bar.st_full(st));
          bulk_load(vec + BC * 4, p.dsum + bh * npad + c0, BC * 4, bar.st_full(st));
        }
        for (int c = 0; c < 2; ++c) tma_load_3d(dst + (3 + c) * B_CHUNK, &m.b2, bar.st_full(st), c * 64, c0, bh);
      }
      if (*abort_flag) {
        // let copies already in flight land before the CTA's shared memory is released
        WaitCtl drain{nullptr, nullptr, wc.limit_ns};
        mbar_wait(bar.a_full(), 0, drain);
        for (int s = max(0, it - STAGES); s < it; ++s) mbar_wait(bar.st_full(s % STAGES), (s / STAGES) & 1, drain);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    // The whole warp runs it, converged (see mma_ss_w).
    {
      constexpr uint32_t idesc_s = idesc_bf16_f32(BR, BC, 0, 0);
      constexpr uint32_t idesc_a2 = idesc_bf16_f32(BR, DQK, 0, 1);
      constexpr uint32_t idesc_a1 = idesc_bf16_f32(BR, DV, 0, 1);
      auto issue_s = [&](int it) {
        const Desc2 a = desc_sw128(sb + OFF_A1, 16, 1024);
        const Desc2 bd = desc_sw128(sb + OFF_B + (it % STAGES) * STAGE_BYTES, 16, 1024);
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k)
          mma_ss_w(tmem + TM_S + 64 * (it & 1), a, ((k >> 2) * A_CHUNK + (k & 3) * 32) >> 4, bd,
                  ((k >> 2) * B_CHUNK + (k & 3) * 32) >> 4, idesc_s, k > 0);
        mma_commit_w(bar.s_full(it & 1));
      };
      auto issue_dp = [&](int it) {
        const Desc2 a = desc_sw128(sb + OFF_A2, 16, 1024);
        const Desc2 bd = desc_sw128(sb + OFF_B + (it % STAGES) * STAGE_BYTES + 3 * B_CHUNK, 16, 1024);
#pragma unroll
        for (int k = 0; k < DV / 16; ++k)
          mma_ss_w(tmem + TM_DP, a, ((k >> 2) * A_CHUNK + (k & 3) * 32) >> 4, bd,
                  ((k >> 2) * B_CHUNK + (k & 3) * 32) >> 4, idesc_s, k > 0);
        mma_commit_w(bar.dp_full());
      };
      auto issue_acc = [&](int it) {
        const uint32_t t = tmem + TM_S + 64 * (it & 1);
        const uint32_t st = sb + OFF_B + (it % STAGES) * STAGE_BYTES;
        // K step k: columns 16k..16k+15 of P and dS, which the warpgroup of
        // half k / 2 left at 32 (k / 2) (P) and 16 further (dS)
        if (KEYS) {
          const Desc2 b2 = desc_sw128(st + 3 * B_CHUNK, B_CHUNK, 1024);
#pragma unroll
          for (int k = 0; k < BC / 16; ++k)
            mma_ts_w(tmem + TM_ACC1, t + 32 * (k >> 1) + 8 * (k & 1), b2, (k * 16 * 128) >> 4, idesc_a1, it > 0 || k > 0);
        }
        const Desc2 b1 = desc_sw128(st, B_CHUNK, 1024);
#pragma unroll
        for (int k = 0; k < BC / 16; ++k)
          mma_ts_w(tmem + TM_ACC2, t + 32 * (k >> 1) + 16 + 8 * (k & 1), b1, (k * 16 * 128) >> 4, idesc_a2,
                  it > 0 || k > 0);
        mma_commit_w(bar.st_free(it % STAGES));
      };
      bool ok = nsteps > 0 && warp_wait2(bar.a_full(), 0, bar.st_full(0), 0, wc);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        issue_dp(0);
      }
      for (int it = 0; ok && it < nsteps; ++it) {
        const bool more = it + 1 < nsteps;
        if (more) {
          ok = warp_wait(bar.st_full((it + 1) % STAGES), ((it + 1) / STAGES) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          issue_s(it + 1);
        }
        ok = warp_wait(bar.e_full(), it & 1, wc);
        if (!ok) break;
        tc_fence_after();
        if (more) issue_dp(it + 1);
        issue_acc(it);
      }
      // every MMA this thread issued must finish before tensor memory is read or freed
      mma_commit_w(bar.fin());
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      mbar_wait(bar.fin(), 0, drain);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------------------------------------------------- element-wise
    const int half = warp >> 2;
    const int row = threadIdx.x & 127, r = r0 + row;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sl = p.scale * 1.4426950408889634f;
    float row_l2 = 0.f, row_d = 0.f;
    if (!KEYS) {
      const size_t npad = static_cast<size_t>((p.Nq + 127) / 128) * 128;
      row_l2 = p.lse2[bh * npad + r];  // padded to whole tiles
      row_d = p.dsum[bh * npad + r];
    }
    bool ok = true;
    for (int it = 0; it < nsteps; ++it) {
      const uint32_t tS = tl + TM_S + 64 * (it & 1) + 32 * half, tD = tl + TM_DP + 32 * half;
      // (the stage's own barrier too: this thread reads the row terms that it counts)
      if (!warp_wait(bar.s_full(it & 1), (it >> 1) & 1, wc) ||
          (KEYS && !warp_wait(bar.st_full(it % STAGES), (it / STAGES) & 1, wc))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sr[32];
      tmem_ld_32x32b_x32(tS, sr);
      tmem_wait_ld();
      const int c0 = (c_lo + it) * BC + 32 * half;  // first column of this half
      float pr[32];
      const float4* vl = reinterpret_cast<const float4*>(smem + OFF_VEC + (it % STAGES) * VEC_BYTES + half * 128);
#pragma unroll
      for (int c4 = 0; c4 < 8; ++c4) {
        float4 l2 = make_float4(row_l2, row_l2, row_l2, row_l2);
        if (KEYS) l2 = vl[c4];
        const float lv[4] = {l2.x, l2.y, l2.z, l2.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[4 * c4 + e] = ex2_approx(fmaf(__uint_as_float(sr[4 * c4 + e]), sl, lv[e]));
      }
      if (KEYS) {
        // query c0 + c sees key r iff r <= c0 + c + off; the lowest query and highest key of the tile decide whether any pair is masked
        if (p.causal && r0 + BR - 1 > c0 + off) {
          const int first = r - off - c0;
#pragma unroll
          for (int c = 0; c < 32; ++c) pr[c] = c >= first ? pr[c] : 0.f;
        }
      } else {
        // keys past the end read as zeros, and their exp may overflow: masked too
        const int limit = p.causal ? min(p.Nk, r + off + 1) : p.Nk;
        const int low = p.causal ? min(p.Nk, r0 + off + 1) : p.Nk;
        if (c0 + 32 > low) {
#pragma unroll
          for (int c = 0; c < 32; ++c) pr[c] = c0 + c < limit ? pr[c] : 0.f;
        }
      }
      if (KEYS) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(pr[2 * c], pr[2 * c + 1]);
        tmem_st_32x32b_x16(tS, pk);
      }
      if (!warp_wait(bar.dp_full(), it & 1, wc)) {
        tmem_wait_st();
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld_32x32b_x32(tD, sr);
      tmem_wait_ld();
      uint32_t dk[16];
#pragma unroll
      for (int c4 = 0; c4 < 8; ++c4) {
        float4 dv = make_float4(row_d, row_d, row_d, row_d);
        if (KEYS) dv = vl[BC / 4 + c4];
        const float ds0 = pr[4 * c4] * (__uint_as_float(sr[4 * c4]) + dv.x);
        const float ds1 = pr[4 * c4 + 1] * (__uint_as_float(sr[4 * c4 + 1]) + dv.y);
        const float ds2 = pr[4 * c4 + 2] * (__uint_as_float(sr[4 * c4 + 2]) + dv.z);
        const float ds3 = pr[4 * c4 + 3] * (__uint_as_float(sr[4 * c4 + 3]) + dv.w);
        dk[2 * c4] = pack_bf16x2(ds0, ds1);  // one rounding, as the products take bf16
        dk[2 * c4 + 1] = pack_bf16x2(ds2, ds3);
      }
      tmem_st_32x32b_x16(tS + 16, dk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.e_full());
    }
    // -------------------------------------------------------------- output
    const bool have = ok && warp_wait(bar.fin(), 0, wc) && !*abort_flag;
    tc_fence_after();
    // columns [lo, hi) of an accumulator, 32 at a time; zeros where nothing was streamed
    auto load32 = [&](uint32_t col, float mul, float* x) {
      uint32_t o[32];
      if (nsteps > 0) {
        tmem_ld_32x32b_x32(tl + col, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = nsteps > 0 ? __uint_as_float(o[e]) * mul : 0.f;
    };
    auto store_bf16 = [&](void* base, long long elem, const float* x) {
      uint8_t* dst = static_cast<uint8_t*>(base) + elem * 2;
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        st_global_v4(dst + q4 * 16,
                     make_uint4(pack_bf16x2(x[8 * q4], x[8 * q4 + 1]), pack_bf16x2(x[8 * q4 + 2], x[8 * q4 + 3]),
                                pack_bf16x2(x[8 * q4 + 4], x[8 * q4 + 5]), pack_bf16x2(x[8 * q4 + 6], x[8 * q4 + 7])));
    };
    if (have) {
      const long long grow = static_cast<long long>(bh) * n_rows + r;
#pragma unroll 1
      for (int c = 3 * half; c < 3 * half + 3; ++c) {  // acc2: six groups of 32 columns, three a warpgroup
        float x[32];
        load32(TM_ACC2 + 32 * c, p.scale, x);
        if (r >= n_rows) continue;
        if (!KEYS) {
          store_bf16(p.dq, grow * DQK + 32 * c, x);
        } else if (c < 4) {
          store_bf16(p.dkn, grow * DN + 32 * c, x);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.dkr_part + grow * DR + 32 * (c - 4));
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
      if (KEYS) {
#pragma unroll 1
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          float x[32];
          load32(TM_ACC1 + 32 * c, 1.f, x);
          if (r < n_rows) store_bf16(p.dv_out, grow * DV + 32 * c, x);
        }
      }
    }
    tc_fence_before();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!KEYS) pdl_wait();
}

template <bool KEYS>
cudaError_t launch_form(const LatentBwd& p, const BwdMapsL& m, cudaStream_t s) {
  static SmemOnce once;
  const cudaError_t e = once(fa_latent_bwd_sm103_kernel<KEYS>, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.B) * p.H * (((KEYS ? p.Nk : p.Nq) + BR - 1) / BR);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_after(fa_latent_bwd_sm103_kernel<KEYS>, static_cast<unsigned>(blocks), kThreads, SMEM_BYTES, s, m, p);
}

}  // namespace

cudaError_t launch_latent_bwd_sm103(const LatentBwd& p, cudaStream_t s) {
  const long long bh = static_cast<long long>(p.B) * p.H;
  BwdMapsL k, q;
  if (!make_map3(&k.a1, p.kn, DN, p.Nk, bh, BR) || !make_map3(&k.a1r, p.kr, DR, p.Nk, p.B, BR) ||
      !make_map3(&k.a2, p.v, DV, p.Nk, bh, BR) || !make_map3(&k.b1, p.q, DQK, p.Nq, bh, BC) ||
      !make_map3(&k.b2, p.dO, DV, p.Nq, bh, BC) || !make_map3(&q.a1, p.q, DQK, p.Nq, bh, BR) ||
      !make_map3(&q.a2, p.dO, DV, p.Nq, bh, BR) || !make_map3(&q.b1, p.kn, DN, p.Nk, bh, BC) ||
      !make_map3(&q.b1r, p.kr, DR, p.Nk, p.B, BC) || !make_map3(&q.b2, p.v, DV, p.Nk, bh, BC))
    return cudaErrorInvalidValue;
  k.b1r = k.b1;
  q.a1r = q.a1;
  const cudaError_t e = launch_form<true>(p, k, s);
  return e != cudaSuccess ? e : launch_form<false>(p, q, s);
}

}  // namespace fa
