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
//   keys form     item = 128 keys of a head, streams the query tiles that see
//                 them:  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   queries form  item = 128 queries, streams the key tiles they see:
//                 S = Q K^T, dP = dO V^T, dQ += dS K
// (A fused kernel would spend 5 products instead of the 4 + 3 here, but needs
// the 128 x 192 fp32 dQ tiles added up in device memory by every key tile's
// CTA, and beside dK (192 columns) and dV (128) tensor memory has no room for
// them.)
//
// Each form keeps its stationary 128 rows (A1 192 wide, A2 128 wide) in shared
// memory and streams tiles of 64 rows, B1 through four stages and B2 through
// three (one ring of three for both left the tensor core waiting for loads:
// 1930 cycles a step, 1650 of them from a stage's release to its next load's
// arrival):
//   S = A1 B1^T and dP = A2 B2^T (128 x 64), then element-wise P and dS, then
//   acc2 += dS B1 and, in the keys form, acc1 += P B2.
// Tensor memory: acc2 [0,192), acc1 [192,320), S in two buffers [320,384) and
// [384,448), dP [448,512); P and dS (packed bf16, the A operands of the
// accumulating products) overwrite their S, each warpgroup's in the 32
// columns that it alone reads.  Issue order per step i: S_{i+1}, then once the
// element-wise work of step i is published dP_{i+1}, acc1, acc2: the tensor
// core has acc_i and S_{i+2} to run while step i + 1's element-wise work goes on.
// Persistent, one CTA per SM: an item's loads and first products overlap the
// last one's output.  (A CTA an item cost 16,200 cycles an item beside the 1545
// of a step; forward and backward of 4 x 16 x 2048: 394 us, so 365 us.)
// 384 threads: warps 0-7 element-wise (thread = row, warpgroup = half of the
// 64 columns), warp 8 MMA issuer and TMEM owner, warp 9 TMA producer.
//
// Within an item, bound by the tensor core's shared-memory reads: a 128 x 64
// product reads (128 + 64) x 32 bytes of operands a K step (48 cycles at 128
// bytes a cycle) for 32 cycles of multiplying; a step of the keys form takes
// 1545 cycles.  That is three quarters of the kernel: the keys form of 2 x 16 x
// 4096, causal, has 222 steps an SM, 170 to 180 us, and takes 240.  By this count
// the rest, some 9 us for each of a CTA's seven items, goes to their ends: the
// element-wise warps write 128 x 320 outputs before they take up the next item,
// whose stationary rows come into the one buffer that the last item's products
// held.
// Forward and backward of 2 x 16 x 4096: 632 us, 980 TFLOP/s by the formulas'
// products, at the power limit (605 us before it bites).
#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BR = 128;   // stationary rows
constexpr int BC = 64;    // streamed rows per step
constexpr int DQK = 192, DN = 128, DR = 64, DV = 128;
constexpr int kThreads = 384;
constexpr int NS1 = 4, NS2 = 3;                         // stages of B1 and of B2
constexpr int A_CHUNK = BR * 128, B_CHUNK = BC * 128;  // bytes of 64 columns
constexpr int OFF_A1 = 0;
constexpr int OFF_A2 = OFF_A1 + 3 * A_CHUNK;
constexpr int OFF_B1 = OFF_A2 + 2 * A_CHUNK;
constexpr int B1_BYTES = 3 * B_CHUNK, B2_BYTES = 2 * B_CHUNK;
constexpr int OFF_B2 = OFF_B1 + NS1 * B1_BYTES;
constexpr int VEC = BC * 4;                             // keys form: a stage's 64 lse terms (with B1), D terms (with B2)
constexpr int OFF_LSE = OFF_B2 + NS2 * B2_BYTES;
constexpr int OFF_D = OFF_LSE + NS1 * VEC;
constexpr int OFF_BAR = OFF_D + NS2 * VEC;
// a_full, a_free, b1_full[4], b1_free[4], b2_full[3], b2_free[3], s_full[2], dp_full, e_full, acc_full, acc_free, drain
constexpr int NBAR = 2 + 2 * NS1 + 2 * NS2 + 7;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM_USED = OFF_MISC + 8;
constexpr int SMEM_BYTES = SMEM_USED + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(OFF_LSE % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
constexpr uint32_t TM_ACC2 = 0, TM_ACC1 = 192, TM_S = 320, TM_DP = 448;

struct Bars {
  uint32_t base;
  __device__ uint32_t a_full() const { return base; }
  __device__ uint32_t a_free() const { return base + 8; }
  __device__ uint32_t b1_full(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t b1_free(int s) const { return base + 8 * (2 + NS1 + s); }
  __device__ uint32_t b2_full(int s) const { return base + 8 * (2 + 2 * NS1 + s); }
  __device__ uint32_t b2_free(int s) const { return base + 8 * (2 + 2 * NS1 + NS2 + s); }
  __device__ uint32_t at(int k) const { return base + 8 * (2 + 2 * NS1 + 2 * NS2 + k); }
  __device__ uint32_t s_full(int b) const { return at(b); }
  __device__ uint32_t dp_full() const { return at(2); }
  __device__ uint32_t e_full() const { return at(3); }
  __device__ uint32_t acc_full() const { return at(4); }
  __device__ uint32_t acc_free() const { return at(5); }
  __device__ uint32_t drain() const { return at(6); }
};

// keys form: a1 = kn, a1r = kr, a2 = v (128-row boxes); b1 = q, b2 = dO (64-row boxes).
// queries form: a1 = q, a2 = dO; b1 = kn, b1r = kr, b2 = v.
struct BwdMapsL {
  CUtensorMap a1, a1r, a2, b1, b1r, b2;
};

// A work item: 128 stationary rows of one head and the streamed tiles that
// meet them.  Items come in order of length, the longest first, heads varying
// fastest; CTA c of G takes item n G + c in even rounds n, n G + G - 1 - c in
// odd ones, so that the CTAs' sums stay close.
struct BwdItem {
  int bh, r0, c_lo, steps;
};
template <bool KEYS>
__device__ __forceinline__ bool bwd_item(const LatentBwd& p, int n, BwdItem& w) {
  const int heads = p.B * p.H, n_rows = KEYS ? p.Nk : p.Nq, n_cols = KEYS ? p.Nq : p.Nk;
  const int tiles = (n_rows + BR - 1) / BR, G = gridDim.x, c = blockIdx.x;
  const long long i = static_cast<long long>(n) * G + ((n & 1) ? G - 1 - c : c);
  if (i >= static_cast<long long>(heads) * tiles) return false;
  const int tile = KEYS ? static_cast<int>(i / heads) : tiles - 1 - static_cast<int>(i / heads);
  w.bh = static_cast<int>(i % heads);
  w.r0 = tile * BR;
  const int off = p.Nk - p.Nq;  // row i sees keys j <= i + off when causal
  int lo = 0, hi = (n_cols + BC - 1) / BC;
  if (p.causal) {
    if (KEYS)
      lo = min(hi, max(0, w.r0 - off) / BC);
    else
      hi = max(0, min(n_cols, min(n_rows, w.r0 + BR) + off) + BC - 1) / BC;
  }
  w.c_lo = lo;
  w.steps = max(0, hi - lo);
  return true;
}

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
  const int off = p.Nk - p.Nq;
  const int n_rows = KEYS ? p.Nk : p.Nq;

  if (threadIdx.x == 0) {
    mbar_init(bar.a_full(), 1);
    mbar_init(bar.a_free(), 1);
    for (int s = 0; s < NS1; ++s) {
      mbar_init(bar.b1_full(s), 1);
      mbar_init(bar.b1_free(s), 1);
    }
    for (int s = 0; s < NS2; ++s) {
      mbar_init(bar.b2_full(s), 1);
      mbar_init(bar.b2_free(s), 1);
    }
    mbar_init(bar.s_full(0), 1);
    mbar_init(bar.s_full(1), 1);
    mbar_init(bar.dp_full(), 1);
    mbar_init(bar.e_full(), 8);    // one arrive per element-wise warp
    mbar_init(bar.acc_full(), 1);
    mbar_init(bar.acc_free(), 8);
    mbar_init(bar.drain(), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The keys form waits for the row terms and only then lets the queries form
  // start, which takes over SMs as this one's CTAs end and, as the last of the
  // two to end, waits for it (they share no output).
  if (KEYS) {
    pdl_wait();
    pdl_launch();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Every barrier's phase counts on across items: steps (g) for the rings, S,
  // dP and the element-wise work, items with any step (na) for the rest.
  if (warp == 9) {
    // ------------------------------------------------------------------ TMA
    if (lane == 0) {
      const size_t npad = static_cast<size_t>((p.Nq + 127) / 128) * 128;
      BwdItem w;
      int g = 0, na = 0;
      bool ok = true;
      for (int n = 0; ok && bwd_item<KEYS>(p, n, w); ++n) {
        if (w.steps == 0) continue;
        const int b = w.bh / p.H;
        // the last item's S and dP products have read its rows
        if (na > 0 && !mbar_wait(bar.a_free(), (na - 1) & 1, wc)) break;
        mbar_arrive_expect_tx(bar.a_full(), 5 * A_CHUNK);
        for (int c = 0; c < 3; ++c) {
          if (KEYS && c == 2)
            tma_load_3d(sb + OFF_A1 + c * A_CHUNK, &m.a1r, bar.a_full(), 0, w.r0, b);
          else
            tma_load_3d(sb + OFF_A1 + c * A_CHUNK, &m.a1, bar.a_full(), c * 64, w.r0, w.bh);
        }
        for (int c = 0; c < 2; ++c) tma_load_3d(sb + OFF_A2 + c * A_CHUNK, &m.a2, bar.a_full(), c * 64, w.r0, w.bh);
        ++na;
        for (int it = 0; it < w.steps; ++it, ++g) {
          const int c0 = (w.c_lo + it) * BC, s1 = g % NS1, s2 = g % NS2;
          if (g >= NS1 && !mbar_wait(bar.b1_free(s1), ((g / NS1) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t b1 = sb + OFF_B1 + s1 * B1_BYTES, b2 = sb + OFF_B2 + s2 * B2_BYTES;
          mbar_arrive_expect_tx(bar.b1_full(s1), B1_BYTES + (KEYS ? VEC : 0));
          for (int c = 0; c < 3; ++c) {
            if (!KEYS && c == 2)
              tma_load_3d(b1 + c * B_CHUNK, &m.b1r, bar.b1_full(s1), 0, c0, b);
            else
              tma_load_3d(b1 + c * B_CHUNK, &m.b1, bar.b1_full(s1), c * 64, c0, w.bh);
          }
          if (KEYS) bulk_load(sb + OFF_LSE + s1 * VEC, p.lse2 + w.bh * npad + c0, VEC, bar.b1_full(s1));
          if (g >= NS2 && !mbar_wait(bar.b2_free(s2), ((g / NS2) - 1) & 1, wc)) {
            ok = false;
            ++g;  // its B1 is in flight
            break;
          }
          mbar_arrive_expect_tx(bar.b2_full(s2), B2_BYTES + (KEYS ? VEC : 0));
          for (int c = 0; c < 2; ++c) tma_load_3d(b2 + c * B_CHUNK, &m.b2, bar.b2_full(s2), c * 64, c0, w.bh);
          if (KEYS) bulk_load(sb + OFF_D + s2 * VEC, p.dsum + w.bh * npad + c0, VEC, bar.b2_full(s2));
        }
      }
      if (*abort_flag) {
        // let copies already in flight land before the CTA's shared memory is
        // released (a wait for copies that were never issued just runs out)
        WaitCtl drain{nullptr, nullptr, wc.limit_ns};
        if (na > 0) mbar_wait(bar.a_full(), (na - 1) & 1, drain);
        for (int s = max(0, g - NS1); s < g; ++s) mbar_wait(bar.b1_full(s % NS1), (s / NS1) & 1, drain);
        for (int s = max(0, g - NS2); s < g; ++s) mbar_wait(bar.b2_full(s % NS2), (s / NS2) & 1, drain);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    // The whole warp runs it, converged (see mma_ss_w).
    constexpr uint32_t idesc_s = idesc_bf16_f32(BR, BC, 0, 0);
    constexpr uint32_t idesc_a2 = idesc_bf16_f32(BR, DQK, 0, 1);
    constexpr uint32_t idesc_a1 = idesc_bf16_f32(BR, DV, 0, 1);
    const Desc2 a1 = desc_sw128(sb + OFF_A1, 16, 1024), a2 = desc_sw128(sb + OFF_A2, 16, 1024);
    const Desc2 b1k = desc_sw128(sb + OFF_B1, 16, 1024), b1m = desc_sw128(sb + OFF_B1, B_CHUNK, 1024);
    const Desc2 b2k = desc_sw128(sb + OFF_B2, 16, 1024), b2m = desc_sw128(sb + OFF_B2, B_CHUNK, 1024);
    auto issue_s = [&](int g) {
      const uint32_t st = ((g % NS1) * B1_BYTES) >> 4;
#pragma unroll
      for (int k = 0; k < DQK / 16; ++k)
        mma_ss_w(tmem + TM_S + 64 * (g & 1), a1, ((k >> 2) * A_CHUNK + (k & 3) * 32) >> 4, b1k,
                 st + (((k >> 2) * B_CHUNK + (k & 3) * 32) >> 4), idesc_s, k > 0);
      mma_commit_w(bar.s_full(g & 1));
    };
    auto issue_dp = [&](int g, bool last) {
      const uint32_t st = ((g % NS2) * B2_BYTES) >> 4;
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss_w(tmem + TM_DP, a2, ((k >> 2) * A_CHUNK + (k & 3) * 32) >> 4, b2k,
                 st + (((k >> 2) * B_CHUNK + (k & 3) * 32) >> 4), idesc_s, k > 0);
      mma_commit_w(bar.dp_full());
      if (!KEYS) mma_commit_w(bar.b2_free(g % NS2));
      if (last) mma_commit_w(bar.a_free());  // no later product of the item reads its rows
    };
    auto issue_acc = [&](int g, bool first) {
      const uint32_t t = tmem + TM_S + 64 * (g & 1);
      const uint32_t st1 = ((g % NS1) * B1_BYTES) >> 4, st2 = ((g % NS2) * B2_BYTES) >> 4;
      // K step k: columns 16k..16k+15 of P and dS, which the warpgroup of
      // half k / 2 left at 32 (k / 2) (P) and 16 further (dS)
      if (KEYS) {
#pragma unroll
        for (int k = 0; k < BC / 16; ++k)
          mma_ts_w(tmem + TM_ACC1, t + 32 * (k >> 1) + 8 * (k & 1), b2m, st2 + ((k * 16 * 128) >> 4), idesc_a1,
                   !first || k > 0);
        mma_commit_w(bar.b2_free(g % NS2));
      }
#pragma unroll
      for (int k = 0; k < BC / 16; ++k)
        mma_ts_w(tmem + TM_ACC2, t + 32 * (k >> 1) + 16 + 8 * (k & 1), b1m, st1 + ((k * 16 * 128) >> 4), idesc_a2,
                 !first || k > 0);
      mma_commit_w(bar.b1_free(g % NS1));
    };
    BwdItem w;
    int g = 0, na = 0;
    bool ok = true;
    for (int n = 0; ok && bwd_item<KEYS>(p, n, w); ++n) {
      if (w.steps == 0) continue;
      ok = warp_wait2(bar.a_full(), na & 1, bar.b1_full(g % NS1), (g / NS1) & 1, wc);
      if (!ok) break;
      tc_fence_after();
      issue_s(g);
      ok = warp_wait(bar.b2_full(g % NS2), (g / NS2) & 1, wc);
      if (!ok) break;
      tc_fence_after();
      issue_dp(g, w.steps == 1);
      for (int it = 0; it < w.steps; ++it, ++g) {
        const bool more = it + 1 < w.steps;
        if (more) {
          ok = warp_wait(bar.b1_full((g + 1) % NS1), ((g + 1) / NS1) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          issue_s(g + 1);
        }
        ok = more ? warp_wait2(bar.e_full(), g & 1, bar.b2_full((g + 1) % NS2), ((g + 1) / NS2) & 1, wc)
                  : warp_wait(bar.e_full(), g & 1, wc);
        // the last item's accumulators have been read out
        if (ok && it == 0 && na > 0) ok = warp_wait(bar.acc_free(), (na - 1) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        if (more) issue_dp(g + 1, it + 2 == w.steps);
        issue_acc(g, it == 0);
      }
      if (!ok) break;
      mma_commit_w(bar.acc_full());
      ++na;
    }
    // every MMA this warp issued must finish before tensor memory is freed
    mma_commit_w(bar.drain());
    WaitCtl drain{nullptr, nullptr, wc.limit_ns};
    mbar_wait(bar.drain(), 0, drain);
    __syncwarp();
  } else if (warp < 8) {
    // ---------------------------------------------------------- element-wise
    const int half = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sl = p.scale * 1.4426950408889634f;
    const size_t npad = static_cast<size_t>((p.Nq + 127) / 128) * 128;
    BwdItem w;
    int g = 0, na = 0;
    bool ok = true;
    for (int n = 0; ok && bwd_item<KEYS>(p, n, w); ++n) {
      const int r0 = w.r0, r = r0 + row;
      float row_l2 = 0.f, row_d = 0.f;
      if (!KEYS) {
        row_l2 = p.lse2[w.bh * npad + r];  // padded to whole tiles
        row_d = p.dsum[w.bh * npad + r];
      }
      for (int it = 0; it < w.steps; ++it, ++g) {
        const uint32_t tS = tl + TM_S + 64 * (g & 1) + 32 * half, tD = tl + TM_DP + 32 * half;
        // (the stages' own barriers too: this thread reads the row terms that they count)
        if (!warp_wait(bar.s_full(g & 1), (g >> 1) & 1, wc) ||
            (KEYS && !warp_wait(bar.b1_full(g % NS1), (g / NS1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[32];
        tmem_ld_32x32b_x32(tS, sr);
        tmem_wait_ld();
        const int c0 = (w.c_lo + it) * BC + 32 * half;  // first column of this half
        float pr[32];
        const float4* vl = reinterpret_cast<const float4*>(smem + OFF_LSE + (g % NS1) * VEC + half * 128);
        const float4* vd = reinterpret_cast<const float4*>(smem + OFF_D + (g % NS2) * VEC + half * 128);
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          float4 l2 = make_float4(row_l2, row_l2, row_l2, row_l2);
          if (KEYS) l2 = vl[c4];
          const float lv[4] = {l2.x, l2.y, l2.z, l2.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[4 * c4 + e] = ex2_approx(fmaf(__uint_as_float(sr[4 * c4 + e]), sl, lv[e]));
        }
        if (KEYS) {
          // query c0 + c sees key r iff r <= c0 + c + off; the lowest query and
          // highest key of the tile decide whether any pair is masked
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
          for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(pr[2 * c], pr[2 * c + 1]);  // one rounding, for P^T dO
          tmem_st_32x32b_x16(tS, pk);
        }
        if (!warp_wait(bar.dp_full(), g & 1, wc) ||
            (KEYS && !warp_wait(bar.b2_full(g % NS2), (g / NS2) & 1, wc))) {
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
          if (KEYS) dv = vd[c4];
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
      if (!ok) break;
      // ------------------------------------------------------------ output
      // (the next item's loads and first products go on meanwhile)
      if (w.steps > 0 && !warp_wait(bar.acc_full(), na & 1, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool out = __all_sync(0xffffffffu, *abort_flag == 0);
      // 32 columns of an accumulator; zeros where nothing was streamed
      auto load32 = [&](uint32_t col, float mul, float* x) {
        uint32_t o[32];
        if (w.steps > 0) {
          tmem_ld_32x32b_x32(tl + col, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = w.steps > 0 ? __uint_as_float(o[e]) * mul : 0.f;
      };
      // row i of this warp in an array of `width` entries a row, from column col on
      const int rw = r0 + (warp & 3) * 32;
      const long long grow = static_cast<long long>(w.bh) * n_rows + rw;
      auto at = [&](void* base, int size, int width, int col) {
        return [=](int i) -> void* {
          return out && rw + i < n_rows ? static_cast<uint8_t*>(base) + ((grow + i) * width + col) * size : nullptr;
        };
      };
#pragma unroll 1
      for (int c = 3 * half; c < 3 * half + 3; ++c) {  // acc2: six groups of 32 columns, three a warpgroup
        float x[32];
        load32(TM_ACC2 + 32 * c, p.scale, x);
        if (!KEYS)
          store_rows_bf16(x, at(p.dq, 2, DQK, 32 * c));
        else if (c < 4)
          store_rows_bf16(x, at(p.dkn, 2, DN, 32 * c));
        else
          store_rows_f32(x, at(p.dkr_part, 4, DR, 32 * (c - 4)));
      }
      if (KEYS) {
#pragma unroll 1
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          float x[32];
          load32(TM_ACC1 + 32 * c, 1.f, x);
          store_rows_bf16(x, at(p.dv_out, 2, DV, 32 * c));
        }
      }
      tc_fence_before();
      if (w.steps > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.acc_free());
        ++na;
      }
    }
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
  const long long items = static_cast<long long>(p.B) * p.H * (((KEYS ? p.Nk : p.Nq) + BR - 1) / BR);
  const int sms = sm_count();
  if (sms <= 0 || items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  return launch_after(fa_latent_bwd_sm103_kernel<KEYS>, grid, kThreads, SMEM_BYTES, s, m, p);
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
