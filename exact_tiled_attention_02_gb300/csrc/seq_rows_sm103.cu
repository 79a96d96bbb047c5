// seq_rows_sm103.cu -- attention of many query rows over long keys, bf16 in /
// fp32 accumulate, on the tensor cores of GB300 (sm_103a): the expanded
// latent forward (keys of two parts, 128 + 64 wide, the second shared by the
// heads; values 128 wide; causal) and the prefix part of shared-prefix
// attention (every sequence's rows against one prefix).
//
//   S_ij = scale q_i . k_j over the keys j < limit(i),  O_i = sum_j softmax_j v_j
//
// one 128-key tile at a time with the running maximum and sum of "Flash
// attention and efficient attention -- Hinglish notes", "Derivation:
// Incremental Softmax", Steps 1-3.
//
// Work item = two 128-row query tiles of one group against a range of its
// key tiles.  Persistent, one CTA per SM; every barrier's phase counts on
// across items, so an item's loads overlap the previous item's last products
// and output.  384 threads:
//   warps 0-3, 4-7  softmax of query tile 0 / 1: thread = row = TMEM lane
//   warp 8          TMEM owner, issues every tcgen05.mma
//   warp 9          TMA producer
// Tensor memory: S_t (P_t as packed bf16 over its first half) at 128 t, O_t
// at 256 + 128 t.  The two tiles take turns: while one's softmax runs, the
// tensor core works on the other.
// Shared memory: both query tiles, then a ring of 16 KB chunks (128 keys x 64
// dimensions, 128-byte swizzle).  K_j takes CK consecutive chunks, V_j the
// next CV, then K_{j+1}; a chunk is reloaded once the products that read it
// have completed.  At 192 + 128 wide two whole (K, V) tiles would not fit
// beside 96 KB of queries (8 chunks remain, a tile takes 5): sharing one ring
// lets V_{j+1} load as soon as K_j is free and K_{j+2} as soon as V_j is.
//
// Bound by the tensor core and, beside it, the exponentials: per 128 x 128
// scores 64 (DQK + DV) / 16 cycles of products against 16,384 exponentials.
// 16 heads of 8192 tokens, 192 + 128 wide, causal: 241 us, 1430 TFLOP/s, call
// after call at the power limit (225 us in short runs before it bites).  The
// prefix part: 8 groups of 2048 rows over 32768 keys, d = 128, on every SM: 197
// us with its merge, 1395 TFLOP/s.
#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BR = 128;  // rows per query tile
constexpr int BC = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int CHUNK = BC * 128;  // bytes: 128 rows x 64 bf16
// register shares: 384 threads x 168 at launch; the two softmax warpgroups take
// 208, the warpgroup of warps 8-11 88
constexpr int kRegsSoftmax = 208;
constexpr int kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * 168, "register shares must add up to the launch allocation");
constexpr uint32_t tm_s(int t) { return 128u * static_cast<uint32_t>(t); }
constexpr uint32_t tm_o(int t) { return 256u + 128u * static_cast<uint32_t>(t); }
// A row's reference maximum rises only when a score exceeds it by 2^8 in
// linear terms; O / l uses one reference for numerator and denominator.
constexpr float kRescaleThreshold = 8.0f;

template <int DQK, int DV>
struct Cfg {
  static constexpr int CK = (DQK + 63) / 64, CV = (DV + 63) / 64, CT = CK + CV;
  static constexpr int DVP = CV * 64;
  static constexpr int Q_BYTES = CK * CHUNK;
  static constexpr int NCH = CT == 2 ? 8 : (CT == 4 ? 10 : 8);  // ring chunks
  static constexpr int NST = CT == 2 ? 4 : 2;                   // K (V) tiles with a barrier of their own
  static constexpr int OFF_RING = 2 * Q_BYTES;
  static constexpr int OFF_BAR = OFF_RING + NCH * CHUNK;
  static constexpr int NBAR = 4 + 4 * NST + 6 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_USED = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = SMEM_USED + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(NCH >= CT + CK, "K_{j+1} fits beside tile j");
  static_assert(CV <= 2 && (CV == 1 || CHUNK * NCH < (1 << 18)), "V is at most two chunks");
};

template <int NST>
struct Bars {
  uint32_t base;
  __device__ uint32_t q_full(int t) const { return base + 8 * t; }
  __device__ uint32_t q_empty(int t) const { return base + 8 * (2 + t); }
  __device__ uint32_t k_full(int s) const { return base + 8 * (4 + s); }
  __device__ uint32_t v_full(int s) const { return base + 8 * (4 + NST + s); }
  __device__ uint32_t k_empty(int s) const { return base + 8 * (4 + 2 * NST + s); }
  __device__ uint32_t v_empty(int s) const { return base + 8 * (4 + 3 * NST + s); }
  __device__ uint32_t s_full(int t) const { return base + 8 * (4 + 4 * NST + t); }
  __device__ uint32_t p_full(int t) const { return base + 8 * (6 + 4 * NST + t); }
  __device__ uint32_t o_done(int t) const { return base + 8 * (8 + 4 * NST + t); }
  __device__ uint32_t drain() const { return base + 8 * (10 + 4 * NST); }
};

struct RowsMaps {
  CUtensorMap q, k, k2, v;
};

// What the kernel needs beside SeqAttn: how rows fall into tiles.
struct RowsPlan {
  int block_rows;  // rows of a row block (SeqAttn::row_block, or all rows)
  int blocks;      // row blocks of a group
  int per_tile;    // whole blocks in a tile (1 where a block takes several tiles)
  int per_block;   // tiles of a block (1 where a tile takes several blocks)
  int tiles;       // query tiles of a group
  int pairs;
  int n_items;
  int heavy_first;  // causal: later (longer) pairs of every group come first
};

// The n-th item of CTA c of G: rounds of G items, every other one backwards,
// so that where items get shorter along their order (causal) the CTAs' sums
// stay close (512 items of 2 to 64 key tiles on 152 CTAs: longest sum 120
// tiles, mean 111; 144 with all rounds forwards).
__device__ __forceinline__ int nth_item(int n) {
  const int G = gridDim.x, c = blockIdx.x;
  return n * G + ((n & 1) ? G - 1 - c : c);
}

struct Tile {
  int block0, r_off, rows;  // first row block, row within it, valid rows
};

struct Item {
  int g, split, j_lo, ntiles;
  Tile tile[2];
  int hi[2];  // key tiles of each query tile
};

__device__ __forceinline__ int row_limit(const SeqAttn& p, int r) {  // keys that row r of a block sees
  return p.causal ? p.n_keys - (p.n_new - 1 - r % p.n_new) : p.n_keys;
}

__device__ __forceinline__ Item decode_item(const SeqAttn& p, const RowsPlan& w, int item) {
  Item it;
  int pair;
  if (w.heavy_first) {
    it.g = item % p.groups;
    pair = w.pairs - 1 - item / p.groups;
    it.split = 0;
  } else {
    pair = item % w.pairs;
    const int rest = item / w.pairs;
    it.split = rest % p.splits;
    it.g = rest / p.splits;
  }
  const int all = (p.n_keys + BC - 1) / BC;
  it.j_lo = static_cast<int>(static_cast<long long>(all) * it.split / p.splits);
  const int j_end = static_cast<int>(static_cast<long long>(all) * (it.split + 1) / p.splits);
  for (int t = 0; t < 2; ++t) {
    const int n = 2 * pair + t;
    Tile& x = it.tile[t];
    x.block0 = 0;
    x.r_off = 0;
    x.rows = 0;
    it.hi[t] = 0;
    if (n >= w.tiles) continue;
    if (w.per_block > 1) {
      x.block0 = n / w.per_block;
      x.r_off = (n % w.per_block) * BR;
      x.rows = min(BR, w.block_rows - x.r_off);
    } else {
      x.block0 = n * w.per_tile;
      x.rows = min(w.per_tile, w.blocks - x.block0) * w.block_rows;
    }
    // limits rise along the rows of a causal tile (it lies in one block of new tokens)
    const int seen = max(0, row_limit(p, x.r_off + x.rows - 1));
    it.hi[t] = max(0, min(j_end, (seen + BC - 1) / BC) - it.j_lo);
  }
  it.ntiles = max(it.hi[0], it.hi[1]);
  return it;
}

template <int DQK, int DV, int D2, bool PART>
__global__ void __launch_bounds__(kThreads, 1)
    fa_seq_rows_sm103_kernel(const __grid_constant__ RowsMaps maps, const __grid_constant__ SeqAttn p,
                             const __grid_constant__ RowsPlan plan) {
  using C = Cfg<DQK, DV>;
  constexpr int CK = C::CK, CV = C::CV, CT = C::CT, NCH = C::NCH, NST = C::NST;
  constexpr int CK1 = CK - D2 / 64;  // chunks of the first key part
  extern __shared__ uint8_t smem_raw[];
  pdl_launch();  // what reads these results waits for this kernel's end
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  if (pad + C::SMEM_USED > static_cast<uint32_t>(C::SMEM_BYTES)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusLayout);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sQ = sb, sR = sb + C::OFF_RING;
  const Bars<NST> bar{sb + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const WaitCtl wc{p.status, abort_flag, p.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar.q_full(t), 1);
      mbar_init(bar.q_empty(t), 1);
      mbar_init(bar.s_full(t), 1);
      mbar_init(bar.p_full(t), 4);
      mbar_init(bar.o_done(t), 1);
    }
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar.k_full(s), 1);
      mbar_init(bar.v_full(s), 1);
      mbar_init(bar.k_empty(s), 1);
      mbar_init(bar.v_empty(s), 1);
    }
    mbar_init(bar.drain(), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int n_items = plan.n_items;

  // ring slot of chunk c of V_j's pair: where the pair wraps round the ring
  // the two swap, so that the second is always at the higher address
  auto v_slot = [&](int j, int c) {
    const int s0 = (j * CT + CK) % NCH;
    if (CV == 1) return s0;
    return s0 + 1 < NCH ? s0 + c : (c == 0 ? 0 : NCH - 1);
  };

  auto role_tma = [&]() {
    // ------------------------------------------------------------------ TMA
    if (lane == 0) {
      prefetch_tensormap(&maps.q);
      prefetch_tensormap(&maps.k);
      if (D2 > 0) prefetch_tensormap(&maps.k2);
      prefetch_tensormap(&maps.v);
      const uint32_t q_box = static_cast<uint32_t>(min(BR, plan.block_rows) * plan.per_tile) * 128u;
      bool ok = true;
      int j = 0;                      // key tiles issued (all items)
      int nq = 0;                     // items whose queries were issued
      int k_freed = 0, v_freed = 0;   // tiles known to be released
      auto free_k = [&](int upto) {   // waits until K tiles .. upto are released
        for (; ok && k_freed <= upto; ++k_freed)
          ok = mbar_wait_backoff(bar.k_empty(k_freed % NST), (k_freed / NST) & 1, wc);
      };
      auto free_v = [&](int upto) {
        for (; ok && v_freed <= upto; ++v_freed)
          ok = mbar_wait_backoff(bar.v_empty(v_freed % NST), (v_freed / NST) & 1, wc);
      };
      auto free_chunk = [&](int x) {  // the ring chunk that chunk x of the stream overwrites (and all before it)
        x -= NCH;
        if (x < 0) return;
        if (x % CT >= CK)
          free_v(x / CT);
        else
          free_k(x / CT);
      };
      for (int item; ok && (item = nth_item(nq)) < n_items; ++nq) {
        const Item w = decode_item(p, plan, item);
        for (int t = 0; ok && t < 2; ++t) {
          if (nq > 0 && !mbar_wait_backoff(bar.q_empty(t), (nq - 1) & 1, wc)) {
            ok = false;
            break;
          }
          if (w.tile[t].rows == 0) {
            mbar_arrive(bar.q_full(t));
            continue;
          }
          mbar_arrive_expect_tx(bar.q_full(t), CK * q_box);
#pragma unroll
          for (int c = 0; c < CK; ++c)
            tma_load_4d(sQ + t * C::Q_BYTES + c * CHUNK, &maps.q, bar.q_full(t), c * 64, w.tile[t].r_off, w.g,
                        w.tile[t].block0);
        }
        for (int it = 0; ok && it < w.ntiles; ++it, ++j) {
          const int kv0 = (w.j_lo + it) * BC, s = j % NST;
          free_k(j - NST);
          free_chunk(j * CT + CK - 1);
          if (!ok) break;
          mbar_arrive_expect_tx(bar.k_full(s), CK * CHUNK);
#pragma unroll
          for (int c = 0; c < CK; ++c) {
            const uint32_t dst = sR + ((j * CT + c) % NCH) * CHUNK;
            if (c < CK1)
              tma_load_3d(dst, &maps.k, bar.k_full(s), c * 64, kv0, w.g);
            else
              tma_load_3d(dst, &maps.k2, bar.k_full(s), (c - CK1) * 64, kv0, w.g / p.k2_div);
          }
          free_v(j - NST);
          free_chunk(j * CT + CT - 1);
          if (!ok) {  // K_j is in flight: its copies land below
            ++j;
            break;
          }
          mbar_arrive_expect_tx(bar.v_full(s), CV * CHUNK);
#pragma unroll
          for (int c = 0; c < CV; ++c) tma_load_3d(sR + v_slot(j, c) * CHUNK, &maps.v, bar.v_full(s), c * 64, kv0, w.g);
        }
      }
      if (*abort_flag) {
        // let copies already in flight land before the CTA's shared memory is
        // released; each wait is bounded, and one for a copy that was never
        // issued just runs out
        WaitCtl drain{nullptr, nullptr, wc.limit_ns};
        if (nq > 0) {
          mbar_wait(bar.q_full(0), (nq - 1) & 1, drain);
          mbar_wait(bar.q_full(1), (nq - 1) & 1, drain);
        }
        for (int s = max(0, j - NST); s < j; ++s) {
          mbar_wait(bar.k_full(s % NST), (s / NST) & 1, drain);
          mbar_wait(bar.v_full(s % NST), (s / NST) & 1, drain);
        }
      }
    }
    __syncwarp();
  };
  auto role_mma = [&]() {
    // ------------------------------------------------------------------ MMA
    // The whole warp runs it, converged (see mma_ss_w).
    {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BR, BC, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BR, C::DVP, 0, 1);
      int j0 = 0, nq = 0;
      int cnt[2] = {0, 0};  // key tiles each query tile has passed (all items)
      auto issue_s = [&](const Item& w, int t, int it) {  // S_t = Q_t K_it^T
        const Desc2 dq = desc_sw128(sQ + t * C::Q_BYTES, 16, 1024);
        const int j = j0 + it;
#pragma unroll
        for (int c = 0; c < CK; ++c) {
          const Desc2 dk = desc_sw128(sR + ((j * CT + c) % NCH) * CHUNK, 16, 1024);
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            if (c * 64 + k4 * 16 >= DQK) break;
            mma_ss_w(tmem + tm_s(t), dq, (c * CHUNK + k4 * 32) >> 4, dk, (k4 * 32) >> 4, idesc_qk, c + k4 > 0);
          }
        }
        mma_commit_w(bar.s_full(t));
        if (it >= w.hi[t ^ 1] || t == 1) mma_commit_w(bar.k_empty(j % NST));  // the last reader of K_j
        if (it == w.hi[t] - 1) mma_commit_w(bar.q_empty(t));                  // the last product that reads Q_t
      };
      auto issue_pv = [&](const Item& w, int t, int it) {  // O_t (+)= P_t V_it
        const int j = j0 + it;
        const uint32_t lbo = CV == 1 ? CHUNK : (v_slot(j, 1) - v_slot(j, 0)) * CHUNK;
        const Desc2 dv = desc_sw128(sR + v_slot(j, 0) * CHUNK, lbo, 1024);
#pragma unroll
        for (int kk = 0; kk < BC / 16; ++kk)
          mma_ts_w(tmem + tm_o(t), tmem + tm_s(t) + kk * 8, dv, (kk * 16 * 128) >> 4, idesc_pv, it > 0 || kk > 0);
        mma_commit_w(bar.o_done(t));
        if (it >= w.hi[t ^ 1] || t == 1) mma_commit_w(bar.v_empty(j % NST));  // the last reader of V_j
      };
      bool ok = true;
      for (int item; ok && (item = nth_item(nq)) < n_items; ++nq) {
        const Item w = decode_item(p, plan, item);
        ok = warp_wait2(bar.q_full(0), nq & 1, bar.q_full(1), nq & 1, wc);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
          if (w.hi[t] == 0) mma_commit_w(bar.q_empty(t));  // no product of this item reads Q_t
        if (w.ntiles > 0) {
          ok = warp_wait(bar.k_full(j0 % NST), (j0 / NST) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          for (int t = 0; t < 2; ++t)
            if (w.hi[t] > 0) issue_s(w, t, 0);
        }
        for (int it = 0; ok && it < w.ntiles; ++it) {
          const int j = j0 + it;
          bool v_in = false, k_in = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || it >= w.hi[t]) continue;
            const uint32_t pp = (cnt[t] + it) & 1;
            ok = v_in ? warp_wait(bar.p_full(t), pp, wc)
                      : warp_wait2(bar.v_full(j % NST), (j / NST) & 1, bar.p_full(t), pp, wc);
            if (!ok) break;
            v_in = true;
            tc_fence_after();
            issue_pv(w, t, it);
            if (it + 1 < w.hi[t]) {
              if (!k_in && !warp_wait(bar.k_full((j + 1) % NST), ((j + 1) / NST) & 1, wc)) {
                ok = false;
                break;
              }
              k_in = true;
              tc_fence_after();
              issue_s(w, t, it + 1);
            }
          }
        }
        cnt[0] += w.hi[0];
        cnt[1] += w.hi[1];
        j0 += w.ntiles;
      }
      // every MMA this thread issued must finish before tensor memory is freed
      mma_commit_w(bar.drain());
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      mbar_wait(bar.drain(), 0, drain);
    }
    __syncwarp();
  };
  auto role_softmax = [&]() {
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = tl + tm_s(t), tO = tl + tm_o(t);
    const float sl = p.scale * 1.4426950408889634f;
    bool ok = true;
    int n = 0;  // key tiles this warpgroup has processed (all items)
    int ni = 0;  // items passed
    for (int item; ok && (item = nth_item(ni)) < n_items; ++ni) {
      const Item w = decode_item(p, plan, item);
      const Tile x = w.tile[t];
      const int rb = x.r_off + row % plan.block_rows;  // row within its block
      const int limit = row < x.rows ? row_limit(p, plan.per_block > 1 ? x.r_off + row : rb) : p.n_keys;
      const int low = row_limit(p, x.r_off);  // the lowest limit of the tile
      // l: row sum of the unrounded P (lse uses it); lc: the bf16 rounding
      // error of each tile's largest P, which O's normaliser adds (below)
      float m_ref = -INFINITY, l = 0.f, lc = 0.f;
      for (int it = 0; it < w.hi[t]; ++it, ++n) {
        if (!warp_wait(bar.s_full(t), n & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[BC];
#pragma unroll
        for (int c = 0; c < BC / 32; ++c) tmem_ld_32x32b_x32(tS + c * 32, &sr[c * 32]);
        tmem_wait_ld();
        float s[BC];
#pragma unroll
        for (int c = 0; c < BC; ++c) s[c] = __uint_as_float(sr[c]);
        const int kv0 = (w.j_lo + it) * BC;
        if (kv0 + BC > low) {
          const int hi = limit - kv0;
#pragma unroll
          for (int c = 0; c < BC; ++c) s[c] = c < hi ? s[c] : -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) mx[a] = fmaxf(s[a], s[a + 4]);
#pragma unroll
        for (int c = 8; c < BC; c += 8)
#pragma unroll
          for (int a = 0; a < 4; ++a) mx[a] = fmax3(mx[a], s[c + a], s[c + 4 + a]);
        const float smax = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
        const float mt = smax * sl;
        float alpha = 1.f;
        if (mt > m_ref + kRescaleThreshold) {
          alpha = ex2_approx(m_ref - mt);  // 0 when m_ref = -inf
          m_ref = mt;
        }
        const float nref = (m_ref == -INFINITY) ? 0.f : -m_ref;
        // P V multiplies bf16-rounded P while the row sum adds the unrounded
        // values; where one key dominates a row, that key's rounding is the
        // whole mismatch, and adding it to O's normaliser cancels it
        const float pmax = ex2_approx(fmaf(smax, sl, nref));
        lc = lc * alpha + (bf16_round(pmax) - pmax);
        const float2 sl2 = make_float2(sl, sl), nref2 = make_float2(nref, nref);
        float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int gq = 0; gq < BC / 32; ++gq) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int e = 32 * gq + 2 * c;
            const float2 y = __ffma2_rn(make_float2(s[e], s[e + 1]), sl2, nref2);
            const float2 pv = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            rs[c & 3] = __fadd2_rn(rs[c & 3], pv);
            pk[c] = pack_bf16x2(pv.x, pv.y);
          }
          tmem_st_32x32b_x16(tS + 16 * gq, pk);
        }
        const float rsum = (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y) + (rs[2].x + rs[2].y) + (rs[3].x + rs[3].y);
        // O may be rescaled only once this item's previous P V into it has
        // completed: the only one that can be outstanding (S_it was issued
        // after P_{it-1} V_{it-1}, and P_it is not yet published)
        if (it > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!warp_wait(bar.o_done(t), (n - 1) & 1, wc)) {
            tmem_wait_st();
            ok = false;
            break;
          }
          tc_fence_after();
          const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
          for (int c = 0; c < C::DVP / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2);
              o[e] = __float_as_uint(v.x);
              o[e + 1] = __float_as_uint(v.y);
            }
            tmem_st_32x32b_x32(tO + c * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.p_full(t));
        l = l * alpha + rsum;
      }
      if (!ok) break;
      // ------------------------------------------------------------ output
      if (w.hi[t] > 0 && !warp_wait(bar.o_done(t), (n - 1) & 1, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool out = __all_sync(0xffffffffu, *abort_flag == 0);
      const bool mine = out && row < x.rows;
      const long long group_row = (w.g / p.group_div) * p.q_s1 + (w.g % p.group_div) * p.q_s2;
      auto out_row = [&](int i) -> long long {  // of row i of the tile
        return plan.per_block > 1 ? group_row + x.block0 * p.q_s3 + x.r_off + i
                                  : group_row + (x.block0 + i / plan.block_rows) * p.q_s3 + i % plan.block_rows;
      };
      const long long orow = out_row(row), prow = (p.part0 + w.split) * p.total + orow;
      const float norm = l + lc;
      const float inv_l = l == 0.f ? 0.f : 1.f / norm;
      // the rows that this lane stores for its group of four (store_rows64)
      uint8_t* dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = (row & ~3) + i;
        const long long at = PART ? (p.part0 + w.split) * p.total + out_row(rr) : out_row(rr);
        dst[i] = !out || rr >= x.rows ? nullptr
                                      : (PART ? reinterpret_cast<uint8_t*>(p.part_o) : static_cast<uint8_t*>(p.o)) +
                                            at * DV * (PART ? 4 : 2);
      }
#pragma unroll 1
      for (int c = 0; c < DV / 32; ++c) {
        uint32_t o[32];
        if (w.hi[t] > 0) {
          tmem_ld_32x32b_x32(tO + c * 32, o);
          tmem_wait_ld();
        }
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * inv_l;  // no key seen: 0
        auto at = [&](int i) -> void* {
          uint8_t* q = dst[i & 3];
          return q == nullptr ? nullptr : q + c * 32 * (PART ? 4 : 2);
        };
        if constexpr (PART)
          store_rows_f32(v, at);
        else
          store_rows_bf16(v, at);
      }
      if (mine) {
        const float mref = (m_ref == -INFINITY) ? 0.f : m_ref;
        const float lse = (mref + __log2f(l)) * 0.69314718055994531f;
        if constexpr (PART)
          p.part_lse[prow] = lse;
        else if (p.lse != nullptr)
          p.lse[orow] = lse;
      }
      tc_fence_before();
    }
  };
  if (warp >= 8) {
    regs_decrease<kRegsOther>();
    if (warp == 9)
      role_tma();
    else if (warp == 8)
      role_mma();
  } else {
    regs_increase<kRegsSoftmax>();
    role_softmax();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

RowsPlan rows_plan(int rows, int row_block, bool causal) {
  RowsPlan w{};
  w.block_rows = row_block == kAllRows ? rows : row_block;
  w.blocks = rows / w.block_rows;
  w.per_tile = w.block_rows <= BR ? BR / w.block_rows : 1;
  if (causal) w.per_tile = 1;  // a causal tile lies in one block
  if (w.per_tile > w.blocks) w.per_tile = w.blocks;
  w.per_block = (w.block_rows + BR - 1) / BR;
  w.tiles = w.per_block > 1 ? w.blocks * w.per_block : (w.blocks + w.per_tile - 1) / w.per_tile;
  w.pairs = (w.tiles + 1) / 2;
  return w;
}

template <int DQK, int DV, int D2, bool PART>
cudaError_t launch_rows(const SeqAttn& p, cudaStream_t s) {
  using C = Cfg<DQK, DV>;
  static SmemOnce once;
  cudaError_t e = once(fa_seq_rows_sm103_kernel<DQK, DV, D2, PART>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  RowsPlan w = rows_plan(p.rows, p.row_block, p.causal != 0);
  w.heavy_first = p.causal;
  const long long items = static_cast<long long>(w.pairs) * p.groups * p.splits;
  if (items > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  w.n_items = static_cast<int>(items);
  RowsMaps m;
  // queries [blocks][groups][block rows][DQK]
  const long long qd[4] = {DQK, w.block_rows, p.groups, w.blocks};
  const int qb[4] = {64, w.block_rows < BR ? w.block_rows : BR, 1, w.per_tile};
  const int keys = p.n_keys > 0 ? p.n_keys : 1;
  if (!make_map(&m.q, p.q, 4, qd, qb) || !make_map3(&m.k, p.k1, DQK - D2, keys, p.groups, BC) ||
      !make_map3(&m.v, p.v, DV, keys, p.groups, BC))
    return cudaErrorInvalidValue;
  m.k2 = m.k;
  if (D2 > 0 && !make_map3(&m.k2, p.k2, D2, keys, p.groups / p.k2_div, BC)) return cudaErrorInvalidValue;
  int ctas = sm_count();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  if (p.ctas > 0 && p.ctas < ctas) ctas = p.ctas;
  const int grid = w.n_items < ctas ? w.n_items : ctas;
  fa_seq_rows_sm103_kernel<DQK, DV, D2, PART><<<grid, kThreads, C::SMEM_BYTES, s>>>(m, p, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_rows(const SeqAttn& p, cudaStream_t s) {
  if (p.part_o == nullptr)
    return p.d2 == 64 && p.d1 == 128 && p.dv == 128 ? launch_rows<192, 128, 64, false>(p, s) : cudaErrorInvalidValue;
  if (p.d1 == 64) return launch_rows<64, 64, 0, true>(p, s);
  if (p.d1 == 96) return launch_rows<96, 96, 0, true>(p, s);
  if (p.d1 == 128) return launch_rows<128, 128, 0, true>(p, s);
  return cudaErrorInvalidValue;
}

// How long the prefix's part takes (us) on n CTAs, its keys in `splits`
// ranges.  Measured at d = 128: 7.5 us to launch, load and write out, 1.45 us
// a 128-key tile of two query tiles; 1.5 us a further item.
double seq_rows_time(int groups, int rows, int row_block, int n_keys, int d, int n, int splits) {
  const RowsPlan w = rows_plan(rows, row_block, false);
  const long long items = static_cast<long long>(w.pairs) * groups * splits;
  const int tiles = (n_keys + BC - 1) / BC;
  const double rounds = static_cast<double>((items + n - 1) / n);
  const double tile = 0.35 + 0.0086 * d;
  return 7.5 + rounds * ((tiles + splits - 1) / splits * tile) + (rounds - 1.0) * 1.5;
}
int seq_rows_items(int groups, int rows, int row_block) { return rows_plan(rows, row_block, false).pairs * groups; }

}  // namespace fa
