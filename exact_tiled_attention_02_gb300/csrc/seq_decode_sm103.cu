// seq_decode_sm103.cu -- attention of few query rows over long caches, bf16 in
// / fp32 accumulate, on the tensor cores of GB300 (sm_103a): the absorbed
// latent form over a paged cache (one 576- or 320-wide vector a token, whose
// first 512 or 256 entries are also the value), and the sequences' own part
// of shared-prefix attention (separate keys and values).
//
//   S_ij = scale q_i . k_j over the keys j < nk - lag(i),  O_i = sum_j softmax_j v_j
//
// Every token's vector is read once for up to NR = 64 query rows, so the
// bound is the cache's bytes until the rows fill the tensor core.  The
// products are taken transposed, keys and value dimensions as the long (M)
// side and query rows as the short (N) side, which may be as small as 16:
//   S^T [64 keys x NR]          = K Q^T    (A = the tile as loaded, K-major)
//   O^T [128 dims x NR] per 128 value dimensions += V^T P^T
//                                           (A = the same tile, MN-major)
// so one copy of a tile in shared memory serves both products, and O takes
// NR columns of tensor memory per 128 dimensions (4 x 64 at 512).
//
// A sequence's softmax statistics run down the columns here, across lanes.
// Per tile a thread (one key) only checks whether any of its scores exceeds
// its column's reference by 2^8; if none of the 64 keys' does (one barrier
// with an OR) the tile is exponentiated as it is.  Otherwise the column
// maxima are reduced across lanes and warps and O is rescaled.  Row sums stay
// per thread until a piece ends.
//
// Work: the tiles of all sequences, laid end to end, are cut into equal
// ranges, one a CTA (per group of rows: heads beyond 64, key/value heads), so
// ragged batches and single long sequences both fill the GPU, and the cut
// depends on the lengths alone.  A CTA's share of one sequence is a piece; a
// sequence that is one whole piece is written out directly where the caller
// asked for that, others as fp32 partial results that a second kernel merges
// in a fixed order.
//
// 320 threads: warps 0-7 softmax (a 64-row accumulator occupies lanes 0-15 of
// each quarter of tensor memory, so key 16 w + l is in lane l < 16 of warps w
// and w + 4; warps 0-3 take the first half of the columns, 4-7 the second),
// warp 8 MMA issuer and TMEM owner, warp 9 TMA producer.
// Shared memory: Q, P, a ring of M units (64 tokens x 128 dimensions; shared
// form: key and value, otherwise values) and one of X units (shared form: the
// rotary part; otherwise keys).
//
// 64 sequences of 500 to 8200 tokens of 512 + 64, 16 heads: 60 us, 5.4 TB/s.
// 128 heads x 2 tokens, up to 16384: 411 us the call, 753 TFLOP/s; there the
// cache passes to four groups of rows, 21 bytes a cycle into every SM (25 to 27
// were the most seen), and the ring of two tiles that fits beside 64 rows of
// queries covers no more: 3170 cycles a tile for 1918 of products.
#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BC = 64;            // keys per tile
constexpr int CB = BC * 128;      // bytes of a chunk: 64 tokens x 64 entries
constexpr int kSoftmax = 256;    // threads of warps 0-7
constexpr int kThreads = 320;
constexpr float kUnset = 3e38f;   // negated reference of a row that has seen no key
constexpr float kRescaleThreshold = 8.0f;

// DM: entries of an M part; DX: of an X part; SHARED: keys are [M | X] and values M.
template <int DM, int DX, bool SHARED, int NR>
struct Cfg {
  static constexpr int UC = DM >= 128 ? 2 : (DM + 63) / 64;    // chunks of an M unit
  static constexpr int UM = SHARED ? DM / 128 : 1;             // M units of a tile
  static constexpr int XC = (DX + 63) / 64;                    // chunks of an X unit
  static constexpr int QC = SHARED ? UM * UC + XC : XC;        // chunks of a query row
  static constexpr int UDIM = UC * 64;                         // value dimensions of an M unit: the M of its product
  static constexpr int Q_BYTES = QC * NR * 128;
  static constexpr int P_BYTES = NR * 128;
  static constexpr int M_BYTES = UC * CB, X_BYTES = XC * CB;
  static constexpr int CTAS = SHARED ? 1 : 2;                  // a SM
  static constexpr int BUDGET = CTAS == 1 ? 227 * 1024 : 113 * 1024;
  static constexpr int BARS = DM == 512 && NR == 64 ? 27 : 40;
  static constexpr int MISC = 3 * NR * 4 + 4 * NR * 4 + 8 * BARS + 24;  // stats, warp scratch, barriers, start
  static constexpr int FREE = BUDGET - 1024 - Q_BYTES - P_BYTES - MISC;
  static constexpr int TILE = UM * M_BYTES + X_BYTES;
  // rings: as many whole tiles as fit (at most four), then M units into what is left
  static constexpr int NT = FREE / TILE < 4 ? FREE / TILE : 4;
  static constexpr int NX = NT + (SHARED && FREE - NT * TILE >= X_BYTES + M_BYTES && NT < 4 ? 1 : 0);
  static constexpr int LEFT = FREE - NT * UM * M_BYTES - NX * X_BYTES;
  static constexpr int EXTRA = SHARED && NT < 4 ? LEFT / M_BYTES : 0;
  static constexpr int NM = NT * UM + EXTRA;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_M = OFF_P + P_BYTES;
  static constexpr int OFF_X = OFF_M + NM * M_BYTES;
  static constexpr int OFF_STAT = OFF_X + NX * X_BYTES;  // nref, alpha (or 1/l), lag: [NR] each
  static constexpr int OFF_RED = OFF_STAT + 3 * NR * 4;  // [4][NR]
  static constexpr int OFF_BAR = OFF_RED + 4 * NR * 4;
  static constexpr int NBAR = 2 * NM + 2 * NX + 7;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_USED = OFF_MISC + 24;
  static constexpr int SMEM_BYTES = SMEM_USED + 1024;
  static constexpr int TM_S = UM * NR;
  static constexpr int TM_NEED = UM * NR + 2 * NR;
  static constexpr int TM_COLS = TM_NEED <= 32 ? 32 : TM_NEED <= 64 ? 64 : TM_NEED <= 128 ? 128 : TM_NEED <= 256 ? 256 : 512;
  static_assert(NT >= 2, "two tiles in flight");
  static_assert(SMEM_BYTES <= BUDGET, "shared memory budget");
  static_assert(NBAR <= BARS, "barriers fit in MISC");
  static_assert(!SHARED || DM % 128 == 0, "whole M units");
};

template <int NM, int NX>
struct Bars {
  uint32_t base;
  __device__ uint32_t m_full(int s) const { return base + 8 * s; }
  __device__ uint32_t m_free(int s) const { return base + 8 * (NM + s); }
  __device__ uint32_t x_full(int s) const { return base + 8 * (2 * NM + s); }
  __device__ uint32_t x_free(int s) const { return base + 8 * (2 * NM + NX + s); }
  __device__ uint32_t q_full() const { return base + 8 * (2 * NM + 2 * NX); }
  __device__ uint32_t q_free() const { return base + 8 * (2 * NM + 2 * NX + 1); }
  __device__ uint32_t s_full(int b) const { return base + 8 * (2 * NM + 2 * NX + 2 + b); }
  __device__ uint32_t p_full() const { return base + 8 * (2 * NM + 2 * NX + 4); }
  __device__ uint32_t o_done() const { return base + 8 * (2 * NM + 2 * NX + 5); }
  __device__ uint32_t drain() const { return base + 8 * (2 * NM + 2 * NX + 6); }
};

struct DecodeMaps {
  CUtensorMap q, m, x;
};

__device__ __forceinline__ int seq_len(const SeqAttn& p, int b, bool report) {
  const int n = p.lens[b];
  const int nk = min(max(n, 0), p.n_keys);
  if (report && n != nk) atomicOr(p.status, kStatusInput);
  return nk;
}
__host__ __device__ __forceinline__ int tiles_of(int nk) { return (nk + BC - 1) / BC; }

// Whole warp: the sum over sequences before `b` of their tiles, and over all.
// The launcher keeps totals below 2^31 / cuts (32-bit products below).
__device__ __forceinline__ void tile_sums(const SeqAttn& p, int n_seq, int b, unsigned& before, unsigned& total) {
  const int lane = threadIdx.x & 31;
  unsigned x = 0, y = 0;
  for (int i = lane; i < n_seq; i += 32) {
    const unsigned t = tiles_of(seq_len(p, i, false));
    y += t;
    if (i < b) x += t;
  }
  before = __reduce_add_sync(0xffffffffu, x);
  total = __reduce_add_sync(0xffffffffu, y);
}
// ranges of `total` tiles that `cuts` CTAs take: none of them empty
__device__ __forceinline__ unsigned range_count(unsigned total, unsigned cuts) { return total < cuts ? total : cuts; }
// first tile of range c of n
__device__ __forceinline__ unsigned range_start(unsigned total, unsigned c, unsigned n) { return total * c / n; }
// the range that holds tile x
__device__ __forceinline__ int owner(unsigned total, unsigned x, unsigned n) {
  return static_cast<int>(((x + 1) * n - 1) / total);
}

// Columns v[0..N) of the 16 lanes of a half-warp reduced over them: lane l
// ends with max(1, N / 16) columns in v[0 ..), from column reduce_col<N>() on.
template <int H, int BIT, int N, typename Op>
__device__ __forceinline__ void reduce_step(float (&v)[N], Op op) {
  if constexpr (BIT >= 1) {
    const bool up = (threadIdx.x & BIT) != 0;
    if constexpr (H >= 1) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, BIT));
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], BIT));
    }
    reduce_step<H / 2, BIT / 2>(v, op);
  }
}
template <int N, typename Op>
__device__ __forceinline__ void reduce16(float (&v)[N], Op op) {
  reduce_step<N / 2, 8>(v, op);
}
template <int N>
__device__ __forceinline__ int reduce_col() {
  int col = 0;
#pragma unroll
  for (int h = N / 2, bit = 8; h >= 1; h /= 2, bit /= 2)
    if (threadIdx.x & bit) col += h;
  return col;
}

__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, %2, %3, p;\n"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

template <int DM, int DX, bool SHARED, int NR>
__global__ void __launch_bounds__(kThreads, Cfg<DM, DX, SHARED, NR>::CTAS)
    fa_seq_decode_sm103_kernel(const __grid_constant__ DecodeMaps maps, const __grid_constant__ SeqAttn p,
                               const DecodePlan plan) {
  using C = Cfg<DM, DX, SHARED, NR>;
  constexpr int UM = C::UM, UC = C::UC, XC = C::XC, NM = C::NM, NX = C::NX, DV = DM;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  pdl_launch();  // the merge waits for this kernel's end before it reads
  if (pad + C::SMEM_USED > static_cast<uint32_t>(C::SMEM_BYTES)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusLayout);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sQ = sb + C::OFF_Q, sP = sb + C::OFF_P, sM = sb + C::OFF_M, sX = sb + C::OFF_X;
  const Bars<NM, NX> bar{sb + C::OFF_BAR};
  float* s_nref = reinterpret_cast<float*>(smem + C::OFF_STAT);
  float* s_alpha = s_nref + NR;
  int* s_lag = reinterpret_cast<int*>(s_alpha + NR);
  float* s_red = reinterpret_cast<float*>(smem + C::OFF_RED);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // first sequence, its first tile, tiles of this CTA
  const WaitCtl wc{p.status, abort_flag, p.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // this CTA: rows r0 .. of head `head` of every sequence (group b * heads + head), range `cut` of `cuts`
  const int grp = blockIdx.x / plan.cuts, cut = blockIdx.x % plan.cuts;
  const int head = grp / plan.row_groups, r0 = (grp % plan.row_groups) * NR;
  const int n_rows = min(NR, p.rows - r0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NM; ++s) {
      mbar_init(bar.m_full(s), 1);
      mbar_init(bar.m_free(s), 1);
    }
    for (int s = 0; s < NX; ++s) {
      mbar_init(bar.x_full(s), 1);
      mbar_init(bar.x_free(s), 1);
    }
    mbar_init(bar.q_full(), 1);
    mbar_init(bar.q_free(), 1);
    mbar_init(bar.s_full(0), 1);
    mbar_init(bar.s_full(1), 1);
    mbar_init(bar.p_full(), 8);
    mbar_init(bar.o_done(), 1);
    mbar_init(bar.drain(), 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  if (warp == 9) {
    // where this CTA's range of the tiles, laid end to end, begins
    unsigned before, total;
    tile_sums(p, plan.n_seq, 0, before, total);
    const unsigned ranges = range_count(total, plan.cuts);
    const bool some = cut < static_cast<int>(ranges);
    const unsigned t0 = some ? range_start(total, cut, ranges) : total;
    const unsigned t1 = some ? range_start(total, cut + 1, ranges) : total;
    unsigned base = 0;
    int b0 = 0, first = 0;
    bool found = false;
    for (int i0 = 0; i0 < plan.n_seq && !found; i0 += 32) {
      const int i = i0 + lane;
      const unsigned t = i < plan.n_seq ? tiles_of(seq_len(p, i, true)) : 0;
      unsigned inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned end = base + inc;
      const unsigned hit = __ballot_sync(0xffffffffu, end > t0);
      if (hit) {
        const int l = __ffs(hit) - 1;
        const unsigned beg = __shfl_sync(0xffffffffu, end - t, l);
        b0 = i0 + l;
        first = static_cast<int>(t0 - beg);
        found = true;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      s_start[0] = b0;
      s_start[1] = first;
      s_start[2] = found ? static_cast<int>(t1 - t0) : 0;
    }
  } else if (threadIdx.x < NR) {
    s_lag[threadIdx.x] = p.n_new - 1 - (r0 + static_cast<int>(threadIdx.x)) % p.n_new;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int start_b = __shfl_sync(0xffffffffu, s_start[0], 0), start_t = __shfl_sync(0xffffffffu, s_start[1], 0),
            n_tiles = __shfl_sync(0xffffffffu, s_start[2], 0);

  // walks the pieces, a whole warp at a time: f(sequence, its keys, first tile, tiles) until it returns false
  auto pieces = [&](auto f) {
    int b = start_b, t = start_t, left = n_tiles;
    while (left > 0) {
      const int nk = __shfl_sync(0xffffffffu, seq_len(p, b, false), 0);
      const int take = min(left, tiles_of(nk) - t);
      if (take > 0) {
        if (!f(b, nk, t, take)) return;
        left -= take;
      }
      ++b;
      t = 0;
    }
  };

  if (warp == 9) {
    // ------------------------------------------------------------------ TMA
    // The whole warp walks, converged; a tile is one box of 64 tokens, or 2 or 4
    // where pages are not whole tiles.  Lane i looks box i's page up.
    const int box = plan.box, per = BC / box;
    int g = 0, nq = 0;  // tiles and pieces issued
    int ms = 0, xs = 0;            // next slots of the rings, and the parity their release completes
    uint32_t mp = 1, xp = 1;
    auto wait = [&](uint32_t bar_addr, uint32_t parity) { return warp_wait(bar_addr, parity, wc); };
    pieces([&](int b, int nk, int t0, int n) -> bool {
      const int group = b * plan.heads + head;
      if (nq > 0 && !wait(bar.q_free(), (nq - 1) & 1)) return false;
      mbar_arrive_expect_tx_w(bar.q_full(), C::Q_BYTES);
      for (int c = 0; c < C::QC; ++c) tma_load_3d_w(sQ + c * NR * 128, &maps.q, bar.q_full(), c * 64, r0, group);
      ++nq;
      // this lane's box of a tile: token within its page, page (as the table has it)
      auto place = [&](int tile, int& tok, int& page) {
        const int j = tile * BC + lane * box;
        tok = 0;
        page = group;
        if (lane >= per || j >= nk) return;
        tok = j;
        if (p.table != nullptr) {
          const int q = j / p.page_size;
          tok = j - q * p.page_size;
          page = p.table[static_cast<long long>(b) * p.max_pages + q];
        }
      };
      int tok, page;
      place(t0, tok, page);
      for (int i = 0; i < n; ++i, ++g) {
        const int valid = min(BC, nk - (t0 + i) * BC);
        const int boxes = (valid + box - 1) / box;
        int tok1 = 0, page1 = 0;
        if (i + 1 < n) place(t0 + i + 1, tok1, page1);  // the next tile's pages, while this one loads
        if (p.table != nullptr && lane < boxes && (page < 0 || page >= p.n_pages)) {
          atomicOr(p.status, kStatusInput);
          page = p.n_pages;  // outside the cache: reads as zeros
        }
        int box_tok[4], box_page[4];  // the boxes' places, in every lane
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          box_tok[k] = __shfl_sync(0xffffffffu, tok, k);
          box_page[k] = __shfl_sync(0xffffffffu, page, k);
        }
        auto load_x = [&]() -> bool {
          if (!wait(bar.x_free(xs), xp)) return false;
          mbar_arrive_expect_tx_w(bar.x_full(xs), boxes * box * 128 * XC);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= boxes) break;
#pragma unroll
            for (int c = 0; c < XC; ++c)
              tma_load_3d_w(sX + xs * C::X_BYTES + c * CB + i * box * 128, &maps.x, bar.x_full(xs),
                            (SHARED ? DM : 0) + c * 64, box_tok[i], box_page[i]);
          }
          if (++xs == NX) {
            xs = 0;
            xp ^= 1;
          }
          return true;
        };
        if (!SHARED && !load_x()) return false;
        for (int u = 0; u < UM; ++u) {
          if (!wait(bar.m_free(ms), mp)) return false;
          mbar_arrive_expect_tx_w(bar.m_full(ms), boxes * box * 128 * UC);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= boxes) break;
#pragma unroll
            for (int c = 0; c < UC; ++c)
              tma_load_3d_w(sM + ms * C::M_BYTES + c * CB + i * box * 128, &maps.m, bar.m_full(ms), (u * UC + c) * 64,
                            box_tok[i], box_page[i]);
          }
          if (++ms == NM) {
            ms = 0;
            mp ^= 1;
          }
        }
        if (SHARED && !load_x()) return false;
        tok = tok1;
        page = page1;
      }
      return true;
    });
    if (*abort_flag && lane == 0) {
      // let copies already in flight land before the CTA's shared memory is
      // released; a wait for copies that were never issued just runs out
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      if (nq > 0) mbar_wait(bar.q_full(), (nq - 1) & 1, drain);
      for (int k = max(0, (g + 1) * UM - NM); k < (g + 1) * UM; ++k) mbar_wait(bar.m_full(k % NM), (k / NM) & 1, drain);
      for (int k = max(0, g + 1 - NX); k < g + 1; ++k) mbar_wait(bar.x_full(k % NX), (k / NX) & 1, drain);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    // The whole warp runs it, converged (see mma_ss_w).  Two streams of work:
    // S^T of tile after tile, a ring unit at a time as its loads land, at most
    // one tile ahead of the values (two S buffers); and O^T of a tile once its
    // P is published.  Whichever is ready goes first, so that a late load
    // does not hold up the product that frees ring space for later ones.
    constexpr uint32_t idesc_s = idesc_bf16_f32(BC, NR, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16_f32(C::UDIM, NR, 1, 0);
    constexpr int UNITS = SHARED ? UM + 1 : 1;  // ring units that S^T of a tile reads
    const Desc2 dq = desc_sw128(sQ, 16, 1024), dp = desc_sw128(sP, 16, 1024);
    const Desc2 dm_k = desc_sw128(sM, 16, 1024), dx = desc_sw128(sX, 16, 1024), dm_v = desc_sw128(sM, CB, 1024);
    bool ok = true;
    int nq = 0;
    int ms = 0, xs = 0, vs = 0;  // M and X slots of the next S^T unit, M slot of the next value unit
    uint32_t mp = 0, xp = 0, vp = 0, sbuf = 0, pp = 0;
    pieces([&](int, int, int, int n) -> bool {
      if (!(ok = warp_wait(bar.q_full(), nq & 1, wc))) return false;
      tc_fence_after();
      int s_tile = 0, s_unit = 0, o_tile = 0;  // progress within the piece
      unsigned long long since = 0;
      while (o_tile < n) {
        bool moved = false;
        if (s_tile < n && s_tile <= o_tile + 1) {
          const bool x_unit = s_unit == UNITS - 1;
          if (x_unit ? warp_test(bar.x_full(xs), xp) : warp_test(bar.m_full(ms), mp)) {
            moved = true;
            tc_fence_after();
            const uint32_t dt = tmem + C::TM_S + NR * sbuf;
            if (x_unit) {
              constexpr int QX = SHARED ? UM * UC : 0;
              const uint32_t at = (xs * C::X_BYTES) >> 4;
#pragma unroll
              for (int kk = 0; kk < DX / 16; ++kk)
                mma_ss_w(dt, dx, at + (((kk >> 2) * CB + (kk & 3) * 32) >> 4), dq,
                         ((QX + (kk >> 2)) * NR * 128 + (kk & 3) * 32) >> 4, idesc_s, SHARED || kk > 0);
              mma_commit_w(bar.x_free(xs));
              mma_commit_w(bar.s_full(sbuf));
              if (++xs == NX) {
                xs = 0;
                xp ^= 1;
              }
              sbuf ^= 1;
              s_unit = 0;
              if (++s_tile == n) mma_commit_w(bar.q_free());  // no later product of this piece reads Q
            } else {
              const uint32_t at = (ms * C::M_BYTES) >> 4, qo = (s_unit * UC * NR * 128) >> 4;
#pragma unroll
              for (int kk = 0; kk < UC * 4; ++kk)
                mma_ss_w(dt, dm_k, at + (((kk >> 2) * CB + (kk & 3) * 32) >> 4), dq,
                         qo + (((kk >> 2) * NR * 128 + (kk & 3) * 32) >> 4), idesc_s, s_unit > 0 || kk > 0);
              ++s_unit;
              if (++ms == NM) {
                ms = 0;
                mp ^= 1;
              }
            }
          }
        }
        if (o_tile < s_tile && warp_test(bar.p_full(), pp)) {
          bool values = true;
          if (!SHARED) values = warp_test(bar.m_full(vs), vp);
          if (values) {
            moved = true;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < UM; ++u) {
              const uint32_t at = (vs * C::M_BYTES) >> 4;
#pragma unroll
              for (int kk = 0; kk < BC / 16; ++kk)
                mma_ss_w(tmem + u * NR, dm_v, at + ((kk * 16 * 128) >> 4), dp, (kk * 32) >> 4, idesc_o,
                         o_tile > 0 || kk > 0);
              mma_commit_w(bar.m_free(vs));
              if (++vs == NM) {
                vs = 0;
                vp ^= 1;
              }
            }
            mma_commit_w(bar.o_done());
            pp ^= 1;
            ++o_tile;
          }
        }
        if (moved) {
          since = 0;
        } else if (since == 0) {
          since = globaltimer_ns();
        } else {
          // neither stream has moved: the wait is bounded like every other
          bool late = globaltimer_ns() - since > wc.limit_ns;
          late = __any_sync(0xffffffffu, late);
          if (late) record_timeout(wc);
          if (__any_sync(0xffffffffu, late || *abort_flag != 0)) return ok = false;
        }
      }
      ++nq;
      return true;
    });
    // every MMA this warp issued must finish before tensor memory is freed
    mma_commit_w(bar.drain());
    WaitCtl drain{nullptr, nullptr, wc.limit_ns};
    mbar_wait(bar.drain(), 0, drain);
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    // Tensor memory hands a key's scores to a lane below 16; lane + 16 takes
    // half of its warp's columns over, so that every lane has NH = NR / 4
    // columns of one key.
    // Once a wait has run out, waits return at once and the loops run on to
    // their ends (barriers count every warp); nothing is written out then.
    constexpr int NH = NR / 4;
    constexpr int LW = NR / 2 < 32 ? NR / 2 : 32;  // columns per tensor-memory access
    constexpr int OC = UM * NR / 2;                // columns of O that a warp handles
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int key = quarter * 16 + (lane & 15), col = wg * (NR / 2) + (lane < 16 ? 0 : NH);
    const float sl = p.scale * 1.4426950408889634f;
    // P is [row][64 keys], 128-byte rows, 16-byte chunks swizzled by row % 8.
    // Lanes of an even and an odd key pair up: the even one writes both keys'
    // P of an even column, the odd one those of the column after it.
    const int odd = lane & 1;
    constexpr int PA = NH / 2 < 4 ? NH / 2 : 4;
    uint32_t p_at[PA];
#pragma unroll
    for (int q = 0; q < PA; ++q) {
      const int row = col + 2 * q + odd;
      p_at[q] = sP + row * 128 + (((key >> 3) ^ (row & 7)) << 4) + (key & 6) * 2;
    }
    const int my_col = col + reduce_col<NH>();  // the column this lane owns after reduce16
    int g = 0;

    pieces([&](int b, int nk, int t0, int n) -> bool {
      const int group = b * plan.heads + head;
      float l[NH], lr[NH];  // this key's share of the row sums: of P, and of P rounded to bf16 (what multiplies V)
#pragma unroll
      for (int c = 0; c < NH; ++c) l[c] = lr[c] = 0.f;
      if (threadIdx.x < NR) s_nref[threadIdx.x] = kUnset;
      named_bar_sync(1, kSoftmax);
      for (int i = 0; i < n; ++i, ++g) {
        warp_wait(bar.s_full(g & 1), (g >> 1) & 1, wc);
        tc_fence_after();
        float s[NH];
        {
          uint32_t r[2 * NH];
          tmem_ld<2 * NH>(tl + C::TM_S + NR * (g & 1) + wg * (NR / 2), r);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            const uint32_t far = __shfl_xor_sync(0xffffffffu, r[c + NH], 16);
            s[c] = __uint_as_float(lane < 16 ? r[c] : far);
          }
        }
        const int j0 = (t0 + i) * BC;
        if (j0 + BC > nk - (p.n_new - 1)) {
          const int room = nk - (j0 + key);  // > lag: the row sees this key
#pragma unroll
          for (int c = 0; c < NH; ++c) s[c] = s_lag[col + c] < room ? s[c] : -INFINITY;
        }
        // values past the sequence's end multiply zero probabilities: they must be finite
        const int valid = min(BC, nk - j0);
        if (valid < BC) {
          if (!SHARED) warp_wait(bar.m_full(g % NM), (g / NM) & 1, wc);
          const int rows = BC - valid;
          for (int x = threadIdx.x; x < rows * UM * UC * 8; x += kSoftmax) {
            const int row = valid + x / (UM * UC * 8), y = x % (UM * UC * 8);
            const int u = y / (UC * 8), z = y % (UC * 8);
            st_shared_v4(sM + ((g * UM + u) % NM) * C::M_BYTES + (z >> 3) * CB + row * 128 + (z & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        float over = -INFINITY;
#pragma unroll
        for (int c = 0; c < NH; c += 4) {
          const float4 nr = *reinterpret_cast<const float4*>(s_nref + col + c);
          over = fmax3(over, fmaf(s[c], sl, nr.x), fmaf(s[c + 1], sl, nr.y));
          over = fmax3(over, fmaf(s[c + 2], sl, nr.z), fmaf(s[c + 3], sl, nr.w));
        }
        if (bar_any(1, kSoftmax, over > kRescaleThreshold)) {
          // some row's reference rises: column maxima over the 64 keys
          {
            float v[NH];
#pragma unroll
            for (int c = 0; c < NH; ++c) v[c] = s[c] * sl;
            reduce16<NH>(v, [](float x, float y) { return fmaxf(x, y); });
            s_red[quarter * NR + my_col] = v[0];
          }
          named_bar_sync(1, kSoftmax);
          if (threadIdx.x < NR) {
            const int c = threadIdx.x;
            const float mx = fmaxf(fmaxf(s_red[c], s_red[NR + c]), fmaxf(s_red[2 * NR + c], s_red[3 * NR + c]));
            const float old = s_nref[c];
            float alpha = 1.f;
            if (mx + old > kRescaleThreshold) {  // old = kUnset: the first key that the row sees
              alpha = old == kUnset ? 0.f : ex2_approx(-old - mx);
              s_nref[c] = -mx;
            }
            s_alpha[c] = alpha;
          }
          named_bar_sync(1, kSoftmax);
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            const float a = s_alpha[col + c];
            l[c] *= a;
            lr[c] *= a;
          }
          if (i > 0) {
            warp_wait(bar.o_done(), (g - 1) & 1, wc);
            tc_fence_after();
#pragma unroll 1
            for (int c = wg * OC; c < (wg + 1) * OC; c += LW) {
              uint32_t o[LW];
              tmem_ld<LW>(tl + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < LW; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s_alpha[c % NR + e]);
              tmem_st<LW>(tl + c, o);
            }
            tmem_wait_st();
          }
        }
        uint32_t pk[NH / 2];
#pragma unroll
        for (int c = 0; c < NH; c += 4) {
          const float4 nr = *reinterpret_cast<const float4*>(s_nref + col + c);
          const float p0 = ex2_approx(fmaf(s[c], sl, nr.x)), p1 = ex2_approx(fmaf(s[c + 1], sl, nr.y));
          const float p2 = ex2_approx(fmaf(s[c + 2], sl, nr.z)), p3 = ex2_approx(fmaf(s[c + 3], sl, nr.w));
          // P is rounded to bf16, the products' type, half a step of 2^-8 each; O is
          // divided by the sum of the rounded values, lse takes the unrounded ones
          const uint32_t a = pack_bf16x2(p0, p1), bq = pack_bf16x2(p2, p3);
          l[c] += p0;
          l[c + 1] += p1;
          l[c + 2] += p2;
          l[c + 3] += p3;
          lr[c] += __uint_as_float(a << 16);
          lr[c + 1] += __uint_as_float(a & 0xffff0000u);
          lr[c + 2] += __uint_as_float(bq << 16);
          lr[c + 3] += __uint_as_float(bq & 0xffff0000u);
          const uint32_t ya = __shfl_xor_sync(0xffffffffu, a, 1), yb = __shfl_xor_sync(0xffffffffu, bq, 1);
          pk[c / 2] = odd ? __byte_perm(ya, a, 0x7632) : __byte_perm(a, ya, 0x5410);
          pk[c / 2 + 1] = odd ? __byte_perm(yb, bq, 0x7632) : __byte_perm(bq, yb, 0x5410);
        }
        // P_{g-1} has been read once its P V has completed
        if (g > 0) warp_wait(bar.o_done(), (g - 1) & 1, wc);
#pragma unroll
        for (int c = 0; c < NH / 2; ++c)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_at[c % PA] + (c / PA) * 1024), "r"(pk[c]) : "memory");
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.p_full());
      }
      // ------------------------------------------------------------ output
      float ref = 0.f, sum = 0.f;  // of row threadIdx.x
      reduce16<NH>(l, [](float x, float y) { return x + y; });
      reduce16<NH>(lr, [](float x, float y) { return x + y; });
      s_red[quarter * NR + my_col] = l[0];
      named_bar_sync(1, kSoftmax);
      if (threadIdx.x < NR) {
        const int c = threadIdx.x;
        sum = (s_red[c] + s_red[NR + c]) + (s_red[2 * NR + c] + s_red[3 * NR + c]);
        ref = s_nref[c] == kUnset ? 0.f : -s_nref[c];
      }
      named_bar_sync(1, kSoftmax);
      s_red[quarter * NR + my_col] = lr[0];
      named_bar_sync(1, kSoftmax);
      const bool whole = plan.direct && t0 == 0 && n == tiles_of(nk);
      const long long slot = static_cast<long long>(grp) * (plan.cuts + plan.n_seq) + cut + b;
      const long long orow0 = (group / p.group_div) * p.q_s1 + (group % p.group_div) * p.q_s2 + r0;
      if (threadIdx.x < NR) {
        const int c = threadIdx.x;
        const float sum_r = (s_red[c] + s_red[NR + c]) + (s_red[2 * NR + c] + s_red[3 * NR + c]);
        s_alpha[c] = sum_r == 0.f ? 0.f : 1.f / sum_r;
        const float lse = (ref + __log2f(sum)) * 0.69314718055994531f;  // -inf where no key was seen
        if (c < n_rows && !*abort_flag) {
          if (!whole)
            p.part_lse[slot * NR + c] = lse;
          else if (p.lse != nullptr)
            p.lse[orow0 + c] = lse;
        }
      }
      named_bar_sync(1, kSoftmax);
      warp_wait(bar.o_done(), (g - 1) & 1, wc);
      tc_fence_after();
      const int d0 = C::UDIM == 128 ? quarter * 32 + lane : quarter * 16 + lane;  // this lane's dimension of an M unit
      const bool has_dim = (C::UDIM == 128 || lane < 16) && d0 < DV;
#pragma unroll 1
      for (int c = wg * OC; c < (wg + 1) * OC; c += LW) {
        if (c % NR >= n_rows) continue;
        uint32_t o[LW];
        tmem_ld<LW>(tl + c, o);
        tmem_wait_ld();
        const int d = (c / NR) * 128 + d0, row = c % NR;
        if (!has_dim || *abort_flag) continue;
#pragma unroll
        for (int e = 0; e < LW; ++e) {
          if (row + e >= n_rows) break;
          const float a = s_alpha[row + e];
          const float v = a == 0.f ? 0.f : __uint_as_float(o[e]) * a;
          if (whole)
            static_cast<__nv_bfloat16*>(p.o)[(orow0 + row + e) * DV + d] = __float2bfloat16_rn(v);
          else
            p.part_o[(slot * NR + row + e) * DV + d] = v;
        }
      }
      tc_fence_before();
      named_bar_sync(1, kSoftmax);  // the statistics are free for the next piece
      return true;
    });
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  pdl_wait();  // the prefix's kernel runs beside this one: the merge waits for both
}

// Merges the pieces of each sequence, and the partial results [pre][total] of
// another set of keys beside them (the prefix), row by row: see
// seq_combine.cu for the formula.  One warp per row and W of its 128-column
// slices (all of them where there are rows enough to fill the GPU); lane i
// holds the weight of part i, so that the parts' loads do not wait for one
// another.  Rows of a sequence that was written directly are left alone.
template <int NR, int W>
__global__ void __launch_bounds__(128)
    fa_seq_decode_merge_kernel(const __grid_constant__ SeqAttn p, const DecodePlan plan, const float* __restrict__ pre_o,
                               const float* __restrict__ pre_lse, int pre) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned slices = (p.dv + 128 * W - 1) / (128 * W);
  const unsigned idx = blockIdx.x * 4 + warp;  // (sequence, head, row, slices)
  const unsigned rows = p.rows;
  const unsigned row_idx = idx / slices, slice = idx - row_idx * slices;
  const unsigned group = row_idx / rows, r = row_idx - group * rows;
  if (group >= static_cast<unsigned>(plan.n_seq * plan.heads)) {
    pdl_wait();
    return;
  }
  const int b = group / plan.heads, head = group % plan.heads;
  unsigned before, total;
  tile_sums(p, plan.n_seq, b, before, total);
  const int nt = tiles_of(seq_len(p, b, true));
  int c0 = 0, n = 0;
  if (nt > 0) {
    const unsigned ranges = range_count(total, plan.cuts);
    c0 = owner(total, before, ranges);
    n = owner(total, before + nt - 1, ranges) - c0 + 1;
  }
  pdl_wait();
  if (plan.direct && n == 1) return;
  const int grp = head * plan.row_groups + r / NR;
  const long long slot0 = (static_cast<long long>(grp) * (plan.cuts + plan.n_seq) + c0 + b) * NR + r % NR;
  const long long row = (group / p.group_div) * p.q_s1 + (group % p.group_div) * p.q_s2 + r;
  n += pre;
  auto part_lse = [&](int i) {
    return i < pre ? pre_lse[i * p.total + row] : p.part_lse[slot0 + static_cast<long long>(i - pre) * NR];
  };
  const float mine = lane < n ? part_lse(lane) : -INFINITY;
  float m = mine;
  for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, part_lse(i));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = lane < n ? expf(mine - ref) : 0.f;
  for (int i = lane + 32; i < n; i += 32) sum += expf(part_lse(i) - ref);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int c = slice * 128 * W + 4 * lane;
  float4 acc[W];
#pragma unroll
  for (int w = 0; w < W; ++w) acc[w] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float ls = i0 == 0 ? mine : (i0 + lane < n ? part_lse(i0 + lane) : -INFINITY);
    const float wl = expf(ls - ref) * inv;
    const int k = min(32, n - i0);
#pragma unroll 8
    for (int i = 0; i < k; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wl, i);
      const int part = i0 + i;
      const float* src = (part < pre ? pre_o + (part * p.total + row) * p.dv
                                     : p.part_o + (slot0 + static_cast<long long>(part - pre) * NR) * p.dv) + c;
      if (wi == 0.f) continue;  // a part without keys holds zeros or nothing
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (c + 128 * w >= p.dv) break;
        const float4 v = *reinterpret_cast<const float4*>(src + 128 * w);
        acc[w].x = fmaf(wi, v.x, acc[w].x);
        acc[w].y = fmaf(wi, v.y, acc[w].y);
        acc[w].z = fmaf(wi, v.z, acc[w].z);
        acc[w].w = fmaf(wi, v.w, acc[w].w);
      }
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (c + 128 * w < p.dv)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + row * p.dv + c + 128 * w) =
          make_uint2(pack_bf16x2(acc[w].x, acc[w].y), pack_bf16x2(acc[w].z, acc[w].w));
  if (slice == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = m + logf(sum);
}

template <int DM, int DX, bool SHARED, int NR>
cudaError_t launch_nr(const SeqAttn& p, const DecodePlan& plan, bool beside, cudaStream_t s) {
  using C = Cfg<DM, DX, SHARED, NR>;
  static SmemOnce once;
  cudaError_t e = once(fa_seq_decode_sm103_kernel<DM, DX, SHARED, NR>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  DecodeMaps m;
  const int width = p.d1;
  const long long pages = p.page_size > 0 ? p.n_pages : p.groups;
  const int page = p.page_size > 0 ? p.page_size : p.n_keys;
  if (!make_map3(&m.q, p.q, width, p.rows, p.groups, NR) || !make_map3(&m.x, p.k1, width, page, pages, plan.box))
    return cudaErrorInvalidValue;
  m.m = m.x;
  if (!SHARED && !make_map3(&m.m, p.v, DM, page, pages, plan.box)) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(plan.heads) * plan.row_groups * plan.cuts;
  if (beside) return launch_after(fa_seq_decode_sm103_kernel<DM, DX, SHARED, NR>, grid, kThreads, C::SMEM_BYTES, s, m, p, plan);
  fa_seq_decode_sm103_kernel<DM, DX, SHARED, NR><<<grid, kThreads, C::SMEM_BYTES, s>>>(m, p, plan);
  return cudaGetLastError();
}

template <int NR>
cudaError_t launch_merge(const SeqAttn& p, const DecodePlan& w, const float* pre_o, const float* pre_lse, int pre,
                         bool after, cudaStream_t s) {
  // A warp takes a whole row of 512 where the rows alone give every SM 32 warps
  // (the whole call at 16384 rows: 105 us, 117 with a warp a slice; at 1024
  // rows 71 and 68; at 16 rows 18.9 and 15.4).
  const long long rows = static_cast<long long>(w.n_seq) * w.heads * p.rows;
  const bool wide = p.dv > 128 && rows >= 152 * 32;
  const long long warps = rows * (wide ? (p.dv + 511) / 512 : (p.dv + 127) / 128);
  if (warps > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
  if (!after) {  // no kernel of this call before it: the lengths may only now be complete
    fa_seq_decode_merge_kernel<NR, 1><<<static_cast<unsigned>((rows * ((p.dv + 127) / 128) + 3) / 4), 128, 0, s>>>(
        p, w, pre_o, pre_lse, pre);
    return cudaGetLastError();
  }
  return wide ? launch_after(fa_seq_decode_merge_kernel<NR, 4>, blocks, 128, 0, s, p, w, pre_o, pre_lse, pre)
              : launch_after(fa_seq_decode_merge_kernel<NR, 1>, blocks, 128, 0, s, p, w, pre_o, pre_lse, pre);
}

}  // namespace

DecodePlan decode_plan(int n_seq, int heads, int rows, bool shared, int box, int sms) {
  DecodePlan w{};
  w.n_seq = n_seq;
  w.heads = heads;
  // The narrowest product that holds the rows (64 sequences of 4000 to 8000
  // tokens of 512 + 64, 16 heads: 84, 86, 92 us with 16, 32, 64 columns; 32
  // heads: 125, 92, 97; separate keys and values, 128 x 8 heads of 2048, d =
  // 128: 16 rows 150, 169, 290; 32 rows 244, 181, 306).
  w.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  w.row_groups = (rows + w.nr - 1) / w.nr;
  const int ctas = shared ? sms : 2 * sms;  // one CTA an SM, or two
  const long long groups = static_cast<long long>(heads) * w.row_groups;
  w.cuts = groups < ctas ? static_cast<int>(ctas / groups) : 1;
  w.direct = shared;
  w.box = box;
  return w;
}
size_t decode_slots(const DecodePlan& w) {
  return static_cast<size_t>(w.heads) * w.row_groups * (static_cast<size_t>(w.cuts) + w.n_seq) * w.nr;
}

cudaError_t launch_seq_decode(const SeqAttn& p, const DecodePlan& w, bool beside, cudaStream_t s) {
  if (static_cast<long long>(w.heads) * w.row_groups * w.cuts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // tile counts are summed, and multiplied by the number of cuts, in 32 bits
  if (static_cast<long long>(w.n_seq) * tiles_of(p.n_keys) * (w.cuts + 1LL) > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
#define FA_DECODE(DM, DX, SH)                                                          \
  (w.nr == 16 ? launch_nr<DM, DX, SH, 16>(p, w, beside, s)                             \
              : w.nr == 32 ? launch_nr<DM, DX, SH, 32>(p, w, beside, s) : launch_nr<DM, DX, SH, 64>(p, w, beside, s))
  if (w.direct) {
    if (p.dv == 512) return FA_DECODE(512, 64, true);
    if (p.dv == 256) return FA_DECODE(256, 64, true);
  } else {
    if (p.dv == 64) return FA_DECODE(64, 64, false);
    if (p.dv == 96) return FA_DECODE(96, 96, false);
    if (p.dv == 128) return FA_DECODE(128, 128, false);
  }
#undef FA_DECODE
  return cudaErrorInvalidValue;
}

cudaError_t launch_seq_decode_merge(const SeqAttn& p, const DecodePlan& w, const float* pre_o, const float* pre_lse,
                                    int pre, bool after, cudaStream_t s) {
  if (w.nr == 16) return launch_merge<16>(p, w, pre_o, pre_lse, pre, after, s);
  if (w.nr == 32) return launch_merge<32>(p, w, pre_o, pre_lse, pre, after, s);
  return launch_merge<64>(p, w, pre_o, pre_lse, pre, after, s);
}

}  // namespace fa
