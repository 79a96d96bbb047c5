// cache4_decode_sm103.cu -- attention of few query rows over the 4-bit key/value
// cache, bf16 in / fp32 accumulate, on the tensor cores of GB300 (sm_103a).
//
//   S_ij = scale k_scale (q_i . K_j) over the keys j < len - lag(i),
//   O_i = v_scale sum_j softmax_j(S_i) V_j,   K, V = code * scale
//
// A tile is 128 keys.  The products are taken transposed, keys and channels as
// the long (M) side and the query rows of a key/value head as the short one:
//   S^T [128 keys x NR] = K Q^T,   O^T [128 channels x NR] += V^T P^T
// and their A operands, K and V^T, come from tensor memory, where the threads
// put them as they unpack the codes: one thread a key, then one a channel, each
// a row of its own; nothing of the unpacked tile passes through shared memory.
// code * scale is exact in fp16 (at most 6 significant bits, 2^-10 to 2688), so
// fp16 it is, and Q and P with it: a row of Q is bf16 (8 bits) times a power of
// two that brings its largest entry to 2^14 .. 2^15, exact down to 2^-31 of that;
// P is rounded to 11 bits where bf16 would keep 8.
//
// W warpgroups take the tiles in turn, each with operands, scores and an O of
// its own in tensor memory and its own running reference, so that one's
// products and waits overlap another's unpacking; they meet at the end of a
// piece (a CTA's share of a sequence) only, where every warpgroup adds up some
// columns of all O.  Per tile a warpgroup: unpacks K, starts S^T, unpacks V
// meanwhile, takes the softmax, writes P, starts O^T.
//
// Statistics run down the columns, across lanes.  Per tile a thread (one key)
// only checks whether any of its scores exceeds its column's reference by 2^8;
// if no key's does (one barrier with an OR) the tile is exponentiated as it is.
// Otherwise the column maxima are reduced across lanes and warps and O rescaled.
//
// One more warp loads: a tile's blocks, one bulk copy for each run of them in
// a page, into a ring of as many tiles as fit.  The work is split as
// seq_ranges.cuh says; a sequence that is one whole piece goes straight to o.
#include <cmath>

#include "cache4.cuh"
#include "seq_ranges.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BC = 128;  // keys per tile
constexpr float kUnset = 3e38f;  // negated reference of a row that has seen no key
constexpr float kRescaleThreshold = 8.0f;

template <int D, int NR>
struct Cfg {
  static constexpr int KC = D / 2;                   // columns of K in tensor memory, then 64 of V^T, S^T, O^T
  static constexpr int COLS = KC + 64 + 2 * NR;      // of a warpgroup
  static constexpr int W = 512 / COLS < 4 ? 512 / COLS : 4;
  static constexpr int THREADS = W * 128 + 32;
  static constexpr int QC = (D + 63) / 64;           // 64-channel chunks of Q
  static constexpr int RB = NR * 2;                  // bytes of a key's row of P
  static constexpr int TILE = 144 * D;               // bytes: 8 blocks of 18 D
  static constexpr int Q_BYTES = QC * NR * 128;
  static constexpr int P_BYTES = 128 * RB;           // a warpgroup
  static constexpr int STATS = (2 + 3 * W) * NR * 4  // lag, column scale; reference, sum and factor of each warpgroup
                               + W * 4 * NR * 4;     // warps' column results
  static constexpr int MISC = STATS + 512;
  static constexpr int SLOTS_FIT = (227 * 1024 - 1024 - Q_BYTES - W * P_BYTES - MISC) / TILE;
  static constexpr int SLOTS = SLOTS_FIT < 12 ? SLOTS_FIT : 12;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_RING = OFF_P + W * P_BYTES;
  static constexpr int OFF_STAT = OFF_RING + SLOTS * TILE;
  static constexpr int OFF_BAR = OFF_STAT + STATS;
  static constexpr int NBAR = 2 * SLOTS + 3 * W;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tensor memory base, abort flag, start, then the slots' missing blocks
  static constexpr int SMEM_USED = OFF_MISC + 24 + SLOTS * 4;
  static constexpr int SMEM_BYTES = SMEM_USED + 1024;
  static constexpr int TM_K = 0, TM_V = KC, TM_S = KC + 64, TM_O = TM_S + NR;
  static_assert(W >= 2 && SLOTS >= 2 * W, "two tiles a warpgroup in flight");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(OFF_P % 1024 == 0 && P_BYTES % 1024 == 0 && OFF_RING % 1024 == 0 && TILE % 16 == 0, "alignment");
};

// fp16 operands: formats 0 in the bf16 descriptor's fields
constexpr uint32_t idesc_f16(int M, int N, int b_mn) { return idesc_bf16_f32(M, N, 0, b_mn) & ~((7u << 7) | (7u << 10)); }

// Shared-memory descriptor of P: key-major rows of RB bytes, swizzled over RB.
template <int RB>
__device__ __forceinline__ Desc2 desc_p(uint32_t saddr) {
  const Desc2 d = desc_sw128(saddr, 16, 8 * RB);
  return Desc2{d.lo, (d.hi & 0x1fffffffu) | (RB == 32 ? 6u : RB == 64 ? 4u : 2u) << 29};
}
// The 16-byte chunk where chunk c of key t's row stands.
template <int RB>
__device__ __forceinline__ int p_chunk(int t, int c) {
  return RB == 32 ? c ^ ((t >> 2) & 1) : RB == 64 ? c ^ ((t >> 1) & 3) : c ^ (t & 7);
}

// Columns v[0..N) reduced over the 32 lanes: lane l ends with max(1, N / 32)
// columns in v[0 ..), from column first_col<N>() on.
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
template <int N>
__device__ __forceinline__ int first_col() {
  int col = 0;
#pragma unroll
  for (int h = N / 2, bit = 16; h >= 1 && bit >= 1; h /= 2, bit /= 2)
    if (threadIdx.x & bit) col += h;
  return col;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg<D, NR>::THREADS, 1)
    fa_cache4_decode_kernel(const __grid_constant__ SeqAttn p, const __grid_constant__ Cache4 cache,
                            const DecodePlan plan) {
  using C = Cfg<D, NR>;
  constexpr int W = C::W, SLOTS = C::SLOTS, GROUPS = D / 16;
  constexpr int kConsumers = W * 128;
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
  const uint32_t sQ = sb + C::OFF_Q, sRing = sb + C::OFF_RING;
  int* s_lag = reinterpret_cast<int*>(smem + C::OFF_STAT);           // [NR]
  float* s_cs = reinterpret_cast<float*>(s_lag + NR);                // [NR] log2-domain scale of a column
  float* s_ref = s_cs + NR;                                          // [W][NR] negated references
  float* s_sum = s_ref + W * NR;                                     // [W][NR]
  float* s_fac = s_sum + W * NR;                                     // [W][NR] alpha, then the factor of an O
  float* s_red = s_fac + W * NR;                                     // [W][4][NR]
  const uint32_t bars = sb + C::OFF_BAR;
  auto full = [&](int s) { return bars + 8 * s; };
  auto free_ = [&](int s) { return bars + 8 * (SLOTS + s); };
  auto s_done = [&](int w) { return bars + 8 * (2 * SLOTS + w); };
  auto o_done = [&](int w) { return bars + 8 * (2 * SLOTS + W + w); };
  auto drain_bar = [&](int w) { return bars + 8 * (2 * SLOTS + 2 * W + w); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // first sequence, its first tile, tiles of this CTA
  volatile int* s_missing = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 24);  // [SLOTS] blocks without a page
  const WaitCtl wc{p.status, abort_flag, p.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // this CTA: rows r0 .. of head `head` of every sequence (group b * heads + head), range `cut` of `cuts`
  const int grp = blockIdx.x / plan.cuts, cut = blockIdx.x % plan.cuts;
  const int head = grp / plan.row_groups, r0 = (grp % plan.row_groups) * NR;
  const int n_rows = min(NR, p.rows - r0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(free_(s), 4);
    }
    for (int w = 0; w < W; ++w) {
      mbar_init(s_done(w), 1);
      mbar_init(o_done(w), 1);
      mbar_init(drain_bar(w), 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 4 * W) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 4 * W - 1) {
    int b0, first, count;
    find_range<BC>(p, plan, cut, b0, first, count);
    if (lane == 0) {
      s_start[0] = b0;
      s_start[1] = first;
      s_start[2] = count;
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

  // walks the pieces, a whole warp at a time: f(sequence, its keys, first tile, tiles, next sequence or -1)
  auto pieces = [&](auto f) {
    int b = start_b, t = start_t, left = n_tiles;
    while (left > 0 && b < plan.n_seq) {
      const int nk = __shfl_sync(0xffffffffu, seq_len(p, b, false), 0);
      const int take = min(left, tiles_of<BC>(nk) - t);
      if (take > 0) {
        left -= take;
        int next = -1;
        if (left > 0) {  // the next sequence with keys
          next = b + 1;
          while (next + 1 < plan.n_seq && seq_len(p, next, false) == 0) ++next;
        }
        if (!f(b, nk, t, take, next)) return;
      }
      ++b;
      t = 0;
    }
  };

  if (warp == 4 * W) {
    // ---------------------------------------------------------------- loads
    // Lane i (of 8) looks block i of a tile up; the first lane of every run of
    // blocks that lie side by side in a page copies the run.
    int g = 0;  // tiles issued
    const int per_page = cache.page_size / 16;
    pieces([&](int b, int nk, int t0, int n, int) -> bool {
      const int blocks = (nk + 15) / 16;
      // this lane's block of a tile: its page as the table has it (-1: past the end), its place there
      auto place = [&](int tile, int& page, int& at) {
        const int i = tile * 8 + lane;
        page = at = -1;
        if (lane >= 8 || i >= blocks) return;
        const int q = i / per_page;
        at = i - q * per_page;
        page = cache.table != nullptr ? cache.table[static_cast<long long>(b) * cache.max_pages + q] : b;
        if (page < 0 || page >= cache.n_pages) page = -2;
      };
      int page, at;
      place(t0, page, at);
      for (int i = 0; i < n; ++i, ++g) {
        int page1 = -1, at1 = -1;
        if (i + 1 < n) place(t0 + i + 1, page1, at1);  // the next tile's pages, while this one loads
        const int slot = g % SLOTS;
        if (g >= SLOTS && !warp_wait(free_(slot), (g / SLOTS - 1) & 1, wc)) return false;
        const bool here = page >= 0;
        if (page == -2) atomicOr(p.status, kStatusInput);
        const unsigned missing = __ballot_sync(0xffffffffu, page == -2);
        const unsigned have = __ballot_sync(0xffffffffu, here);
        const int before = __shfl_up_sync(0xffffffffu, page, 1);
        const bool starts = here && (lane == 0 || before != page || at == 0);
        const unsigned heads = __ballot_sync(0xffffffffu, starts);
        if (lane == 0) {
          s_missing[slot] = static_cast<int>(missing);
          mbar_arrive_expect_tx(full(slot), __popc(have) * 18 * D);
        }
        __syncwarp();
        if (starts) {
          const unsigned ends = (heads | ~have) & (0xfffffffeu << lane);  // never empty: lanes from 8 on have none
          const int run = __ffs(ends) - 1 - lane;
          const long long src = ((static_cast<long long>(page) * cache.Hkv + head) * per_page + at) * (18 * D);
          bulk_load(sRing + slot * C::TILE + lane * 18 * D, cache.cache + src, run * 18 * D, full(slot));
        }
        page = page1;
        at = at1;
      }
      return true;
    });
    if (*abort_flag) {
      // let copies already in flight land before the CTA's shared memory is
      // released; a wait for copies that were never issued just runs out
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      for (int k = max(0, g - SLOTS); k < g; ++k) mbar_wait(full(k % SLOTS), (k / SLOTS) & 1, drain);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------- unpacking, products, softmax
    // Once a wait has run out, waits return at once and the loops run on to
    // their ends (barriers count every warp); nothing is written out then.
    const int w = warp >> 2, quarter = warp & 3, id = threadIdx.x & 127;  // id: a key, then a channel
    const uint32_t tw = tmem + w * C::COLS;                               // this warpgroup's columns
    const uint32_t tl = tw + (static_cast<uint32_t>(quarter * 32) << 16);  // and this warp's lanes
    const uint32_t sP = sb + C::OFF_P + w * C::P_BYTES;
    const Desc2 dq = desc_sw128(sQ, 16, 1024), dp = desc_p<C::RB>(sP);
    constexpr uint32_t idesc_s = idesc_f16(128, NR, 0), idesc_o = idesc_f16(128, NR, 1);
    float* ref = s_ref + w * NR;
    float* fac = s_fac + w * NR;
    float* red = s_red + w * 4 * NR;
    constexpr int RCOLS = NR > 32 ? NR / 32 : 1;  // columns that a lane owns after a reduction
    const int my_col = first_col<NR>();
    auto put = [&](float* dst, const float* v) {  // this warp's column results
#pragma unroll
      for (int i = 0; i < RCOLS; ++i) dst[quarter * NR + my_col + i] = v[i];
    };
    auto wg_sync = [&]() { named_bar_sync(1 + w, 128); };
    auto all_sync = [&]() { named_bar_sync(8, kConsumers); };
    int g = 0, mine = 0;  // tiles of the CTA so far, and of this warpgroup

    // Q rows of a sequence: a warp takes rows warp, warp + 4 W, ...; a lane 4 channels of one
    constexpr int QR = (NR + 4 * W - 1) / (4 * W);
    uint2 qv[QR];
    auto load_q = [&](int b) {
      const long long row0 = (b * plan.heads + head) / p.group_div * p.q_s1 + (b * plan.heads + head) % p.group_div * p.q_s2 + r0;
#pragma unroll
      for (int i = 0; i < QR; ++i) {
        const int r = warp + 4 * W * i;
        qv[i] = make_uint2(0, 0);
        if (r < n_rows && 4 * lane < D)
          qv[i] = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + (row0 + r) * D + 4 * lane);
      }
    };
    auto put_q = [&]() {
#pragma unroll
      for (int i = 0; i < QR; ++i) {
        const int r = warp + 4 * W * i;
        if (r >= NR) break;
        const uint32_t m2 = __vmaxu2(qv[i].x & 0x7fff7fffu, qv[i].y & 0x7fff7fffu);
        const uint32_t amax = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
        // the power of two that brings the row's largest entry to 2^14 .. 2^15 (its
        // exponent field is e; rows below 2^-112 are brought as far as fp32 reaches)
        const int e = amax >> 7;
        const int up = amax == 0 ? 0 : min(141 - e, 126);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        const uint32_t lo = pack_f16x2(__uint_as_float(qv[i].x << 16) * f, __uint_as_float(qv[i].x & 0xffff0000u) * f);
        const uint32_t hi = pack_f16x2(__uint_as_float(qv[i].y << 16) * f, __uint_as_float(qv[i].y & 0xffff0000u) * f);
        if (4 * lane < D) {
          const int ch = 4 * lane, c16 = (ch & 63) >> 3;
          const uint32_t at = sQ + (ch >> 6) * NR * 128 + r * 128 + ((c16 ^ (r & 7)) << 4) + (ch & 4) * 2;
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(lo), "r"(hi) : "memory");
        }
        if (lane == 0)
          s_cs[r] = fmaxf(p.scale * cache.k_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23),
                          1.5e-45f);  // not 0, for the masked scores' sake
      }
      fence_proxy_async_smem();
    };

    bool begun = false;
    pieces([&](int b, int nk, int t0, int n, int next) -> bool {
      const int group = b * plan.heads + head;
      if (!begun) {
        begun = true;
        load_q(b);
        put_q();
        all_sync();
      }
      if (next >= 0) load_q(next);  // lands while this piece goes on
      float l[NR];
#pragma unroll
      for (int c = 0; c < NR; ++c) l[c] = 0.f;
      if (id < NR) ref[id] = kUnset;
      bool any = false;  // this warpgroup has had a tile of the piece
      for (int i = 0; i < n; ++i, ++g) {
        if (g % W != w) continue;
        const int slot = g % SLOTS;
        warp_wait(full(slot), (g / SLOTS) & 1, wc);
        const uint32_t base = sRing + slot * C::TILE;
        const int missing = s_missing[slot];
        const int j0 = (t0 + i) * BC, valid = min(BC, nk - j0);
        // ---- K: a thread a key
        {
          const uint32_t blk = base + (id >> 4) * (18 * D), t = id & 15;
          const bool gone = (missing >> (id >> 4)) & 1;  // no page: zeros
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint2 a = ld_shared_v2(blk + (2 * c) * 128 + t * 8), e = ld_shared_v2(blk + (2 * c + 1) * 128 + t * 8);
            uint32_t sc[2];
            cache4::scales_f16(gone ? 0u : ld_shared_u16(blk + 8 * D + t * GROUPS + 2 * c), sc);
            const uint32_t s0 = __byte_perm(sc[0], 0, 0x1010), s1 = __byte_perm(sc[0], 0, 0x3232);
            uint32_t o[16];
            cache4::codes_f16(a.x, o);
            cache4::codes_f16(a.y, o + 4);
            cache4::codes_f16(e.x, o + 8);
            cache4::codes_f16(e.y, o + 12);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              o[x] = cache4::mul_f16x2(o[x], s0);
              o[8 + x] = cache4::mul_f16x2(o[8 + x], s1);
            }
            tmem_st_32x32b_x16(tl + C::TM_K + 16 * c, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        wg_sync();
        if (quarter == 0) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_w(tw + C::TM_S, tw + C::TM_K + 8 * kk, dq, ((kk >> 2) * NR * 128 + (kk & 3) * 32) >> 4, idesc_s, kk > 0);
          mma_commit_w(s_done(w));
        }
        // ---- V: a thread a channel.  The last product of this warpgroup has read V^T and P.
        if (mine > 0) warp_wait(o_done(w), (mine - 1) & 1, wc);
        tc_fence_after();
        if (quarter * 32 < D) {
          const uint32_t cb = base + 9 * D + id * 8, cs = base + 17 * D + (id >> 4) * 16;
          const int part = valid < BC || missing != 0 ? 0 : BC;  // below: some tokens are to be zeros
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t o[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = 2 * x + h;
              const uint2 a = ld_shared_v2(cb + k * 18 * D);
              const uint4 s4 = ld_shared_v4(cs + k * 18 * D);
              uint32_t sc[8];
              cache4::scales_f16(s4.x, sc);
              cache4::scales_f16(s4.y, sc + 2);
              cache4::scales_f16(s4.z, sc + 4);
              cache4::scales_f16(s4.w, sc + 6);
              if (part == 0) {
                const int room = (missing >> k) & 1 ? 0 : valid - 16 * k;
#pragma unroll
                for (int y = 0; y < 8; ++y)
                  sc[y] &= (2 * y < room ? 0xffffu : 0u) | (2 * y + 1 < room ? 0xffff0000u : 0u);
              }
              cache4::codes_f16(a.x, o + 8 * h);
              cache4::codes_f16(a.y, o + 8 * h + 4);
#pragma unroll
              for (int y = 0; y < 8; ++y) o[8 * h + y] = cache4::mul_f16x2(o[8 * h + y], sc[y]);
            }
            tmem_st_32x32b_x16(tl + C::TM_V + 16 * x, o);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(free_(slot));
        // ---- scores
        warp_wait(s_done(w), mine & 1, wc);
        tc_fence_after();
        float s[NR];
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tl + C::TM_S + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; ++x) s[c + x] = __uint_as_float(r[x]);
        }
        if (j0 + BC > nk - (p.n_new - 1)) {
          const int room = nk - (j0 + id);  // > lag: the row sees this key
#pragma unroll
          for (int c = 0; c < NR; ++c) s[c] = s_lag[c] < room ? s[c] : -INFINITY;
        }
        float over = -INFINITY;
#pragma unroll
        for (int c = 0; c < NR; c += 4) {
          const float4 nr = *reinterpret_cast<const float4*>(ref + c), cs = *reinterpret_cast<const float4*>(s_cs + c);
          over = fmax3(over, fmaf(s[c], cs.x, nr.x), fmaf(s[c + 1], cs.y, nr.y));
          over = fmax3(over, fmaf(s[c + 2], cs.z, nr.z), fmaf(s[c + 3], cs.w, nr.w));
        }
        if (bar_any(1 + w, 128, over > kRescaleThreshold)) {
          // some row's reference rises: column maxima over the 128 keys
          {
            float v[NR];
#pragma unroll
            for (int c = 0; c < NR; ++c) v[c] = s[c] * s_cs[c];
            reduce_step<NR / 2, 16>(v, [](float x, float y) { return fmaxf(x, y); });
            put(red, v);
          }
          wg_sync();
          if (id < NR) {
            const float mx = fmaxf(fmaxf(red[id], red[NR + id]), fmaxf(red[2 * NR + id], red[3 * NR + id]));
            const float old = ref[id];
            float alpha = 1.f;
            if (mx + old > kRescaleThreshold) {  // old = kUnset: the first key that the row sees
              alpha = old == kUnset ? 0.f : ex2_approx(-old - mx);
              ref[id] = -mx;
            }
            fac[id] = alpha;
          }
          wg_sync();
#pragma unroll
          for (int c = 0; c < NR; ++c) l[c] *= fac[c];
          if (any) {
#pragma unroll 1
            for (int c = 0; c < NR; c += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(tl + C::TM_O + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fac[c + x]);
              tmem_st_32x32b_x16(tl + C::TM_O + c, o);
            }
          }
        }
        // ---- P
#pragma unroll
        for (int c = 0; c < NR; c += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            const float4 nr = *reinterpret_cast<const float4*>(ref + c + x);
            const float4 cs = *reinterpret_cast<const float4*>(s_cs + c + x);
            const float p0 = ex2_approx(fmaf(s[c + x], cs.x, nr.x)), p1 = ex2_approx(fmaf(s[c + x + 1], cs.y, nr.y));
            const float p2 = ex2_approx(fmaf(s[c + x + 2], cs.z, nr.z)), p3 = ex2_approx(fmaf(s[c + x + 3], cs.w, nr.w));
            l[c + x] += p0;
            l[c + x + 1] += p1;
            l[c + x + 2] += p2;
            l[c + x + 3] += p3;
            // P is rounded to fp16, the products' type: half a step of 2^-11 each
            pk[x / 2] = pack_f16x2(p0, p1);
            pk[x / 2 + 1] = pack_f16x2(p2, p3);
          }
          st_shared_v4(sP + id * C::RB + p_chunk<C::RB>(id, c / 8) * 16, pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        tmem_wait_st();
        tc_fence_before();
        wg_sync();
        if (quarter == 0) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BC / 16; ++kk)
            mma_ts_w(tw + C::TM_O, tw + C::TM_V + 8 * kk, dp, (kk * 16 * C::RB) >> 4, idesc_o, any || kk > 0);
          mma_commit_w(o_done(w));
        }
        any = true;
        ++mine;
      }
      // ------------------------------------------------------------ output
      if (any) warp_wait(o_done(w), (mine - 1) & 1, wc);
      tc_fence_after();
      reduce_step<NR / 2, 16>(l, [](float x, float y) { return x + y; });
      put(red, l);
      wg_sync();
      if (id < NR) s_sum[w * NR + id] = (red[id] + red[NR + id]) + (red[2 * NR + id] + red[3 * NR + id]);
      tc_fence_before();
      all_sync();
      tc_fence_after();
      const bool whole = t0 == 0 && n == tiles_of<BC>(nk);
      const long long slot = static_cast<long long>(grp) * (plan.cuts + plan.n_seq) + cut + b;
      const long long orow0 = (group / p.group_div) * p.q_s1 + (group % p.group_div) * p.q_s2 + r0;
      if (threadIdx.x < NR) {  // the warpgroups' O share one reference: the largest
        const int c = threadIdx.x;
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int y = 0; y < W; ++y)
          if (s_ref[y * NR + c] != kUnset) m = fmaxf(m, -s_ref[y * NR + c]);
        float f[W];
#pragma unroll
        for (int y = 0; y < W; ++y) {
          f[y] = s_ref[y * NR + c] == kUnset ? 0.f : ex2_approx(-s_ref[y * NR + c] - m);
          sum += f[y] == 0.f ? 0.f : f[y] * s_sum[y * NR + c];
        }
        const float inv = sum == 0.f ? 0.f : cache.v_scale / sum;
#pragma unroll
        for (int y = 0; y < W; ++y) s_fac[y * NR + c] = f[y] * inv;
        const float lse = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994531f;
        if (c < n_rows && !*abort_flag) {
          if (!whole)
            p.part_lse[slot * NR + c] = lse;
          else if (p.lse != nullptr)
            p.lse[orow0 + c] = lse;
        }
      }
      if (next >= 0) put_q();  // every product with this piece's Q has completed
      all_sync();
#pragma unroll 1
      for (int c = 8 * w; c < n_rows; c += 8 * W) {
        float acc[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] = 0.f;
#pragma unroll
        for (int y = 0; y < W; ++y) {
          __syncwarp();
          if (n < W && (g - 1 - y + W * (n + W)) % W >= n) continue;  // warpgroup y had no tile
          uint32_t o[8];
          tmem_ld_32x32b_x8(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + y * C::COLS + C::TM_O + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float f = s_fac[y * NR + c + x];
            if (f != 0.f) acc[x] = fmaf(__uint_as_float(o[x]), f, acc[x]);
          }
        }
        if (id >= D || *abort_flag) continue;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (c + x >= n_rows) break;
          if (whole)
            static_cast<__nv_bfloat16*>(p.o)[(orow0 + c + x) * D + id] = __float2bfloat16_rn(acc[x]);
          else
            p.part_o[(slot * NR + c + x) * D + id] = acc[x];
        }
      }
      tc_fence_before();
      all_sync();  // statistics and accumulators are free for the next piece
      return true;
    });
    // every product this warp issued must finish before tensor memory is freed
    if (quarter == 0) {
      mma_commit_w(drain_bar(w));
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      mbar_wait(drain_bar(w), 0, drain);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4 * W) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int NR>
cudaError_t launch_nr(const SeqAttn& p, const Cache4& c, const DecodePlan& plan, cudaStream_t s) {
  using C = Cfg<D, NR>;
  static SmemOnce once;
  const cudaError_t e = once(fa_cache4_decode_kernel<D, NR>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(plan.heads) * plan.row_groups * plan.cuts;
  fa_cache4_decode_kernel<D, NR><<<grid, C::THREADS, C::SMEM_BYTES, s>>>(p, c, plan);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const SeqAttn& p, const Cache4& c, const DecodePlan& w, cudaStream_t s) {
  return w.nr == 16 ? launch_nr<D, 16>(p, c, w, s) : w.nr == 32 ? launch_nr<D, 32>(p, c, w, s) : launch_nr<D, 64>(p, c, w, s);
}

}  // namespace

DecodePlan cache4_plan(int n_seq, int heads, int rows, int sms) {
  DecodePlan w{};
  w.n_seq = n_seq;
  w.heads = heads;
  w.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  w.row_groups = (rows + w.nr - 1) / w.nr;
  const long long groups = static_cast<long long>(heads) * w.row_groups;
  w.cuts = groups < sms ? static_cast<int>(sms / groups) : 1;  // a CTA an SM
  w.direct = 1;
  return w;
}

cudaError_t launch_cache4_decode(const SeqAttn& p, const Cache4& c, const DecodePlan& w, cudaStream_t s) {
  if (static_cast<long long>(w.heads) * w.row_groups * w.cuts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // tile counts are summed, and multiplied by the number of cuts, in 32 bits
  if (static_cast<long long>(w.n_seq) * tiles_of<BC>(p.n_keys) * (w.cuts + 1LL) > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  if (c.d == 64) return launch_d<64>(p, c, w, s);
  if (c.d == 96) return launch_d<96>(p, c, w, s);
  if (c.d == 128) return launch_d<128>(p, c, w, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache4_merge(const SeqAttn& p, const DecodePlan& w, cudaStream_t s) {
  if (w.nr == 16) return launch_merge<BC, 16>(p, w, nullptr, nullptr, 0, true, s);
  if (w.nr == 32) return launch_merge<BC, 32>(p, w, nullptr, nullptr, 0, true, s);
  return launch_merge<BC, 64>(p, w, nullptr, nullptr, 0, true, s);
}

}  // namespace fa
