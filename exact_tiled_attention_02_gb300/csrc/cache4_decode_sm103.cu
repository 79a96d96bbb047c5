// cache4_decode_sm103.cu -- attention of few query rows over the 4-bit key/value
// cache, bf16 or float32 in / fp32 accumulate, on the tensor cores of GB300
// (sm_103a).
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
// W teams of eight warps, each with a range of the tiles, a ring, operands,
// scores and an O in tensor memory of its own: they share nothing, so that
// one's waits (products, the end of a sequence) overlap another's unpacking.  Of
// a team half unpacks K, a thread a key, half V, a thread a channel; the first
// takes the softmax, or both a half of the columns where there are more than 16.
// One more warp issues all products, told by mbarriers, so that the warps of a
// team do not wait for one another around them.
//
// Statistics run down the columns, across lanes.  Per tile a thread (one key)
// only checks whether any P of it would exceed 2^15, that is whether a score is
// 15 above its column's reference (log2 domain), 8 above the score that set it;
// if no key's is (one barrier with an OR) the tile is exponentiated as it is.
// Otherwise the column maxima are reduced across lanes and warps and O rescaled.
//
// A warp a team loads: a tile's blocks, one bulk copy for each run of them in a
// page.  (One warp for all teams waited for each tile's pages before it turned to
// the next team; with pages of 16 tokens, where every tile's entries are in a
// sector of their own, 64 sequences of 500 to 8200 took 79 us for 64 now.)  The
// work is split as seq_ranges.cuh says, a range a team; a sequence that is one
// whole piece goes straight to o.
//
// Unpacking costs two instructions a pair of codes (a conversion and a product, in
// pipes that take 2.6 cycles for both), 330 cycles a tile of d = 128 for the 830
// that its 18 KB take at the copy rate; at 4 rows the whole tile is 640
// instructions a scheduler.  64 sequences of 4096 to 32768 tokens, 32 / 8 heads,
// d = 128: 216 us, 6.3 TB/s (93% of the copy rate).  500 to 8200 tokens: 66 us, 7
// of them before its first tile has come (length, page, tile: three dependent
// loads), after its last, and for the merge.  With 32 rows two teams fit tensor
// memory instead of three, and the softmax's instructions come to 300 a tile more:
// 32 sequences, 64 / 8 heads x 4 tokens, 1000 to 16384: 99 us.  (S^T in columns of
// V^T made room for three teams, whose S^T then waited for the last O^T: 107 for
// 96.)  512 tokens, 64 rows a group: 125 us, 565 TFLOP/s, two thirds of the issue
// slots.
#include <cmath>
#include <type_traits>

#include "cache4.cuh"
#include "seq_ranges.cuh"

namespace fa {
namespace {

using namespace seq;

constexpr int BC = 128;  // keys per tile
// A row's reference is 7 (log2 domain: a factor 2^7) below the largest score when
// it was set, and rises once a score is 8 above that one: P is at most 2^15, and
// fp16's smallest half step, 2^-25, at most 2^-32 of the largest P.
constexpr float kBelow = 7.0f, kRescaleThreshold = kBelow + 8.0f;

// F32: float32 q and o.  Q is then three fp16 terms and P two, 2^-33 and 2^-22
// relative, which the products take one after the other, the smallest first.  A
// product that adds to what an accumulator holds drops bits of it, to the same
// side each time, so O^T is of one tile only, and the tiles are added up in
// registers (6 x 32 heads x 3 tokens, up to 3001 tokens, d = 96: 4e-7 of O,
// 1.1e-6 with O^T kept on and the largest terms first; float32 sums 6.6e-7).
template <int D, int NR, int NA, bool F32>
struct Cfg {
  static constexpr int QT = F32 ? 3 : 1, PT = F32 ? 2 : 1;
  static constexpr int KC = D / 2;                   // columns of K in tensor memory, then 64 of V^T, S^T, O^T
  static constexpr int COLS = KC + 64 + 2 * NR;      // of a team
  static constexpr int W = 512 / COLS < 3 ? 512 / COLS : 3;
  // Query rows in use: NA of the product's NR columns (16 is the narrowest; what
  // stands in the others reaches no row).  Past 16 both halves of a team take
  // half of the softmax, else the half that unpacks K takes all of it.
  static constexpr bool SPLIT = NR > 16;
  static constexpr int NH = SPLIT ? NR / 2 : NA;     // columns of a thread
  static constexpr int THREADS = W * 256 + 32 + W * 32;
  static constexpr int QC = (D + 63) / 64;           // 64-channel chunks of Q
  static constexpr int RB = NR * 2;                  // bytes of a key's row of P
  static constexpr int TILE = 144 * D;               // bytes: 8 blocks of 18 D
  static constexpr int Q_BYTES = QC * NR * 128;      // a term
  static constexpr int P_BYTES = 128 * RB;           // a term of a team
  static constexpr int VS_BYTES = W * 4 * 512;       // a warp's value scales in fp16: [2 groups][128 keys]
  static constexpr int STATS = 4 * NR * 4                  // a team: lag, column scale, reference, factor
                               + 4 * NR * 4;               // and warps' column results
  static constexpr int MISC = VS_BYTES + W * STATS + 512;
  static constexpr int FIT = (227 * 1024 - 1024 - W * (QT * Q_BYTES + PT * P_BYTES) - MISC) / TILE / W;
  static constexpr int SL = FIT < 4 ? FIT : 4;             // ring slots of a team
  static constexpr int SLOTS = W * SL;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + W * QT * Q_BYTES;
  static constexpr int OFF_RING = OFF_P + W * PT * P_BYTES;
  static constexpr int OFF_VS = OFF_RING + SLOTS * TILE;
  static constexpr int OFF_STAT = OFF_VS + VS_BYTES;
  static constexpr int OFF_BAR = OFF_STAT + W * STATS;
  static constexpr int NBAR = 2 * SLOTS + 4 * W + 1;
  // tensor memory base, abort flag; where the teams begin (6 words each), first-tile flags; slots' missing blocks
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_USED = OFF_MISC + 8 + W * 28 + SLOTS * 4;
  static constexpr int SMEM_BYTES = SMEM_USED + 1024;
  static constexpr int TM_K = 0, TM_V = KC, TM_S = KC + 64, TM_O = TM_S + NR;
  static_assert(W >= 2 && SL >= 2, "two tiles a team in flight");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0 && OFF_RING % 1024 == 0 && TILE % 16 == 0, "alignment");
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
// The N scales (4, 6 or 8) of a key, the first in the lowest byte.
template <int N>
__device__ __forceinline__ uint2 ld_scales(uint32_t addr) {
  uint2 v = make_uint2(0, 0);
  if constexpr (N == 8) {
    v = ld_shared_v2(addr);
  } else if constexpr (N == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.x) : "r"(addr) : "memory");
  } else {
    asm volatile("{\n.reg .b16 a, b, c;\nld.shared.b16 a, [%2];\nld.shared.b16 b, [%2+2];\nld.shared.b16 c, [%2+4];\n"
                 "mov.b32 %0, {a, b};\ncvt.u32.u16 %1, c;\n}"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(addr)
                 : "memory");
  }
  return v;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_ld_x4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four or two products in a row, K steps of 16: A steps 8 columns, B's start STEP
// units of 16 bytes.  One election for all of them: the issuing warp shares its
// scheduler with a quarter of the others.
template <int N, int STEP>
__device__ __forceinline__ void mma_ts_steps(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                             uint32_t acc) {
  static_assert(N == 2 || N == 4, "steps");
  if constexpr (N == 4)
    asm volatile(
        "{\n.reg .pred p, q, e;\n.reg .b64 b0, b1, b2, b3;\n.reg .b32 x;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, %5, %5;\n"
        "mov.b64 b0, {%2, %3};\n"
        "add.u32 x, %2, %6;\nmov.b64 b1, {x, %3};\n"
        "add.u32 x, %2, %7;\nmov.b64 b2, {x, %3};\n"
        "add.u32 x, %2, %8;\nmov.b64 b3, {x, %3};\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 8], b1, %4, q;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 16], b2, %4, q;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 24], b3, %4, q;\n}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p, q, e;\n.reg .b64 b0, b1;\n.reg .b32 x;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %5, 0;\nsetp.eq.b32 q, %5, %5;\n"
        "mov.b64 b0, {%2, %3};\n"
        "add.u32 x, %2, %6;\nmov.b64 b1, {x, %3};\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 8], b1, %4, q;\n}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "n"(STEP)
        : "memory");
}

// A whole warp's wait.  The first try is where the warp goes on at once; what
// follows is kept out of line, and out of the instruction cache.
__device__ __noinline__ void wait_longer(uint32_t bar, uint32_t parity, unsigned int* status, volatile int* abort_flag,
                                         unsigned long long limit_ns) {
  mbar_wait(bar, parity, WaitCtl{status, abort_flag, limit_ns});
}
__device__ __forceinline__ void wait_for(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (!mbar_try_wait(bar, parity)) wait_longer(bar, parity, w.status, w.abort_flag, w.limit_ns);
  __syncwarp();
}

template <int D, int NR, int NA, bool F32>
__global__ void __launch_bounds__(Cfg<D, NR, NA, F32>::THREADS, 1)
    fa_cache4_decode_kernel(const __grid_constant__ SeqAttn p, const __grid_constant__ Cache4 cache,
                            const DecodePlan plan) {
  using C = Cfg<D, NR, NA, F32>;
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int W = C::W, SLOTS = C::SLOTS, GROUPS = D / 16, NH = C::NH;
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
  const uint32_t bars = sb + C::OFF_BAR;
  auto full = [&](int s) { return bars + 8 * s; };
  auto free_ = [&](int s) { return bars + 8 * (SLOTS + s); };
  auto k_ready = [&](int w) { return bars + 8 * (2 * SLOTS + w); };
  auto s_done = [&](int w) { return bars + 8 * (2 * SLOTS + W + w); };
  auto p_ready = [&](int w) { return bars + 8 * (2 * SLOTS + 2 * W + w); };
  auto o_done = [&](int w) { return bars + 8 * (2 * SLOTS + 3 * W + w); };
  const uint32_t drain_bar = bars + 8 * (2 * SLOTS + 4 * W);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);    // [W][6] a team's first head, row group, sequence and tile, its tiles, range
  volatile int* s_first = reinterpret_cast<volatile int*>(s_start + 6 * W);  // [W] a team's tile is its first of a piece
  volatile int* s_missing = s_first + W;                                     // [SLOTS] blocks without a page
  const WaitCtl wc{p.status, abort_flag, p.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // A group of rows is rows NR rg .. of key/value head `head`.
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(free_(s), 8);
    }
    for (int w = 0; w < W; ++w) {
      mbar_init(k_ready(w), C::SPLIT ? 8 : 4);
      mbar_init(s_done(w), 1);
      mbar_init(p_ready(w), 8);
      mbar_init(o_done(w), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8 * W) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp < 8 * W && (warp & 7) == 0) {
    // (teams in the order of the ranges: few tiles spread over the SMs)
    const int r = (warp >> 3) * gridDim.x + blockIdx.x;
    int grp, b0, first, count;
    find_flat<BC>(p, plan, r, grp, b0, first, count);
    if (lane == 0) {
      int* at = s_start + 6 * (warp >> 3);
      at[0] = grp / plan.row_groups;
      at[1] = grp % plan.row_groups;
      at[2] = b0;
      at[3] = first;
      at[4] = count;
      at[5] = r;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Steps to the next sequence with keys, of the next group of rows past the
  // last one; its keys.
  auto next_seq = [&](int& head, int& rg, int& b) -> int {
    for (int i = 0; i < plan.n_seq; ++i) {
      if (++b == plan.n_seq) {
        b = 0;
        if (++rg == plan.row_groups) {
          rg = 0;
          ++head;
        }
      }
      const int n = seq_len(p, b, false);
      if (n > 0) return n;
    }
    return 0;
  };

  if (warp > 8 * W) {
    // ---------------------------------------------------------------- loads
    // A warp a team: lane i (of 8) looks block i of a tile up, and the first lane
    // of every run of blocks that lie side by side in a page copies the run.
    const int w = warp - 8 * W - 1;
    const int per_page = cache.page_size / 16;
    const int* start = s_start + 6 * w;  // the next tile's head, row group, sequence and place there; tiles to go
    int head = start[0], rg = start[1], b = start[2], t = start[3], left = start[4];
    int n = left > 0 ? seq_len(p, b, false) : 0;  // keys of sequence b
    int page = -1, at = -1;  // of this lane's block: -1 past the end, -2 no such page
    auto place = [&]() {
      const int blk = t * 8 + lane;
      page = at = -1;
      if (left <= 0 || lane >= 8 || blk * 16 >= n) return;
      const int q = blk / per_page;
      at = blk - q * per_page;
      page = cache.table != nullptr ? cache.table[static_cast<long long>(b) * cache.max_pages + q] : b;
      if (page < 0 || page >= cache.n_pages) page = -2;
    };
    place();
    int slot = w * C::SL, used = 0;  // the next ring slot, tiles issued
    uint32_t par = 1;                // of the slot's release: the first round waits for none
    while (left > 0) {
      if (!warp_wait(free_(slot), par, wc)) break;
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
      --left;
      ++used;
      if (++slot == (w + 1) * C::SL) {
        slot = w * C::SL;
        par ^= 1;
      }
      if (++t * BC >= n) {  // the next sequence with keys
        t = 0;
        n = left > 0 ? next_seq(head, rg, b) : 0;
      }
      place();  // the next tile's pages, while this one loads
      __syncwarp();
    }
    if (*abort_flag && lane == 0) {
      // let copies already in flight land before the CTA's shared memory is
      // released; a wait for copies that were never issued just runs out
      WaitCtl drain{nullptr, nullptr, wc.limit_ns};
      for (int k = max(0, used - C::SL); k < used; ++k) mbar_wait(full(w * C::SL + k % C::SL), (k / C::SL) & 1, drain);
    }
    __syncwarp();
  } else if (warp == 8 * W) {
    // ------------------------------------------------------------- products
    // The whole warp runs it, converged (see mma_ts_w): S^T of a team's tile
    // once its K is in place, O^T once its V^T and P are, whichever is ready.
    constexpr uint32_t idesc_s = idesc_f16(128, NR, 0), idesc_o = idesc_f16(128, NR, 1);
    const Desc2 dq = desc_sw128(sQ, 16, 1024), dp = desc_p<C::RB>(sb + C::OFF_P);
    int left = 0;  // products to issue
#pragma unroll
    for (int w = 0; w < W; ++w) left += 2 * __shfl_sync(0xffffffffu, s_start[6 * w + 4], 0);
    // lane l < W looks for K of team l, lane W + l for its P
    const uint32_t my_bar = lane < W ? k_ready(lane) : p_ready(lane < 2 * W ? lane - W : 0);
    uint32_t par = 0;
    unsigned long long since = 0;
    while (left > 0) {
      uint32_t ok;
      asm volatile(
          "{\n.reg .pred p;\n"
          "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
          "selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(ok)
          : "r"(my_bar), "r"(par)
          : "memory");
      const unsigned ready = __ballot_sync(0xffffffffu, lane < 2 * W && ok != 0);
      const bool moved = ready != 0;
      if (ready >> lane & 1) par ^= 1;
      left -= __popc(ready);
      if (moved) tc_fence_after();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t tw = tmem + w * C::COLS;
        if (ready >> w & 1) {
#pragma unroll
          for (int t = 0; t < C::QT; ++t)
#pragma unroll
            for (int c = 0; c < C::QC; ++c) {  // 64 channels, or what is left of them
              constexpr int LAST = D / 16 - (C::QC - 1) * 4;
              const uint32_t at = dq.lo + (((w * C::QT + C::QT - 1 - t) * C::Q_BYTES + c * NR * 128) >> 4);
              if (c < C::QC - 1)
                mma_ts_steps<4, 2>(tw + C::TM_S, tw + C::TM_K + 32 * c, at, dq.hi, idesc_s, t > 0 || c > 0);
              else
                mma_ts_steps<LAST, 2>(tw + C::TM_S, tw + C::TM_K + 32 * c, at, dq.hi, idesc_s, t > 0 || c > 0);
            }
          mma_commit_w(s_done(w));
        }
        if (ready >> (W + w) & 1) {
          const uint32_t more = !F32 && s_first[w] == 0;
#pragma unroll
          for (int t = 0; t < C::PT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              mma_ts_steps<4, C::RB>(tw + C::TM_O, tw + C::TM_V + 32 * c,
                                     dp.lo + (((w * C::PT + C::PT - 1 - t) * C::P_BYTES + c * 64 * C::RB) >> 4), dp.hi, idesc_o,
                                     t > 0 || c > 0 ? 1u : more);
          mma_commit_w(o_done(w));
        }
      }
      if (moved) {
        since = 0;
      } else if (since == 0) {
        since = globaltimer_ns();
      } else {
        // no team has moved: the wait is bounded like every other
        const bool late = __any_sync(0xffffffffu, globaltimer_ns() - since > wc.limit_ns);
        if (late) record_timeout(wc);
        if (__any_sync(0xffffffffu, late || *abort_flag != 0)) break;
      }
    }
    // every product must finish before tensor memory is freed
    mma_commit_w(drain_bar);
    WaitCtl drain{nullptr, nullptr, wc.limit_ns};
    mbar_wait(drain_bar, 0, drain);
    __syncwarp();
  } else {
    // ----------------------------------------------------- unpacking, softmax
    // Once a wait has run out, waits return at once and the loops run on to
    // their ends (barriers count every warp); nothing is written out then.
    const int w = warp >> 3, quarter = warp & 3;
    const bool keys = (warp & 4) == 0;     // this half of the team unpacks K, the other V
    const bool rows = keys || C::SPLIT;    // and has columns of the softmax
    const int id = threadIdx.x & 127;      // a key, or a channel
    const uint32_t tl = tmem + w * C::COLS + (static_cast<uint32_t>(quarter * 32) << 16);  // this team's columns, this warp's lanes
    const uint32_t sP = sb + C::OFF_P + w * C::PT * C::P_BYTES;
    const uint32_t sVS = sb + C::OFF_VS + (w * 4 + quarter) * 512;
    const int c0 = C::SPLIT && !keys ? NH : 0;  // this thread's columns: c0 .. c0 + NH - 1
    int* lag = reinterpret_cast<int*>(smem + C::OFF_STAT + w * C::STATS);  // [NR]
    float* cscale = reinterpret_cast<float*>(lag + NR);  // [NR] log2-domain scale of a column
    float* ref = cscale + NR;                            // [NR] negated reference
    float* fac = ref + NR;                               // [NR] alpha, then 1 / sum
    float* red = fac + NR;                               // [4][NR] warps' column results
    constexpr int kRows = C::SPLIT ? 256 : 128;   // threads of a team with columns
    constexpr int RCOLS = NH > 32 ? NH / 32 : 1;  // columns that a lane owns after a reduction
    const int my_col = c0 + first_col<NH>();
    const int tid = threadIdx.x & 255;  // within the team
    auto rows_sync = [&]() { named_bar_sync(1 + w, kRows); };
    int mine = 0, slot = w * C::SL;  // tiles so far, the next ring slot
    uint32_t phase = 0;

    // Q rows of a sequence: a warp with columns takes every QW-th; a lane 4 channels of one
    constexpr int QW = kRows / 32, QR = (NA + QW - 1) / QW;
    const int qwarp = warp & (QW - 1);
    using Four = typename std::conditional<F32, uint4, uint2>::type;
    Four qv[QR];
    auto row_of = [&](int head, int rg, int b) {  // the group's first row of q, o and lse
      return b * p.q_s1 + head * p.q_s2 + rg * NR;
    };
    auto load_q = [&](int head, int rg, int b) {
      const long long row0 = row_of(head, rg, b);
      const int n_rows = min(NR, p.rows - rg * NR);
#pragma unroll
      for (int i = 0; i < QR; ++i) {
        const int r = qwarp + QW * i;
        qv[i] = Four{};
        if (r < n_rows && 4 * lane < D)
          qv[i] = *reinterpret_cast<const Four*>(static_cast<const T*>(p.q) + (row0 + r) * D + 4 * lane);
      }
    };
    auto put_q = [&]() {
#pragma unroll
      for (int i = 0; i < QR; ++i) {
        const int r = qwarp + QW * i;
        if (r >= NA) break;
        float x[4];
        if constexpr (F32) {
          x[0] = __uint_as_float(qv[i].x), x[1] = __uint_as_float(qv[i].y);
          x[2] = __uint_as_float(qv[i].z), x[3] = __uint_as_float(qv[i].w);
        } else {
          x[0] = __uint_as_float(qv[i].x << 16), x[1] = __uint_as_float(qv[i].x & 0xffff0000u);
          x[2] = __uint_as_float(qv[i].y << 16), x[3] = __uint_as_float(qv[i].y & 0xffff0000u);
        }
        const uint32_t amax = __reduce_max_sync(
            0xffffffffu, __float_as_uint(fmaxf(fmax3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), fabsf(x[3]))));
        // the power of two that brings the row's largest entry to 2^14 .. 2^15 (its
        // exponent field is e; rows below 2^-112 are brought as far as fp32 reaches)
        const int e = amax >> 23;
        const int up = amax == 0 ? 0 : min(141 - e, 126);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] *= f;
        const int ch = 4 * lane, c16 = (ch & 63) >> 3;
        const uint32_t at = sQ + w * C::QT * C::Q_BYTES + (ch >> 6) * NR * 128 + r * 128 + ((c16 ^ (r & 7)) << 4) + (ch & 4) * 2;
#pragma unroll
        for (int t = 0; t < C::QT; ++t) {
          const uint32_t lo = pack_f16x2(x[0], x[1]), hi = pack_f16x2(x[2], x[3]);
          if (ch < D) st_shared_v2(at + t * C::Q_BYTES, lo, hi);
          const float2 a = cache4::floats(lo), b = cache4::floats(hi);
          x[0] -= a.x, x[1] -= a.y, x[2] -= b.x, x[3] -= b.y;
        }
        if (lane == 0)
          cscale[r] = fmaxf(p.scale * cache.k_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23),
                          1.5e-45f);  // not 0, for the masked scores' sake
      }
      fence_proxy_async_smem();
    };

    auto next_slot = [&]() {
      if (++slot == (w + 1) * C::SL) {
        slot = w * C::SL;
        phase ^= 1;
      }
    };
    // K of the next tile, a thread a key: S^T of the tile before must have read
    // the last one, and this thread have its scores
    auto unpack_k = [&]() {
      wait_for(full(slot), phase, wc);
      const uint32_t t = id & 15, blk = sRing + slot * C::TILE + (id >> 4) * (18 * D);
      const bool gone = (s_missing[slot] >> (id >> 4)) & 1;  // no page: zeros
      const uint32_t sa = blk + 8 * D + t * GROUPS, ka = blk + t * 8;
      uint2 code[GROUPS];
      uint2 s8 = ld_scales<GROUPS>(sa);
      if (gone) s8 = make_uint2(0, 0);
#pragma unroll
      for (int c = 0; c < GROUPS; ++c) code[c] = ld_shared_v2(ka + c * 128);
      uint32_t sc[4];
      cache4::scales_f16(s8.x, sc);
      if (GROUPS > 4) cache4::scales_f16(s8.y, sc + 2);
#pragma unroll
      for (int c = 0; c < GROUPS; c += 2) {
        const uint32_t s0 = __byte_perm(sc[c / 2], 0, 0x1010), s1 = __byte_perm(sc[c / 2], 0, 0x3232);
        uint32_t o[16];
        cache4::codes_f16(code[c].x, o);
        cache4::codes_f16(code[c].y, o + 4);
        cache4::codes_f16(code[c + 1].x, o + 8);
        cache4::codes_f16(code[c + 1].y, o + 12);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          o[x] = cache4::mul_f16x2(o[x], s0);
          o[8 + x] = cache4::mul_f16x2(o[8 + x], s1);
        }
        tmem_st_32x32b_x16(tl + C::TM_K + 8 * c, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_ready(w));
        mbar_arrive(free_(slot));
      }
      next_slot();
    };
    const int* start = s_start + 6 * w;
    int head = __shfl_sync(0xffffffffu, start[0], 0), rg = __shfl_sync(0xffffffffu, start[1], 0);
    int b = __shfl_sync(0xffffffffu, start[2], 0), t0 = __shfl_sync(0xffffffffu, start[3], 0);
    int left = __shfl_sync(0xffffffffu, start[4], 0), lag_of = -1;  // the row group that lag[] is of
    const int range = __shfl_sync(0xffffffffu, start[5], 0);
    int nk = left > 0 ? __shfl_sync(0xffffffffu, seq_len(p, b, false), 0) : 0;
    if (rows && left > 0) load_q(head, rg, b);
    // a piece at a time: tiles t0 .. t0 + n - 1 of sequence b
    while (left > 0) {
      const int n = min(left, tiles_of<BC>(nk) - t0);
      left -= n;
      int next_head = head, next_rg = rg, next = b, next_nk = 0;
      if (left > 0) next_nk = __shfl_sync(0xffffffffu, next_seq(next_head, next_rg, next), 0);
      if (next_nk == 0) left = 0;
      const int n_rows = min(NR, p.rows - rg * NR);
      const int all_seen = nk - (p.n_new - 1);  // keys that every row sees
      float l[NH];
#pragma unroll
      for (int c = 0; c < NH; ++c) l[c] = 0.f;
      float acc[F32 ? NH : 1];  // float32: O of the tiles so far, this thread's channel
#pragma unroll
      for (int c = 0; c < (F32 ? NH : 1); ++c) acc[c] = 0.f;
      auto add_tile = [&]() {
        if constexpr (F32) {
          uint32_t o[NH];
          if constexpr (NH == 4)
            tmem_ld_x4(tl + C::TM_O, o);
          else
            tmem_ld<NH>(tl + C::TM_O + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NH; ++c) acc[c] += __uint_as_float(o[c]);
        }
      };
      if (rows) {
        put_q();  // every product with the last piece's Q has completed
        if (left > 0) load_q(next_head, next_rg, next);  // lands while this piece goes on
        if (tid < NA) {
          ref[tid] = 0.f;  // set by the piece's first tile
          if (rg != lag_of) lag[tid] = p.n_new - 1 - (rg * NR + tid) % p.n_new;
        }
        rows_sync();
        if (keys)
          unpack_k();
        else if (lane == 0)
          mbar_arrive(k_ready(w));  // (split: this half has read the last scores, and its rows of Q are in place)
      }
      for (int i = 0; i < n; ++i) {
        const int j0 = (t0 + i) * BC;
        if (keys) {
        } else if (quarter * 32 >= D) {
          if (mine > 0) wait_for(o_done(w), (mine - 1) & 1, wc);  // arrive for this tile, not for the last one
        } else {
          // ---- V: a thread a channel.  First the scales of the warp's two groups,
          // zeros past the sequence's end and in missing pages.
          wait_for(full(slot), phase, wc);
          const uint32_t base = sRing + slot * C::TILE;
          const int missing = s_missing[slot], valid = min(BC, nk - j0);
          {
            const int k = (lane & 15) >> 1, t = (lane & 1) * 8;  // block, first of eight keys
            uint32_t sc[4];
            const uint2 s8 = ld_shared_v2(base + k * 18 * D + 17 * D + (2 * quarter + (lane >> 4)) * 16 + t);
            cache4::scales_f16(s8.x, sc);
            cache4::scales_f16(s8.y, sc + 2);
            if (valid < BC || missing != 0) {
              const int room = (missing >> k) & 1 ? 0 : valid - 16 * k - t;
#pragma unroll
              for (int y = 0; y < 4; ++y)
                sc[y] &= (2 * y < room ? 0xffffu : 0u) | (2 * y + 1 < room ? 0xffff0000u : 0u);
            }
            st_shared_v4(sVS + lane * 16, sc[0], sc[1], sc[2], sc[3]);
          }
          const uint32_t cb = base + 9 * D + id * 8, cs = sVS + (lane >> 4) * 256;
          uint2 code[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) code[k] = ld_shared_v2(cb + k * 18 * D);
          __syncwarp();
          // the last product of this team has read V^T
          if (mine > 0) wait_for(o_done(w), (mine - 1) & 1, wc);
          tc_fence_after();
          uint4 sa = ld_shared_v4(cs), se = ld_shared_v4(cs + 16);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t o[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = 2 * x + h;
              uint32_t* y = o + 8 * h;
              cache4::codes_f16(code[k].x, y);
              cache4::codes_f16(code[k].y, y + 4);
              y[0] = cache4::mul_f16x2(y[0], sa.x);
              y[1] = cache4::mul_f16x2(y[1], sa.y);
              y[2] = cache4::mul_f16x2(y[2], sa.z);
              y[3] = cache4::mul_f16x2(y[3], sa.w);
              y[4] = cache4::mul_f16x2(y[4], se.x);
              y[5] = cache4::mul_f16x2(y[5], se.y);
              y[6] = cache4::mul_f16x2(y[6], se.z);
              y[7] = cache4::mul_f16x2(y[7], se.w);
              if (k < 7) {
                sa = ld_shared_v4(cs + (k + 1) * 32);
                se = ld_shared_v4(cs + (k + 1) * 32 + 16);
              }
            }
            tmem_st_32x32b_x16(tl + C::TM_V + 16 * x, o);
          }
        }
        if (!keys) {
          if (!C::SPLIT) {
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(free_(slot));
            if (!C::SPLIT) mbar_arrive(p_ready(w));
          }
          next_slot();
        }
        if (rows) {
          // ---- scores, in the log2 domain and against the row's reference
          wait_for(s_done(w), mine & 1, wc);
          tc_fence_after();
          float x[NH];
          {
            uint32_t r[NH];
            if constexpr (NH == 4)
              tmem_ld_x4(tl + C::TM_S, r);
            else
              tmem_ld<NH>(tl + C::TM_S + c0, r);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NH; ++c) x[c] = __uint_as_float(r[c]);
          }
          if (i + 1 < n) {  // the next tile's S^T goes on while this one's scores are dealt with
            if (keys) {
              unpack_k();
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(k_ready(w));
            }
          }
          if (j0 + BC > all_seen) {  // some row does not see the whole tile
            const int room = nk - (j0 + id);   // > lag: the row sees this key
#pragma unroll
            for (int c = 0; c < NH; ++c) x[c] = lag[c0 + c] < room ? x[c] : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < NH; c += 4) {
            const float4 nr = *reinterpret_cast<const float4*>(ref + c0 + c);
            const float4 cs = *reinterpret_cast<const float4*>(cscale + c0 + c);
            x[c] = fmaf(x[c], cs.x, nr.x);
            x[c + 1] = fmaf(x[c + 1], cs.y, nr.y);
            x[c + 2] = fmaf(x[c + 2], cs.z, nr.z);
            x[c + 3] = fmaf(x[c + 3], cs.w, nr.w);
          }
          float over = -INFINITY;
#pragma unroll
          for (int c = 0; c < NH; c += 2) over = fmax3(over, x[c], x[c + 1]);
          const bool o_ready = mine == 0 || mbar_try_wait(o_done(w), (mine - 1) & 1);  // (asked ahead of the barrier)
          const bool rises = bar_any(1 + w, kRows, i == 0 || over > kRescaleThreshold);
          // the last product of this team has read P (and O is complete)
          if (!o_ready) wait_longer(o_done(w), (mine - 1) & 1, wc.status, wc.abort_flag, wc.limit_ns);
          __syncwarp();
          if (F32 && i > 0) {
            tc_fence_after();
            add_tile();
          }
          if (rises) {
            // the piece's first tile sets the references (a row that sees any key of
            // the piece sees its first one), in others some rise: column maxima over
            // the 128 keys
            tc_fence_after();
            {
              float v[NH];
#pragma unroll
              for (int c = 0; c < NH; ++c) v[c] = x[c];
              reduce_step<NH / 2, 16>(v, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
              for (int y = 0; y < RCOLS; ++y) red[quarter * NR + my_col + y] = v[y];
            }
            rows_sync();
            if (tid < NA) {
              const float mx = fmaxf(fmaxf(red[tid], red[NR + tid]), fmaxf(red[2 * NR + tid], red[3 * NR + tid]));
              const bool up = i == 0 ? mx != -INFINITY : mx > kRescaleThreshold;
              fac[tid] = up ? kBelow - mx : 0.f;  // what the column's scores, and the logarithms of P and O, change by
              ref[tid] += fac[tid];
            }
            rows_sync();
#pragma unroll
            for (int c = 0; c < NH; ++c) {
              const float f = fac[c0 + c];
              x[c] += f;
              const float alpha = ex2_approx(fminf(f, 0.f));  // (the first tile finds zeros)
              l[c] *= alpha;
              if constexpr (F32) acc[c] *= alpha;
            }
            if (!F32 && i > 0) {
#pragma unroll 1
              for (int c = c0; c < c0 + NH; c += 8) {
                uint32_t o[8];
                tmem_ld_32x32b_x8(tl + C::TM_O + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * ex2_approx(fac[c + y]));
                tmem_st_32x32b_x8(tl + C::TM_O + c, o);
              }
            }
          }
          // ---- P
          constexpr int PW = NH < 8 ? NH : 8;  // columns of a store
#pragma unroll
          for (int c = 0; c < NH; c += PW) {
#pragma unroll
            for (int y = 0; y < PW; ++y) {
              x[c + y] = ex2_approx(x[c + y]);
              l[c + y] += x[c + y];
            }
            // P is rounded to fp16, the products' type: half a step of 2^-11 each
            // (of a second term too, where there is one: 2^-22)
            const uint32_t at = sP + id * C::RB + p_chunk<C::RB>(id, (c0 + c) / 8) * 16;
#pragma unroll
            for (int t = 0; t < C::PT; ++t) {
              uint32_t pk[PW / 2];
#pragma unroll
              for (int y = 0; y < PW / 2; ++y) {
                pk[y] = pack_f16x2(x[c + 2 * y], x[c + 2 * y + 1]);
                if (t + 1 < C::PT) {
                  const float2 h = cache4::floats(pk[y]);
                  x[c + 2 * y] -= h.x;
                  x[c + 2 * y + 1] -= h.y;
                }
              }
              if constexpr (PW == 8)
                st_shared_v4(at + t * C::P_BYTES, pk[0], pk[1], pk[2], pk[3]);
              else
                st_shared_v2(at + t * C::P_BYTES, pk[0], pk[1]);
            }
          }
          if (tid == 0) s_first[w] = i == 0;
          fence_proxy_async_smem();
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready(w));
        }
        ++mine;
      }
      // ------------------------------------------------------------ output
      if (rows) {
        reduce_step<NH / 2, 16>(l, [](float x, float y) { return x + y; });
        rows_sync();  // the last tile's column results have been read
#pragma unroll
        for (int x = 0; x < RCOLS; ++x) red[quarter * NR + my_col + x] = l[x];
        rows_sync();
        const bool whole = t0 == 0 && n == tiles_of<BC>(nk);
        const long long part = static_cast<long long>(head * plan.row_groups + rg) * plan.n_seq + b + range;
        const long long orow0 = row_of(head, rg, b);
        if (tid < NA) {
          const float sum = (red[tid] + red[NR + tid]) + (red[2 * NR + tid] + red[3 * NR + tid]);
          fac[tid] = sum == 0.f ? 0.f : __frcp_rn(sum);
          // (one product in 64 bits: the reference may be large beside the logarithm; no key seen: -inf)
          const float lse = sum == 0.f ? -INFINITY : static_cast<float>(logf(sum) - ref[tid] * 0.69314718055994531);
          if (tid < n_rows && !*abort_flag) {
            if (!whole)
              p.part_lse[part * NR + tid] = lse;
            else if (p.lse != nullptr)
              p.lse[orow0 + tid] = lse;
          }
        }
        wait_for(o_done(w), (mine - 1) & 1, wc);
        tc_fence_after();
        rows_sync();
        auto put_o = [&](int row, float y) {
          y *= cache.v_scale;  // (not part of fac: v_scale / sum may be too small a number where O is not)
          if (!whole)
            p.part_o[(part * NR + row) * D + id] = y;
          else if constexpr (F32)
            static_cast<float*>(p.o)[(orow0 + row) * D + id] = y;
          else
            static_cast<__nv_bfloat16*>(p.o)[(orow0 + row) * D + id] = __float2bfloat16_rn(y);
        };
        if constexpr (F32) {
          add_tile();
          if (id < D && !*abort_flag) {
#pragma unroll
            for (int c = 0; c < NH; ++c)
              if (c0 + c < n_rows) put_o(c0 + c, fac[c0 + c] == 0.f ? 0.f : acc[c] * fac[c0 + c]);
          }
        } else {
#pragma unroll 1
          for (int c = c0; c < min(c0 + NH, n_rows); c += 8) {
            uint32_t o[8];
            __syncwarp();
            tmem_ld_32x32b_x8(tl + C::TM_O + c, o);
            tmem_wait_ld();
            if (id >= D || *abort_flag) continue;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              if (c + x >= n_rows) break;
              const float f = fac[c + x];
              put_o(c + x, f == 0.f ? 0.f : __uint_as_float(o[x]) * f);
            }
          }
        }
        __syncwarp();
        tc_fence_before();
      }
      lag_of = rg;
      head = next_head;
      rg = next_rg;
      b = next;
      t0 = 0;
      nk = next_nk;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8 * W) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int NR, int NA, bool F32>
cudaError_t launch_nr(const SeqAttn& p, const Cache4& c, const DecodePlan& plan, cudaStream_t s) {
  using C = Cfg<D, NR, NA, F32>;
  static SmemOnce once;
  const cudaError_t e = once(fa_cache4_decode_kernel<D, NR, NA, F32>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(plan.cuts / C::W);
  fa_cache4_decode_kernel<D, NR, NA, F32><<<grid, C::THREADS, C::SMEM_BYTES, s>>>(p, c, plan);
  return cudaGetLastError();
}
template <int D, bool F32>
cudaError_t launch_d(const SeqAttn& p, const Cache4& c, const DecodePlan& w, cudaStream_t s) {
  if (w.nr == 16) {
    if (p.rows <= 4) return launch_nr<D, 16, 4, F32>(p, c, w, s);
    return p.rows <= 8 ? launch_nr<D, 16, 8, F32>(p, c, w, s) : launch_nr<D, 16, 16, F32>(p, c, w, s);
  }
  if constexpr (!F32)
    if (w.nr == 64) return launch_nr<D, 64, 64, F32>(p, c, w, s);
  return launch_nr<D, 32, 32, F32>(p, c, w, s);
}
template <bool F32>
cudaError_t launch_type(const SeqAttn& p, const Cache4& c, const DecodePlan& w, cudaStream_t s) {
  if (c.d == 64) return launch_d<64, F32>(p, c, w, s);
  if (c.d == 96) return launch_d<96, F32>(p, c, w, s);
  if (c.d == 128) return launch_d<128, F32>(p, c, w, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// Teams of a CTA.
template <bool F32>
static int teams(int d, int nr) {
  if (nr == 16) return d == 64 ? Cfg<64, 16, 16, F32>::W : d == 96 ? Cfg<96, 16, 16, F32>::W : Cfg<128, 16, 16, F32>::W;
  if (nr == 32) return d == 64 ? Cfg<64, 32, 32, F32>::W : d == 96 ? Cfg<96, 32, 32, F32>::W : Cfg<128, 32, 32, F32>::W;
  return 2;
}

DecodePlan cache4_plan(int n_seq, int heads, int rows, int d, fa_dtype dt, int sms) {
  DecodePlan w{};
  w.n_seq = n_seq;
  w.heads = heads;
  // The narrowest product that holds the rows (32 sequences of 1000 to 16384
  // tokens, 8 heads, d = 128: 4 rows 61, 92, 119 us with 16, 32, 64 columns; 16
  // rows 73, 93, 121; 24 rows, in two groups of 16, 130, 95, 125; 32 rows 132, 96,
  // 126; 64 rows 247, 178, 133).  float32: at most 32, whose terms of Q and P leave
  // the ring its room.
  w.nr = rows <= 16 ? 16 : rows <= 32 || dt == FA_DTYPE_F32 ? 32 : 64;
  w.row_groups = (rows + w.nr - 1) / w.nr;
  w.cuts = sms * (dt == FA_DTYPE_F32 ? teams<true>(d, w.nr) : teams<false>(d, w.nr));  // a CTA an SM, a range a team
  w.direct = 1;
  return w;
}

cudaError_t launch_cache4_decode(const SeqAttn& p, const Cache4& c, const DecodePlan& w, fa_dtype dt, cudaStream_t s) {
  // the sequences' tiles are summed in 32 bits, a range's tiles are counted in 31
  const long long tiles = static_cast<long long>(w.n_seq) * tiles_of<BC>(p.n_keys);
  if (tiles > 0x7fffffffLL || tiles * w.heads * w.row_groups / w.cuts >= 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return dt == FA_DTYPE_F32 ? launch_type<true>(p, c, w, s) : launch_type<false>(p, c, w, s);
}

template <typename T>
static cudaError_t merge_of(const SeqAttn& p, const DecodePlan& w, cudaStream_t s) {
  if (w.nr == 16) return launch_merge<BC, 16, T, true>(p, w, nullptr, nullptr, 0, true, s);
  if constexpr (sizeof(T) == 2)  // (float32 has at most 32: cache4_plan)
    if (w.nr == 64) return launch_merge<BC, 64, T, true>(p, w, nullptr, nullptr, 0, true, s);
  return launch_merge<BC, 32, T, true>(p, w, nullptr, nullptr, 0, true, s);
}
cudaError_t launch_cache4_merge(const SeqAttn& p, const DecodePlan& w, fa_dtype dt, cudaStream_t s) {
  return dt == FA_DTYPE_F32 ? merge_of<float>(p, w, s) : merge_of<__nv_bfloat16>(p, w, s);
}

}  // namespace fa
