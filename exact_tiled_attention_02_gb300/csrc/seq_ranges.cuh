// seq_ranges.cuh -- work split of the decoding kernels: the tiles of BC keys of
// all sequences, laid end to end, cut into equal ranges, one a CTA (per group
// of rows), and the kernel that merges the pieces of sequences that several
// CTAs share.  The cut depends on the lengths alone.  The flat form lays the
// tiles of all groups of rows end to end too: any number of groups fills the
// GPU, at the price of a few divisions (in 64 bits only where tiles pass 32).
#pragma once

#include <cmath>

#include "seq_sm103.cuh"

namespace fa {
namespace seq {

__device__ __forceinline__ int seq_len(const SeqAttn& p, int b, bool report) {
  const int n = p.lens[b];
  const int nk = min(max(n, 0), p.n_keys);
  if (report && n != nk) atomicOr(p.status, kStatusInput);
  return nk;
}
template <int BC>
__host__ __device__ __forceinline__ int tiles_of(int nk) {
  return (nk + BC - 1) / BC;
}

// Whole warp: the sum over sequences before `b` of their tiles, and over all.
// The launcher keeps totals below 2^31 / cuts (32-bit products below).
template <int BC>
__device__ __forceinline__ void tile_sums(const SeqAttn& p, int n_seq, int b, unsigned& before, unsigned& total) {
  const int lane = threadIdx.x & 31;
  unsigned x = 0, y = 0;
  for (int i = lane; i < n_seq; i += 32) {
    const unsigned t = tiles_of<BC>(seq_len(p, i, false));
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

// Whole warp: where range `cut` begins (a sequence and one of its tiles), and how
// many tiles it has; reports lengths out of range.
template <int BC>
__device__ __forceinline__ void find_range(const SeqAttn& p, const DecodePlan& plan, int cut, int& b0, int& first,
                                           int& count) {
  const int lane = threadIdx.x & 31;
  unsigned before, total;
  tile_sums<BC>(p, plan.n_seq, 0, before, total);
  const unsigned ranges = range_count(total, plan.cuts);
  const bool some = cut < static_cast<int>(ranges);
  const unsigned t0 = some ? range_start(total, cut, ranges) : total;
  const unsigned t1 = some ? range_start(total, cut + 1, ranges) : total;
  unsigned base = 0;
  b0 = first = count = 0;
  for (int i0 = 0; i0 < plan.n_seq; i0 += 32) {
    const int i = i0 + lane;
    const unsigned t = i < plan.n_seq ? tiles_of<BC>(seq_len(p, i, true)) : 0;
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
      count = static_cast<int>(t1 - t0);
      return;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
}

// The flat form: plan.cuts ranges of all groups' tiles, none of them empty, the
// first `rem` a tile longer than the others.  U: 32 bits where they hold the tiles.
template <typename U>
struct FlatCut {
  U n, q, rem;
  __device__ __forceinline__ FlatCut(U all, unsigned cuts) {
    n = all < cuts ? all : cuts;
    q = n > 0 ? all / n : 0;
    rem = all - q * n;
  }
  __device__ __forceinline__ U start(U r) const { return r * q + (r < rem ? r : rem); }
  __device__ __forceinline__ int owner(U x) const {
    return static_cast<int>(x < rem * (q + 1) ? x / (q + 1) : rem + (x - rem * (q + 1)) / q);
  }
};
// f(all groups' tiles, in 32 bits where they fit)
template <typename F>
__device__ __forceinline__ void flat_tiles(const DecodePlan& plan, unsigned total, F f) {
  const unsigned long long all = static_cast<unsigned long long>(plan.heads) * plan.row_groups * total;
  if (all >> 32 == 0)
    f(static_cast<unsigned>(all));
  else
    f(all);
}
// Of range r: where it begins (group of rows, sequence, tile) and its tiles.
template <int BC>
__device__ __forceinline__ void find_flat(const SeqAttn& p, const DecodePlan& plan, int r, int& grp, int& b0, int& first,
                                          int& count) {
  const int lane = threadIdx.x & 31;
  unsigned before, total;
  tile_sums<BC>(p, plan.n_seq, 0, before, total);
  grp = b0 = first = count = 0;
  unsigned t0 = 0;
  flat_tiles(plan, total, [&](auto all) {
    using U = decltype(all);
    const FlatCut<U> cut(all, plan.cuts);
    if (static_cast<U>(r) >= cut.n) return;
    const U x0 = cut.start(r);
    grp = static_cast<int>(x0 / total);
    t0 = static_cast<unsigned>(x0 - static_cast<U>(grp) * total);
    count = static_cast<int>(cut.start(r + 1) - x0);
  });
  if (count == 0) return;
  unsigned base = 0;
  for (int i0 = 0; i0 < plan.n_seq; i0 += 32) {
    const int i = i0 + lane;
    const unsigned t = i < plan.n_seq ? tiles_of<BC>(seq_len(p, i, true)) : 0;
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
      b0 = i0 + l;
      first = static_cast<int>(t0 - __shfl_sync(0xffffffffu, end - t, l));
      return;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
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

// Merges the pieces of each sequence, and the partial results [pre][total] of
// another set of keys beside them (the prefix), row by row: see
// seq_combine.cu for the formula.  One warp per row and W of its 128-column
// slices (all of them where there are rows enough to fill the GPU); lane i
// holds the weight of part i, so that the parts' loads do not wait for one
// another.  Rows of a sequence that was written directly are left alone.
template <int BC, int NR, int W, typename T, bool FLAT>
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
  tile_sums<BC>(p, plan.n_seq, b, before, total);
  const int nt = tiles_of<BC>(seq_len(p, b, true));
  const int grp = head * plan.row_groups + r / NR;
  int c0 = 0, n = 0;
  if (nt > 0) {
    if constexpr (FLAT) {
      flat_tiles(plan, total, [&](auto all) {
        using U = decltype(all);
        const FlatCut<U> cut(all, plan.cuts);
        const U at = static_cast<U>(grp) * total + before;
        c0 = cut.owner(at);
        n = cut.owner(at + nt - 1) - c0 + 1;
      });
    } else {
      const unsigned ranges = range_count(total, plan.cuts);
      c0 = owner(total, before, ranges);
      n = owner(total, before + nt - 1, ranges) - c0 + 1;
    }
  }
  pdl_wait();
  if (plan.direct && n == 1) return;
  const long long slot0 =
      (static_cast<long long>(grp) * (FLAT ? plan.n_seq : plan.cuts + plan.n_seq) + c0 + b) * NR + r % NR;
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
  constexpr int U = W == 1 ? 4 : 2;
  float4 acc[W];
#pragma unroll
  for (int w = 0; w < W; ++w) acc[w] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float ls = i0 == 0 ? mine : (i0 + lane < n ? part_lse(i0 + lane) : -INFINITY);
    const float wl = expf(ls - ref) * inv;
    const unsigned holds = __ballot_sync(0xffffffffu, ls != -INFINITY);  // a part without keys holds zeros or nothing
    const int k = min(32, n - i0);
#pragma unroll 1
    for (int i = 0; i < k; i += U) {  // the loads of U parts do not wait for one another
      float wi[U];
      float4 v[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        wi[u] = __shfl_sync(0xffffffffu, wl, (i + u) & 31);
        const bool on = i + u < k && (holds >> ((i + u) & 31) & 1);
        const int part = i0 + i + u;
        const float* src = (part < pre ? pre_o + (part * p.total + row) * p.dv
                                       : p.part_o + (slot0 + static_cast<long long>(part - pre) * NR) * p.dv) + c;
#pragma unroll
        for (int w = 0; w < W; ++w)
          v[u][w] = on && c + 128 * w < p.dv ? *reinterpret_cast<const float4*>(src + 128 * w)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u >= k) break;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          acc[w].x = fmaf(wi[u], v[u][w].x, acc[w].x);
          acc[w].y = fmaf(wi[u], v[u][w].y, acc[w].y);
          acc[w].z = fmaf(wi[u], v[u][w].z, acc[w].z);
          acc[w].w = fmaf(wi[u], v[u][w].w, acc[w].w);
        }
      }
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (c + 128 * w >= p.dv) break;
    T* dst = static_cast<T*>(p.o) + row * p.dv + c + 128 * w;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(dst) = acc[w];
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[w].x, acc[w].y), pack_bf16x2(acc[w].z, acc[w].w));
  }
  if (slice == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = m + logf(sum);
}

template <int BC, int NR, typename T = __nv_bfloat16, bool FLAT = false>
cudaError_t launch_merge(const SeqAttn& p, const DecodePlan& w, const float* pre_o, const float* pre_lse, int pre,
                         bool after, cudaStream_t s) {
  // A warp takes a whole row of 512 where the rows alone give every SM 32 warps
  // (the whole call at 16384 rows: 105 us, 117 with a warp a slice; at 1024
  // rows 71 and 68; at 16 rows 18.9 and 15.4).
  const long long rows = static_cast<long long>(w.n_seq) * w.heads * p.rows;
  const bool wide = !FLAT && p.dv > 128 && rows >= 152 * 32;  // (the flat form's rows are of 128 at most)
  const long long warps = rows * (wide ? (p.dv + 511) / 512 : (p.dv + 127) / 128);
  if (warps > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
  if constexpr (FLAT) {
    return launch_after(fa_seq_decode_merge_kernel<BC, NR, 1, T, true>, blocks, 128, 0, s, p, w, pre_o, pre_lse, pre);
  } else {
    if (!after) {  // no kernel of this call before it: the lengths may only now be complete
      fa_seq_decode_merge_kernel<BC, NR, 1, T, false><<<static_cast<unsigned>((rows * ((p.dv + 127) / 128) + 3) / 4), 128, 0, s>>>(
          p, w, pre_o, pre_lse, pre);
      return cudaGetLastError();
    }
    return wide ? launch_after(fa_seq_decode_merge_kernel<BC, NR, 4, T, false>, blocks, 128, 0, s, p, w, pre_o, pre_lse, pre)
                : launch_after(fa_seq_decode_merge_kernel<BC, NR, 1, T, false>, blocks, 128, 0, s, p, w, pre_o, pre_lse, pre);
  }
}

}  // namespace seq
}  // namespace fa
