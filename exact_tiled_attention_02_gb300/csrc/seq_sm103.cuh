// seq_sm103.cuh -- what the language-model kernels share on top of
// sm103.cuh: split shared-memory descriptors, 4-D TMA loads, host-side tensor
// maps and per-device launch state.
#pragma once

#include <atomic>

#include "seq_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace seq {

using namespace sm103;

// Shared-memory descriptor in its two 32-bit words: the start address (bits
// 0-13, 16-byte units) lives in the low word, so stepping through a tile is
// one 32-bit add (every address is below 256 KB, so the field never carries).
struct Desc2 {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc2 desc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  const uint64_t d = sdesc_sw128(saddr, lbo_bytes, sbo_bytes);
  return Desc2{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
// tcgen05 instructions for a whole converged warp: every lane runs the code
// around them, one elected lane (always the same) issues.  Kept converged, the
// descriptors live in uniform registers; issued from one lane of a diverged
// warp they are moved there for every instruction.  Measured, cycles a
// product, back to back: diverged 46 or more at any size (80-120 with the
// descriptor arithmetic of a real loop); converged 24 at M = 64 N = 16, 32 at
// M = 64 N = 64, 48 at M = 128 N = 64, 64 at M = N = 128: the operands' bytes
// over 128 a cycle, or M N 16 / 4096.
__device__ __forceinline__ void mma_ss_w(uint32_t d_tmem, Desc2 a, uint32_t a_off, Desc2 b, uint32_t b_off,
                                         uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 da, db;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "mov.b64 da, {%1, %2};\nmov.b64 db, {%3, %4};\n"
      "setp.ne.b32 p, %6, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d_tmem),
      "r"(a.lo + a_off), "r"(a.hi), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts_w(uint32_t d_tmem, uint32_t a_tmem, Desc2 b, uint32_t b_off, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 db;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "mov.b64 db, {%2, %3};\n"
      "setp.ne.b32 p, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit_w(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// TMA load and expected-bytes arrive by one elected lane of a converged warp.
__device__ __forceinline__ void tma_load_3d_w(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                              int c2) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_w(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
// Waits by a whole warp; the answer is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}
__device__ __forceinline__ bool warp_wait2(uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2, const WaitCtl& w) {
  return __all_sync(0xffffffffu, mbar_wait2(b1, p1, b2, p2, w));
}
// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 8, 16 or 32 columns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "columns of one access");
  if constexpr (N == 8)
    tmem_ld_32x32b_x8(taddr, r);
  else if constexpr (N == 16)
    tmem_ld_32x32b_x16(taddr, r);
  else
    tmem_ld_32x32b_x32(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "columns of one access");
  if constexpr (N == 8)
    tmem_st_32x32b_x8(taddr, r);
  else if constexpr (N == 16)
    tmem_st_32x32b_x16(taddr, r);
  else
    tmem_st_32x32b_x32(taddr, r);
}

// Rows out of tensor memory: a lane holds 64 bytes (four 16-byte pieces) of a
// row of its own.  The lanes of every group of four swap pieces so that lane
// l stores piece l % 4 of each of the group's rows: a store instruction then
// touches 8 rows' lines instead of 32, and costs a cycle for each (measured
// at 128 rows of 320 columns by eight warps: 9,000 cycles row by row).
// row(i): where row i of the warp (0 .. 31) goes, null where it is not wanted.
template <typename R>
__device__ __forceinline__ void store_rows64(uint4 (&v)[4], R row) {
  const int lane = threadIdx.x & 31;
  auto swap = [](uint4 x, int bit) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, x.x, bit), __shfl_xor_sync(0xffffffffu, x.y, bit),
                      __shfl_xor_sync(0xffffffffu, x.z, bit), __shfl_xor_sync(0xffffffffu, x.w, bit));
  };
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint4 got = swap(odd ? v[i] : v[i + 1], 1);
    if (odd)
      v[i] = got;
    else
      v[i + 1] = got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 got = swap(high ? v[i] : v[i + 2], 2);
    if (high)
      v[i] = got;
    else
      v[i + 2] = got;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint8_t* dst = static_cast<uint8_t*>(row((lane & ~3) + i));
    if (dst != nullptr) st_global_v4(dst + (lane & 3) * 16, v[i]);
  }
}
// 32 values of a lane's row as bf16 (64 bytes), or as fp32 (128 bytes).
template <typename R>
__device__ __forceinline__ void store_rows_bf16(const float* x, R row) {
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                      pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  store_rows64(v, row);
}
template <typename R>
__device__ __forceinline__ void store_rows_f32(const float* x, R row) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* y = x + 16 * h + 4 * i;
      v[i] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
    }
    store_rows64(v, [&](int i) -> void* {
      uint8_t* dst = static_cast<uint8_t*>(row(i));
      return dst == nullptr ? nullptr : dst + 64 * h;
    });
  }
}

// A bf16 map of up to four dimensions, innermost first (dims[0] contiguous),
// rows packed; box of 64 columns, 128-byte swizzle, zeros outside.
inline bool make_map(CUtensorMap* m, const void* base, int rank, const long long* dims, const int* box) {
  const EncodeTiledFnPtr fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t b[4];
  const cuuint32_t es[4] = {1, 1, 1, 1};
  unsigned long long bytes = 2;
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    bytes *= static_cast<unsigned long long>(dims[i]);
    if (i + 1 < rank) st[i] = bytes;
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, b, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool make_map3(CUtensorMap* m, const void* base, long long d0, long long d1, long long d2, int box1) {
  const long long dims[3] = {d0, d1, d2};
  const int box[3] = {64, box1, 1};
  return make_map(m, base, 3, dims, box);
}

// Programmatic dependent launch: the next kernel of a call may be put on the
// SMs as this one's blocks let go of them.  pdl_launch lets it start;
// pdl_wait returns once the kernels before this one have completed and their
// results can be read.  A kernel launched this way waits before it reads what
// they wrote and, in any case, before it ends, so that its own completion
// implies theirs.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch that may overlap the kernel before it on the stream (see pdl_wait),
// which must be one of the same call.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Raises a kernel's dynamic shared memory limit once per device.
struct SmemOnce {
  std::atomic<unsigned long long> done{0};
  template <typename F>
  cudaError_t operator()(F kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
  }
};

inline int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = cached[dev].load()) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cached[dev].store(n);
  return n;
}

}  // namespace seq
}  // namespace fa
