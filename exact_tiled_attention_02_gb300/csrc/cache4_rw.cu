// cache4_rw.cu -- writing new tokens into the 4-bit key/value cache, and
// reading cached tokens back as dense keys and values.
//
// Both are a pass over memory: a warp takes one block (16 tokens of a head),
// whose 18 d bytes and whose rows it moves in whole 16- and 32-byte pieces.
// 8 prompts of 900 to 8192 tokens, 8 heads, d = 128, bf16: written in 40 us (191
// MB, 4.8 TB/s: three dependent loads, length, page and rows, before a warp has
// anything to do, at 7 warps a scheduler), read back in 53 (309 MB, 5.8 TB/s).
// One token for each of 64 sequences: 4 us each, latency.
#include <cmath>

#include "cache4.cuh"

namespace fa {
namespace {

using namespace cache4;

constexpr int kWarps = 4;

// Sixteen entries as they are in memory, and as numbers.
template <typename T>
struct Raw {
  uint4 v[sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void numbers(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          x[4 * i + j] = __uint_as_float(w[j]);
        } else {
          x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    }
  }
};
static_assert(sizeof(Raw<float>) == 64 && sizeof(Raw<__nv_bfloat16>) == 32, "sixteen entries");
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// N consecutive entries of a row (N a multiple of 4)
template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(bf16x2(x[8 * i], x[8 * i + 1]), bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                                  bf16x2(x[8 * i + 4], x[8 * i + 5]), bf16x2(x[8 * i + 6], x[8 * i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<uint2*>(p)[i] = make_uint2(bf16x2(x[4 * i], x[4 * i + 1]), bf16x2(x[4 * i + 2], x[4 * i + 3]));
  }
}

// Blocks that Nn consecutive positions can touch.
__host__ __device__ __forceinline__ int blocks_of(int n) { return (n + kBlock - 2) / kBlock + 1; }

// One warp a block.  A lane quantises whole groups of 16 channels of a token;
// the values' codes change places through shared memory, since the cache
// holds the tokens of a channel together.  Tokens of the block that are not
// new keep their codes and scales: where a byte of value codes is shared with
// one of them it is read and put together again.
template <typename T, Quotient Q>
__global__ void __launch_bounds__(kWarps * 32)
    fa_cache4_write_kernel(const __grid_constant__ Cache4 c, const T* __restrict__ k, const T* __restrict__ v,
                           const int* __restrict__ n_new, int Nn, float k_scale, float v_scale) {
  extern __shared__ uint2 smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = c.d, groups = d / 16;
  uint2* codes = smem + warp * d;  // [16 tokens][d/16]
  const int per = blocks_of(Nn);
  const long long at = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int b = static_cast<int>(at / (static_cast<long long>(per) * c.Hkv));
  if (b >= c.B) return;
  const int rest = static_cast<int>(at - static_cast<long long>(b) * per * c.Hkv);
  const int h = rest / per;
  const int len = c.lens[b];
  if (len < 0 || len > capacity(c)) {  // nowhere to put them
    if (lane == 0) atomicOr(c.status, kStatusInput);
    return;
  }
  int n = Nn;
  if (n_new != nullptr) {
    n = min(max(n_new[b], 0), Nn);
    if (n != n_new[b] && lane == 0) atomicOr(c.status, kStatusInput);
  }
  if (n == 0) return;  // not even its last block's own bits are put back: another sequence may be writing to that page
  const int p0 = max(len - n, 0);  // positions p0 .. len - 1 are written
  const int blk = p0 / kBlock + rest % per;
  if (blk >= (len + kBlock - 1) / kBlock) return;  // (in blocks: a position past the end may pass 32 bits)
  const int page = page_of(c, b, blk);
  if (page < 0) return;
  uint8_t* dst = c.cache + block_at(c, page, h, blk);
  const int t0 = max(p0 - blk * kBlock, 0), t1 = min(len - blk * kBlock, kBlock);  // new tokens of the block
  // token t of the block is row t + row0 of the sequence's new ones
  const long long row0 = (static_cast<long long>(b) * c.Hkv + h) * Nn + (Nn - len) + blk * kBlock;

  for (int i = lane; i < d; i += 32) {
    const int t = i / groups, g = i - t * groups;
    if (t < t0 || t >= t1) continue;
    Raw<T> kr, vr;  // both on their way before either is used
    kr.load(k + (row0 + t) * d + g * 16);
    vr.load(v + (row0 + t) * d + g * 16);
    float x[16];
    uint2 w;
    kr.numbers(x);
    uint8_t s = quantise16<Q>(x, k_scale, w);
    *reinterpret_cast<uint2*>(dst + (g * 16 + t) * 8) = w;
    dst[off_k_scale(d) + t * groups + g] = s;
    vr.numbers(x);
    s = quantise16<Q>(x, v_scale, w);
    codes[i] = w;
    dst[off_v_scale(d) + g * 16 + t] = s;
  }
  __syncwarp();
  // a lane takes the 16 tokens of eight channels
  unsigned long long keep = 0;  // nibbles of the tokens that stay
  if (t0 > 0) keep |= (1ull << (4 * t0)) - 1;
  if (t1 < kBlock) keep |= ~0ull << (4 * t1);
  const uint32_t keep_lo = static_cast<uint32_t>(keep), keep_hi = static_cast<uint32_t>(keep >> 32);
  const uint32_t* rows = reinterpret_cast<const uint32_t*>(codes);  // [16 tokens][d/8]
  for (int i = lane; i < d / 8; i += 32) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      lo[t] = rows[t * (d / 8) + i];
      hi[t] = rows[(t + 8) * (d / 8) + i];
    }
    transpose_codes(lo);
    transpose_codes(hi);
    uint4* out = reinterpret_cast<uint4*>(dst + off_v(d) + i * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 w = make_uint4(lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1]);
      if (keep != 0) {
        const uint4 o = out[j];
        w = make_uint4((o.x & keep_lo) | (w.x & ~keep_lo), (o.y & keep_hi) | (w.y & ~keep_hi),
                       (o.z & keep_lo) | (w.z & ~keep_lo), (o.w & keep_hi) | (w.w & ~keep_hi));
      }
      out[j] = w;
    }
  }
}

// One warp a block of the cache that the positions touch; positions outside a
// sequence are zeros.  Registers are held to what eight CTAs an SM have (bf16: 60
// us with 5, 53 with 8; float32, with rows twice as long in flight, 8.8 and 10.3).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 8 : 5)
    fa_cache4_read_kernel(const __grid_constant__ Cache4 c, const int* __restrict__ first, T* __restrict__ k,
                          T* __restrict__ v, int N) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = c.d, groups = d / 16;
  const int per = blocks_of(N);
  const long long at = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int b = static_cast<int>(at / (static_cast<long long>(per) * c.Hkv));
  if (b >= c.B) return;
  const int rest = static_cast<int>(at - static_cast<long long>(b) * per * c.Hkv);
  const int h = rest / per;
  const int len = length(c, b, lane == 0);
  const long long p0 = first != nullptr ? first[b] : 0;                 // position of row 0
  const long long q0 = (p0 >= 0 ? p0 : p0 - (kBlock - 1)) / kBlock * kBlock + rest % per * kBlock;  // of the block's token 0
  const long long row0 = (static_cast<long long>(b) * c.Hkv + h) * N + (q0 - p0);
  const int t0 = static_cast<int>(max(p0 - q0, 0ll)), t1 = static_cast<int>(min(p0 + N - q0, static_cast<long long>(kBlock)));
  if (t1 <= t0) return;
  const uint8_t* src = nullptr;
  if (q0 >= 0 && q0 < len) {
    const int page = page_of(c, b, static_cast<int>(q0 / kBlock));
    if (page >= 0) src = c.cache + block_at(c, page, h, static_cast<int>(q0 / kBlock));
  }
  const int held = src != nullptr ? static_cast<int>(min(len - q0, static_cast<long long>(kBlock))) : 0;

  for (int i = lane; i < d; i += 32) {
    const int t = i / groups, g = i - t * groups;
    if (t < t0 || t >= t1) continue;
    float x[16];
    if (t < held) {
      const uint2 w = *reinterpret_cast<const uint2*>(src + (g * 16 + t) * 8);
      const uint32_t s = src[off_k_scale(d) + t * groups + g];
      uint32_t o[8], sc[2];
      scales_f16(s | s << 8, sc);
      codes_f16(w.x, o);
      codes_f16(w.y, o + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = floats(mul_f16x2(o[j], sc[0]));
        x[2 * j] = f.x * c.k_scale;
        x[2 * j + 1] = f.y * c.k_scale;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = 0.f;
    }
    store_row(k + (row0 + t) * d + g * 16, x);
  }
  // a lane takes four channels
  for (int i = lane; i < d / 4; i += 32) {
    const int ch = 4 * i;
    uint4 a = make_uint4(0, 0, 0, 0), e = a, s = a;
    if (held > 0) {
      a = *reinterpret_cast<const uint4*>(src + off_v(d) + ch * 8);
      e = *reinterpret_cast<const uint4*>(src + off_v(d) + ch * 8 + 16);
      s = *reinterpret_cast<const uint4*>(src + off_v_scale(d) + (ch >> 4) * 16);
    }
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, e.x, e.y, e.z, e.w}, sw[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {  // tokens 8 hf .. 8 hf + 7
      uint32_t o[4][4], sc[4];
      scales_f16(sw[2 * hf], sc);
      scales_f16(sw[2 * hf + 1], sc + 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) codes_f16(w[2 * q + hf], o[q]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = floats(mul_f16x2(o[q][j], sc[j]));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = 8 * hf + 2 * j + y;
          if (t < t0 || t >= t1) continue;
          float x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) x[q] = t < held ? (y == 0 ? f[q].x : f[q].y) * c.v_scale : 0.f;
          store_row(v + (row0 + t) * d + ch, x);
        }
      }
    }
  }
}

// A power of two whose reciprocal is a normal number, and so can stand for the division by it.
bool power_of_two(float x) {
  int e;
  return std::frexp(x, &e) == 0.5f && e > -100 && e < 100;
}

template <typename T>
cudaError_t launch_write(const Cache4& c, const void* k, const void* v, const int* n_new, int Nn, cudaStream_t s) {
  const long long warps = static_cast<long long>(c.B) * c.Hkv * blocks_of(Nn);
  const long long blocks = (warps + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  const int smem = kWarps * c.d * 8;
  const T *kt = static_cast<const T*>(k), *vt = static_cast<const T*>(v);
  constexpr Quotient kFast = sizeof(T) == 2 ? kShort : kMultiply;
  if (power_of_two(c.k_scale) && power_of_two(c.v_scale))
    fa_cache4_write_kernel<T, kFast><<<grid, kWarps * 32, smem, s>>>(c, kt, vt, n_new, Nn, 1.f / c.k_scale, 1.f / c.v_scale);
  else
    fa_cache4_write_kernel<T, kDivide><<<grid, kWarps * 32, smem, s>>>(c, kt, vt, n_new, Nn, c.k_scale, c.v_scale);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_read(const Cache4& c, const int* first, void* k, void* v, int N, cudaStream_t s) {
  const long long warps = static_cast<long long>(c.B) * c.Hkv * blocks_of(N);
  const long long blocks = (warps + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  fa_cache4_read_kernel<T><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(c, first, static_cast<T*>(k),
                                                                                static_cast<T*>(v), N);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache4_write(const Cache4& c, const void* k, const void* v, const int* n_new, int Nn, fa_dtype dt,
                                cudaStream_t s) {
  return dt == FA_DTYPE_BF16 ? launch_write<__nv_bfloat16>(c, k, v, n_new, Nn, s)
                             : launch_write<float>(c, k, v, n_new, Nn, s);
}
cudaError_t launch_cache4_read(const Cache4& c, const int* first, void* k, void* v, int N, fa_dtype dt, cudaStream_t s) {
  return dt == FA_DTYPE_BF16 ? launch_read<__nv_bfloat16>(c, first, k, v, N, s) : launch_read<float>(c, first, k, v, N, s);
}

}  // namespace fa
