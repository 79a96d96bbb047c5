// cache4_fwd_simt.cu -- attention of a sequence's last tokens over the 4-bit
// cache, fp32 on CUDA cores: bf16 and float32 tensors of the head widths that
// the tensor-core kernel does not take (all but 64, 96 and 128).
//
//   S_ij = scale k_scale (q_i . K_j),  O_i = v_scale sum_j softmax_j(S_i) V_j
//
// over the keys j < len - (n_new - 1 - t) of the row's token t, with K = code *
// scale exact in fp32, the row's running maximum and sum, and the accurate expf
// and logf.  A row that sees no key gives O = 0, lse = -inf.
//
// One CTA of 128 threads per 8 query rows of a key/value head and split of its
// keys; tiles of 64 keys are unpacked to shared memory.
//
// For completeness of widths, not for speed: every CTA unpacks its keys for 8
// rows at most (4 in use at 4 query heads a key head), four CTAs of four warps an
// SM at d = 80 and one at 256, with five barriers a tile.  64 sequences of 500 to
// 8200 tokens, 32 / 8 heads, either type: d = 80 1100 us, 112 1520, 256 6160, where
// the bytes take 30, 42 and 95 and the tensor-core kernel 67 at d = 128.
#include <cmath>

#include "cache4.cuh"
#include "seq_sm103.cuh"

namespace fa {
namespace {

using namespace cache4;

constexpr int BK = 64, TR = 8, kThreads = 128;

__host__ __device__ constexpr int ld_of(int d) { return d + 4; }  // rows 16-byte aligned, 8 of them apart in 32 banks
constexpr int smem_floats(int d) { return TR * d + 2 * BK * ld_of(d) + BK * TR + TR * BK + 2 * TR; }

template <typename T, int NC>  // NC: channels of O a thread
__global__ void __launch_bounds__(kThreads) fa_cache4_fwd_simt_kernel(const __grid_constant__ Cache4Attn p) {
  extern __shared__ float4 smem4[];
  seq::pdl_launch();
  const Cache4& c = p.c;
  const int d = c.d, LDK = ld_of(d), groups = d / 16;
  float* Qs = reinterpret_cast<float*>(smem4);  // [TR][d]
  float* Ks = Qs + TR * d;                      // [BK][LDK]
  float* Vs = Ks + BK * LDK;                    // [BK][LDK]
  float* Ss = Vs + BK * LDK;                    // [TR][BK] scores
  float* Ps = Ss + TR * BK;                     // [BK][TR] probabilities
  float* alpha = Ps + BK * TR;                  // [TR] factor of a row's O, then 1 / its sum
  const int G = p.Hq / c.Hkv, rows = G * p.n_new, row_tiles = (rows + TR - 1) / TR;
  const int group = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * TR;
  const int b = group / c.Hkv, h = group % c.Hkv, split = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nk = length(c, b, tid == 0);
  const int tiles = (nk + BK - 1) / BK;
  const int j0 = static_cast<int>(static_cast<long long>(tiles) * split / p.splits);
  const int j1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / p.splits);
  const long long row0 = (static_cast<long long>(b) * p.Hq + h * G) * p.n_new + r0;  // of q, o and lse
  const T* q = static_cast<const T*>(p.q) + row0 * d;
  for (int i = tid; i < TR * d; i += kThreads) {
    float x = 0.f;
    if (r0 + i / d < rows) {
      if constexpr (sizeof(T) == 2)
        x = __bfloat162float(q[i]);
      else
        x = q[i];
    }
    Qs[i] = x;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of rows 2 warp, 2 warp + 1
  int limit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) limit[i] = nk - (p.n_new - 1 - (r0 + 2 * warp + i) % p.n_new);
  float acc[NC][TR];
#pragma unroll
  for (int x = 0; x < NC; ++x)
#pragma unroll
    for (int r = 0; r < TR; ++r) acc[x][r] = 0.f;
  const float sl = p.scale * c.k_scale;

  for (int j = j0; j < j1; ++j) {
    __syncthreads();  // the last tile has been read
    for (int i = tid; i < BK * groups; i += kThreads) {  // 16 channels of a key
      const int t = i % BK, g = i / BK, pos = j * BK + t;
      uint2 w = make_uint2(0, 0);
      uint32_t s = 0;
      if (pos < nk) {
        const int page = page_of(c, b, pos / kBlock);
        if (page >= 0) {
          const uint8_t* src = c.cache + block_at(c, page, h, pos / kBlock);
          w = *reinterpret_cast<const uint2*>(src + (g * 16 + pos % kBlock) * 8);
          s = src[off_k_scale(d) + pos % kBlock * groups + g];
        }
      }
      uint32_t o[8], sc[2];
      scales_f16(s | s << 8, sc);
      codes_f16(w.x, o);
      codes_f16(w.y, o + 4);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f0 = floats(mul_f16x2(o[2 * x], sc[0])), f1 = floats(mul_f16x2(o[2 * x + 1], sc[0]));
        *reinterpret_cast<float4*>(Ks + t * LDK + g * 16 + 4 * x) = make_float4(f0.x, f0.y, f1.x, f1.y);
      }
    }
    for (int i = tid; i < (BK / 8) * d; i += kThreads) {  // 8 tokens of a channel
      const int ch = i % d, t8 = i / d, pos = j * BK + 8 * t8;
      uint32_t w = 0;
      uint2 s = make_uint2(0, 0);
      if (pos < nk) {
        const int page = page_of(c, b, pos / kBlock);
        if (page >= 0) {
          const uint8_t* src = c.cache + block_at(c, page, h, pos / kBlock);
          const int half = pos / 8 % 2;
          w = *reinterpret_cast<const uint32_t*>(src + off_v(d) + ch * 8 + 4 * half);
          s = *reinterpret_cast<const uint2*>(src + off_v_scale(d) + (ch >> 4) * 16 + 8 * half);
        }
      }
      uint32_t o[4], sc[4];
      scales_f16(s.x, sc);
      scales_f16(s.y, sc + 2);
      codes_f16(w, o);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = floats(mul_f16x2(o[x], sc[x]));
        // past the end: zeros, whatever the scales there
        Vs[(8 * t8 + 2 * x) * LDK + ch] = pos + 2 * x < nk ? f.x : 0.f;
        Vs[(8 * t8 + 2 * x + 1) * LDK + ch] = pos + 2 * x + 1 < nk ? f.y : 0.f;
      }
    }
    __syncthreads();
    {  // a thread: one key, four rows
      const int t = tid % BK, rr = tid / BK * 4;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int x = 0; x < d; x += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(Ks + t * LDK + x);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(Qs + (rr + r) * d + x);
          s[r] = fmaf(kv.w, qv.w, fmaf(kv.z, qv.z, fmaf(kv.y, qv.y, fmaf(kv.x, qv.x, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) Ss[(rr + r) * BK + t] = s[r];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // a warp: two rows, two keys a lane
      const int r = 2 * warp + i;
      float x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x[e] = j * BK + lane + 32 * e < limit[i] ? Ss[r * BK + lane + 32 * e] * sl : -INFINITY;
      float mx = fmaxf(x[0], x[1]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m[i], mx), ref = m_new == -INFINITY ? 0.f : m_new;
      const float a = expf(m[i] - ref);  // 0 while the row has seen no key
      const float p0 = expf(x[0] - ref), p1 = expf(x[1] - ref);
      float sum = p0 + p1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      Ps[lane * TR + r] = p0;
      Ps[(lane + 32) * TR + r] = p1;
      l[i] = l[i] * a + sum;
      m[i] = m_new;
      if (lane == 0) alpha[r] = a;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NC; ++x) {
      const int ch = tid + x * kThreads;
      if (ch >= d) break;
#pragma unroll
      for (int r = 0; r < TR; ++r) acc[x][r] *= alpha[r];
#pragma unroll 4
      for (int t = 0; t < BK; ++t) {
        const float vv = Vs[t * LDK + ch];
        const float4 a = *reinterpret_cast<const float4*>(Ps + t * TR), e = *reinterpret_cast<const float4*>(Ps + t * TR + 4);
        const float pr[8] = {a.x, a.y, a.z, a.w, e.x, e.y, e.z, e.w};
#pragma unroll
        for (int r = 0; r < TR; ++r) acc[x][r] = fmaf(pr[r], vv, acc[x][r]);
      }
    }
  }
  __syncthreads();
  const long long total = static_cast<long long>(c.B) * p.Hq * p.n_new;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * warp + i;
      alpha[r] = l[i] == 0.f ? 0.f : 1.f / l[i];
      if (r0 + r >= rows) continue;
      const float lse = m[i] + logf(l[i]);  // no key: -inf
      if (p.splits > 1)
        p.part_lse[split * total + row0 + r] = lse;
      else if (p.lse != nullptr)
        p.lse[row0 + r] = lse;
    }
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < NC; ++x) {
    const int ch = tid + x * kThreads;
    if (ch >= d) break;
#pragma unroll
    for (int r = 0; r < TR; ++r) {
      if (r0 + r >= rows) break;
      const float y = alpha[r] == 0.f ? 0.f : acc[x][r] * alpha[r] * c.v_scale;  // (v_scale / l may be too small a number)
      if (p.splits > 1)
        p.part_o[(split * total + row0 + r) * d + ch] = y;
      else if constexpr (sizeof(T) == 2)
        static_cast<T*>(p.o)[(row0 + r) * d + ch] = __float2bfloat16_rn(y);
      else
        static_cast<T*>(p.o)[(row0 + r) * d + ch] = y;
    }
  }
}

template <typename T, int NC>
cudaError_t launch_nc(const Cache4Attn& p, cudaStream_t s) {
  static seq::SmemOnce once;
  const cudaError_t e = once(fa_cache4_fwd_simt_kernel<T, NC>, smem_floats(NC * kThreads) * 4);
  if (e != cudaSuccess) return e;
  const long long blocks =
      static_cast<long long>(p.c.B) * p.c.Hkv * ((p.Hq / p.c.Hkv * static_cast<long long>(p.n_new) + TR - 1) / TR);
  if (blocks > 0x7fffffffLL || p.splits > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), p.splits);
  fa_cache4_fwd_simt_kernel<T, NC><<<grid, kThreads, smem_floats(p.c.d) * 4, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_t(const Cache4Attn& p, cudaStream_t s) {
  if (p.c.d <= 128) return launch_nc<T, 1>(p, s);
  if (p.c.d <= 256) return launch_nc<T, 2>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// Splits of the keys: as many CTAs as fit the SMs at once, or a tile a split.
int cache4_simt_splits(int B, int Hq, int Hkv, int n_new, int n_keys, int d) {
  const long long blocks =
      static_cast<long long>(B) * Hkv * ((static_cast<long long>(Hq / Hkv) * n_new + TR - 1) / TR);
  const int tiles = (n_keys + BK - 1) / BK, fit = 227 * 1024 / (smem_floats(d) * 4 + 1024);
  long long n = fit * 152LL / blocks;
  if (n > tiles) n = tiles;
  if (n > 64) n = 64;
  return n < 1 ? 1 : static_cast<int>(n);
}

cudaError_t launch_cache4_simt(const Cache4Attn& p, fa_dtype dt, cudaStream_t s) {
  return dt == FA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace fa
