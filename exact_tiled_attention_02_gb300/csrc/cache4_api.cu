// cache4_api.cu -- the C ABI of the 4-bit key/value cache declared in
// include/fa.h: writing new tokens, reading tokens back, attention over it.
// Argument checks, workspace layouts, dispatch.  Nothing here allocates device
// memory or synchronises.
#include "seq_checks.h"

namespace fa {
namespace {

constexpr int kMaxD = 256;

fa_status cache_check(const void* cache, const int* table, const int* lens, int B, int Hkv, int n_pages, int page_size,
                      int max_pages, int d, float k_scale, float v_scale, fa_dtype dt) {
  if (!cache || !lens || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4)) return FA_ERR_INVALID;
  if (!sizes_ok(n_pages, Hkv, page_size, d) || !sizes_ok(B, Hkv) || max_pages < 1) return FA_ERR_INVALID;
  if (!sizes_ok(B, max_pages) || paged_keys(page_size, max_pages) < 0) return FA_ERR_INVALID;
  if (!table && (max_pages != 1 || n_pages < B)) return FA_ERR_INVALID;
  if (!scale_ok(k_scale) || !scale_ok(v_scale) || !dtype_ok(dt)) return FA_ERR_INVALID;
  if (page_size % 16 != 0 || d % 16 != 0 || d > kMaxD) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}
// a warp a block of 16 tokens and head, four a CTA; a sequence's are counted in 31 bits
bool blocks_ok(int B, int Hkv, int n) {
  if (!sizes_ok(B, Hkv, n) || n > 0x3fffffff) return false;
  const long long per = static_cast<long long>(Hkv) * ((n + 14) / 16 + 1);
  return per <= 0x7fffffffLL && static_cast<double>(B) * per < 4.0 * 0x7ffffff0;
}
Cache4 cache_of(const void* cache, const int* table, const int* lens, int B, int Hkv, int n_pages, int page_size,
                int max_pages, int d, float k_scale, float v_scale) {
  Cache4 c{};
  c.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  c.table = table;
  c.lens = lens;
  c.B = B;
  c.Hkv = Hkv;
  c.d = d;
  c.page_size = page_size;
  c.max_pages = max_pages;
  c.n_pages = n_pages;
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  return c;
}

bool attn_sizes_ok(int B, int Hq, int Hkv, int Nq, int page_size, int max_pages, int d) {
  if (Hkv < 1 || Hq % Hkv != 0 || page_size < 1 || d > kMaxD) return false;
  const long long keys = paged_keys(page_size, max_pages);
  return sizes_ok(B, Hq, Nq, d) && sizes_ok(B, max_pages) && keys > 0 &&
         static_cast<long long>(B) * Hq * Nq <= 0x7fffffffLL / 8 &&
         tiles_ok(B, keys) &&  // and a CTA's tiles of 128, at least 304 ranges sharing those of all groups of rows
         B * ((keys + 127) / 128) * Hkv / 304 < 0x7fffffffLL / ((static_cast<long long>(Hq / Hkv) * Nq + 15) / 16);
}
PartLayout attn_layout(int B, int Hq, int Hkv, int Nq, int n_keys, int d) {
  return part_layout(cache4_simt_splits(B, Hq, Hkv, Nq, n_keys, d), 0, static_cast<long long>(B) * Hq * Nq, d);
}
// on the tensor cores: the pieces of sequences that several CTAs share
bool tensor_cores(int d) { return d == 64 || d == 96 || d == 128; }
DecodePlan attn_plan(int B, int Hq, int Hkv, int Nq, int d, fa_dtype dt) {
  return cache4_plan(B, Hkv, Hq / Hkv * Nq, d, dt, 152);
}
PartLayout attn_layout_tc(const DecodePlan& plan, int d) {
  const long long pieces = static_cast<long long>(plan.heads) * plan.row_groups * plan.n_seq + plan.cuts;
  return part_layout(1, 0, pieces * plan.nr, d);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cache_fp4_bytes(int n_pages, int Hkv, int page_size, int d) {
  if (!sizes_ok(n_pages, Hkv, page_size, d) || page_size % 16 != 0 || d % 16 != 0 || d > kMaxD) return 0;
  return static_cast<size_t>(n_pages) * Hkv * page_size * (9 * d / 8);
}

fa_status fa_cache_fp4_write(const void* k, const void* v, void* cache, const int* block_table, const int* lens,
                             const int* n_new, int B, int Hkv, int Nn, int n_pages, int page_size, int max_pages,
                             int d, float k_scale, float v_scale, fa_dtype dt, void* stream) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(n_new, 4)) return FA_ERR_INVALID;
  const fa_status st =
      cache_check(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale, dt);
  if (st != FA_OK) return st;
  if (!sizes_ok(B, Hkv, Nn, d) || !blocks_ok(B, Hkv, Nn)) return FA_ERR_INVALID;
  Cache4 c = cache_of(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale);
  if (device_status_ptr(&c.status) != cudaSuccess) return FA_ERR_CUDA;
  return of(launch_cache4_write(c, k, v, n_new, Nn, dt, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_fp4_read(const void* cache, const int* block_table, const int* lens, const int* first, void* k,
                            void* v, int B, int Hkv, int N, int n_pages, int page_size, int max_pages, int d,
                            float k_scale, float v_scale, fa_dtype dt, void* stream) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(first, 4)) return FA_ERR_INVALID;
  const fa_status st =
      cache_check(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale, dt);
  if (st != FA_OK) return st;
  if (!sizes_ok(B, Hkv, N, d) || !blocks_ok(B, Hkv, N)) return FA_ERR_INVALID;
  Cache4 c = cache_of(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale);
  if (device_status_ptr(&c.status) != cudaSuccess) return FA_ERR_CUDA;
  return of(launch_cache4_read(c, first, k, v, N, dt, static_cast<cudaStream_t>(stream)));
}

size_t fa_fwd_cache_fp4_workspace_bytes(int B, int Hq, int Hkv, int Nq, int page_size, int max_pages, int d) {
  if (!attn_sizes_ok(B, Hq, Hkv, Nq, page_size, max_pages, d)) return 0;
  if (tensor_cores(d)) {
    const size_t f32 = attn_layout_tc(attn_plan(B, Hq, Hkv, Nq, d, FA_DTYPE_F32), d).bytes;
    const size_t bf16 = attn_layout_tc(attn_plan(B, Hq, Hkv, Nq, d, FA_DTYPE_BF16), d).bytes;
    return f32 > bf16 ? f32 : bf16;
  }
  return attn_layout(B, Hq, Hkv, Nq, static_cast<int>(paged_keys(page_size, max_pages)), d).bytes;
}

fa_status fa_fwd_cache_fp4(const void* q, const void* cache, const int* block_table, const int* lens, void* o,
                           float* lse, int B, int Hq, int Hkv, int Nq, int n_pages, int page_size, int max_pages,
                           int d, float scale, float k_scale, float v_scale, fa_dtype dt, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!q || !o || !workspace || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
    return FA_ERR_INVALID;
  if (!attn_sizes_ok(B, Hq, Hkv, Nq, page_size, max_pages, d) && d <= kMaxD) return FA_ERR_INVALID;
  const fa_status st =
      cache_check(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale, dt);
  if (st != FA_OK) return st;
  if (!scale_ok(scale) || !std::isnormal(scale * k_scale) || !std::isfinite(scale * k_scale * 1.4426950408889634f))
    return FA_ERR_INVALID;  // scores are multiplied with these in float32
  if (workspace_bytes < fa_fwd_cache_fp4_workspace_bytes(B, Hq, Hkv, Nq, page_size, max_pages, d))
    return FA_ERR_INVALID;
  Cache4 c = cache_of(cache, block_table, lens, B, Hkv, n_pages, page_size, max_pages, d, k_scale, v_scale);
  if (device_status_ptr(&c.status) != cudaSuccess) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tensor_cores(d)) {
    const DecodePlan plan = attn_plan(B, Hq, Hkv, Nq, d, dt);
    SeqAttn a{};
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.groups = B * Hkv;
    a.rows = Hq / Hkv * Nq;
    a.group_div = Hkv;
    a.row_block = kAllRows;
    a.n_new = Nq;
    a.q_s1 = static_cast<long long>(Hq) * Nq;
    a.q_s2 = a.rows;
    a.d1 = a.dv = d;
    a.n_keys = page_size * max_pages;
    a.lens = lens;
    a.lens_div = Hkv;
    a.causal = 1;
    a.scale = scale;
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + attn_layout_tc(plan, d).off_lse);
    a.total = static_cast<long long>(B) * Hq * Nq;
    a.status = c.status;
    a.wait_ns = device_wait_ns();
    cudaError_t e = launch_cache4_decode(a, c, plan, dt, s);
    if (e == cudaSuccess) e = launch_cache4_merge(a, plan, dt, s);
    return of(e);
  }
  const PartLayout w = attn_layout(B, Hq, Hkv, Nq, page_size * max_pages, d);
  Cache4Attn p{};
  p.c = c;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.Hq = Hq;
  p.n_new = Nq;
  p.scale = scale;
  p.splits = w.splits_a;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.off_lse);
  const cudaError_t e = launch_cache4_simt(p, dt, s);
  if (e != cudaSuccess || p.splits == 1) return of(e);
  return of(launch_seq_combine(p.part_o, p.part_lse, p.splits, static_cast<long long>(B) * Hq * Nq, d, o, dt, lse, s));
}

}  // extern "C"
