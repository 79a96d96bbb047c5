// seq_api.cu -- the C ABI of the language-model operators declared in
// include/fa.h: latent attention (expanded forward and backward, absorbed)
// and shared-prefix attention.  Argument checks, workspace layouts, dispatch.
// Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "seq_checks.h"

namespace fa {
namespace {

PartLayout prefix_layout(int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d) {
  const int G = Hq / Hkv;
  // The prefix's kernel and the sequences' run side by side, a CTA an SM each
  // (7 x 8 heads x 3 tokens, 2999 + 333 keys, d = 80: 37.6 us; two each, 46.6).
  const int sp = seq_simt_splits(Hkv, B * G * Nq, Np, Ns > 0 ? 1 : 2);
  const int ss = seq_simt_splits(static_cast<long long>(B) * Hkv, G * Nq, Ns, Np > 0 ? 1 : 2);
  return part_layout(sp, ss, static_cast<long long>(B) * Hq * Nq, d);
}
// bf16: the prefix's splits [splits][rows], then the pieces of the sequences
struct PrefixLayout {
  int splits, ctas;  // of the prefix's part
  DecodePlan plan;
  size_t off_pre_lse, off_o, off_lse, bytes;
};
// The prefix's part is bound by the tensor cores, the sequences' own part by
// memory, and a CTA of the first takes a whole SM: so they run side by side on
// SMs of their own (n and 152 - n) where that is faster than one after the
// other, by measured rates: the first as seq_rows_time, the second 5 us and a
// time an SM for a 64-key tile by its row columns (16, 32, 64), up to 6.2 TB/s
// of keys and values, the merge 4 us and 5 TB/s of partial results.  While the
// second runs, the first takes 1.5 times as long where one item reads a prefix
// tile (2.2 us a tile for 1.45), 1.25 times where two share it, and so on.
// The host does not see the lengths: the plan takes every sequence as three
// quarters of its room, and the kernels keep its division whatever they are.
// us, side by side by that plan and one after the other, with lengths of 2, 25,
// 50, 75 and 100% of the room:
//   128 x 32 heads x 4 tokens, 32768 + 2048 keys, d = 128:
//     255 258 260 265 300   and   213 248 286 322 360
//   64 x 32 x 1, 16384 + 1024:
//     45 50 55 60 71        and   51 61 74 83 93
// So a batch of drafted tokens that has just begun to generate in a large room
// loses by the division up to about a third of the room, and gains from there on.
PrefixLayout prefix_layout_bf16(int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d) {
  PrefixLayout w{};
  const int G = Hq / Hkv, R = B * G * Nq, block = G * Nq, kSms = 152;
  const size_t rows = static_cast<size_t>(B) * Hq * Nq;
  const double own_bytes = 0.75 * 4.0 * B * Hkv * d * Ns;  // the sequences' keys and values
  const int nr = decode_plan(B, Hkv, block, false, 64, kSms).nr;
  const double sm_rate = 256.0 * d / (nr == 16 ? 0.36 : nr == 32 ? 0.42 : 0.69);  // bytes a us
  auto own_time = [&](int sms) {
    const double rate = sm_rate * sms < 6.2e6 ? sm_rate * sms : 6.2e6;
    return own_bytes > 0 ? 5.0 + own_bytes / rate : 0.0;
  };
  int own_sms = kSms;
  if (Np > 0) {
    const int items = seq_rows_items(Hkv, R, block), tiles = (Np + 127) / 128;
    const double slow = 0.5 * Hkv / items;  // items a head read the same prefix through L2
    double best = 1e30;
    for (int n = kSms; n >= 8; n -= 8) {
      if (n < kSms && Ns == 0) break;
      for (int k = 1; k <= 4; ++k) {  // rounds of items to aim at
        int s = static_cast<int>(static_cast<long long>(k) * n / items);
        if (s < 1) s = 1;
        if (s > tiles) s = tiles;
        if (s > 64) s = 64;
        const double r = seq_rows_time(Hkv, R, block, Np, d, n, s), own = own_time(n == kSms ? kSms : kSms - n);
        const double merge = 4.0 + static_cast<double>(s) * rows * d * 8.0 / 5e6;
        const double all = r * (1.0 + slow), part = r + own * slow / (1.0 + slow), beside = all < part ? all : part;
        const double t = merge + (n == kSms ? r + own : beside > own ? beside : own);
        if (t < best) {
          best = t;
          w.splits = s;
          w.ctas = n;
        }
      }
    }
    if (w.ctas < kSms) own_sms = kSms - w.ctas;
  }
  w.plan = decode_plan(B, Hkv, block, false, 64, own_sms);
  const size_t slots = Ns > 0 ? decode_slots(w.plan) : 0;
  w.off_pre_lse = up256(w.splits * rows * d * 4);
  w.off_o = w.off_pre_lse + up256(w.splits * rows * 4);
  w.off_lse = w.off_o + up256(slots * d * 4);
  w.bytes = w.off_lse + up256(slots * 4);
  return w;
}
bool prefix_sizes_ok(int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d) {
  // (Np past 2^31 - 256 would round up to tiles past 32 bits; Ns is held lower by tiles_ok)
  if (Np < 0 || Np > 0x7fffff00 || Ns < 0 || Hkv < 1 || Hq % Hkv != 0) return false;
  return sizes_ok(B, Hq, Nq, d) && sizes_ok(B, Hkv, Ns > 0 ? Ns : 1, d) && sizes_ok(Hkv, Np > 0 ? Np : 1, d) &&
         static_cast<long long>(B) * Hq * Nq <= 0x7fffffffLL / 8 && tiles_ok(B, Ns);
}

PartLayout absorbed_layout(int B, int H, int Nq, int n_keys, int dc) {
  // Twice as many CTAs as SMs.  Past 128 value columns one CTA fills an SM, and
  // these are two rounds: that evens ragged lengths out where a CTA has few
  // tiles, and costs parts to merge where it has many.  us with two and with one
  // CTA an SM, lengths from 0 to the room and (in brackets) all equal to it:
  // 5 x 12 heads, 2047 tokens of 192 + 40: 25 33 (33 34); of 512 + 64: 40 62 (60
  // 62); 2 x 48, 3000 of 512 + 64: 62 81 (82 83); 4 x 20, 6000 of 192 + 40: 58 51
  // (69 51); 8 x 16, 2500 of 512 + 64: 84 79 (110 79).
  const int sp = seq_simt_splits(B, H * Nq, n_keys, 2);
  return part_layout(sp, 0, static_cast<long long>(B) * H * Nq, dc);
}
// bf16: the pieces of sequences that several CTAs share
PartLayout absorbed_layout_bf16(const DecodePlan& plan, int dc) {
  return part_layout(1, 0, static_cast<long long>(decode_slots(plan)), dc);
}
DecodePlan absorbed_plan(int B, int H, int Nq, int page_size, bool table) {
  const int box = !table || page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  return decode_plan(B, 1, H * Nq, true, box, 152);
}
// What the layouts and plans above count on (rows and tiles in 32 bits): the
// workspace query's check and part of the call's.
bool absorbed_sizes_ok(int B, int H, int Nq, int page_size, int max_pages, int dc) {
  if (!sizes_ok(B, H, Nq, dc) || dc > 4096 || !sizes_ok(B, max_pages) || page_size < 1) return false;
  const long long keys = paged_keys(page_size, max_pages);
  return static_cast<long long>(B) * H * Nq <= 0x7fffffffLL / 8 && keys > 0 && tiles_ok(B, keys);
}

bool expanded_sizes_ok(int B, int H, int Nq, int Nk, int dn, int dr, int dv) {
  return sizes_ok(B, H, Nq, dn) && sizes_ok(B, H, Nq, dr) && sizes_ok(B, H, Nq, dv) && sizes_ok(B, H, Nk, dn) &&
         sizes_ok(B, H, Nk, dr) && sizes_ok(B, H, Nk, dv) && dn <= 4096 && dr <= 4096 && dv <= 4096 &&
         static_cast<long long>(B) * H <= 0x7fffffffLL && Nq <= 0x3fffffff && Nk <= 0x3fffffff;
}
// and the backward's rows, padded to 128 a head: four a block of the float32 prep
bool expanded_bwd_sizes_ok(int B, int H, int Nq, int Nk, int dn, int dr, int dv) {
  return expanded_sizes_ok(B, H, Nq, Nk, dn, dr, dv) &&
         static_cast<long long>(B) * H <= ((1LL << 33) - 1) / ((Nq + 127) / 128 * 128LL);
}
fa_status expanded_check(int B, int H, int Nq, int Nk, int dn, int dr, int dv, float scale, int causal, fa_dtype dt) {
  if (!expanded_sizes_ok(B, H, Nq, Nk, dn, dr, dv)) return FA_ERR_INVALID;
  if (!scale_ok(scale) || !dtype_ok(dt) || (causal != 0 && causal != 1)) return FA_ERR_INVALID;
  if (dt == FA_DTYPE_BF16 && !(dn == 128 && dr == 64 && dv == 128)) return FA_ERR_UNSUPPORTED;
  if (dt == FA_DTYPE_F32 && (dn + dr > 256 || dv > 128)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d) {
  if (!prefix_sizes_ok(B, Hq, Hkv, Nq, Np, Ns, d)) return 0;
  const size_t f32 = prefix_layout(B, Hq, Hkv, Nq, Np, Ns, d).bytes;
  const size_t bf16 = prefix_layout_bf16(B, Hq, Hkv, Nq, Np, Ns, d).bytes;
  return f32 > bf16 ? f32 : bf16;
}

fa_status fa_fwd_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                               const int* lens, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Np, int Ns,
                               int d, float scale, fa_dtype dt, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!prefix_sizes_ok(B, Hq, Hkv, Nq, Np, Ns, d)) return FA_ERR_INVALID;
  if (!q || !o || !lens || !workspace || (Np > 0 && (!k_prefix || !v_prefix)) || (Ns > 0 && (!k || !v)))
    return FA_ERR_INVALID;
  const void* ptrs[] = {q, o, k_prefix, v_prefix, k, v};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return FA_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(lens, 4) || !aligned(workspace, 256)) return FA_ERR_INVALID;
  if (!scale_ok(scale) || !dtype_ok(dt)) return FA_ERR_INVALID;
  if (dt == FA_DTYPE_BF16 && d != 64 && d != 96 && d != 128) return FA_ERR_UNSUPPORTED;
  if (dt == FA_DTYPE_F32 && d > 128) return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < fa_fwd_shared_prefix_workspace_bytes(B, Hq, Hkv, Nq, Np, Ns, d)) return FA_ERR_INVALID;

  const int G = Hq / Hkv;
  SeqAttn p{};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.n_new = Nq;
  p.d1 = d;
  p.dv = d;
  p.v_stride = d;
  p.k2_div = 1;
  p.lens_div = 1;
  p.scale = scale;
  p.total = static_cast<long long>(B) * Hq * Nq;
  p.wait_ns = device_wait_ns();
  if (device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // the prefix: one group per key/value head, the rows of every sequence
  SeqAttn a = p;
  a.groups = Hkv;
  a.rows = B * G * Nq;
  a.group_div = Hkv;
  a.row_block = G * Nq;
  a.q_s2 = G * Nq;
  a.q_s3 = static_cast<long long>(Hq) * Nq;
  a.k1 = k_prefix;
  a.v = v_prefix;
  a.n_keys = Np;
  // the sequences' own keys: one group per sequence and key/value head
  SeqAttn b = p;
  b.groups = B * Hkv;
  b.rows = G * Nq;
  b.group_div = Hkv;
  b.row_block = kAllRows;
  b.q_s1 = static_cast<long long>(Hq) * Nq;
  b.q_s2 = G * Nq;
  b.k1 = k;
  b.v = v;
  b.n_keys = Ns;
  b.lens = lens;
  b.lens_div = Hkv;
  b.causal = 1;
  char* base = static_cast<char*>(workspace);
  if (dt == FA_DTYPE_BF16) {
    const PrefixLayout w = prefix_layout_bf16(B, Hq, Hkv, Nq, Np, Ns, d);
    a.part_o = reinterpret_cast<float*>(base);
    a.part_lse = reinterpret_cast<float*>(base + w.off_pre_lse);
    a.splits = w.splits;
    a.ctas = w.ctas;
    b.part_o = reinterpret_cast<float*>(base + w.off_o);
    b.part_lse = reinterpret_cast<float*>(base + w.off_lse);
    cudaError_t e = cudaSuccess;
    if (Np > 0) e = launch_seq_rows(a, s);
    if (e == cudaSuccess && Ns > 0) e = launch_seq_decode(b, w.plan, Np > 0, s);
    if (e == cudaSuccess) e = launch_seq_decode_merge(b, w.plan, a.part_o, a.part_lse, w.splits, Np > 0 || Ns > 0, s);
    return of(e);
  }
  const PartLayout w = prefix_layout(B, Hq, Hkv, Nq, Np, Ns, d);
  a.part_o = b.part_o = reinterpret_cast<float*>(base);
  a.part_lse = b.part_lse = reinterpret_cast<float*>(base + w.off_lse);
  a.splits = w.splits_a;
  a.part0 = 0;
  b.splits = w.splits_b;
  b.part0 = w.splits_a;
  cudaError_t e = launch_seq_simt(a, false, s);
  if (e == cudaSuccess) e = launch_seq_simt(b, true, s);
  if (e == cudaSuccess)
    e = launch_seq_combine(a.part_o, a.part_lse, w.splits_a + w.splits_b, p.total, d, o, dt, lse, s);
  return of(e);
}

size_t fa_fwd_latent_absorbed_workspace_bytes(int B, int H, int Nq, int page_size, int max_pages, int dc) {
  if (!absorbed_sizes_ok(B, H, Nq, page_size, max_pages, dc)) return 0;
  const size_t f32 = absorbed_layout(B, H, Nq, static_cast<int>(paged_keys(page_size, max_pages)), dc).bytes;
  const size_t bf16 = absorbed_layout_bf16(absorbed_plan(B, H, Nq, page_size, true), dc).bytes;
  return f32 > bf16 ? f32 : bf16;
}

fa_status fa_fwd_latent_absorbed(const void* q, const void* cache, const int* block_table, const int* lens, void* o,
                                 float* lse, int B, int H, int Nq, int n_pages, int page_size, int max_pages, int dc,
                                 int dr, float scale, fa_dtype dt, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!q || !cache || !lens || !o || !workspace) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(o, 16) || !aligned(workspace, 256)) return FA_ERR_INVALID;
  if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return FA_ERR_INVALID;
  if (!absorbed_sizes_ok(B, H, Nq, page_size, max_pages, dc)) return FA_ERR_INVALID;
  if (!sizes_ok(B, H, Nq, dr) || dr > 4096 || !sizes_ok(n_pages, page_size, dc + dr)) return FA_ERR_INVALID;
  if (!block_table && (max_pages != 1 || n_pages < B)) return FA_ERR_INVALID;
  if (!scale_ok(scale) || !dtype_ok(dt)) return FA_ERR_INVALID;
  if (dt == FA_DTYPE_BF16 && !((dc == 256 || dc == 512) && dr == 64)) return FA_ERR_UNSUPPORTED;
  if (dt == FA_DTYPE_BF16 && block_table && page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (dt == FA_DTYPE_F32 && (dc > 512 || dr > 128)) return FA_ERR_UNSUPPORTED;
  const int n_keys = static_cast<int>(paged_keys(page_size, max_pages));
  if (workspace_bytes < fa_fwd_latent_absorbed_workspace_bytes(B, H, Nq, page_size, max_pages, dc))
    return FA_ERR_INVALID;

  SeqAttn p{};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.groups = B;
  p.rows = H * Nq;
  p.group_div = 1;
  p.row_block = kAllRows;
  p.n_new = Nq;
  p.q_s1 = static_cast<long long>(H) * Nq;
  p.k1 = cache;
  p.v = cache;
  p.d1 = dc + dr;
  p.dv = dc;
  p.v_stride = dc + dr;
  p.n_keys = n_keys;
  p.k2_div = 1;
  p.lens = lens;
  p.lens_div = 1;
  p.table = block_table;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.causal = 1;
  p.scale = scale;
  p.total = static_cast<long long>(B) * H * Nq;
  p.wait_ns = device_wait_ns();
  if (device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.part_o = static_cast<float*>(workspace);
  if (dt == FA_DTYPE_BF16) {
    const DecodePlan plan = absorbed_plan(B, H, Nq, page_size, block_table != nullptr);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + absorbed_layout_bf16(plan, dc).off_lse);
    cudaError_t e = launch_seq_decode(p, plan, false, s);
    if (e == cudaSuccess) e = launch_seq_decode_merge(p, plan, nullptr, nullptr, 0, true, s);
    return of(e);
  }
  const PartLayout w = absorbed_layout(B, H, Nq, n_keys, dc);
  p.splits = w.splits_a;
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.off_lse);
  if (w.splits_a == 1) p.part_o = p.part_lse = nullptr;
  const cudaError_t e = launch_seq_simt(p, false, s);
  if (e != cudaSuccess || w.splits_a == 1) return of(e);
  return of(launch_seq_combine(p.part_o, p.part_lse, w.splits_a, p.total, dc, o, dt, lse, s));
}

fa_status fa_fwd_latent(const void* q, const void* k_nope, const void* k_rope, const void* v, void* o, float* lse,
                        int B, int H, int Nq, int Nk, int dn, int dr, int dv, float scale, int causal, fa_dtype dt,
                        void* stream) {
  const void* ptrs[] = {q, k_nope, k_rope, v, o};
  for (const void* x : ptrs)
    if (!x || !aligned(x, 16)) return FA_ERR_INVALID;
  if (!aligned(lse, 4)) return FA_ERR_INVALID;
  const fa_status c = expanded_check(B, H, Nq, Nk, dn, dr, dv, scale, causal, dt);
  if (c != FA_OK) return c;
  SeqAttn p{};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.groups = B * H;
  p.rows = Nq;
  p.group_div = 1;
  p.row_block = kAllRows;
  p.n_new = Nq;
  p.q_s1 = Nq;
  p.k1 = k_nope;
  p.k2 = k_rope;
  p.v = v;
  p.d1 = dn;
  p.d2 = dr;
  p.dv = dv;
  p.v_stride = dv;
  p.n_keys = Nk;
  p.k2_div = H;
  p.lens_div = 1;
  p.causal = causal;
  p.scale = scale;
  p.splits = 1;
  p.total = static_cast<long long>(B) * H * Nq;
  p.wait_ns = device_wait_ns();
  if (device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return of(dt == FA_DTYPE_BF16 ? launch_seq_rows(p, s) : launch_seq_simt(p, false, s));
}

size_t fa_bwd_latent_workspace_bytes(int B, int H, int Nq, int Nk, int dn, int dr, int dv) {
  if (!expanded_bwd_sizes_ok(B, H, Nq, Nk, dn, dr, dv)) return 0;
  return latent_bwd_workspace_layout(B, H, Nq, Nk, dr, nullptr, nullptr);
}

fa_status fa_bwd_latent(const void* q, const void* k_nope, const void* k_rope, const void* v, const void* o,
                        const float* lse, const void* dO, void* dq, void* dk_nope, void* dk_rope, void* dv_out, int B,
                        int H, int Nq, int Nk, int dn, int dr, int dv, float scale, int causal, fa_dtype dt,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const void* ptrs[] = {q, k_nope, k_rope, v, o, dO, dq, dk_nope, dk_rope, dv_out};
  for (const void* x : ptrs)
    if (!x || !aligned(x, 16)) return FA_ERR_INVALID;
  if (!lse || !aligned(lse, 4) || !workspace || !aligned(workspace, 256)) return FA_ERR_INVALID;
  if (!expanded_bwd_sizes_ok(B, H, Nq, Nk, dn, dr, dv)) return FA_ERR_INVALID;
  const fa_status c = expanded_check(B, H, Nq, Nk, dn, dr, dv, scale, causal, dt);
  if (c != FA_OK) return c;
  if (workspace_bytes < fa_bwd_latent_workspace_bytes(B, H, Nq, Nk, dn, dr, dv)) return FA_ERR_INVALID;
  LatentBwd p{};
  p.q = q;
  p.kn = k_nope;
  p.kr = k_rope;
  p.v = v;
  p.o = o;
  p.dO = dO;
  p.lse = lse;
  p.dq = dq;
  p.dkn = dk_nope;
  p.dkr = dk_rope;
  p.dv_out = dv_out;
  p.B = B;
  p.H = H;
  p.Nq = Nq;
  p.Nk = Nk;
  p.dn = dn;
  p.dr = dr;
  p.dv = dv;
  p.causal = causal;
  p.scale = scale;
  size_t off_dsum = 0, off_part = 0;
  latent_bwd_workspace_layout(B, H, Nq, Nk, dr, &off_dsum, &off_part);
  p.lse2 = static_cast<float*>(workspace);
  p.dsum = reinterpret_cast<float*>(static_cast<char*>(workspace) + off_dsum);
  p.dkr_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + off_part);
  p.wait_ns = device_wait_ns();
  if (device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_latent_bwd_prep(p, dt, s);
  if (e == cudaSuccess) e = dt == FA_DTYPE_BF16 ? launch_latent_bwd_sm103(p, s) : launch_latent_bwd_simt(p, s);
  if (e == cudaSuccess) e = launch_latent_bwd_dkr(p, dt, s);
  return of(e);
}

}  // extern "C"
