// seq_kernels.h -- internal interface between the C-ABI layer (seq_api.cu)
// and the kernels of the language-model operators: latent attention
// (expanded and absorbed) and shared-prefix attention.  Not part of the
// public ABI.
#pragma once

#include "kernels.h"

namespace fa {

// Status bit: a length or page index in device memory was out of range (not read past).
constexpr unsigned int kStatusInput = 1u;  // matches FA_ERR_INVALID
constexpr int kAllRows = 0x7fffffff;  // SeqAttn::row_block of a problem whose rows are one block

// One attention problem family: groups of query rows, each group against its
// own keys.  Every index is in rows (tokens), never in bytes.
struct SeqAttn {
  // query row r of group g is row
  //   (g / group_div) * q_s1 + (g % group_div) * q_s2 + (r / row_block) * q_s3 + r % row_block
  // of q, o and lse (q rows have dk = d1 + d2 entries, o rows dv), and token
  // r % n_new of its sequence's n_new new ones
  const void* q;
  void* o;
  float* lse;  // may be null
  int groups, rows;
  int group_div, row_block, n_new;
  long long q_s1, q_s2, q_s3;
  // keys j < nk: nk = n_keys, or lens[g / lens_div] where lens is given
  // (clamped to 0 .. n_keys).  A key's entries are k1 row (g * n_keys + j) and
  // k2 row ((g / k2_div) * n_keys + j); its value is v row (g * n_keys + j).
  // With page_size > 0 the k1 and v row is page * page_size + j % page_size
  // instead, page = table[g * max_pages + j / page_size], or g without a table.
  const void* k1;
  const void* k2;
  const void* v;
  int d1, d2, dv, v_stride;  // v rows are v_stride entries apart
  int n_keys, k2_div;
  const int* lens;
  int lens_div;
  const int* table;
  int page_size, max_pages, n_pages;
  // a row sees keys j < nk - (causal ? n_new - 1 - r % n_new : 0)
  int causal;
  float scale;
  // splits > 1 or part_o given: results go to part_o [part0 + split][total][dv]
  // and part_lse [part0 + split][total] (fp32) instead of o and lse
  int splits;
  float* part_o;
  float* part_lse;
  int part0;
  long long total;  // rows of o
  int ctas;         // rows kernel: at most so many CTAs (0: one an SM)
  unsigned int* status;
  unsigned long long wait_ns;
};

// float32 on CUDA cores (seq_fwd_simt.cu).  beside: the kernel before it on the
// stream is the same call's and independent.
cudaError_t launch_seq_simt(const SeqAttn& p, bool beside, cudaStream_t s);
// Splits of the keys that give the launch `ctas` blocks an SM.
int seq_simt_splits(long long groups, int rows, int max_keys, int ctas);

// bf16 on the tensor cores, many rows a group (seq_rows_sm103.cu): no lens, no
// pages; the expanded latent shape to o and lse, or d = 64, 96, 128 to partial
// results.
cudaError_t launch_seq_rows(const SeqAttn& p, cudaStream_t s);
// The work items of a partial-result call before its keys are split, and the
// time (us) it takes on n CTAs.
int seq_rows_items(int groups, int rows, int row_block);
double seq_rows_time(int groups, int rows, int row_block, int n_keys, int d, int n, int splits);

// bf16 on the tensor cores, few rows a group over (paged) caches
// (seq_decode_sm103.cu).  Groups are (sequence, head) pairs, lens per
// sequence; the tiles of all sequences are cut into `cuts` ranges per head and
// group of nr rows.  Pieces go to part_o [slot][dv] and part_lse [slot], slot
// = ((row group * (cuts + n_seq)) + cut + sequence) * nr + row.
struct DecodePlan {
  int n_seq, heads;
  int nr;          // query rows of a CTA: 16, 32 or 64
  int row_groups;  // of nr rows each
  int cuts;
  int direct;      // keys and values shared (the latent form): whole sequences go straight to o and lse
  int box;         // tokens of one load: 64, or 32 or 16 where pages are not whole tiles
};
DecodePlan decode_plan(int n_seq, int heads, int rows, bool shared, int box, int sms);
size_t decode_slots(const DecodePlan& w);  // rows of part_o
// beside: as launch_seq_simt
cudaError_t launch_seq_decode(const SeqAttn& p, const DecodePlan& w, bool beside, cudaStream_t s);
// o, lse = the pieces merged, with the partial results pre_o [pre][total][dv]
// of other keys.  after: the kernels before it on the stream, back to one that
// was launched normally, are the same call's.
cudaError_t launch_seq_decode_merge(const SeqAttn& p, const DecodePlan& w, const float* pre_o, const float* pre_lse,
                                    int pre, bool after, cudaStream_t s);

// o, lse = the merged partial results [splits][total] (seq_combine.cu).
cudaError_t launch_seq_combine(const float* part_o, const float* part_lse, int splits, long long total, int dv,
                               void* o, fa_dtype dt, float* lse, cudaStream_t s);

// A key/value cache in 4 bits (layout and helpers: cache4.cuh).
struct Cache4 {
  uint8_t* cache;    // [n_pages][Hkv][page_size / 16] blocks of 18 d bytes
  const int* table;  // [B][max_pages], or null: sequence b is page b
  const int* lens;   // [B]
  int B, Hkv, d;
  int page_size, max_pages, n_pages;
  float k_scale, v_scale;
  unsigned int* status;
};
// New tokens k, v [B,Hkv,Nn,d] to the positions before lens (cache4_rw.cu).
cudaError_t launch_cache4_write(const Cache4& c, const void* k, const void* v, const int* n_new, int Nn, fa_dtype dt,
                                cudaStream_t s);
// Positions first[b] .. first[b] + N - 1 (from 0 where first is null) to k, v [B,Hkv,N,d].
cudaError_t launch_cache4_read(const Cache4& c, const int* first, void* k, void* v, int N, fa_dtype dt, cudaStream_t s);

// Attention of each sequence's last n_new tokens, q and o [B,Hq,n_new,d], over
// the cache.
struct Cache4Attn {
  Cache4 c;
  const void* q;
  void* o;
  float* lse;  // may be null
  int Hq, n_new;
  float scale;
  // splits > 1: results go to part_o [split][B Hq n_new][d] and part_lse [split][B Hq n_new] instead of o and lse
  int splits;
  float* part_o;
  float* part_lse;
};
// On CUDA cores, any type and d (cache4_fwd_simt.cu).
cudaError_t launch_cache4_simt(const Cache4Attn& p, fa_dtype dt, cudaStream_t s);
int cache4_simt_splits(int B, int Hq, int Hkv, int n_new, int n_keys, int d);

// On the tensor cores, d = 64, 96 or 128 (cache4_decode_sm103.cu).  p: as for
// launch_seq_decode, groups (sequence, key/value head), page fields and k1, v unused.
// Ranges are flat (seq_ranges.cuh): plan.cuts of them over all groups of rows; slot = range + row group * n_seq + sequence.
DecodePlan cache4_plan(int n_seq, int heads, int rows, int d, fa_dtype dt, int sms);
cudaError_t launch_cache4_decode(const SeqAttn& p, const Cache4& c, const DecodePlan& w, fa_dtype dt, cudaStream_t s);
cudaError_t launch_cache4_merge(const SeqAttn& p, const DecodePlan& w, fa_dtype dt, cudaStream_t s);

// Expanded latent attention's backward.
struct LatentBwd {
  const void* q;   // [B,H,Nq,dn+dr]
  const void* kn;  // [B,H,Nk,dn]
  const void* kr;  // [B,Nk,dr]
  const void* v;   // [B,H,Nk,dv]
  const void* o;
  const void* dO;  // [B,H,Nq,dv]
  const float* lse;
  void* dq;
  void* dkn;
  void* dkr;
  void* dv_out;
  int B, H, Nq, Nk, dn, dr, dv;
  int causal;
  float scale;
  // workspace: lse2 and dsum [B*H][Nq rounded up to 128] fp32 (-lse log2 e and
  // -D; rows past Nq: -inf and 0), dkr_part [B*H][Nk][dr] fp32
  float* lse2;
  float* dsum;
  float* dkr_part;
  unsigned int* status;
  unsigned long long wait_ns;
};
size_t latent_bwd_workspace_layout(int B, int H, int Nq, int Nk, int dr, size_t* off_dsum, size_t* off_part);
cudaError_t launch_latent_bwd_prep(const LatentBwd& p, fa_dtype dt, cudaStream_t s);
// bf16 on the tensor cores (latent_bwd_sm103.cu)
cudaError_t launch_latent_bwd_sm103(const LatentBwd& p, cudaStream_t s);
cudaError_t launch_latent_bwd_simt(const LatentBwd& p, cudaStream_t s);  // float32
// dkr = the sum over heads of dkr_part
cudaError_t launch_latent_bwd_dkr(const LatentBwd& p, fa_dtype dt, cudaStream_t s);

// From fa_api.cu: the device status word of the current device, the time
// limit of device-side waits, cuTensorMapEncodeTiled.
cudaError_t device_status_ptr(unsigned int** out);
unsigned long long device_wait_ns();
EncodeTiledFnPtr encode_tiled_fn();

}  // namespace fa
