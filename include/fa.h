/*
 * fa.h -- C ABI of the exact tiled attention library (libfa.so) for NVIDIA
 * GB300 (sm_103a).
 *
 * The operation is exact scaled-dot-product attention, per (batch, head):
 *
 *     S = Q K^T * scale,   P = softmax_row(S),   O = P V,
 *     lse_i = ln sum_j exp(S_ij)
 *
 * as stated in "Flash attention and efficient attention -- Hinglish notes",
 * section "The Standard Attention Problem" (the page's "S / d_k" reads as
 * S / sqrt(d_k): its worked example's 0.707 for d = 2 needs the square root),
 * computed one tile at a time with running max / running sum statistics as in
 * that page's "Derivation: Incremental Softmax" (Steps 1-3) and in "Compute
 * attention one tile at a time" (TensorViz), step "tiles", so the N x N score
 * matrix never reaches device memory.  The optional local window follows the
 * notes' "Worked example Local Attention Window": query i attends to key j
 * iff |i - j| <= (window - 1) / 2.  The backward pass recomputes S and P on
 * chip from Q, K, V, O, dO and the saved lse ("Backward Pass: Recomputation").
 *
 * Common conventions for every entry point
 * ----------------------------------------
 * Layout     Q, K, V, O, dO, dQ, dK, dV are dense, contiguous, row-major
 *            [B, H, N, d] arrays in device memory; lse is [B, H, N] float32.
 *            Every base pointer must be 16-byte aligned.
 * dtype      FA_DTYPE_BF16: Q/K/V/O/dO/dQ/dK/dV are bfloat16, arithmetic is
 *            fp32-accumulated tensor-core math with P rounded to bf16 before
 *            the P V product; d must be 64, 96, 128 or 256 (256: forward
 *            only).
 *            FA_DTYPE_F32: all arrays are float32 and all arithmetic is exact
 *            fp32 on CUDA cores with the accurate expf/logf; 1 <= d <= 128.
 * scale      finite and > 0; usually 1/sqrt(d).
 * window     <= 0: unmasked.  Otherwise an odd full width w; r = (w - 1) / 2.
 *            Even widths are rejected (the pages give them no meaning).
 * stream     a cudaStream_t passed as void*; NULL is the legacy default
 *            stream.  All work is enqueued on it; no call synchronises except
 *            fa_last_device_status().
 * Ownership  the caller owns every buffer.  The library allocates no device
 *            memory and keeps no pointer after a call returns.
 * Errors     argument errors are detected on the host before anything is
 *            launched and return FA_ERR_INVALID or FA_ERR_UNSUPPORTED with no
 *            side effect.  A failed launch returns FA_ERR_CUDA.  Every wait
 *            inside the kernels is bounded in time; a wait that runs out
 *            records FA_ERR_TIMEOUT in the library's device status word and
 *            the kernel returns early (its outputs are then undefined), which
 *            fa_last_device_status() reports.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID = 1,      /* bad pointer, size, alignment, scale or window */
  FA_ERR_UNSUPPORTED = 2,  /* valid request this build does not implement (dtype/d) */
  FA_ERR_CUDA = 3,         /* a CUDA runtime/driver call or launch failed */
  FA_ERR_TIMEOUT = 4       /* a bounded device-side wait ran out */
} fa_status;

typedef enum { FA_DTYPE_F32 = 0, FA_DTYPE_BF16 = 1 } fa_dtype;

/*
 * Forward pass: O = softmax(Q K^T * scale) V, and lse.
 *   q, k, v  [B,H,N,d] inputs (read only).
 *   o        [B,H,N,d] output, same dtype as the inputs.
 *   lse      [B,H,N] float32 output (natural log of the row sum of exp over
 *            the scaled, masked scores), or NULL if not wanted.
 * Sources: the notes' "The Standard Attention Problem" (what is computed),
 * "Derivation: Incremental Softmax" Steps 1-3 and TensorViz step "tiles" (how:
 * running max m, running sum l, rescale when m rises, divide by l at the end),
 * "Worked example Local Attention Window" (window; key tiles wholly outside
 * the band are never loaded).
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int H, int N, int d, float scale, int window, fa_dtype dt,
                 void* stream);

/*
 * Size in bytes of the workspace fa_bwd needs for a problem of this shape:
 * a float32 [B,H,N,d] dQ accumulator, then two [B,H,Npad] arrays derived
 * from lse_i and from D_i = sum_k dO_ik O_ik (Npad = N rounded up to a
 * multiple of 128; 4 bytes per row, or 16 bytes per row at d = 64, where
 * each value is kept as three bf16 terms), each section 256-byte aligned;
 * at d = 64, 96 and 128 then float32 dV and dK rows for up to 128 key tiles of
 * 128 keys (min(B*H*ceil(N/128), 128) * 2 * 128 * d * 4 bytes), which the
 * backward uses when it splits the key tiles of a last, partly filled wave
 * of CTAs in two.  Returns 0 for non-positive sizes.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * The same forward pass as fa_fwd, evaluated in the key-major loop order that
 * "Compute attention one tile at a time" (TensorViz), fidelity note,
 * attributes to the original Algorithm 1: the outer loop runs over 128-key
 * tiles (one launch each, in order on `stream`), and each launch merges that
 * tile into every query tile's running statistics (the notes' "Derivation:
 * Incremental Softmax", Steps 2-3), which live in `workspace` between
 * launches: fp32 unnormalised O~ [B,H,N,d], then m and l [B,H,N], each
 * section 256-byte aligned; a last launch writes O = O~ / l and lse.  It is
 * kept as a measured comparison point: every step reads and writes O~ in
 * device memory, which fa_fwd keeps on chip.
 *   workspace        at least fa_fwd_key_major_workspace_bytes() bytes,
 *                    256-byte aligned, owned by the caller; contents on entry
 *                    do not matter and are undefined on return.
 * bf16 with d = 64 or 128 only (others return FA_ERR_UNSUPPORTED); other
 * arguments, results and errors as fa_fwd.
 */
fa_status fa_fwd_key_major(const void* q, const void* k, const void* v, void* o, float* lse,
                           int B, int H, int N, int d, float scale, int window, fa_dtype dt,
                           void* workspace, size_t workspace_bytes, void* stream);
size_t fa_fwd_key_major_workspace_bytes(int B, int H, int N, int d);

/*
 * The float32 forward on the tensor cores.  Same operation, layouts, window
 * and results as fa_fwd with FA_DTYPE_F32 (q, k, v, o float32 [B,H,N,d], lse
 * float32 [B,H,N] or NULL), for 1 <= d <= 128.  The tensor cores multiply
 * tf32 values (11 significant bits), so every float32 operand x is split as
 * hi = tf32(x), lo = tf32(x - hi) and each product is taken as
 * hi*hi + hi*lo + lo*hi (the "3xTF32" scheme): S = Q K^T from split Q and K,
 * O += P V from split P and V, fp32 accumulation, fp32 output.  The dropped
 * lo*lo term and the rounding of lo are below 2^-21 relative.  fa_fwd with
 * FA_DTYPE_F32 stays the exact CUDA-core path; this entry point trades a
 * little of that accuracy for tensor-core speed.
 *   workspace        at least fa_fwd_f32_3xtf32_workspace_bytes() bytes,
 *                    256-byte aligned, owned by the caller (it receives the
 *                    split copies of Q, K and V: 6 x 4 x B*H*N*64 bytes for
 *                    d <= 64; for 64 < d <= 128 those of K and V only, 4 x 4
 *                    x B*H*N*128 bytes, the kernel splitting Q itself; N
 *                    rounded up to 64 for V); contents on entry do not
 *                    matter and are undefined on return.
 * d > 128 returns FA_ERR_UNSUPPORTED; other arguments and errors as fa_fwd.
 */
fa_status fa_fwd_f32_3xtf32(const float* q, const float* k, const float* v, float* o, float* lse,
                            int B, int H, int N, int d, float scale, int window,
                            void* workspace, size_t workspace_bytes, void* stream);
size_t fa_fwd_f32_3xtf32_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward pass by recomputation: given Q, K, V, the forward output O, its
 * lse and the output gradient dO, writes dQ, dK, dV (same dtype and layout
 * as Q).  S and P are rebuilt on chip from Q, K and lse; nothing of size
 * N x N is read or written.  Sources: the notes' "Backward Pass:
 * Recomputation" (recompute, do not store, S and P); the gradient formulas
 * are the derivative of the forward definition (the pages print none):
 * dV = P^T dO, dP = dO V^T, D_i = sum_j P_ij dP_ij = sum_k dO_ik O_ik,
 * dS = P o (dP - D), dQ = scale dS K, dK = scale dS^T Q.
 *   workspace        device scratch of at least fa_bwd_workspace_bytes(),
 *                    owned by the caller, 256-byte aligned; its contents on
 *                    entry do not matter and are undefined on return.
 *   workspace_bytes  its size; smaller than required -> FA_ERR_INVALID.
 * bf16 with d = 64, 96 or 128 (other d, 256 included, return
 * FA_ERR_UNSUPPORTED), or float32
 * with 1 <= d <= 128 (CUDA cores; one warp per query row for dQ and one per
 * key row for dK and dV, so dK and dV need no atomics and the float32 path
 * is bitwise repeatable).
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dO, void* dq, void* dk, void* dv,
                 int B, int H, int N, int d, float scale, int window, fa_dtype dt,
                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_bwd for callers that cannot allocate device memory (code running where
 * device allocation is not permitted, or with no allocator to call): the same
 * arguments and results as fa_bwd, minus the workspace, which is replaced by
 * a fixed 64 MiB scratch array inside the library.  This function calls no
 * allocator.  The pages describe no such variant; it is a deployment aid.
 *   - Arguments are checked as fa_bwd checks them, with the same status
 *     codes; then problems with fa_bwd_workspace_bytes(B,H,N,d) > 64 MiB
 *     return FA_ERR_UNSUPPORTED.  Nothing is launched in either case.
 *   - Under CUDA's lazy module loading (the default), the array is brought
 *     onto a device, and its 64 MiB committed there, by the first call on
 *     that device; it then stays until the process exits.  That first call
 *     may therefore allocate and synchronise inside the CUDA driver: make it
 *     outside any region where allocation or stream capture is forbidden.
 *   - All calls share the one array: calls whose work overlaps on the GPU
 *     (e.g. on two concurrent streams) race on it; calls in order on one
 *     stream are fine.  Each call re-initialises what must start at zero.
 *   - The first call on each device looks up the array's device address;
 *     make that first call before any stream capture.
 */
fa_status fa_bwd_static_workspace(const void* q, const void* k, const void* v, const void* o,
                                  const float* lse, const void* dO, void* dq, void* dk, void* dv,
                                  int B, int H, int N, int d, float scale, int window, fa_dtype dt,
                                  void* stream);

/*
 * Attention for language models: shared prefix, latent keys and values
 * -------------------------------------------------------------------
 * The calls below compute the same softmax attention with the head layouts,
 * caches and masks of a language model.  The pages describe none of them;
 * they are written from the formulas given here.  Common to all:
 *   - bf16 runs on the tensor cores (fp32 accumulation; P and, in the backward,
 *     dS are rounded to bf16, the products' type, before they multiply, and D
 *     comes from the rounded o), float32 on CUDA cores in plain fp32.
 *   - "New tokens": a sequence's Nq query tokens are its last ones, so query
 *     token t sees the keys j < n - (Nq - 1 - t) of its n keys.  A query row
 *     that sees no key (t too early, or an empty sequence) gets O = 0 and
 *     lse = -inf, and adds nothing to any gradient.
 *   - lens and block_table are int32 arrays in device memory, read when the
 *     kernels run (a captured graph sees their contents at replay).  A length
 *     below 0 counts as 0, one above the capacity as the capacity, a page
 *     index outside the cache as a page of zeros; each is reported by
 *     fa_last_device_status() as FA_ERR_INVALID.  Nothing out of range is read.
 *   - Entries of K, V and the cache at positions a sequence's length does not
 *     cover may hold anything (NaN included).  Everything else must be finite,
 *     the padding of the expanded form included: a masked probability is 0,
 *     and 0 times an infinity or a NaN is not.
 *   - Outputs must not overlap inputs, nor the workspace anything.  A workspace
 *     serves one call at a time: calls (and replays of graphs) that share one
 *     must run in order.
 *   - Sizes: every tensor at most 2^40 elements; expanded also B H < 2^31 and
 *     Nq, Nk < 2^30, and in the backward B H Nq, Nq rounded up to 128, < 2^33;
 *     shared prefix and absorbed B H Nq < 2^28 rows and, for float32 as for
 *     bf16, at most 7,040,929 tiles of 64 tokens in the batch's rooms, every
 *     sequence's room (Ns, or max_pages * page_size) rounded up to whole tiles
 *     (4.5e8 tokens where rooms are long, 7,040,929 sequences where they are
 *     short).  Past these FA_ERR_INVALID, and 0 from the queries.
 *   - The order of every sum is fixed by the shapes and the lengths: results
 *     repeat bit for bit.
 */

/*
 * Attention of a decoding batch whose sequences begin with one shared prefix.
 * The prefix's keys and values are stored, and read, once for the whole
 * batch.  Query head h uses key/value head h / (Hq / Hkv).
 *   q            [B,Hq,Nq,d], a sequence's Nq new tokens.
 *   k_prefix, v_prefix  [Hkv,Np,d]: seen by every query row.  Np may be 0
 *                (then both may be NULL), at most 2^31 - 256.
 *   k, v         [B,Hkv,Ns,d]: each sequence's own keys and values after the
 *                prefix, those of the new tokens included; positions
 *                j < lens[b] are valid.  Ns may be 0 (then both may be NULL).
 *   lens         int32 [B], 0 <= lens[b] <= Ns.
 *   o, lse       [B,Hq,Nq,d] and float32 [B,Hq,Nq] (or NULL), over the
 *                prefix's and the sequence's own keys together.
 *   workspace    at least fa_fwd_shared_prefix_workspace_bytes() bytes,
 *                256-byte aligned; contents on entry do not matter and are
 *                undefined on return.
 * Hq must be a multiple of Hkv.  bf16 with d = 64, 96 or 128; float32 with
 * 1 <= d <= 128; others return FA_ERR_UNSUPPORTED.  Forward only: a serving
 * call.
 */
fa_status fa_fwd_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k,
                               const void* v, const int* lens, void* o, float* lse,
                               int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d, float scale, fa_dtype dt,
                               void* workspace, size_t workspace_bytes, void* stream);
size_t fa_fwd_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Np, int Ns, int d);

/*
 * Latent attention, absorbed form (serving): every head attends to one shared
 * vector per token, c = [latent | rotary] of dc + dr entries, as the key, and
 * to its first dc entries as the value:
 *     S_ij = scale q_i . c_j,  O_i = sum_j softmax_j(S_i) c_j[:dc]
 * (the per-head up-projections are folded into q before, and applied to O
 * after, the call).
 *   q            [B,H,Nq,dc+dr], a sequence's Nq new tokens.
 *   cache        [n_pages,page_size,dc+dr].
 *   block_table  int32 [B,max_pages]: page of the sequence's tokens
 *                p * page_size ...; entries past its length are not read.
 *                NULL: sequence b is page b (then max_pages must be 1 and
 *                n_pages >= B).
 *   lens         int32 [B], tokens in the cache, the new ones included,
 *                0 <= lens[b] <= max_pages * page_size.
 *   o, lse       [B,H,Nq,dc] and float32 [B,H,Nq] (or NULL).
 *   scale        of the expanded head, usually 1/sqrt(its q and k width).
 *   workspace    at least fa_fwd_latent_absorbed_workspace_bytes() bytes,
 *                256-byte aligned, as above.
 * bf16 with dc = 256 or 512, dr = 64 and, with a table, page_size a multiple
 * of 16; float32 with dc <= 512, dr <= 128; others return
 * FA_ERR_UNSUPPORTED.  Forward only: training uses the expanded form.
 */
fa_status fa_fwd_latent_absorbed(const void* q, const void* cache, const int* block_table, const int* lens,
                                 void* o, float* lse, int B, int H, int Nq, int n_pages, int page_size,
                                 int max_pages, int dc, int dr, float scale, fa_dtype dt,
                                 void* workspace, size_t workspace_bytes, void* stream);
size_t fa_fwd_latent_absorbed_workspace_bytes(int B, int H, int Nq, int page_size, int max_pages, int dc);

/*
 * Latent attention, expanded form (training and prefill): each head's keys
 * are [k_nope | k_rope], the rotary part shared by the heads of a token, and
 * its values have a width of their own:
 *     S_ij = scale (q_i[:dn] . k_nope_j + q_i[dn:] . k_rope_j)
 *   q            [B,H,Nq,dn+dr].
 *   k_nope, v    [B,H,Nk,dn], [B,H,Nk,dv].     k_rope  [B,Nk,dr].
 *   o, lse       [B,H,Nq,dv] and float32 [B,H,Nq] (or NULL).
 *   causal       1: query row i sees keys j <= i + Nk - Nq (rows are the last
 *                Nq of Nk tokens; with Nq > Nk the first Nq - Nk rows see
 *                none); 0: every key.
 * A batch of unequal lengths after pasts of one length (Nk - Nq tokens, 0 with
 * Nq = Nk) is padded on the right, with finite values: with causal = 1 no real
 * token sees the padding behind it, and rows whose dO is 0 add nothing to the
 * gradients.  Sequences whose pasts differ cannot share a call: the mask is
 * aligned at the end of the padded lengths, so that a row of a shorter past
 * would see the padding, or miss keys of its own.
 * bf16 with dn = 128, dr = 64, dv = 128; float32 with dn + dr <= 256,
 * dv <= 128; others return FA_ERR_UNSUPPORTED.
 */
fa_status fa_fwd_latent(const void* q, const void* k_nope, const void* k_rope, const void* v, void* o, float* lse,
                        int B, int H, int Nq, int Nk, int dn, int dr, int dv, float scale, int causal, fa_dtype dt,
                        void* stream);

/*
 * Its backward, by recomputation from the forward's o and lse:
 *     dV = P^T dO, dS = P o (dO V^T - D), D_i = dO_i . O_i,
 *     dq = scale dS [k_nope | k_rope], dk_nope = scale dS^T q[:dn],
 *     dk_rope = scale (sum over heads) dS^T q[dn:].
 *   dq, dk_nope, dk_rope, dv_out   shapes and dtype of q, k_nope, k_rope, v.
 *   workspace    at least fa_bwd_latent_workspace_bytes() bytes, 256-byte
 *                aligned, as above.
 * No atomics: gradients repeat bit for bit.  Other arguments as fa_fwd_latent.
 */
fa_status fa_bwd_latent(const void* q, const void* k_nope, const void* k_rope, const void* v, const void* o,
                        const float* lse, const void* dO, void* dq, void* dk_nope, void* dk_rope, void* dv_out,
                        int B, int H, int Nq, int Nk, int dn, int dr, int dv, float scale, int causal, fa_dtype dt,
                        void* workspace, size_t workspace_bytes, void* stream);
size_t fa_bwd_latent_workspace_bytes(int B, int H, int Nq, int Nk, int dn, int dr, int dv);

/*
 * A key/value cache in 4 bits, and the attention that reads it
 * ------------------------------------------------------------
 * Keys and values of a decoding batch with key/value heads shared by query
 * heads, held at 4.5 bits an entry (9 d bytes for 8 tokens of a head, keys and
 * values together: bf16 takes 32 d).
 *   Format     16 neighbouring entries x of a token's key (or value) of one head
 *              are a group.  With y = x / k_scale (x / v_scale; float32), the
 *              group's scale is s = amax |y| / 6 rounded to e4m3 (nearest, ties
 *              to even, at most 448; up to 2^-10 it is 0, and so is the group),
 *              and an entry's code is the e2m1 number nearest to y / s: one of
 *              +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to even, at most 6.  It
 *              stands for code * s * k_scale.  So an entry is off by at most
 *              amax / 6 but for what s is rounded (1/16).  k_scale and v_scale
 *              map the tensors onto what a scale can hold, 2^-9 to 448: entries
 *              up to 2688 k_scale, larger ones (infinities too) become that.  A
 *              group that holds a NaN is NaN.
 *              The write takes half of the time for bf16 tensors, three quarters
 *              for float32 ones, where both are powers of two between 2^-100 and
 *              2^98 (no divisions by them); results follow the definition with any.
 *   cache      uint8 [n_pages][Hkv][page_size][9 d / 8], 16-byte aligned.  Of
 *              every page and head, 16 tokens are a block of 18 d bytes: key
 *              codes [d/16][16 tokens][8], key scales [16 tokens][d/16], value
 *              codes [d][8] (a channel's 16 tokens), value scales [d/16][16
 *              tokens].  The first of the two codes in a byte is in its low half.
 *   block_table, lens  as for the absorbed form: int32 [B,max_pages] (NULL:
 *              sequence b is page b; then max_pages must be 1 and n_pages >= B)
 *              and int32 [B], the tokens in the cache, new ones included.  Of
 *              the conventions above those on new tokens, device-side lengths
 *              and pages, uncovered positions (any bytes), workspaces and sizes
 *              hold here too, with Nq for new queries, unless stated otherwise.
 *   Sizes      page_size and d multiples of 16, d <= 256 (others return
 *              FA_ERR_UNSUPPORTED).  Rows written or read, n a sequence: n <
 *              2^30, Hkv (floor((n + 14) / 16) + 1) < 2^31, and B times that
 *              below 2^33 - 64 (the blocks that they can touch).
 */

/* Bytes of a cache, or 0 for sizes that the calls refuse. */
size_t fa_cache_fp4_bytes(int n_pages, int Hkv, int page_size, int d);

/*
 * Writes a step's keys and values into the cache.
 *   k, v         [B,Hkv,Nn,d], bf16 or float32: row t of sequence b is the token
 *                at position lens[b] - Nn + t.
 *   n_new        int32 [B], or NULL: how many of the Nn rows, the last ones, are
 *                tokens of sequence b (0 <= n_new[b] <= Nn; clamped and reported
 *                as lens is); the rows before them are padding and not read.
 *                NULL: all.  Rows whose position is below 0 are padding too.
 *   lens         a length out of range is reported, and nothing of that
 *                sequence written.
 * Other tokens of the cache keep their bits.  A byte holds codes of two
 * neighbouring tokens: calls that write to one page must run in order, and a
 * page must not appear twice among those that a call writes to (a sequence
 * writes to the pages of its new tokens' positions, and to none without any).
 */
fa_status fa_cache_fp4_write(const void* k, const void* v, void* cache, const int* block_table, const int* lens,
                             const int* n_new, int B, int Hkv, int Nn, int n_pages, int page_size, int max_pages,
                             int d, float k_scale, float v_scale, fa_dtype dt, void* stream);

/*
 * Reads cached tokens back as the numbers they stand for.
 *   first        int32 [B], or NULL (0): row t of sequence b is position
 *                first[b] + t.
 *   k, v         [B,Hkv,N,d], bf16 or float32; rows at positions below 0 or from
 *                lens[b] on are zeros.
 */
fa_status fa_cache_fp4_read(const void* cache, const int* block_table, const int* lens, const int* first, void* k,
                            void* v, int B, int Hkv, int N, int n_pages, int page_size, int max_pages, int d,
                            float k_scale, float v_scale, fa_dtype dt, void* stream);

/*
 * Attention of each sequence's last Nq tokens over the cache: query token t
 * sees the keys j < lens[b] - (Nq - 1 - t), query head h uses key/value head
 * h / (Hq / Hkv).
 *   q, o         [B,Hq,Nq,d], bf16 or float32.   lse  float32 [B,Hq,Nq] or NULL.
 *   workspace    at least fa_fwd_cache_fp4_workspace_bytes() bytes, 256-byte
 *                aligned, as above.
 * Hq must be a multiple of Hkv; Hkv ceil(Hq / Hkv Nq / 16) B tiles of 128
 * tokens / 304 must stay below 2^31 too.  Forward only: a serving call.
 * scale k_scale and scale k_scale / ln 2 must be normal float32 numbers (others
 * return FA_ERR_INVALID).
 * d = 64, 96 and 128 run on the tensor cores, with fp32 accumulation: code * s
 * is exact in fp16, a row of q is brought to fp16 by a power of two (bf16: exact
 * down to 2^-31 of its largest entry; float32: as three terms), and P, rounded
 * to fp16 (float32: as two terms), multiplies the values: 2^-11 relative
 * (2^-22), and 2^-32 of the largest P at the least.  Other d run on CUDA cores
 * in plain fp32, at a small part of that speed (a serving batch at d = 80 takes 16
 * times as long as at d = 128).  The workspace has room for the rows of every
 * sequence and key/value head, rounded up to 16, 32 or a multiple of 64, in fp32
 * and whatever the lengths: 8 MB for B = 64, Hkv = 8, d = 128 and up to 16 rows,
 * 545 MB for B = 8192.
 */
fa_status fa_fwd_cache_fp4(const void* q, const void* cache, const int* block_table, const int* lens, void* o,
                           float* lse, int B, int Hq, int Hkv, int Nq, int n_pages, int page_size, int max_pages,
                           int d, float scale, float k_scale, float v_scale, fa_dtype dt, void* workspace,
                           size_t workspace_bytes, void* stream);
size_t fa_fwd_cache_fp4_workspace_bytes(int B, int Hq, int Hkv, int Nq, int page_size, int max_pages, int d);

/*
 * Synchronises `stream` (as void* cudaStream_t), then reads and clears the
 * device status word that the kernels set when a bounded wait runs out.
 * Returns FA_OK, FA_ERR_TIMEOUT, FA_ERR_INVALID (a length or page index in
 * device memory was out of range), or FA_ERR_CUDA if synchronising failed or
 * a kernel refused to run on the device (a layout check failed).
 */
fa_status fa_last_device_status(void* stream);

/*
 * Sets the time limit, in microseconds, of every device-side wait in kernels
 * launched afterwards by this process (default 1,000,000 = 1 s; values <= 0
 * restore the default).  Returns the previous limit.
 */
long long fa_set_wait_limit_us(long long limit_us);

/*
 * Self-test of the bounded wait: launches one block that waits on a shared
 * memory barrier nothing ever arrives on, for `limit_us` microseconds
 * (1..100000), then gives up, records FA_ERR_TIMEOUT in the status word and
 * returns.  A caller checks fa_last_device_status() == FA_ERR_TIMEOUT.
 */
fa_status fa_selftest_wait_timeout(int limit_us, void* stream);

/* Static, human-readable name of a status code. */
const char* fa_status_string(fa_status s);

/* Library version as major*10000 + minor*100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
