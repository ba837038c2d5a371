/*
 * bss_attn.h - C ABI of libbss_attn.so: exact, causal, block-sparse and
 * chunk-merged softmax attention on GB300 (sm_103a), forward and backward.
 *
 * Operation.  For every batch b and head h, with Q [Lq, d], K and V [Lk, d]:
 *     S = scale * Q K^T,   O = softmax_row(S over the allowed keys) V,
 *     LSE_i = ln sum_{j allowed} exp(S_ij)
 * computed tile by tile with the online-softmax state (m, l, A) so that S and
 * P never reach device memory ("Exact Blocks, Rings, and Sparsity", sections 1
 * and 2; "FlashAttention: Fast and Memory Efficient Exact Attention with IO
 * Awareness", section 5.2 and Theorem 1).
 *
 * Conventions shared by every entry point.
 *   - Tensors are contiguous row-major [B, H, L, d] (d fastest), bf16 unless
 *     stated; LSE, partial states and delta are fp32.  d must be 64 or 128.
 *   - Grouped heads: H query heads read H_kv K/V heads (1 <= H_kv <= H, H_kv
 *     divides H; H_kv = H is ordinary multi-head attention).  q, o, dout, dq,
 *     lse and delta have H heads; k, v, dk and dv have H_kv heads, and query
 *     head h reads K/V head h / (H / H_kv) ("Exact Blocks, Rings, and
 *     Sparsity", section 6: query heads that share one physical KV head).
 *     dk and dv are summed over the query heads of their group.  Otherwise
 *     ATTN_ERR_INVALID_ARG.
 *   - All pointers to tensors are DEVICE pointers, 16-byte aligned, owned by
 *     the caller.  The library never allocates, frees or synchronises device
 *     memory (attn_poll_status excepted) and keeps no pointer after a call
 *     returns.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Work is only
 *     enqueued; results are ready when the stream reaches it.
 *   - Masks follow the pages' semantics: a masked pair contributes exactly
 *     zero; a query row with no allowed key gets O = 0 and LSE = -inf (and
 *     zero gradient); causal visibility is key + k_offset <= query + q_offset.
 *   - LSE is the natural log of the normaliser of the scaled logits.
 *   - Every call returns an attn_status_t; nothing is thrown or aborted across
 *     the ABI.  Errors found inside a kernel (a block index out of range, a
 *     watchdog timeout) are recorded in a per-library device word read by
 *     attn_poll_status.
 */
#ifndef BSS_ATTN_H_
#define BSS_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, non-finite or non-positive scale */
  ATTN_ERR_UNSUPPORTED = 2,   /* d not in {64,128}, block != 128, size beyond a stated limit */
  ATTN_ERR_BAD_BLOCKLIST = 3, /* malformed CSR: row_ptr not monotone, index out of range, nnz mismatch */
  ATTN_ERR_CUDA = 4,          /* a CUDA runtime/driver call or kernel launch failed */
  ATTN_ERR_TIMEOUT = 5,       /* a kernel's bounded wait expired (watchdog); the kernel returned early */
  ATTN_ERR_WORKSPACE = 6,     /* workspace missing or smaller than attn_bwd_workspace_bytes() */
  ATTN_ERR_BAD_PAGES = 7,     /* paged cache: a page, sequence, length or position out of range */
  ATTN_ERR_NO_PAGES = 8       /* paged cache: fewer free pages than asked for; nothing was changed */
} attn_status_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* attn_status_string(int status);

/* Library ABI version (major*100 + minor). */
int attn_version(void);

/* Text of the last CUDA/driver failure seen by this thread (for ATTN_ERR_CUDA
 * diagnostics); empty string if none.  Static per-thread storage. */
const char* attn_last_error_message(void);

/*
 * attn_fwd - exact attention forward, dense or causal.
 * "Exact Blocks, Rings, and Sparsity", section 2 ('What the forward kernel
 * keeps on chip'); causal element mask on the diagonal tiles only, tiles wholly
 * in the future skipped (section 4, last paragraph).
 *   q [B,H,Lq,d], k/v [B,H,Lk,d] bf16 in; o [B,H,Lq,d] bf16 out; lse [B,H,Lq] fp32 out.
 *   causal != 0 applies key + k_offset <= query + q_offset (offsets >= 0).
 *   scale must be finite and > 0 (the pages use d^-1/2).
 */
attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                       int B, int H, int H_kv, int Lq, int Lk, int d, float scale, int causal,
                       int64_t q_offset, int64_t k_offset, void* stream);

/*
 * attn_fwd_partial - unnormalised online-softmax state over one KV chunk.
 * "Exact Blocks, Rings, and Sparsity", section 2 (state m, l, A and its merge
 * invariant) and section 4 (one Ring-Attention step on a KV block).
 *   Writes, per query row, m = max allowed scaled logit (natural-log units),
 *   l = sum exp(s - m), acc = sum exp(s - m) V over the keys of this chunk.
 *   Rows with no allowed key get the empty state m = -inf, l = 0; their acc
 *   row is left untouched (an empty state is identified by m = -inf and is
 *   never read by attn_merge_states).
 *   m, l: fp32 [B,H,Lq]; acc: fp32 [B,H,Lq,d].  Other arguments as attn_fwd;
 *   k_offset is the absolute position of the chunk's first key.
 */
attn_status_t attn_fwd_partial(const void* q, const void* k, const void* v,
                               float* m, float* l, float* acc,
                               int B, int H, int H_kv, int Lq, int Lk, int d, float scale,
                               int causal,
                               int64_t q_offset, int64_t k_offset, void* stream);

/*
 * attn_merge_states - combine C partial states over disjoint key sets.
 * "Exact Blocks, Rings, and Sparsity", section 4 (the associative merge of two
 * ring steps); "FlashAttention ..." section 5.1 (block-wise m and l).
 *   m, l: fp32 [C,B,H,L]; acc: fp32 [C,B,H,L,d] (as written by attn_fwd_partial,
 *   chunk-major).  Out: o bf16 [B,H,L,d] = A* / l*, lse fp32 [B,H,L] = m* + ln l*.
 *   Empty states (m = -inf) are skipped without reading their acc rows; a row
 *   whose states are all empty gets O = 0, LSE = -inf.  1 <= C <= 64.
 */
attn_status_t attn_merge_states(int C, const float* m, const float* l, const float* acc,
                                void* o, float* lse, int B, int H, int L, int d, void* stream);

/*
 * attn_fwd_splitkv_workspace_bytes - workspace of attn_fwd_splitkv: the fp32
 * partial states (m, l, acc) of every key chunk, 0 for invalid arguments.
 */
size_t attn_fwd_splitkv_workspace_bytes(int B, int H, int Lq, int Lk, int d, int n_chunks);

/*
 * attn_fwd_splitkv - exact attention with the keys split into chunks whose
 * partial states are computed in one launch and then merged: the split-KV
 * (decode-shaped) forward.
 * "Exact Blocks, Rings, and Sparsity", section 4 (each Ring step folds one KV
 * block into the state (m, l, A); the merge is associative and order-free)
 * and section 2 (the merge invariant).
 *   Arguments and results as attn_fwd; n_chunks in [1, 64].  The keys are cut
 *   into chunks of ceil(Lk / n_chunks) keys rounded up to a multiple of 128
 *   (so there may be fewer chunks than asked), each read in place from k and
 *   v.  A chunk wholly in the causal future of a query tile is skipped for
 *   that tile (its state is empty and the merge ignores it).  Meant for
 *   shapes with few query tiles against many keys, e.g. decoding: Lq of one
 *   to a few hundred queries against a long cache, q_offset = Lk - Lq under a
 *   causal mask.
 *   workspace: device, 16-byte aligned, >= attn_fwd_splitkv_workspace_bytes
 *   bytes; contents on entry irrelevant.  Two launches on the stream: the
 *   partial states, then attn_merge_states.
 */
attn_status_t attn_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                               void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                               int Lq,
                               int Lk, int d, float scale, int causal, int64_t q_offset,
                               int64_t k_offset, int n_chunks, void* stream);

/*
 * attn_blocklist_normalize - HOST function: canonical form of a CSR block list.
 * Block-sparse attention patterns page, 'Count active blocks and acknowledge the
 * changed operator' (duplicate entries never count twice; order carries no meaning).
 *   In: row_ptr[n_qblk+1], col_idx[row_ptr[n_qblk]] (host memory, any order,
 *   duplicates allowed).  Out: out_row_ptr[n_qblk+1] and out_col_idx (capacity
 *   >= row_ptr[n_qblk]) hold each row's set of key blocks in ascending order;
 *   *out_nnz = total unique entries.  Returns ATTN_ERR_BAD_BLOCKLIST if row_ptr
 *   does not start at 0, decreases, or an index is outside [0, n_kblk).
 */
attn_status_t attn_blocklist_normalize(const int32_t* row_ptr, const int32_t* col_idx,
                                       int n_qblk, int n_kblk, int32_t* out_row_ptr,
                                       int32_t* out_col_idx, int32_t* out_nnz);

/*
 * attn_fwd_blocksparse - attention over a per-query-block list of key blocks,
 * renormalised over the sparse domain.
 * "Exact Blocks, Rings, and Sparsity", section 5 ('Why the sparse unit is
 * usually a block': the outer loop visits only the listed tiles) and section 6
 * (drop-and-renormalise); block-sparse attention patterns page (triangular
 * element mask inside diagonal blocks, partial blocks, duplicates, empty rows).
 *   q/k/v/o/lse as attn_fwd with Lq = Lk = L.  block must be 128.
 *   row_ptr [n_lists][n_qblk+1], col_idx [nnz]: DEVICE int32 CSR, n_qblk =
 *   ceil(L/128), raw form accepted (any order, duplicates counted once).
 *   n_lists >= 1 lists share the B*H heads in consecutive groups: head
 *   (b*H + h) uses list (b*H + h) / (B*H / n_lists), so n_lists must divide
 *   B*H (1: one list for every head; B*H: one per head; B*H_kv with grouped
 *   query heads: one per KV head).  Each list's row_ptr holds offsets into
 *   the one col_idx array (else ATTN_ERR_BAD_BLOCKLIST).  A listed block
 *   wholly in the causal future contributes nothing (attn_blocklist_stats
 *   counts such blocks, with the list's pairs and tiles).  An entry outside
 *   [0, ceil(L/128)) is ignored and reported as ATTN_ERR_BAD_BLOCKLIST by
 *   attn_poll_status; so is a row whose row_ptr range is not inside [0, nnz]
 *   (that row is then treated as empty).  A query block with an empty list
 *   gets O = 0, LSE = -inf.  L <= 4096*128 (at most 4096 key blocks).
 *   Lists of one set (any order, any duplicates) give bit-identical results.
 *   At d = 128 with at most 2048 key blocks the launch runs the kernel with
 *   256-key score tiles, otherwise the two-tile kernel (speed only: both
 *   agree with the dense forward within rounding).
 */
attn_status_t attn_fwd_blocksparse(const void* q, const void* k, const void* v, void* o,
                                   float* lse, int B, int H, int H_kv, int L, int d, float scale,
                                   int causal, int block, const int32_t* row_ptr,
                                   const int32_t* col_idx, int n_lists, int n_qblk, int nnz,
                                   void* stream);

/*
 * attn_blocklist_stats - what a block list asks the block-sparse kernels to do.
 * Block-sparse attention patterns page, 'Count active blocks and acknowledge the
 * changed operator' (report the logical allowed pairs beside the executed tile
 * work; under a causal mask the token rule applies inside every listed block,
 * so a listed block wholly in the causal future contributes nothing: it is
 * flagged here, not rejected).
 *   row_ptr, col_idx, n_lists, n_qblk, nnz, L, causal, block: as
 *   attn_fwd_blocksparse (DEVICE int32 CSR, raw form accepted, block 128).
 *   Out: stats, DEVICE int64 [n_lists][4], 8-byte aligned, per list:
 *     [0] listed (query block, key block) pairs, duplicates counted once;
 *     [1] executed tiles: listed pairs holding at least one allowed pair;
 *     [2] listed pairs wholly in the causal future (key block after query
 *         block; 0 without a causal mask), which the kernels skip;
 *     [3] logical allowed (query, key) pairs of the realised mask.
 *   [0] = [1] + [2].  Malformed rows and entries are skipped and reported as
 *   ATTN_ERR_BAD_BLOCKLIST by attn_poll_status, as in attn_fwd_blocksparse.
 *   One launch on the stream; stats is fully written (zeros when L = 0).
 */
attn_status_t attn_blocklist_stats(const int32_t* row_ptr, const int32_t* col_idx, int n_lists,
                                   int n_qblk, int nnz, int L, int causal, int block,
                                   int64_t* stats, void* stream);

/*
 * attn_select_blocks - block lists for attn_fwd_blocksparse from mean-pooled
 * scores (a selector that needs no trained weights).
 * "Exact Blocks, Rings, and Sparsity", section 5 ('Why the sparse unit is
 * usually a block': the selector must score something cheaper than Q K^T, and
 * it chooses an exact set: selected blocks united with a mandatory local
 * window; 'Fixed pooling: a cheap proxy, not the true block mass') and
 * section 6 (query heads that share a KV head share the block choice).
 *   q [B,H,L,d], k [B,H_kv,L,d] bf16 (device).  Per 128-row block the query
 *   and key rows are averaged (fp32); query block a scores key block c by the
 *   sum, over the query heads that share a list, of scale * qbar_a . kbar_c
 *   (the block pair's mean logit), query head h pooling the keys of K/V head
 *   h / (H / H_kv).  Row a keeps the local window a, a-1, .., a-local_blocks+1
 *   (those >= 0) and the top_r other candidates (under a causal mask only
 *   blocks <= a), larger score first, the lower index on equal scores, listed
 *   in ascending order.  n_lists as in attn_fwd_blocksparse.
 *   Out (device): row_ptr [n_lists][n+1] (offsets into col_idx),
 *   col_idx [attn_select_blocks_nnz(...)] int32 - the input format of
 *   attn_fwd_blocksparse and attn_bwd_blocksparse.
 *   block must be 128; top_r + local_blocks <= 256; ceil(L/128) <= 4096 and
 *   n_lists * entries per list < 2^31 (else ATTN_ERR_UNSUPPORTED).
 *   workspace: device, 16-byte aligned, >= attn_select_blocks_workspace_bytes.
 */
size_t attn_select_blocks_workspace_bytes(int B, int H, int L, int d);
int64_t attn_select_blocks_nnz(int L, int top_r, int local_blocks, int causal, int n_lists);
attn_status_t attn_select_blocks(const void* q, const void* k, int B, int H, int H_kv, int L,
                                 int d,
                                 float scale, int causal, int block, int top_r, int local_blocks,
                                 int n_lists, int32_t* row_ptr, int32_t* col_idx, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * attn_bwd_workspace_bytes - size of the caller-provided workspace of attn_bwd
 * (an fp32 dQ accumulator of B*H*L*d elements).
 */
size_t attn_bwd_workspace_bytes(int B, int H, int L, int d);

/*
 * attn_bwd - gradients by recomputation from the saved LSE.
 * "Exact Blocks, Rings, and Sparsity", section 3 (D_i = dO_i . O_i;
 * P = exp(S - LSE); dS = P o (dP - D); dQ = scale dS K; dK = scale dS^T Q;
 * dV = P^T dO; KV-owned traversal with accumulated dQ, 'The ownership
 * conflict between dQ and dK, dV'); "FlashAttention ..." section 5.3.
 *   q,k,v,o,dout bf16 [B,H,L,d]; lse fp32 [B,H,L] from attn_fwd with the same
 *   scale and mask.  Out: dq, dk, dv bf16 [B,H,L,d]; delta fp32 [B,H,L].
 *   workspace: device, >= attn_bwd_workspace_bytes(B,H,L,d) bytes, contents
 *   on entry irrelevant (it is cleared on the stream).
 */
attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv,
                       float* delta, void* workspace, size_t workspace_bytes,
                       int B, int H, int H_kv, int L, int d, float scale, int causal,
                       void* stream);

/*
 * attn_bwd_blocksparse_workspace_bytes - size of the caller-provided workspace
 * of attn_bwd_blocksparse: the fp32 dQ accumulator (B*H*L*d elements, rounded
 * up to 256 bytes), a key-major bitmap of each of the n_lists block lists
 * (ceil(L/128) columns of ceil(ceil(L/128)/32) 32-bit words, rounded up to
 * 256 bytes) and the launch order of the key tiles (B*H*ceil(L/128) int32);
 * 0 when n_lists does not divide B*H.
 */
size_t attn_bwd_blocksparse_workspace_bytes(int B, int H, int L, int d, int n_lists);

/*
 * attn_bwd_blocksparse - gradients of attn_fwd_blocksparse by recomputation.
 * "Exact Blocks, Rings, and Sparsity", section 3 (the backward of section 2
 * over the same allowed set) and section 6 (gradients flow only through the
 * kept blocks: the dropped ones have P = 0, and renormalising over the sparse
 * domain is what the saved LSE already encodes); block-sparse attention
 * patterns page (compare gradients too, duplicates counted once, empty rows).
 *   Arguments as attn_bwd plus the block list of attn_fwd_blocksparse (block
 *   128, DEVICE int32 CSR, raw form accepted) and the same causal flag; lse
 *   must come from attn_fwd_blocksparse with that list.  Each key tile walks
 *   the query blocks that list it (the list's transpose, built in the
 *   workspace on the stream, with the key tiles' launch order: columns far
 *   longer than the mean first).  A key block no query block lists gets
 *   dK = dV = 0; a query block with an empty list gets dQ = 0.  Malformed
 *   entries are handled and reported as in attn_fwd_blocksparse.  With
 *   grouped heads the query heads of one K/V head must share one list
 *   (B*H/n_lists a multiple of H/H_kv), else ATTN_ERR_BAD_BLOCKLIST.
 *   workspace: device, >= attn_bwd_blocksparse_workspace_bytes(B,H,L,d,n_lists).
 */
attn_status_t attn_bwd_blocksparse(const void* q, const void* k, const void* v, const void* o,
                                   const float* lse, const void* dout, void* dq, void* dk,
                                   void* dv, float* delta, void* workspace, size_t workspace_bytes,
                                   int B, int H, int H_kv, int L, int d, float scale, int causal,
                                   int block,
                                   const int32_t* row_ptr, const int32_t* col_idx, int n_lists,
                                   int n_qblk, int nnz, void* stream);

/*
 * attn_bwd_noalloc - attn_bwd for callers that cannot allocate device memory.
 * The source pages have no counterpart: this entry exists for callers that
 * may not call cudaMalloc or own a workspace (an allocator that forbids new
 * device allocations, a host process that hands out none).  The fp32 dQ
 * accumulator lives in a static device array inside the library, 32 MiB
 * (8388608 floats).  Arguments and results are those of attn_bwd without the
 * workspace.
 *   - B*H*L*d above 8388608 is rejected with ATTN_ERR_WORKSPACE before any
 *     device work (attn_last_error_message says why).
 *   - The array sits in a module of its own.  Under lazy module loading (the
 *     CUDA default) the driver reserves its 32 MiB on a device during the
 *     first attn_bwd_noalloc call there, which also looks up the array's
 *     address (cudaGetSymbolAddress); the device then holds it until the
 *     process exits.  Processes that never call this entry do not hold it
 *     (unless CUDA_MODULE_LOADING=EAGER, which loads it at context creation).
 *     Make one first call per device before fixing a memory budget and before
 *     any stream capture (L = 0 with non-null, 16-byte aligned pointers does
 *     the set-up and no device work).
 *   - The cached address assumes the device's context is not reset
 *     (cudaDeviceReset) while the library is in use.
 *   - Every call shares the one array and clears it on the stream before use.
 *     Calls that can overlap on the GPU (different streams, no ordering) race
 *     on it and give wrong gradients; serialise them.
 *   - Nothing is allocated or freed by the call itself (no cudaMalloc, cudaFree
 *     or allocating library routine).
 */
attn_status_t attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                               const float* lse, const void* dout, void* dq, void* dk, void* dv,
                               float* delta, int B, int H, int H_kv, int L, int d, float scale,
                               int causal,
                               void* stream);

/*
 * attn_fwd_window - attention forward with a sliding window and sinks: query
 * i sees key j when 0 <= t and (t < window or j + k_offset < sinks), with t =
 * (i + q_offset) - (j + k_offset): the last `window` positions up to its own,
 * and the sequence's first `sinks` positions that are not in its future.
 * "Exact Blocks, Rings, and Sparsity", section 5 (a mandatory local window
 * united with a few global blocks) at the granularity of single keys; the
 * block-sparse attention patterns page, 'Block-sparse attention' (local +
 * global patterns).
 *   q [B,H,Lq,d], k/v [B,H_kv,Lk,d] bf16 in; o [B,H,Lq,d] bf16 out; lse
 *   [B,H,Lq] fp32 out; window >= 1, sinks >= 0, offsets >= 0.  A query that
 *   sees no key gets O = 0, LSE = -inf.  window >= every distance gives the
 *   causal attn_fwd (within rounding).
 *   Work is proportional to the visible 128-key blocks: the blocks that meet a
 *   128-query tile's window, and the sink blocks.
 *   Keys and values are taken as finite: a NaN or infinity in v reaches the
 *   queries of every 128-query tile that reads its block.
 *   Scores, maxima, sums and O are fp32; the probabilities are rounded to bf16
 *   for their product with v, as in attn_fwd (O comes out about 1.9e-3 off in
 *   norm, of which rounding O itself is 1.65e-3).
 */
attn_status_t attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int H, int H_kv, int Lq, int Lk, int d, float scale,
                              int64_t window, int64_t sinks, int64_t q_offset, int64_t k_offset,
                              void* stream);

/*
 * attn_bwd_window - gradients of attn_fwd_window by recomputation from the
 * saved LSE ("Exact Blocks, Rings, and Sparsity", section 3, over the
 * window's allowed pairs).
 *   q, o, dout [B,H,Lq,d], k, v [B,H_kv,Lk,d] bf16, lse fp32 [B,H,Lq] from
 *   attn_fwd_window with the same window, sinks, offsets and scale.  Out: dq
 *   [B,H,Lq,d], dk, dv [B,H_kv,Lk,d] bf16 (dk and dv summed over the query
 *   heads of their group), delta fp32 [B,H,Lq]: dO . O, and for queries of few
 *   keys (up to 64 near the first and past the last key; all of them when
 *   window and sinks are at most 32 keys together) sum_j P_ij (dO_i . V_j),
 *   the same without O's rounding.  A query that sees no key gets dq = 0; a
 *   key that no query sees gets dk = dv = 0.  Inputs are taken as finite, as in
 *   attn_fwd_window.
 *   P and dS are rounded to bf16 for their products, as in attn_bwd, all else
 *   is fp32 (gradients about 2.4e-3 off in norm, of which rounding them is
 *   1.65e-3; more where one key has most of a query's weight, by the rounding
 *   of O in delta).  With up to 8 sinks in the call, whose dk and dv add up
 *   every later query, the pairs with a sink take P and dS in two bf16 parts
 *   (2^-15).
 *   dk and dv are the same in every run.  dq is accumulated in fp32 in the
 *   order the key tiles finish, so its last bit may differ from run to run.
 *   workspace: device, 16-byte aligned, >= attn_bwd_window_workspace_bytes
 *   bytes (0 for invalid arguments and for lengths that the call refuses): the
 *   fp32 dQ accumulator, and fp32 parts of dK and dV of sinks and of key tiles
 *   whose queries several CTAs share; contents on entry irrelevant.  Calls that can overlap need a workspace each.
 */
size_t attn_bwd_window_workspace_bytes(int B, int H, int H_kv, int Lq, int Lk, int d,
                                       int64_t window, int64_t sinks, int64_t q_offset,
                                       int64_t k_offset);
attn_status_t attn_bwd_window(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dout, void* dq, void* dk, void* dv,
                              float* delta, void* workspace, size_t workspace_bytes, int B, int H,
                              int H_kv, int Lq, int Lk, int d, float scale, int64_t window,
                              int64_t sinks, int64_t q_offset, int64_t k_offset, void* stream);

/*
 * Paged key/value caches (attn_decode_paged, attn_fwd_paged, attn_select_pages,
 * attn_decode_selected and the attn_kv_ calls).
 *   - k_cache, v_cache [n_pages][H_kv][page_size][d], bf16 (ATTN_KV_BF16) or
 *     e4m3 (ATTN_KV_E4M3); a page is contiguous, pages lie k_page_stride /
 *     v_page_stride elements apart (a multiple of 16 bytes, at least a page).
 *     page_size: a power of two in [16, 1024].  An e4m3 element x of K/V head
 *     h stands for x * k_scale[h] (v_scale[h]), fp32 device arrays [H_kv] of
 *     positive scales; both are NULL for bf16 caches.
 *   - page_table [S][max_pages] int32: entry m of row s is the page of tokens
 *     m * page_size .. of sequence s, -1 where it holds none.  seq_lens [S]
 *     int32: tokens.  refs [n_pages] int32: table entries holding the page
 *     (0: free).  S <= 65536, n_pages <= 2^30, a length at most 0x7FFFFF00.
 *     A fresh cache has every entry -1, every length and every count 0.
 *   - The attn_kv_ calls keep these consistent: a page that is not full is
 *     held once, pages are taken from the lowest free index up, in order of
 *     the sequences (or forks), and a call that cannot be met changes nothing.
 *   - What is wrong in the arrays (a page, sequence, length or position out of
 *     range) is skipped and reported as ATTN_ERR_BAD_PAGES by
 *     attn_poll_status; too few free pages as ATTN_ERR_NO_PAGES.
 */
enum { ATTN_KV_BF16 = 0, ATTN_KV_E4M3 = 1 };

/*
 * attn_decode_paged - attention of one new token per sequence over a paged
 * cache, split over its length and joined ("Exact Blocks, Rings, and
 * Sparsity", section 4: partial states over key chunks and their associative
 * merge).
 *   q [S][H][d] bf16, rows q_stride elements apart (a multiple of 8, at least
 *   H*d); o [S][H][d] bf16 and lse [S][H] fp32 out, contiguous.  The query of
 *   sequence s stands at position seq_lens[s] - 1 (its key is in the cache)
 *   and sees the keys j < seq_lens[s], with window > 0 only those with j >=
 *   seq_lens[s] - window or j < sinks; window = 0: every key (sinks must be
 *   0).  H_kv divides H; query head h reads K/V head h / (H / H_kv).  A
 *   sequence of length 0 gets O = 0, LSE = -inf.
 *   What the table's entries of unseen keys and the caches' rows that are not
 *   seen (past the length, or outside window and sinks) hold does not matter.
 *   A seen page outside [0, n_pages) is skipped and reported, a length past
 *   max_pages * page_size (or 0x7FFFFF00) is cut to it and reported.
 *   workspace: device, 16-byte aligned, >= attn_decode_paged_workspace_bytes
 *   (it does not depend on the lengths: 0 for invalid arguments and for small
 *   calls, which take NULL; at most 16 MB for groups of up to 8 query heads,
 *   31 MB for larger ones), contents on entry irrelevant.  Calls that can
 *   overlap need a workspace each.
 *   S >= 1.  The same lengths give the same bits in every run.
 *   Scores, maxima, sums and O are fp32; the probabilities enter their product
 *   in two bf16 parts (2^-15) over bf16 pages, as fp16 (2^-11) over e4m3 ones.
 */
size_t attn_decode_paged_workspace_bytes(int S, int H, int H_kv, int d, int max_pages,
                                         int page_size);
attn_status_t attn_decode_paged(const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, int64_t k_page_stride, int64_t v_page_stride,
                                int kv_dtype, const float* k_scale, const float* v_scale,
                                const int32_t* page_table, const int32_t* seq_lens, void* o,
                                float* lse, void* workspace, size_t workspace_bytes, int S, int H,
                                int H_kv, int d, int max_pages, int n_pages, int page_size,
                                float scale, int64_t window, int64_t sinks, void* stream);

/*
 * attn_fwd_paged - attention of a chunk of new tokens per sequence over a paged
 * cache ("Exact Blocks, Rings, and Sparsity", section 4: the new tokens'
 * queries against key chunks, cached ones and their own): a prompt's next
 * chunk, a few tokens to verify, or both beside single tokens in one batch.
 *   q [T][H][d] bf16, rows q_stride elements apart (a multiple of 8, at least
 *   H*d); o [T][H][d] bf16 and lse [T][H] fp32 out, contiguous.  Rows cu_q[s] ..
 *   cu_q[s+1]-1 (cu_q [S+1] int32, ascending) are the last tokens of sequence s,
 *   whose keys are in the cache: row t stands at position
 *       i = seq_lens[s] - (cu_q[s+1] - t)
 *   and sees the keys j <= i, with window > 0 only those with j > i - window or
 *   j < sinks; window = 0: every key (sinks must be 0).  H_kv divides H, at most
 *   128 query heads share a K/V head; query head h reads K/V head h / (H / H_kv).
 *   Rows before cu_q[0] or from cu_q[S] on belong to no sequence: their o and
 *   lse are left as they were (all rows' where cu_q does not ascend, which is
 *   reported).  A row before its sequence's first token (more
 *   new tokens than the sequence has) gets O = 0, LSE = -inf and is reported.
 *   What the table's entries of keys that no row of a sequence sees hold does
 *   not matter, nor what the caches hold past a sequence's length.  A seen page
 *   outside [0, n_pages) is reported (its keys are left out), a length past
 *   max_pages * page_size (or 0x7FFFFF00) is cut to it and reported.  As in
 *   attn_fwd_window, a V that is infinite or NaN reaches every row whose block of
 *   128 keys it lies in.
 *   workspace: device, 16-byte aligned, >= attn_fwd_paged_workspace_bytes (it
 *   depends on none of the device's arrays; 0 for invalid arguments), contents
 *   on entry irrelevant.  Calls that can overlap need a workspace each.
 *   T >= 0, S >= 1, T * H < 2^31.  The same lengths give the same bits in every
 *   run.  With a window, attn_kv_evict is for after this call: a chunk's first tokens
 *   still see what its last one does not.
 *   Scores, maxima, sums and O are fp32, parts are joined in fp32.  The
 *   probabilities enter their product as bf16 (2^-8) over bf16 pages, as fp16
 *   (2^-11, and 2^-32 of the row's largest) over e4m3 ones, where q enters its
 *   own as two 8-bit parts (all of an element down to 2^-13 of its row's largest,
 *   below that off by 2^-21 of that one at most).
 */
size_t attn_fwd_paged_workspace_bytes(int T, int S, int H, int H_kv, int d, int max_pages,
                                      int page_size);
attn_status_t attn_fwd_paged(const void* q, int64_t q_stride, const void* k_cache,
                             const void* v_cache, int64_t k_page_stride, int64_t v_page_stride,
                             int kv_dtype, const float* k_scale, const float* v_scale,
                             const int32_t* page_table, const int32_t* seq_lens,
                             const int32_t* cu_q, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, int T, int S, int H, int H_kv, int d,
                             int max_pages, int n_pages, int page_size, float scale,
                             int64_t window, int64_t sinks, void* stream);

/*
 * attn_kv_pool - the mean keys that attn_select_pages scores ("Exact Blocks,
 * Rings, and Sparsity", section 5, 'Fixed pooling').  k_means
 * [n_pages][H_kv][d] fp32, contiguous: of every page of sequence s that became
 * full between start[s] and seq_lens[s] tokens (start as attn_kv_reserve gives
 * it), the mean over its page_size keys, times k_scale[h] over an e4m3 cache, is
 * written, rounded once; other pages' are left as they are.  Sequences with
 * start[s] < 0 and pages given back (-1) are passed over.  With start[s] = 0 all
 * of a sequence's pages are pooled, as after attn_kv_copy_pages has moved pages
 * (attn_kv_compact; what attn_kv_fork copies is not full).  S >= 1.
 */
attn_status_t attn_kv_pool(const void* k_cache, int64_t k_page_stride, int kv_dtype,
                           const float* k_scale, float* k_means, const int32_t* page_table,
                           const int32_t* start, const int32_t* seq_lens, int S, int max_pages,
                           int n_pages, int H_kv, int d, int page_size, void* stream);

/*
 * attn_select_pages - for each new token and K/V head the pages it reads: the
 * first first_pages pages of its sequence, the last local_pages (its own among
 * them, so local_pages >= 1), and of the others the top_r with the highest score
 *   (sum of the query heads that share the K/V head) . k_means[page]
 * ("Exact Blocks, Rings, and Sparsity", sections 5 and 6, as attn_select_blocks
 * scores blocks; ties to the lower place, a NaN last).  What fp32 cannot decide is
 * decided in whole numbers of 128 bits: a score is exact where no product of a
 * query's element and a mean's is below 2^-60 times the largest of both, but 0 (what
 * is lower may be left out of it), and the same products score alike in any order.
 * q, cu_q, seq_lens and page_table as for attn_fwd_paged; a row sees the pages of
 * the tokens up to its own.  Pages given back (-1) are left out.  Where cu_q does not
 * ascend, which is reported, a row is one of some sequence or of none.
 *   pages [T][H_kv][R] int32 out, R = first_pages + local_pages + top_r: the pages
 *   in ascending order of their place, then -1.  lens [T] int32 out: the tokens
 *   in them (every page but the row's own counts whole); -1 for a row of no
 *   sequence, 0 for one before its sequence's first token (reported).
 *   workspace: as for attn_fwd_paged (attn_select_pages_workspace_bytes).
 *   max_pages <= 32768, T * H_kv * R < 2^31.  T >= 0, S >= 1.
 */
size_t attn_select_pages_workspace_bytes(int T, int S, int H, int H_kv, int d, int max_pages,
                                         int page_size, int top_r, int local_pages,
                                         int first_pages);
attn_status_t attn_select_pages(const void* q, int64_t q_stride, const float* k_means,
                                const int32_t* page_table, const int32_t* seq_lens,
                                const int32_t* cu_q, int32_t* pages, int32_t* lens,
                                void* workspace, size_t workspace_bytes, int T, int S, int H,
                                int H_kv, int d, int max_pages, int n_pages, int page_size,
                                int top_r, int local_pages, int first_pages, void* stream);

/*
 * attn_decode_selected - attn_decode_paged for rows that read pages of their own
 * per K/V head: row t's query heads of K/V head h see the first lens[t] tokens of
 * the pages pages[t][h][0 .. max_pages-1] ([T][H_kv][max_pages] int32, as
 * attn_select_pages gives them), in fp32 and bf16 parts as there.  q [T][H][d], o,
 * lse, caches, scales, workspace (attn_decode_paged_workspace_bytes(T, H, H_kv,
 * d, max_pages, page_size)) and errors as for attn_decode_paged with S = T; a row
 * with lens[t] < 0 is of no sequence, its o and lse are left as they were.
 * 1 <= T <= 65536 (a longer batch, which attn_select_pages takes, in parts of rows).
 */
attn_status_t attn_decode_selected(const void* q, int64_t q_stride, const void* k_cache,
                                   const void* v_cache, int64_t k_page_stride,
                                   int64_t v_page_stride, int kv_dtype, const float* k_scale,
                                   const float* v_scale, const int32_t* pages,
                                   const int32_t* lens, void* o, float* lse, void* workspace,
                                   size_t workspace_bytes, int T, int H, int H_kv, int d,
                                   int max_pages, int n_pages, int page_size, float scale,
                                   void* stream);

/*
 * attn_kv_reserve - room for n_new[s] >= 0 more tokens in every sequence: new
 * pages enter the table, seq_lens grows.  start [S] out: the position of the
 * first new token, or -1 for every sequence when the call was refused (too
 * few free pages, or a sequence past max_pages * page_size or 0x7FFFFF00).
 * S >= 1.
 */
attn_status_t attn_kv_reserve(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                              const int32_t* n_new, int32_t* start, int S, int max_pages,
                              int n_pages, int page_size, void* stream);

/*
 * attn_kv_write - keys and values of new tokens into their pages.  k_new,
 * v_new [T][H_kv][d] bf16, rows k_new_stride / v_new_stride elements apart (a
 * multiple of 8, at least H_kv*d).  Rows cu_new[s] .. cu_new[s+1]-1 (cu_new
 * [S+1] int32, ascending) are sequence s's tokens start[s], start[s]+1, ...;
 * rows before cu_new[0] or from cu_new[S] on are left out, and so are
 * sequences with start[s] < 0.  An e4m3 cache gets round(x / scale[h]),
 * saturated at 448.
 */
attn_status_t attn_kv_write(const void* k_new, const void* v_new, int64_t k_new_stride,
                            int64_t v_new_stride, void* k_cache, void* v_cache,
                            int64_t k_page_stride, int64_t v_page_stride, int kv_dtype,
                            const float* k_scale, const float* v_scale, const int32_t* page_table,
                            const int32_t* start, const int32_t* cu_new, int T, int S,
                            int max_pages, int n_pages, int H_kv, int d, int page_size,
                            void* stream);

/*
 * attn_kv_fork - sequence children[f] becomes a copy of parents[f].  Full
 * pages are shared; of a last page that is not full the child takes a page of
 * its own, and copy_src[f], copy_dst[f] name the copy to make (-1: none) with
 * attn_kv_copy_pages, once per layer's cache.  A child must be empty, occur
 * once and not be a parent too; a parent may occur often.
 */
attn_status_t attn_kv_fork(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                           const int32_t* parents, const int32_t* children, int n_forks,
                           int32_t* copy_src, int32_t* copy_dst, int S, int max_pages, int n_pages,
                           int page_size, void* stream);

/*
 * attn_kv_free - the listed sequences give back their pages and become empty
 * (listed twice: freed once).
 */
attn_status_t attn_kv_free(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                           const int32_t* seqs, int n_seqs, int S, int max_pages, int n_pages,
                           int page_size, void* stream);

/*
 * attn_kv_evict - every sequence gives back the pages that attn_decode_paged
 * with this window and sinks no longer reads, now or at a greater length.
 */
attn_status_t attn_kv_evict(int32_t* page_table, const int32_t* seq_lens, int32_t* refs,
                            int64_t window, int64_t sinks, int S, int max_pages, int n_pages,
                            int page_size, void* stream);

/*
 * attn_kv_compact - the pages in use move to the lowest indices: with n in
 * use, those at n or past it take, in ascending order, the free pages below n.
 * The table and refs follow; copy_src, copy_dst [n_pages] list the copies to
 * make (ascending, then -1) and count [1] their number, for
 * attn_kv_copy_pages.
 */
attn_status_t attn_kv_compact(int32_t* page_table, int32_t* refs, int32_t* copy_src,
                              int32_t* copy_dst, int32_t* count, int S, int max_pages, int n_pages,
                              void* stream);

/*
 * attn_kv_copy_pages - page copy_src[i] of both caches to page copy_dst[i],
 * for i < n_copies, or i < min(n_copies, *count) when count (device) is not
 * NULL.  A pair of two negative entries is left out.  The copies run in any
 * order: no page may be both a source and a destination, and a destination
 * may occur once.
 */
attn_status_t attn_kv_copy_pages(void* k_cache, void* v_cache, int64_t k_page_stride,
                                 int64_t v_page_stride, int kv_dtype, const int32_t* copy_src,
                                 const int32_t* copy_dst, int n_copies, const int32_t* count,
                                 int n_pages, int H_kv, int d, int page_size, void* stream);

/*
 * attn_poll_status - synchronise `stream`, then return and clear the first
 * error any kernel of this library recorded on the current device since the
 * last poll (ATTN_OK if none).
 */
attn_status_t attn_poll_status(void* stream);

/*
 * attn_bwd_time_main - measurement aid: the backward calls (attn_bwd,
 * attn_bwd_blocksparse, attn_bwd_noalloc) launch three kernels, the row
 * statistic D = rowsum(dO * O), the main kernel that recomputes the score
 * tiles and produces dK, dV and the dQ accumulator ("Exact Blocks, Rings, and
 * Sparsity", section 3), and the dQ conversion to bf16.  While `begin` and
 * `end` are set, every backward call records `begin` on its stream just
 * before the main kernel's launch and `end` just after it, so that the
 * elapsed time between them (cudaEventElapsedTime) is that kernel's own
 * duration.  `begin`, `end`: cudaEvent_t handles owned by the caller, created
 * on the device of the calls (and with timing enabled, for elapsed times).
 * Both NULL switches the recording off.  The setting is process-wide: set and
 * clear it from the thread that makes the calls.  Returns
 * ATTN_ERR_INVALID_ARG when exactly one of the two is NULL, else ATTN_OK.
 */
attn_status_t attn_bwd_time_main(void* begin, void* end);

/*
 * attn_probe_ex2_rate - measurement aid for the softmax's second ceiling:
 * the forward evaluates one exponential per pair ("FlashAttention: Fast and
 * Memory Efficient Exact Attention with IO Awareness", section 5.1, the
 * online softmax), so pairs/s cannot exceed the SMs' ex2 rate.  Launches
 * `blocks` blocks of 256 threads on `stream`; every thread evaluates
 * 8 * `iters` independent ex2.approx exponentials, blocks * 256 * 8 * iters
 * in all.  The caller times the launch.  `sink`: one device float,
 * 4-byte aligned, never written in practice (it keeps the work alive).
 * Returns ATTN_ERR_INVALID_ARG for a null sink or non-positive sizes, else
 * the launch status.
 */
attn_status_t attn_probe_ex2_rate(float* sink, int blocks, int iters, void* stream);

/*
 * attn_watchdog_selftest - launch one block that waits on a barrier nobody
 * arrives at, with a limit of `timeout_cycles` SM clock cycles; the wait gives
 * up, records ATTN_ERR_TIMEOUT and the block returns.  Lets a test observe the
 * watchdog path without hanging or faulting the GPU.  Returns the launch status.
 */
attn_status_t attn_watchdog_selftest(unsigned long long timeout_cycles, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSS_ATTN_H_ */
