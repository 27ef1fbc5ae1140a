/*
 * attn.h -- C ABI of libattn, a GB300 (sm_103a) fused attention forward pass.
 *
 * The operation is scaled-dot-product attention as the JAX Pallas page
 * (attention_mgpu.py) defines it in `attention_reference`, with the caller's
 * softmax scale applied to the logits, grouped-query heads mapped as in that
 * page's `_attention_forward` (kv_head = q_head / (Hq / Hkv)), and the
 * log-sum-exp residual that page stores for the backward pass:
 *
 *     S   = scale * Q K^T              (per batch b, query head h, kv head g)
 *     O   = softmax(S [+ causal mask]) V
 *     LSE = ln sum_j exp(S_ij)         (natural log, fp32)
 *
 * It is computed tile by tile with an online softmax (running row max m, row
 * sum l and an fp32 accumulator, exp2 of pre-scaled logits, one final division
 * by l), the schedule of the Pallas page's kernel loop and of the Choreo
 * tutorial's non-persistent FA kernel, on Blackwell tensor cores (tcgen05).
 *
 * Plain pointers and sizes only; no framework types.  All functions are
 * thread-safe.  No call allocates device memory: scratch memory, where a path
 * needs some, is passed in by the caller.  The library's own device state is
 * static: a 4-byte status word and the 40 MiB scratch array of
 * attn_fwd_splitkv_noalloc, which every GPU that loads the library holds until
 * the process exits (one copy per GPU), whether or not that entry point is
 * ever called.
 */
#ifndef LIBATTN_ATTN_H_
#define LIBATTN_ATTN_H_

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment, scale or flag; nothing launched */
    ATTN_ERR_UNSUPPORTED = 2, /* valid request this build does not implement (head size)  */
    ATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call or the kernel launch failed       */
    ATTN_ERR_TIMEOUT = 4      /* a device-side bounded wait ran out (see attn_last_device_status) */
} attn_status_t;

/*
 * attn_fwd -- O = softmax(scale * Q K^T [+ mask]) V and LSE, asynchronously on `stream`.
 *
 * q    device pointer, bf16, [B, Sq, Hq, D], D contiguous (row stride Hq*D elements)
 * k, v device pointers, bf16, [B, Skv, Hkv, D]
 * o    device pointer, bf16, [B, Sq, Hq, D]   (written; round-to-nearest-even of O)
 * lse  device pointer, fp32, [B, Hq, Sq], or NULL to skip it
 * B, Sq, Skv, Hq, Hkv, D  sizes; every one >= 1, Hq a multiple of Hkv, D 64, 128 or 256
 *      (other head sizes: ATTN_ERR_UNSUPPORTED).
 *      Sq and Skv may be any length (ragged tails are handled in the kernel).
 * causal 0: every key visible.  1: key j visible from query i iff
 *      j <= i + (Skv - Sq) (bottom-right aligned, as in chunked prefill).
 *      2: iff j <= i (top-left aligned, the Pallas page's reference mask).
 *      1 and 2 coincide when Sq == Skv.  A query row that sees no key gets
 *      O = 0 and LSE = -inf.
 * scale  finite, > 0 (typically 1/sqrt(D)).
 * stream CUDA stream the kernel runs on (0 = legacy default stream).
 *
 * Ownership: the caller owns every buffer; nothing is retained after return.
 * q, k, v, o must be 16-byte aligned (TMA).  o must not alias q, k or v.
 * Returns ATTN_OK once the kernel is enqueued; a device-side wait that runs out
 * is reported later through attn_last_device_status.  On any error return,
 * nothing was launched and no output was written.
 */
attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int Sq, int Skv, int Hq, int Hkv, int D, int causal, float scale,
                       cudaStream_t stream);

/* Element type of q, k, v and o for attn_fwd_ex. */
typedef enum {
    ATTN_DTYPE_BF16 = 0, /* bfloat16 (what attn_fwd takes) */
    ATTN_DTYPE_F16 = 1   /* IEEE binary16 */
} attn_dtype_t;

/*
 * attn_fwd_ex -- attn_fwd with a choice of 16-bit element type for q, k, v and
 * o (the Pallas page's forward accepts float16 and bfloat16 alike).  `dtype`
 * is an attn_dtype_t; anything else returns ATTN_ERR_INVALID_ARG.  P is rounded
 * to the same type before the P.V product; accumulation, softmax and LSE stay
 * fp32; O is rounded to nearest-even in that type.  Everything else, including
 * errors, as attn_fwd.
 */
attn_status_t attn_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
                          int B, int Sq, int Skv, int Hq, int Hkv, int D, int causal, float scale,
                          int dtype, cudaStream_t stream);

/*
 * Split-KV forward for problems with too few query tiles to fill the GPU
 * (short query blocks against long key ranges, e.g. chunked prefill).  The
 * same operation and arguments as attn_fwd (bf16), plus a device workspace the
 * caller allocates.  This is the single-GPU form of the kernbench page's group
 * sequence parallelism (`_gqa_attention_prefill_short.py`): the iterations over
 * (query tile pair, KV tile) are cut into equal contiguous shares, one per SM; a
 * tile pair whose KV range straddles shares is computed in pieces whose partial
 * (m, l, O) are merged by that page's `_merge_running` rule in a second kernel.
 *
 * attn_fwd_splitkv_workspace_size: bytes of workspace attn_fwd_splitkv needs
 *   for this problem on the current device (it depends on the SM count); 0 when
 *   no split pays off, and then attn_fwd_splitkv runs exactly what attn_fwd runs.
 *   A split is chosen only when the whole-unit schedule's busiest SM would run at
 *   least 1.35x the KV iterations of an equal share (plus 4): the crossover
 *   measured on GB300 (decode rows and short prefill chunks against long key
 *   ranges split and run several times faster; shapes that already fill the GPU
 *   do not).  This is the entry point to call when scratch can be supplied.
 * attn_fwd_splitkv: workspace device pointer (256-byte aligned, not aliasing
 *   any other argument) of at least that many bytes, or NULL when the size is 0.
 *   The workspace is scratch: its contents are undefined before and after the
 *   call, and two calls that overlap in time on the GPU must not share one.
 *   Errors as attn_fwd; ATTN_ERR_INVALID_ARG also for a missing or short workspace.
 */
attn_status_t attn_fwd_splitkv_workspace_size(int B, int Sq, int Skv, int Hq, int Hkv, int D,
                                              int causal, size_t* bytes);
attn_status_t attn_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                               int B, int Sq, int Skv, int Hq, int Hkv, int D, int causal,
                               float scale, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * attn_fwd_splitkv_noalloc -- attn_fwd_splitkv for callers that cannot
 * allocate device memory where they call attention: code whose device memory
 * all belongs to another allocator (a framework's caching pool, a fixed arena
 * reserved at start-up) or that runs where allocation is not allowed once
 * serving has begun.  The pages have no counterpart of this entry point.
 *
 * Same arguments, semantics and errors as attn_fwd_splitkv, without the
 * workspace: the split-KV scratch is a static 40 MiB device array inside
 * libattn, which every GPU that loads the library holds until the process
 * exits.  The call allocates nothing, on the device or on the host.
 *   - The first call on a device looks up that array's device address (once per
 *     device, with the device current); make that first call before any stream
 *     capture begins.
 *   - Problems whose scratch would exceed 40 MiB return ATTN_ERR_UNSUPPORTED
 *     (on a 152-SM GPU the split plan never needs more than about 38.4 MiB).
 *   - Each GPU has its own copy of the array; every call on one GPU shares that
 *     copy, which keeps the last call's contents.  Nothing in it needs to start
 *     at zero (each call writes every partial slot before it reads it).  Calls
 *     that overlap in time on the same GPU (for example on different streams)
 *     race on it and must be serialised; calls on different GPUs do not share
 *     scratch.
 */
attn_status_t attn_fwd_splitkv_noalloc(const void* q, const void* k, const void* v, void* o,
                                       float* lse, int B, int Sq, int Skv, int Hq, int Hkv, int D,
                                       int causal, float scale, cudaStream_t stream);

/*
 * attn_bwd -- gradients of the attention forward: given dO, the gradient of
 * L = sum dO * O, with O = softmax(scale * Q K^T [+ mask]) V as in attn_fwd
 * (the Pallas page, attention_mgpu.py, `_attention_bwd`):
 *   P = exp(scale * Q K^T - LSE) (masked pairs 0), delta = rowsum(O * dO),
 *   dP = dO V^T, dS = P * (dP - delta),
 *   dQ = scale * dS K,  dK = scale * dS^T Q,  dV = P^T dO,
 * with dK and dV summed over the query heads that share a key/value head.
 *
 * q, k, v   device pointers, the forward's inputs (layouts as attn_fwd).
 * o         device pointer, [B, Sq, Hq, D]: the forward's output.
 * lse       device pointer, fp32 [B, Hq, Sq]: the forward's natural-log LSE
 *           (-inf for rows that see no key).
 * dO        device pointer, [B, Sq, Hq, D]: gradient of the output.
 * dq        device pointer, [B, Sq, Hq, D]     (written)
 * dk, dv    device pointers, [B, Skv, Hkv, D]  (written; every element, zero for
 *           keys no query row sees)
 * B .. scale  as attn_fwd (the same causal mode and scale as the forward call;
 *           the page's backward has no mask, this one applies the forward's);
 *           D 64, 128 or 256; B <= 65535.
 * dtype     ATTN_DTYPE_BF16 or ATTN_DTYPE_F16: the element type of q, k, v, o,
 *           dO, dq, dk and dv.
 * workspace device pointer, 256-byte aligned, of at least
 *           attn_bwd_workspace_size bytes (per-row delta and base-2 LSE);
 *           scratch, contents undefined before and after the call.
 *
 * Arithmetic: operands and P, dS in the element type, fp32 accumulation in
 * tensor memory, fp32 delta; outputs rounded to nearest even once.
 * Ownership: the caller owns every buffer.  q, k, v, o, dO, dq, dk, dv must be
 * 16-byte aligned; lse 4-byte aligned.  dq, dk, dv and the workspace must not
 * overlap any input or each other.  Three kernels are enqueued on `stream`
 * (prep, dK/dV, dQ), four at D = 256 (prep, dV, dK, dQ); errors are reported
 * as for attn_fwd (nothing is launched on any error return; a device-side
 * timeout shows in attn_last_device_status).
 */
attn_status_t attn_bwd_workspace_size(int B, int Sq, int Skv, int Hq, int Hkv, int D, size_t* bytes);
attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* dO, void* dq, void* dk, void* dv, int B, int Sq, int Skv, int Hq,
                       int Hkv, int D, int causal, float scale, int dtype, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * Paged key/value cache: sequences of unlike lengths whose keys and values live in
 * pages, for serving.  (The pages that describe this forward compute attention over
 * dense tensors only; this is the same operation over a cache.)
 *
 * A cache is two tensors, K and V, of n_pages pages of page_size tokens of Hkv heads
 * of D elements.  Element d of head h of row r of page x is at
 *     x * page_stride + r * token_stride + h * head_stride + d   (strides in elements),
 * so pages stored token by token ([page, token, head, D]), head by head ([page, head,
 * token, D]) or with K and V in turn ([page, 2, token, head, D], two base pointers)
 * are all read as they are.  K and V share the strides, which are multiples of 8 and
 * lay no two rows over each other (of an axis of one the stride is ignored).  Base
 * pointers are 16-byte aligned.
 *
 * Token t of sequence s lives in row t % page_size of page
 * block_table[s * table_stride + t / page_size]; the table is int32 with max_pages
 * columns.  Its slot is page * page_size + row.  An entry outside [0, n_pages) names
 * no page: its tokens are not written and not seen.
 *
 * Lengths, tables and slots are device data.  No call reads them on the host, so a
 * captured graph replays with what they hold then.  Values are clamped where they
 * are read; no content of theirs makes a kernel leave its buffers.
 */

/*
 * attn_paged_tables -- the tables of one step, from the lengths of its sequences.
 *
 * Sequence i has ctx_lens[i] tokens in the cache and gets new_lens[i] more (both
 * device int32 [n_seqs]; a negative length counts as zero, and a sequence without new
 * tokens takes no page).  Its row of block_table is extended by the pages that the new
 * tokens start: columns ceil(ctx / page_size) to ceil((ctx + new) / page_size) - 1.
 *
 * free_pages   device int32 [n_free], pages to take in order, sequence after sequence,
 *              from entry *free_head on (device int32; NULL: from the first).  Once
 *              the list is used up, new columns get -1.  n_free 0 needs no list.
 * block_table  device int32 [n_seqs, max_pages], row stride table_stride (in/out; only
 *              the new columns are written, none past max_pages).
 * cu_new       device int32 [n_seqs + 1] (written): sums of the new tokens before each
 *              sequence; the batch's rows of sequence i are cu_new[i] .. cu_new[i+1]-1.
 * kv_lens      device int32 [n_seqs] (written): ctx + new.
 * slot_map     device int64 [max_tokens] (written): the slot of each new token, in the
 *              batch's order; -1 for a token without a page and for every entry behind
 *              the last token.  Tokens past max_tokens get no entry.
 * counts       device int32 [4] (written): new tokens in all; the entry of free_pages
 *              at which the next call starts; pages that were missing; sequences that
 *              do not fit into max_pages columns.
 * Sums past 2^31 - 1 are written as that.
 *
 * Asynchronous on `stream`, one kernel, no workspace.  int32 buffers 4-byte, slot_map
 * 8-byte aligned; no output overlaps an input or another output; every size but
 * n_free is at least 1.  On any error return nothing was launched.
 */
attn_status_t attn_paged_tables(const int* ctx_lens, const int* new_lens, int n_seqs, int page_size,
                                const int* free_pages, int n_free, const int* free_head, int* block_table,
                                int max_pages, long long table_stride, int* cu_new, int* kv_lens,
                                long long* slot_map, int max_tokens, int* counts, cudaStream_t stream);

/*
 * attn_paged_append -- write the keys and values of new tokens into their pages.
 *
 * k, v      device pointers, 16-bit elements, [n_tokens, Hkv, D], heads contiguous, row
 *           strides k_stride and v_stride (elements, multiples of 8, at least Hkv * D:
 *           slices of a fused projection are read in place).
 * slot_map  device int64 [n_tokens]: each row's slot; rows whose slot is outside
 *           [0, n_pages * page_size) are skipped.  If two rows name one slot, the slot
 *           holds elements of either afterwards.
 * k_cache, v_cache, n_pages .. head_stride  the cache, as above; D 64, 128 or 256
 *           (other head sizes: ATTN_ERR_UNSUPPORTED).  It overlaps no other argument.
 *
 * The rows are copied as they are (bf16 and fp16 alike).  Every size is at least 1.
 * Asynchronous on `stream`, one kernel; on any error return nothing was launched.
 */
attn_status_t attn_paged_append(const void* k, const void* v, const long long* slot_map, void* k_cache,
                                void* v_cache, int n_tokens, int Hkv, int D, int n_pages, int page_size,
                                long long k_stride, long long v_stride, long long page_stride,
                                long long token_stride, long long head_stride, cudaStream_t stream);

/*
 * attn_paged_fwd -- attn_fwd for the new tokens of a ragged batch over their cache:
 * whole prompts, chunks of prompts, drafted tokens and single tokens, in one call.
 *
 * q            device pointer, [total_q, Hq, D], heads contiguous, row stride q_stride
 *              (elements, a multiple of 8, at least Hq * D), 16-byte aligned.
 * o            device pointer, [total_q, Hq, D] contiguous, 16-byte aligned (written).
 * lse          device pointer, fp32 [Hq, total_q], or NULL to skip it (written).
 * cu_q         device int32 [n_seqs + 1]: sequence i's rows of q and o are cu_q[i] ..
 *              cu_q[i+1] - 1, cut to [0, total_q); a sequence may have none.  Rows of no
 *              sequence (behind the last one, in a padded batch) are left as they were.
 * kv_lens      device int32 [n_seqs]: keys of sequence i in the cache, its new tokens
 *              among them (append before this call); values below zero count as zero,
 *              values past max_pages * page_size as that.
 * block_table, k_cache, v_cache, n_pages .. head_stride  the cache, as above.
 * max_q_len    the longest sequence's rows, >= 1, as far as the host knows.  It chooses
 *              the kernel (few rows against many; total_q or more: not known); results are
 *              right for any value.
 * causal       0: every key of the sequence is visible.  1: row t of a sequence with n
 *              rows and m keys sees keys j <= t + (m - n).  A row that sees no key gets
 *              O = 0 and LSE = -inf.  What unseen rows of the cache hold (stale rows
 *              behind the last key, NaN or infinities among them) has no influence; a
 *              key that some rows of a sequence see and others do not is expected to be
 *              finite.
 * Hq, Hkv, D, scale, dtype  as attn_fwd_ex.
 * workspace    device pointer, 256-byte aligned, of at least
 *              attn_paged_fwd_workspace_size bytes for the current device (the size for
 *              the same total_q .. page_size).  Scratch: its contents are undefined before
 *              and after the call, and calls that overlap in time on the GPU must not
 *              share one.
 * Every size is at least 1; total_q * Hq is at most 2^31 - 1.
 *
 * Arithmetic as attn_fwd: operands and P in the element type, products and softmax
 * statistics in fp32, O rounded to nearest even once.  Results do not depend on timing:
 * two calls with equal arguments give equal bits.  Asynchronous on `stream`; o, lse and
 * the workspace overlap no input and not each other.  On any error return that is not
 * ATTN_ERR_CUDA nothing was launched; after that one, with up to three kernels in a call, o
 * and lse are undefined (the call may be made again).  A device-side timeout shows in
 * attn_last_device_status.
 */
attn_status_t attn_paged_fwd_workspace_size(int total_q, int max_q_len, int Hq, int Hkv, int D, int page_size,
                                            size_t* bytes);
attn_status_t attn_paged_fwd(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                             const int* block_table, const int* cu_q, const int* kv_lens, int n_seqs,
                             int total_q, int max_q_len, int Hq, int Hkv, int D, int n_pages, int page_size,
                             int max_pages, long long q_stride, long long table_stride, long long page_stride,
                             long long token_stride, long long head_stride, int causal, float scale, int dtype,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Pages that several sequences share.
 *
 * shares  device int32 [n_pages], for every page the rows of the block table that name it
 *         beyond the first: 0 for a page of one row and for a free page, so attn_paged_tables
 *         needs no count.  A buffer of zeros goes with a table without shared pages.  A page
 *         that is shared is not written to: attn_paged_fork leaves only full pages shared.
 */

/*
 * attn_paged_fork -- rows that begin with the tokens of another row (beams, requests with a
 * common beginning).
 *
 * parents   device int32 [n_seqs]: the row that row i takes its first tokens from.  A value
 *           outside [0, n_seqs), and i itself, mean none: the row is left as it is.  A row whose
 *           parent has a parent in the same call is left too, and counted.  Any number of rows
 *           may have one parent.  The pages that a row named before are not given back: free it
 *           first.
 * lens      device int32 [n_seqs]: tokens to take (below zero: none; past the parent's: all), or
 *           NULL for all of the parent's.
 * kv_lens   device int32 [n_seqs] (in/out): tokens of every row (clamped to what a row can name);
 *           a fork's becomes the tokens that it took.
 * free_pages, n_free, free_head  as attn_paged_tables.
 * block_table  device int32 [n_seqs, max_pages], row stride table_stride (in/out).  With t tokens
 *           a fork's first t / page_size columns are its parent's.  A rest of t % page_size tokens
 *           takes a page of the list, in the order of the rows (-1 once it is used up; without a
 *           page of the parent's that holds the rest none is taken, and the entry is the
 *           parent's).  Columns behind are left.
 * shares    (in/out) one more for every column that a fork shares.
 * copies    device int32 [n_seqs, 3] (written): (from page, to page, tokens) of a fork with a
 *           rest, for attn_paged_copy; (-1, -1, 0) for all other rows.
 * counts    device int32 [4] (written): forks; the entry of free_pages at which the next call
 *           starts; pages that were missing; rows that were left since their parent has one.
 *
 * Asynchronous on `stream`, one kernel, no workspace.  All buffers are 4-byte aligned; no output
 * overlaps an input or another output.  On any error return nothing was launched.
 */
attn_status_t attn_paged_fork(const int* parents, const int* lens, int* kv_lens, int n_seqs, int page_size,
                              const int* free_pages, int n_free, const int* free_head, int* block_table,
                              int max_pages, long long table_stride, int* shares, int n_pages, int* copies,
                              int* counts, cudaStream_t stream);

/*
 * attn_paged_free -- pages of rows that end or are cut shorter go back to the free list.
 *
 * kv_lens, keep_lens  device int32 [n_seqs]: tokens that a row has and that it keeps (0: the row
 *             ends; as many as it has or more: nothing changes; below zero counts as 0).  The
 *             columns ceil(keep / page_size) to ceil(kv / page_size) - 1 give up their page.
 * block_table device int32 [n_seqs, max_pages] (read; entries are left as they are).
 * shares      (in/out) one less for every column that gives up a page.  A page whose count would
 *             fall below zero is free and has 0.
 * free_pages  device int32 [n_free] (in/out): the list of attn_paged_tables, whose entries before
 *             *free_head (device int32, read; clamped to [0, n_free]) have been taken.  The freed
 *             pages become the entries in front of it, in ascending order.
 * counts      device int32 [4] (written): pages that were listed; the entry at which the next call
 *             starts; freed pages that found no room in front of free_head (the lowest numbers);
 *             rows cut inside a page that is still shared, which is not to be written to: fork the
 *             row instead.
 *
 * Asynchronous on `stream`, one kernel, or two where the table has 65536 entries (n_seqs * max_pages) or more; no
 * workspace; results do not depend on timing.  All buffers are 4-byte aligned; no output overlaps an input or another
 * output; every size is at least 1.  On any error return that is not ATTN_ERR_CUDA nothing was launched.  After
 * ATTN_ERR_CUDA the first of two kernels may have lowered counts: shares is undefined then, and a second call would
 * lower them again.
 */
attn_status_t attn_paged_free(const int* kv_lens, const int* keep_lens, int n_seqs, int page_size,
                              const int* block_table, int max_pages, long long table_stride, int* shares,
                              int n_pages, int* free_pages, int n_free, const int* free_head, int* counts,
                              cudaStream_t stream);

/*
 * attn_paged_copy -- the first tokens of pages to other pages, in many caches at once.
 *
 * copies    device int32 [n_copies, 3]: (from page, to page, tokens), as attn_paged_fork lists them.
 *           Entries with a page outside [0, n_pages), with no tokens, or from a page to itself are
 *           skipped; tokens past page_size count as that.  If a page is written by one entry and
 *           read or written by another, it holds elements of either afterwards.
 * caches    host array of n_caches device pointers (every layer's K and V, say), read before the
 *           call returns: caches of one layout, of any element type.  They overlap no other argument.
 * row_bytes bytes of a head's row, a multiple of 4 (16-bit caches: 2 D; codes of 4 bits: D / 2; their
 *           scales: D / 16); a page's tokens together are at most 2^31 - 1 bytes.
 * page_stride .. head_stride  in bytes, multiples of 4, laying no two rows over each other.
 *
 * Every size is at least 1.  Asynchronous on `stream`, one kernel for every 256 caches; on any error
 * return that is not ATTN_ERR_CUDA nothing was launched.
 */
attn_status_t attn_paged_copy(const int* copies, int n_copies, void* const* caches, int n_caches, int n_pages,
                              int page_size, int Hkv, int row_bytes, long long page_stride,
                              long long token_stride, long long head_stride, cudaStream_t stream);

/*
 * Paged cache in 4 bits.
 *
 * K and V are each two tensors: codes, of D / 2 bytes a head's row, and scales, of D / 16 bytes.
 * Byte i of a row's codes holds elements 2 i (low half) and 2 i + 1 (high half) as e2m1 (sign bit, then
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6); byte b of its scales is the e4m3 scale of elements 16 b to 16 b + 15.  An
 * element is code * scale * unit, the unit being a number for all of K (k_unit) or V (v_unit): 1 serves
 * rows whose blocks' largest elements lie between 2^-4 and 2688; smaller ones lose precision, larger ones
 * saturate.  4.5 bits an element.
 *
 * Rows lie as in a cache of 16 bits, with strides in bytes: the codes' are multiples of 16, the scales' of
 * D / 16, and so are the base pointers' addresses.  K and V share the strides.  Pages stored head by head
 * ([page, head, token, .]) keep the small scales of a head's tokens together and are read fastest.
 */

/*
 * attn_paged_coded_append -- attn_paged_append into a cache in 4 bits.
 *
 * k, v, slot_map, n_tokens, k_stride, v_stride  as attn_paged_append; dtype is an attn_dtype_t.
 * With y = x / unit (a product with 1 / unit) a block's scale is max |y| / 6 rounded to the nearest
 * e4m3, ties to even, at most 448 and at least 2^-9 unless the block is zero; a code is y / scale
 * rounded to the nearest e2m1, ties to the even code, 6 at most, with y's sign (product and quotients
 * in fp32).  Of a block with a NaN or an infinity the scale is 448, and those are stored as +-6 (a NaN
 * as +6).  Units are positive and finite, and so is 1 / unit in fp32.
 * If two rows name one slot, it holds bytes of either afterwards, codes and scales apart.
 *
 * Errors and the rest as attn_paged_append.
 */
attn_status_t attn_paged_coded_append(const void* k, const void* v, const long long* slot_map, void* k_codes,
                                 void* k_scales, void* v_codes, void* v_scales, int n_tokens, int Hkv, int D,
                                 int n_pages, int page_size, long long k_stride, long long v_stride,
                                 long long code_page_stride, long long code_token_stride,
                                 long long code_head_stride, long long scale_page_stride,
                                 long long scale_token_stride, long long scale_head_stride, float k_unit,
                                 float v_unit, int dtype, cudaStream_t stream);

/*
 * attn_paged_coded_fwd -- attn_paged_fwd over a cache in 4 bits.
 *
 * q, o and lse are bf16 or fp16 and fp32 as there, and so are all other arguments and the workspace (of
 * attn_paged_coded_fwd_workspace_size bytes).  scale * k_unit * log2(e) is a normal number of fp32.
 * Logits times log2(e) are below 2^23 in size: O and LSE of a row with larger ones may be NaN.
 *
 * Arithmetic: K and V become fp16 without rounding, and q in bf16 does but for elements below 2^-28 of its
 * row's largest, which are off by at most 2^-39 of that.  P is rounded to fp16, weights below 2^-21 of their row's
 * largest to 2^-32 of it.  Products and softmax statistics are fp32, O is rounded to nearest even once.  What unseen
 * rows of the cache hold (scales that are NaN among them) has no influence.
 */
attn_status_t attn_paged_coded_fwd_workspace_size(int total_q, int max_q_len, int Hq, int Hkv, int D, int page_size,
                                             size_t* bytes);
attn_status_t attn_paged_coded_fwd(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                              const void* v_scales, void* o, float* lse, const int* block_table, const int* cu_q,
                              const int* kv_lens, int n_seqs, int total_q, int max_q_len, int Hq, int Hkv, int D,
                              int n_pages, int page_size, int max_pages, long long q_stride, long long table_stride,
                              long long code_page_stride, long long code_token_stride, long long code_head_stride,
                              long long scale_page_stride, long long scale_token_stride,
                              long long scale_head_stride, int causal, float scale, float k_unit, float v_unit,
                              int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char* attn_status_str(attn_status_t status);

/*
 * attn_last_device_status -- the device-side outcome of the calls made so far.
 * Every libattn kernel records a bounded wait that ran out in one status word
 * per device (the Pallas page's host boundary returns errors only at call
 * time; this word carries the ones found later, on the GPU).  Waits until all
 * work submitted to the current device has completed (cudaDeviceSynchronize),
 * then reads and clears that device's word.  Returns ATTN_ERR_TIMEOUT if any
 * libattn kernel on the current device gave up a bounded wait since the word
 * was last read (that call's outputs are then invalid), ATTN_ERR_CUDA if
 * synchronisation or the read failed, else ATTN_OK.  The word is per device,
 * not per calling thread: a timeout is reported once, to whichever caller
 * reads it first.
 */
attn_status_t attn_last_device_status(void);

/*
 * attn_check_device_status -- attn_last_device_status that waits only for
 * `stream` (cudaStreamSynchronize) instead of the whole device, for callers
 * whose libattn work all ran on that stream.  Same word, same return values.
 */
attn_status_t attn_check_device_status(cudaStream_t stream);

/* Number of kernels libattn has enqueued in this process (all devices). */
unsigned long long attn_kernel_launches(void);

/*
 * Self-test of the bounded-wait path (failure detection without a GPU fault):
 * launches one CTA that waits on an mbarrier nothing ever arrives on, for at
 * most `poll_limit` polls, then records ATTN_ERR_TIMEOUT in the device status
 * word and returns normally.  The caller then sees ATTN_ERR_TIMEOUT from
 * attn_last_device_status.  poll_limit must be in [1, 1<<20].
 */
attn_status_t attn_debug_wait_timeout(unsigned int poll_limit, cudaStream_t stream);

/*
 * Measured issue rates of the units the attention loop leans on (diagnostic;
 * no page defines it: it checks the design's assumption that the forward's
 * 16384 exponentials per 128x128 tile fit under its 2 x 8 tensor-core products,
 * so that no exponential has to move to the FMA pipe).  Runs one CTA per SM of
 * the current device on `stream` and synchronises it.  out (host, n >=
 * ATTN_UNIT_RATES doubles) receives:
 *   out[0..4]  SM clock cycles per tcgen05.mma kind::f16 with M = 128, K = 16,
 *              bf16 operands, fp32 accumulator, issued back to back by one
 *              thread: [0] both operands in shared memory, N = 128; [1] A in
 *              tensor memory, N = 128; [2] shared memory, N = 256; [3] shared
 *              memory, N = 64; [4] A in tensor memory, N = 64
 *   out[5]     cycles per warp-wide ex2.approx.ftz.f32 on one SM sub-partition
 *              (two warps of independent exponentials per sub-partition)
 *   out[6]     exponentials per cycle per SM (= 4 x 32 / out[5])
 *   out[7]     number of SMs measured
 * Returns ATTN_ERR_INVALID_ARG for a NULL `out` or n < ATTN_UNIT_RATES (nothing
 * is launched), ATTN_ERR_CUDA on a launch or copy failure, ATTN_ERR_TIMEOUT if
 * the MMA completion wait ran out or if an earlier libattn kernel on this device
 * had already recorded a timeout (that earlier timeout is reported here, not
 * lost: the status word is read and cleared before the first rate kernel and
 * again after the last, as attn_check_device_status(stream) does), else ATTN_OK.
 */
#define ATTN_UNIT_RATES 8
attn_status_t attn_debug_unit_rates(double* out, int n, cudaStream_t stream);

/*
 * The forward's unit schedule for a shape (diagnostic; host only, launches
 * nothing).  attn_fwd runs two 128-row query tiles per work unit on a
 * persistent grid of min(#units, sms) CTAs.  For causal shapes of head size
 * 128 with at most 2048 units it takes the units from a table: the units in
 * blocks of heads whose K and V together take at most 48 MB, longest first
 * within a block, each unit handed to the least-loaded CTA.  Otherwise each
 * CTA takes units in a snake order and no table exists.
 *   sms          number of SMs to plan for, in [1, 256]
 *   cta_begin    (host, >= grid + 1 ints, grid = min(#units, sms)) receives
 *                the table's per-CTA start offsets into `units`
 *   units        (host, `cap` ints) receives the unit indices, CTA after CTA,
 *                each CTA's in the order it takes them
 *   n_units_out  receives the number of units in the table, or 0 when the
 *                snake order is used (cta_begin and units are then untouched)
 * Returns ATTN_ERR_INVALID_ARG for invalid sizes, sms out of range, a NULL
 * pointer, or a `cap` smaller than the table; ATTN_ERR_UNSUPPORTED for a head
 * size other than 64, 128 or 256; else ATTN_OK.
 */
attn_status_t attn_debug_unit_schedule(int B, int Sq, int Skv, int Hq, int Hkv, int D, int causal, int sms,
                                       int* cta_begin, int* units, int cap, int* n_units_out);

#ifdef __cplusplus
}
#endif

#endif /* LIBATTN_ATTN_H_ */
