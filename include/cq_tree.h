/*
 * cq_tree.h -- a step of tree speculative decoding over the 8-bit paged cache of
 * cq_kv.h: per-head norms and rotation of queries and keys, masks and positions of
 * a tree of drafted tokens, attention under them, verification of the drafts
 * against the target's probabilities, and the cache put in order afterwards:
 *
 *   cq_kv_plan -> cq_tree_plan -> (each layer: projections -> cq_qk_rope ->
 *   cq_kv_append -> cq_attn_tree -> ...) -> LM head -> cq_tree_verify
 *   -> cq_kv_move (each layer's cache) -> cq_kv_release
 *
 * Boundary rules as in cq.h: DEVICE pointers owned by the caller, every argument
 * checked before any launch (an error means that nothing was written), no
 * synchronisation, no allocation.
 *
 * Sources (web pages on GGUF inference engines): alice-llm docs (WGSL layer
 * shaders: RMSNorm, batch-aware RoPE; speculative decoding with acceptance by
 * probabilities) and cera README (speculative decoding; verification of draft
 * tokens in one pass).
 *
 * A tree: the new tokens of a request, in order, at most CQ_TREE_MAX, each with
 * parent[t], the index among them (0 for the request's first) of the token it
 * follows; -1: it follows the cache alone. A parent comes before its children.
 * For cq_tree_verify token 0 is the last token that was sampled, and the others
 * are drafts.
 */
#ifndef CQ_TREE_H
#define CQ_TREE_H

#include "cq_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CQ_TREE_MAX 64

/* Device status word bits of these calls, in the library's word (cq_read_global_status). */
#define CQ_DEV_TREE   0x100 /* a parent that does not come before its child, a path or count outside the request
                               (cq_kv_move) */
#define CQ_DEV_LOGITS 0x200 /* cq_tree_verify: a row with NaN or +infinity, or without a finite value, was reached */

/*
 * Norm and rotation of queries and keys, one pass. q: T rows of q_heads * head_dim
 * values of `in`, k: of kv_heads * head_dim, rows q_stride / k_stride elements apart
 * (slices of a fused projection's rows work); q_out, k_out: the same rows in `out`.
 * For each head x of a row, in fp32, rounded once at the end:
 *   y = x * w / sqrt(mean(x^2) + eps)    w: q_norm or k_norm, fp32 [head_dim]; NULL: y = x
 *   phi_i = positions[t] * freqs[i]      freqs: fp64 [rot_dim / 2], radians a position
 *   (y_a, y_b) -> (y_a cos phi_i - y_b sin phi_i, y_b cos phi_i + y_a sin phi_i)
 * for the pairs (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) if adjacent = 1;
 * the dimensions from rot_dim on are not turned. phi is reduced without loss: freqs / 2 pi is
 * taken to 2^-62 of a turn, so that phi is as good as that times the position (2^-31 of a turn
 * at 2^31) and its sine and cosine as fp32's. Frequencies are finite, below 2^31 in size.
 * Rows with a negative position (padding) are not written. Sums of squares are fp32: |x|
 * up to 1e18, and any size below. in = out, or in = CQ_F32; q_out may be q and k_out may be k, with the same type and stride
 * (in place); any other overlap of inputs and outputs is a race. Either of q_heads and
 * kv_heads may be 0 (its pointers are not read).
 * head_dim 64 or 128; rot_dim a multiple of 8, 0 to head_dim (0: freqs may be NULL);
 * q_heads, kv_heads <= 1024; T < 2^31; eps >= 0. Rows 16-byte aligned, strides multiples of 16 bytes; norms 16-byte,
 * freqs 8-byte aligned. Asynchronous, one launch, no allocation.
 */
cq_status cq_qk_rope(cq_dtype in, cq_dtype out, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                     int64_t rot_dim, int adjacent, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const int32_t* positions, const double* freqs, const float* q_norm, const float* k_norm, float eps,
                     void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/*
 * Masks and positions of the requests' trees. q_start: int32 [R + 1], kv_len:
 * int32 [R] as cq_kv_plan writes them (kv_len counts the new tokens); parent: int32 [T].
 * For token i of a request of n tokens:
 *   bit j of mask[t] = 1 if token j is token i or an ancestor of it      (uint64 [T])
 *   positions[t] = kv_len - n + the number of its ancestors              (int32 [T])
 * Tokens t outside [q_start[0], q_start[R]) (padding) get mask 0 and position -1. A parent that is not
 * in [-1, i - 1] counts as -1 and is flagged (CQ_DEV_TREE). A request of more than
 * CQ_TREE_MAX tokens is no tree (a prompt, a chunk): its parents are not read, its
 * masks are 0, its positions follow one another. positions below 0 or past 2^31 - 1 are -1.
 * mask or positions may be NULL. R <= 16384, T < 2^31. Asynchronous, one launch, no allocation.
 */
cq_status cq_tree_plan(int64_t R, int64_t T, const int32_t* kv_len, const int32_t* q_start, const int32_t* parent,
                       uint64_t* mask, int32_t* positions, void* stream);

/*
 * cq_attn_paged for trees: token t of a request with n new tokens sees key j when
 * 0 <= j < kv_len - n, or when 0 <= j - (kv_len - n) < n and that bit of mask[t] is set
 * (mask: uint64 [T]; bits from n on are not looked at, any pattern is allowed).
 * A request of more than CQ_TREE_MAX new tokens is causal, its masks are not
 * read: prompts and chunks may stand beside trees. Everything else as there,
 * with no window (max_new, the workspace, precision, rows that see nothing, pages outside the cache), but that
 * max_new <= CQ_TREE_MAX sends a call's requests to one kernel, all of them, and that the probabilities of binary16
 * calls' trees have 21 bits, whatever stands beside them (of longer requests 11 at least). The tensor cores'
 * sums, cut off rather than rounded at each addition of 16 keys, go over 512 keys at most in fp32 calls, 8192 in
 * binary16 and 32768 in bfloat16 ones; what they add up to rounds.
 */
cq_status cq_attn_tree(const cq_kv_cache* cache, cq_dtype dtype, int64_t R, int64_t T, int64_t q_heads,
                       int64_t max_new, const void* q, int64_t q_stride, const int32_t* block_table,
                       int64_t max_blocks, const int32_t* kv_len, const int32_t* q_start, const uint64_t* mask,
                       float scale, void* out, int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Verification of the requests' drafts from given random numbers. logits: fp32
 * [T][V], rows logits_stride elements apart: the target's after each token. tokens: int32 [T].
 * draft (may be NULL): fp32 [T][V], rows draft_stride elements apart, the probabilities
 * that the children of each token were drawn from, independently of one another; not negative. Without them
 * the drafts were not drawn, and q is the point at the child's token. For a request
 * at token c (at first 0) with p = softmax(logits[c] / temperature[r]), r_0 = p and
 * q = draft[c], its children in order, k = 0, 1, ...: with u = u_accept of the child and x its token
 *   u * q(x) < r_k(x): the child is kept, and is the next c
 *   else r_{k+1} = max(r_k - q, 0) / sum of it; where that sum is 0, r_{k+1} = r_k
 * until no child is kept or max_path tokens are (the last one's children are then not
 * looked at):
 *   count[r] = tokens kept, the first included    path[r][0 .. count) = their indices, the rest -1
 *   next[r] = the smallest v with sum of r_k(w) over w <= v > u_sample[r]
 * so that every kept token and the next one are distributed as the target's.
 * temperature: fp32 [R]; below 2^-64 (0, negative, NaN): p is the point at the largest logit, of the smallest
 * index where several are, and so is every draft's q; above 2^64: as 2^64. u are fp32 in [0, 1): below 0 and NaN count as
 * 0, 1 and more as 1 - 2^-24. Tokens outside [0, V) are never kept. -infinity is
 * a logit of probability 0. A row with NaN or +infinity or nothing finite that is
 * reached ends the request there, with next = -1, and is flagged (CQ_DEV_LOGITS). Parents as in cq_tree_plan; drafts whose
 * parent is -1 are never kept. A request without tokens, or of more than CQ_TREE_MAX (no
 * tree: a prompt beside them; nothing of it is read), gets count 0 and next -1.
 * Probabilities are held as whole numbers to 2^-45 of the row's largest, each within 2^-36 of its own
 * size, and summed exactly: results do not depend on timing or on how the work is split.
 * The rows of tokens that are not kept are not read.
 * R <= 16384; 1 <= V <= 262144; T < 2^31; 1 <= max_path <= CQ_TREE_MAX. All 4-byte aligned,
 * strides at least V. path: int32 [R][max_path]. Asynchronous, one launch, no allocation.
 */
cq_status cq_tree_verify(int64_t R, int64_t T, int64_t V, const float* logits, int64_t logits_stride, const float* draft,
                         int64_t draft_stride, const int32_t* tokens, const int32_t* parent, const int32_t* q_start,
                         const float* temperature, const float* u_accept, const float* u_sample, int64_t max_path,
                         int32_t* count, int32_t* path, int32_t* next, void* stream);

/*
 * Rows of the tokens that were kept, moved together in a cache. Request r has n =
 * q_start[r + 1] - q_start[r] new tokens at positions b = kv_len[r] - n and on; for i in
 * [0, count[r]) the row (keys and values, every head) of position b + path[r][i]
 * goes to position b + i (path[r][i] = i stays). Where a page (p, head) gets rows
 * from other places, for keys and values each:
 *   s = the largest of its scale and of the scales of the pages that those rows come from
 *   its other rows: q = rha(q * (s_old / s)); the rows that come: q = rha(q * (s_src / s))
 * (rha: to nearest, halves away from zero; fp32; 0 where s is 0 or NaN). So rows are copied as they are
 * where the scales are alike, and else every value is within s / 2 of what it was. A NaN
 * scale makes s NaN. All rows and scales are taken as they were before the call, so the path may be any; where no
 * source is itself overwritten and no page that gets rows from another one gives any to a third, repeating the call
 * changes nothing.
 *   new_len[r] = b + count[r], at least 0                   (int32 [R]; may be NULL)
 * count[r] is cut to [0, n] and to max_path, a path entry outside [0, n) leaves its row
 * as it is; both are flagged (CQ_DEV_TREE). A request of more than CQ_TREE_MAX tokens is no tree (a prompt beside
 * them): it keeps all of them, count and path are not looked at, new_len[r] = kv_len[r]. Pages outside the cache, and positions outside the table, are
 * skipped and flagged (CQ_DEV_KV_PAGE). The pages that rows come from and go to are the request's own:
 * one page in two requests of a call is a race. block_table as in cq_attn_paged.
 * R <= 16384; 1 <= max_path <= CQ_TREE_MAX. Asynchronous, one launch, no allocation.
 */
cq_status cq_kv_move(const cq_kv_cache* cache, int64_t R, const int32_t* block_table, int64_t max_blocks,
                     const int32_t* kv_len, const int32_t* q_start, const int32_t* count, const int32_t* path,
                     int64_t max_path, int32_t* new_len, void* stream);

/*
 * Pages that requests no longer need, given back: the entries of blocks
 * [ceil(new_len / P), ceil(old_len / P)) of each request, in the order of requests
 * and blocks, to freed[0 .. used[0]); freed[used[0] .. capacity) = -1. new_len 0 gives all of a request's pages
 * back; a new_len of old_len and more none. The table is left as it is (entries past a
 * request's length are not read by the other calls, and cq_kv_plan writes them anew).
 * used[1] = status bits:
 *   CQ_DEV_KV_LENGTH  a negative length, taken as 0
 *   CQ_DEV_KV_BLOCKS  old_len longer than max_blocks pages: taken as max_blocks
 *   CQ_DEV_KV_PAGES   more pages than capacity: those past it are left out
 *   CQ_DEV_KV_PAGE    an entry outside [0, num_pages): -1 in its place
 * (int32 [2]). page_size as in cq_kv.h; R <= 16384; capacity < 2^31; max_blocks * P < 2^31. Asynchronous, one launch,
 * no allocation.
 */
cq_status cq_kv_release(int64_t R, int64_t page_size, const int32_t* block_table, int64_t max_blocks, int64_t num_pages,
                        const int32_t* old_len, const int32_t* new_len, int32_t* freed, int64_t capacity, int32_t* used,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CQ_TREE_H */
