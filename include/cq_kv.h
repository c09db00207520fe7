/*
 * cq_kv.h -- an 8-bit paged key/value cache and attention over it: what a decoder
 * layer needs between the products of cq.h. Boundary rules as there: DEVICE
 * pointers owned by the caller, every argument checked before any launch (an error
 * means that nothing was written), no synchronisation, no allocation.
 *
 * Sources (web pages on GGUF inference engines): alice-llm docs (paged key/value
 * cache, continuous batching, batch-4 speculative decoding) and cera README
 * (tiled attention for long prompts; verification of draft tokens in one pass).
 *
 * The cache is a pool of pages of page_size tokens. k and v hold int8 values
 * [page][kv head][token in page][head_dim]; the token rows of one (page, head)
 * are contiguous, pages are page_stride bytes apart. k_scale and v_scale hold
 * one fp32 scale per (page, kv head), pages scale_stride floats apart: a stored
 * value stands for q * scale. Token i of request r lives in page
 * block_table[r][i / page_size] at row i % page_size; a slot is
 * page * page_size + row.
 *
 * page_size 16, 32, 64 or 128; head_dim 64 or 128; 1 <= kv_heads <= 1024;
 * num_pages < 2^31; page_stride a multiple of 16, at least kv_heads *
 * page_size * head_dim; scale_stride >= kv_heads. k and v 16-byte aligned,
 * scales 4-byte aligned; all DEVICE memory owned by the caller, who may keep k
 * and v in one allocation (page_stride then spans both). Sizes pass 32 bits.
 */
#ifndef CQ_KV_H
#define CQ_KV_H

#include "cq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status word bits of these calls (the others are in cq.h). cq_read_global_status and
 * cq_read_device_status return CQ_ERR_DEVICE_STATUS for the library's word with one of them set. */
#define CQ_DEV_KV_LENGTH 0x08 /* cq_kv_plan: a negative length */
#define CQ_DEV_KV_BLOCKS 0x10 /* cq_kv_plan: a request longer than its block-table row */
#define CQ_DEV_KV_PAGES  0x20 /* cq_kv_plan: the free pages ran out */
#define CQ_DEV_KV_TOKENS 0x40 /* cq_kv_plan: more new tokens than slots */
#define CQ_DEV_KV_PAGE   0x80 /* a page id or slot outside the cache: skipped */

typedef enum { CQ_F32 = 0, CQ_F16 = 1, CQ_BF16 = 30 } cq_dtype;   /* the GGML tensor-type ids */

typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t num_pages;
    int64_t page_stride;
    int64_t scale_stride;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t reserved;        /* 0 */
} cq_kv_cache;

/*
 * Block tables and slot maps of a step, built on the GPU from the requests'
 * lengths. past_len, new_len: int32 [R] (tokens in the cache, tokens of this
 * step); block_table: int32 [R][max_blocks], entries of the past tokens'
 * pages filled in; free_pages: int32 [n_free], taken from the front.
 *   kv_len[r]  = past_len[r] + new_len[r]                      (int32 [R])
 *   q_start    = exclusive sums of new_len                     (int32 [R + 1])
 *   block_table[r][ceil(past/P) .. ceil(kv/P) - 1] = the next free pages, in
 *     request order (other entries are left as they are)
 *   for token t of the step, t in [q_start[r], q_start[r+1]):
 *     positions[t] = past_len[r] + t - q_start[r]              (int32 [T])
 *     slots[t] = the slot of that position                     (int64 [T])
 *   slots[t] = positions[t] = -1 for t in [q_start[R], T) (padding)
 *   used[0] = pages taken, used[1] = status bits               (int32 [2])
 * The same inputs give the same outputs, also after block_table was updated by
 * an earlier call. What does not fit is left out and flagged in used[1]:
 *   CQ_DEV_KV_LENGTH  a negative length, taken as 0
 *   CQ_DEV_KV_BLOCKS  a request longer than max_blocks pages: the tokens past
 *                     them get slot -1, kv_len stops at max_blocks * P; a
 *                     position past 2^31 - 1 is -1
 *   CQ_DEV_KV_PAGES   free_pages used up: table entry -1, slots -1
 *   CQ_DEV_KV_TOKENS  more than T new tokens: those past T are left out, and
 *                     q_start stops at T
 *   CQ_DEV_KV_PAGE    a page id outside [0, num_pages) in the free list (entry
 *                     and slots -1) or in a partly filled page's entry (slots -1)
 * kv_len and the table then count tokens that have no slot: a step with a bit set in used[1] is
 * planned anew with what fits before it is attended to.
 * R <= 16384 (CQ_ERR_SHAPE beyond), T < 2^31, max_blocks * P < 2^31. R = 0 only
 * writes q_start[0], used and the padding. Asynchronous, one launch, no
 * allocation.
 */
cq_status cq_kv_plan(int64_t R, int64_t page_size, int64_t max_blocks, int64_t num_pages, const int32_t* past_len,
                     const int32_t* new_len, const int32_t* free_pages, int64_t n_free, int32_t* block_table,
                     int64_t T, int32_t* kv_len, int32_t* q_start, int64_t* slots, int32_t* positions, int32_t* used,
                     void* stream);

/*
 * Write the keys and values of T new tokens into the cache. k, v: T rows of
 * kv_heads * head_dim values of `dtype`, rows k_stride / v_stride elements
 * apart (slices of a fused projection's rows work), 16-byte aligned with
 * strides a multiple of 16 bytes; slots: int64 [T] as cq_kv_plan writes them.
 * Negative slots are skipped; slots past the cache are skipped and flagged in
 * the library's status word (CQ_DEV_KV_PAGE). Per (page, head), for k and v
 * each, with a = max |x| over the call's new tokens in that page (fp32):
 *   s = max(s_old, a / 127), where s_old = 0 if the first of them is row 0 of
 *       the page, else the stored scale; a / 127 below 2^-126 counts as 0
 *   rows of the page before the first new one: q = rha(q * (s_old / s))
 *   new rows: q = clamp(rha(x * (1 / s)), -127, 127); 0 if s = 0
 * (rha: round to nearest, halves away from zero; all fp32). So a stored value is
 * within s / 2 of what was given, and every later call that raises the page's scale,
 * to s', moves it by up to s' / 2 more: after g of them it is within (g + 1) / 2
 * steps of the last scale. Rows of a prompt come in few calls. Tokens that come one
 * by one raise a page's scale about log(page_size) times if they are alike (128
 * normal rows: 1.5e-2 of them, 2-norm, for 1.0e-2 in one call); rows that grow from
 * token to token raise it each time (by 3% each: 0.6 at pages of 128, 0.05 at 16).
 * Small pages bound this. A value that is
 * not finite makes s NaN, for the whole (page, head), until the page is begun
 * anew. The tokens of one page have to be consecutive, with consecutive slots:
 * one page in two separate runs of one call is a race. Repeating a call leaves
 * the cache as it is. Asynchronous, one launch, no allocation.
 */
cq_status cq_kv_append(const cq_kv_cache* cache, cq_dtype dtype, int64_t T, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const int64_t* slots, void* stream);

/*
 * Cache rows back as numbers: row t of k_out and v_out (T rows of kv_heads *
 * head_dim values of `dtype`, contiguous, 16-byte aligned) is q * scale of slot
 * slots[t], in fp32, rounded once. Negative slots give zero rows; slots past the
 * cache too, flagged in the library's status word (CQ_DEV_KV_PAGE). k_out or v_out may be NULL.
 */
cq_status cq_kv_read(const cq_kv_cache* cache, cq_dtype dtype, int64_t T, const int64_t* slots, void* k_out,
                     void* v_out, void* stream);

/*
 * Attention of a step's tokens over the cache (their own keys and values
 * already appended). q: T rows of q_heads * head_dim values of `dtype`,
 * q_stride elements apart; query head i reads kv head i / (q_heads / kv_heads).
 * Token t of request r (q_start[r] <= t < q_start[r+1], n of them) is at
 * position i = kv_len[r] - n + t - q_start[r] and sees key j when
 *   0 <= j < kv_len[r],  j <= i if causal,  j > i - window if window > 0.
 *   out[t][head] = sum_j softmax_j(scale * q . k_j) v_j   (`dtype`, rows
 *                  out_stride elements apart)
 *   lse[t][head] = log sum_j exp(scale * q . k_j)         (fp32 [T][q_heads]; may be NULL)
 * A row that sees nothing gets out = 0 and lse = -inf; a hidden key never
 * reaches a row, whatever it or its block's scale holds. Rows of no request
 * (t >= q_start[R]) are not written. Softmax statistics and sums are fp32,
 * exponentials and the factors of 16-bit calls' value scales good to 2^-22.
 * What the products take:
 *   fp32 q 22 bits, the probabilities 22 (those below 2^-15 of the row's largest 16 at least)
 *   16-bit q as it is (values below 2^-22 of the row's largest to 2^-33 of it)
 *   bfloat16 calls' probabilities as binary16, 11 bits
 *   binary16 calls' probabilities 22 bits in requests of less than 40 rows (tokens times q_heads /
 *     kv_heads: decoding, drafts), 11 bits in wider ones (prompts, chunks): 2.1e-4 and 2.5e-4 of a
 *     result, 2-norm, against 64 bits
 * As one binary16 a probability, times its value scale (2^-64 for a block of zeros, scale 0), that
 * is below 2^-31 of the row's largest adds nothing to out. Scales are not negative, blocks of
 * scale 0 hold zeros; a q that is not finite makes its own row NaN. Value scales are 0 or 2^-126
 * (the smallest that cq_kv_append writes) to 2^96, and those that one row sees, 2^-64 for 0 among
 * them, within 2^100 of one another: past that, a block of the smaller ones may lose its weight.
 * Pages outside [0, num_pages) are hidden and flagged in the library's status
 * word (CQ_DEV_KV_PAGE); lengths are clipped to the table and to T.
 * max_new: the host's upper bound of any request's new tokens. It chooses kernels and their
 * tiles: too small or too large a bound costs time, results stay right. max_kv: the same of kv_len;
 * it is checked (>= 0) and otherwise not used yet.
 * q, out 16-byte aligned, strides multiples of 16 bytes; q_heads a multiple of
 * kv_heads, at most 1024; R <= 16384; T * q_heads / kv_heads <= 2^30. workspace: cq_attn_workspace_size
 * bytes (0 for arguments the call does not take), 256-byte aligned; its first
 * CQ_ATTN_WORKSPACE_ZERO bytes are zero before its first use, and every call leaves
 * them so (the others may hold anything). Calls that may overlap on the GPU need
 * separate ones. Asynchronous, no allocation; results do not depend on timing.
 */
#define CQ_ATTN_WORKSPACE_ZERO 4096
size_t cq_attn_workspace_size(int64_t q_heads, int64_t kv_heads, int64_t head_dim);
cq_status cq_attn_paged(const cq_kv_cache* cache, cq_dtype dtype, int64_t R, int64_t T, int64_t q_heads,
                        int64_t max_new, int64_t max_kv, const void* q, int64_t q_stride, const int32_t* block_table,
                        int64_t max_blocks, const int32_t* kv_len, const int32_t* q_start, float scale, int causal,
                        int64_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CQ_KV_H */
