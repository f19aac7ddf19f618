/*
 * sv_attention.h -- C ABI of libsvattention: the paged key/value cache of the
 * target model and the attention of a chunk of new tokens over it, on one
 * NVIDIA GB300 (sm_103a).
 *
 * spec_verify.h starts from the logits of the K + 1 positions of every
 * sequence. The layer before it is the target's parallel forward over those
 * positions ("Speculative decoding" lecture notes of Hung-yi Lee's generative
 * AI course, section 3: all drafted positions are scored in one pass): each
 * layer writes the new tokens' keys and values into the sequence's cache and
 * lets their queries attend to everything cached before them and, causally, to
 * one another. A rejected draft costs nothing here: the next call passes the
 * shorter cached length and overwrites what was rejected.
 *
 * The cache. Keys and values lie in pages of page_size tokens. Sequence b's
 * position p is slot p % page_size of page page_table[b][p / page_size].
 *   16-bit formats hold the values themselves.
 *   SV_E4M3 holds, for every (page, slot, head), head_dim e4m3 codes and one
 *   exponent byte e; the values are code * 2^(e - 127), and NaN throughout
 *   when e is 255. On writing, 2^(e - 127) is the smallest power of two (from
 *   2^-117 up) that brings the vector's largest magnitude to 448 or below, and
 *   the codes are rounded to nearest, ties to even. A vector that holds a NaN
 *   or an infinity is stored with e = 255. Every stored value is a bfloat16
 *   number; float16 sources are clamped to +-61440 first so that the stored
 *   value is a float16 number too (below 2^-14 up to float16's own rounding).
 *   Codes 0x7F and 0xFF are never written, and must not be in a cache that was
 *   written by something else.
 *
 * The chunks. Sequence b has cached_lens[b] tokens in the cache and
 * chunk_starts[b + 1] - chunk_starts[b] new ones (none is allowed), which are
 * rows chunk_starts[b] .. of the packed arrays. All of it is read on the
 * device when the kernels run: a call makes no synchronisation and may be
 * captured into a CUDA graph and replayed with other lengths and pages.
 *
 * Bad lengths and pages are found on the device and never followed:
 *   SV_SEQ_BAD_LENGTH  starts that fall or leave [0, tokens], a negative
 *                      cached length, more than max_chunk new tokens, or an
 *                      end beyond max_pages * page_size. The sequence is left
 *                      out: nothing is written to the cache, and its output
 *                      rows, where they lie in the packed arrays, are NaN.
 *   SV_SEQ_OVERLAP     starts that are out of order (then some sequence has
 *                      SV_SEQ_BAD_LENGTH too) give some of the sequence's rows to
 *                      another one; no row has two owners. The sequence is left
 *                      out as above, its rows that are another's excepted.
 *   SV_SEQ_BAD_PAGE    a page outside [0, num_pages) among those needed.
 *                      Its tokens are not written; output rows that would read
 *                      it are NaN.
 *   SV_SEQ_TIMEOUT     (spec_verify.h's) a wait inside the attention ran out
 *                      (about 2 s; never in ordinary operation). It is reported
 *                      for every sequence, and every output of the call is NaN.
 * seq_status, where given, receives 0 or these bits for every sequence.
 *
 * Return codes are spec_verify.h's SV_OK and SV_ERR_*. All calls are
 * asynchronous on `stream` and allocate nothing.
 */
#ifndef SV_ATTENTION_H
#define SV_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types besides spec_verify.h's SV_F32 and SV_BF16. */
#define SV_F16 2
#define SV_E4M3 3

/* seq_status bits besides spec_verify.h's. */
#define SV_SEQ_BAD_PAGE 16
#define SV_SEQ_BAD_LENGTH 32
#define SV_SEQ_OVERLAP 64

/*
 * A paged cache and the chunks of one call. Index 0 of the two-element fields
 * is the keys', index 1 the values'. Strides count elements; the innermost
 * (head_dim) stride is 1; the stride of a dimension of one element (one page, one
 * head; in the packed arrays one token or head) is not looked at.
 *   pages        device, 16-byte aligned; page, slot and head strides are
 *                multiples of 16 bytes, below 2^40.
 *   exps         device bytes, SV_E4M3 only (NULL otherwise), any strides.
 *   num_pages    pages in each of the two arrays, 0 <= num_pages < 2^31.
 *   page_size    a power of two, 8 .. 1024.
 *   head_dim     a multiple of 16, 16 .. 256.
 *   dtype        SV_BF16, SV_F16 or SV_E4M3.
 *   page_table   device int32 [batch][table_stride], the first max_pages of
 *                each row being the sequence's. Entries that no position of
 *                the call needs are not read.
 */
typedef struct sv_paged_cache {
    void* pages[2];
    uint8_t* exps[2];
    int64_t page_stride[2], slot_stride[2], head_stride[2];
    int64_t exp_page_stride[2], exp_slot_stride[2], exp_head_stride[2];
    int64_t num_pages;
    int32_t page_size, kv_heads, head_dim, dtype;
    const int32_t* page_table;
    int64_t table_stride, max_pages;
    const int32_t* cached_lens;
    const int32_t* chunk_starts;
    int64_t batch;
} sv_paged_cache;

/*
 * Write the new tokens' keys and values to positions cached_lens[b] + t.
 *   key, value  device [tokens, kv_heads, head_dim] of `dtype` (SV_BF16 or
 *               SV_F16; the cache's own type unless the cache is SV_E4M3),
 *               16-byte aligned; *_token_stride and *_head_stride in elements,
 *               multiples of 8.
 *   tokens      rows of the packed arrays, 0 <= tokens < 2^31.
 *   seq_status  device int32 [batch] or NULL.
 * One launch (and a memset when seq_status is given).
 */
int sv_kv_append(const sv_paged_cache* cache, const void* key, const void* value, int dtype,
                 int64_t tokens, int64_t key_token_stride, int64_t key_head_stride,
                 int64_t value_token_stride, int64_t value_head_stride, int32_t* seq_status,
                 void* stream);

/*
 * Read positions cached_lens[b] + t back into the packed arrays
 * key, value [tokens, kv_heads, head_dim], contiguous, 16-byte aligned, of
 * `dtype`: the cache's own type, or either 16-bit type from SV_E4M3 (one
 * rounding). Rows of bad sequences or pages, and of no sequence, are NaN.
 * What was written to an e4m3 cache from bfloat16 may be too large for float16.
 * One launch (and a memset when seq_status is given).
 */
int sv_kv_read(const sv_paged_cache* cache, void* key, void* value, int dtype, int64_t tokens,
               int32_t* seq_status, void* stream);

/*
 * Attention of the new tokens over their sequences' caches, which already hold
 * them (sv_kv_append first). Query t of sequence b, at position
 * p = cached_lens[b] + t, sees positions max(0, p - window + 1) .. p (from 0
 * when window is 0):
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = log sum_j exp(scale q.k_j).
 * Query head h reads key/value head h / (q_heads / kv_heads). Values and
 * scores at positions that a query does not see have no influence on it,
 * whatever they are. Rows of no sequence are left as they are.
 *
 * Scores, softmax sums and outputs are accumulated in float32. Roundings: the
 * softmax weights become the query's type (e4m3 caches: float16) for the second
 * product, and float16 weights below 2^-32 (e4m3: 2^-27) of a row's largest may be
 * lost; bfloat16 values above 2^90 may overflow there. Over e4m3 caches bfloat16
 * queries are held as float16 relative to their row's largest element, exact down
 * to 2^-38 of it; keys and values are taken exactly. Where a type's range does not
 * reach (keys or values of neighbouring tokens more than 2^22 apart, or below
 * 448 2^-87 and not zero; keys above 2^60; scores past 2^22) rows are computed again
 * key by key: as exactly, but a hundred times slower and more.
 * Results do not depend on the order in which blocks run.
 *   query       device [tokens, q_heads, head_dim] of `dtype` (SV_BF16 or
 *               SV_F16; the cache's own type unless the cache is SV_E4M3),
 *               16-byte aligned, strides in elements, multiples of 8.
 *   out         like query, contiguous.
 *   lse         device float32 [tokens, q_heads], or NULL.
 *   scale       finite, > 0.
 *   window      0 (none) .. 2^31 - 1.
 *   max_chunk   no sequence has more new tokens than this (0: tokens). The
 *               launches and the workspace are planned with it: 512 single tokens
 *               take 467 us with 1 and 712 with 0, and 43 MB.
 *   workspace   device, 256-byte aligned, sv_chunk_attention_workspace_bytes.
 */
int sv_chunk_attention_workspace_bytes(int64_t batch, int64_t tokens, int64_t q_heads,
                                       int64_t kv_heads, int64_t head_dim, int64_t max_chunk,
                                       size_t* bytes);

int sv_chunk_attention(const sv_paged_cache* cache, const void* query, int dtype, int64_t tokens,
                       int64_t q_heads, int64_t query_token_stride, int64_t query_head_stride,
                       float scale, int64_t window, int64_t max_chunk, void* out, float* lse,
                       int32_t* seq_status, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Test hook for the timeout path: sv_chunk_attention with the values' loads of
 * one thread block held until the device int32 *gate becomes nonzero. That wait
 * is bounded like every other wait in the kernels (about 2 s). When it runs out
 * the thread block gives up and returns with no copy in flight, every sequence of
 * the call is reported as SV_SEQ_TIMEOUT and every output is NaN. The context
 * stays usable.
 * A caller that sets *gate before the wait runs out gets the ordinary results.
 *   block  the thread block, 0 .. SMs - 1; negative: all of them.
 *   gate   device int32, 4-byte aligned (SV_ERR_ARG if NULL, SV_ERR_ALIGN).
 * Other arguments as sv_chunk_attention.
 */
int sv_chunk_attention_gated(const sv_paged_cache* cache, const void* query, int dtype,
                             int64_t tokens, int64_t q_heads, int64_t query_token_stride,
                             int64_t query_head_stride, float scale, int64_t window,
                             int64_t max_chunk, void* out, float* lse, int32_t* seq_status,
                             void* workspace, size_t workspace_bytes, void* stream, int32_t block,
                             const int32_t* gate);

#ifdef __cplusplus
}
#endif

#endif /* SV_ATTENTION_H */
