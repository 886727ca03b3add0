/*
 * inkling_paged_attn.h -- C ABI of the serving form of the learned-relative
 * attention in libinkling_rel_attn.so (same library, status codes and
 * conventions as inkling_rel_attn.h): a key-value cache in pages, and the
 * attention of one new token per request over it.
 *
 * A serving step is three calls, each asynchronous on `stream`, none of which
 * needs the lengths or the tables on the host (so a step can be captured in a
 * CUDA graph and replayed). Nothing is kept between calls but, per device, its number
 * of SMs and whether a kernel's shared-memory limit has been raised:
 *   inkling_kv_plan          pages of the growing requests, slots of the new tokens
 *   inkling_kv_append        new key / value rows into their slots (k clipped, 8 bits)
 *   inkling_rel_attn_decode  attention of each request's last token
 * Not on the Inkling2 pages, which describe the whole-sequence forward: the
 * attention is inkling_rel_attn_fwd's for the last query row of each request
 * (one document, every cached token valid).
 *
 * The cache. K and V are two pools of num_pages pages of page_size tokens. The
 * row of head g of token o of page p holds head_dim contiguous values and begins
 *   p * page_stride + o * token_stride + g * head_stride
 * elements after the pool's base, in both pools. [pages, page_size, heads, D] and
 * [pages, heads, page_size, D] are both of this form. A token's slot is
 * p * page_size + o. Values are BF16, or e4m3 with one FP32 scale per KV head:
 * the value that a code stands for is code * scale[g].
 */
#ifndef INKLING_PAGED_ATTN_H
#define INKLING_PAGED_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "inkling_rel_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    INKLING_KV_BF16 = 0,
    INKLING_KV_E4M3 = 1
} inkling_kv_dtype;

/*
 * num_pages   pages in each pool (1 .. 2^31 - 1)
 * page_size   tokens in a page, any number from 1 (below 2^30); num_pages * page_size <= 2^31
 * heads_kv    Hkv
 * head_dim    D: 64 or 128
 * dtype       inkling_kv_dtype
 * *_stride    in elements; each a multiple of 16 bytes and at least D where its
 *             extent is above 1 (with an extent of 1 the stride is not looked at)
 */
typedef struct {
    int64_t num_pages, page_size, heads_kv, head_dim, dtype, page_stride, token_stride, head_stride;
} inkling_kv_cache_desc;

/*
 * Block tables and slot maps from request lengths.
 *   requests    N (0 .. 16384)
 *   page_size   P tokens in a page
 *   max_pages   M: entries in each row of the block table; N * M * P < 2^31
 *   num_pages   pages in the pool: page numbers are 0 .. num_pages - 1
 *   max_tokens  T: entries of slots and positions, at most 2^30
 */
typedef struct {
    int64_t requests, page_size, max_pages, num_pages, max_tokens;
} inkling_kv_plan_dims;

/*
 *   old_lens    [N]     int32  tokens of each request in the cache (it holds ceil(old / P) pages)
 *   new_lens    [N]     int32  tokens wanted after this step: above old, the difference is
 *                              appended; below it, the request is cut back (0: it has ended)
 *   block_table [N, M]  int32  page numbers, read and updated
 *   free_pages  [num_pages] int32  stack of free pages, read and updated
 *   free_count  [1]     int32  pages on the stack
 *   lens        [N]     int32  tokens after this step
 *   query_start [N + 1] int32  prefix sums of the new tokens (max(0, new - old)) of the requests
 *   slots       [T]     int64  slot of each new token, requests one after another
 *   positions   [T]     int32  its position in its request
 *   info        [4]     int32  pages on the stack afterwards, new tokens, pages that were
 *                              wanted but not there, pages taken
 * Pages of requests that are cut back are pushed first, in the order of the
 * requests and of their tables; growing requests then pop theirs in the order of
 * the requests. A request that gets fewer pages than it wants keeps as many tokens
 * as fit in the pages it has (lens), and the slots of its other new tokens are -1.
 * slots and positions behind the last new token are set to -1 and 0; new tokens
 * beyond T have no entry, though lens counts them (info[1] is how many there are,
 * so T has to be that at least for every token to get its slot). A page belongs to
 * one request: one that stood in two rows would be given back twice. Table entries other than the new pages, and entries of
 * free_pages at or above the new count, stay as they were. Lengths outside
 * [0, M * P] and a count outside [0, num_pages] are taken as the nearest bound; the
 * slots of tokens whose page number is outside the pool are -1. What is written
 * (block_table, free_pages, lens, query_start, slots, positions, info) may not
 * overlap anything else (INKLING_ERR_INVALID_ARG).
 * slots needs 8-byte alignment, the rest 4.
 */
inkling_status inkling_kv_plan(const inkling_kv_plan_dims* dims, const int32_t* old_lens, const int32_t* new_lens,
                               int32_t* block_table, int32_t* free_pages, const int32_t* free_count, int32_t* lens,
                               int32_t* query_start, int64_t* slots, int32_t* positions, int32_t* info,
                               void* stream);

/*
 * Appends T rows to the cache: k_cache[slots[t]] = k[t], v_cache[slots[t]] = v[t].
 * Rows whose slot is outside [0, num_pages * page_size) are skipped. Slots that are
 * stored must differ from each other, and the pools may not overlap, nor a stored
 * slot a row of k or v.
 *   tokens       T
 *   k_row, v_row elements from one token's [Hkv, D] rows to the next one's, multiples
 *                of 8 and at least Hkv * D (the rows of a fused projection)
 *   clip_k       nonzero: k goes through L2Clip (inkling_l2clip.h) on the way, with
 *                threshold >= 0, clip_scale [Hkv, D] FP32 or NULL, tau [T] FP32 or NULL:
 *                inkling_l2clip_fwd's formula, rounded to BF16 like its result
 * With an e4m3 cache, k_scale and v_scale [Hkv] FP32 (positive) are required and the
 * code of x is x / scale[g], at most 448 in magnitude, rounded to nearest even (NaN
 * stays NaN); with a BF16 cache they must be NULL.
 * k, v, the pools and clip_scale are 16-byte aligned, slots 8, tau and the scales 4.
 */
typedef struct {
    int64_t tokens, k_row, v_row, clip_k;
    double threshold;
} inkling_kv_append_dims;

inkling_status inkling_kv_append(const inkling_kv_cache_desc* cache, const inkling_kv_append_dims* dims,
                                 const uint16_t* k, const uint16_t* v, const int64_t* slots, const float* k_scale,
                                 const float* v_scale, const float* clip_scale, const float* tau, void* k_cache,
                                 void* v_cache, void* stream);

/*
 * Attention of one new token per request over its cached tokens. Request n has
 * lens[n] tokens in the cache, its new one (the query) the last of them:
 *   allowed(j) = j < lens[n] && (window == 0 || lens[n] - 1 - j < window)
 *                && the page of token j is inside the pool
 *   d    = lens[n] - 1 - j
 *   z_j  = scale * <q[n,h,:], K[j,g,:]> + (d < rel_extent ? profiles[n,h,d] : 0)
 *   lse[n,h] = log(exp(sink[n,h]) + sum_allowed exp(z_j))
 *   out[n,h,:] = sum_allowed exp(z_j - lse) * V[j,g,:]
 * Token j is on page block_table[n, j / page_size]; entries whose tokens are all
 * outside the window or behind lens[n] are not read. Cached values that no allowed
 * key has (the rest of the last page) may be anything, NaN and infinities included;
 * a value of an allowed key that is not finite makes NaN of its column. Logits are held
 * in units of log 2: profile entries beyond 2.35e38 (BF16's lowest value, as a mask) count
 * as infinite, and where that leaves a row no key, it is one with no allowed key.
 * A request with no allowed key (lens[n] <= 0: a padding row) gets out = 0, lse =
 * sink. A length above max_pages * page_size is taken as that.
 *   requests N, heads_q Hq (a multiple of heads_kv, below 65536), rel_extent R (a
 *   multiple of 8), window W (0: all), max_pages M; scale <= 0 means head_dim^-0.5
 *   q [N,Hq,D] BF16; profiles [N,Hq,R] BF16 (NULL exactly when R == 0); sink [N,Hq]
 *   FP32 or NULL (no sink); block_table [N,M] int32; lens [N] int32;
 *   out [N,Hq,D] FP32; lse [N,Hq] FP32; k_scale, v_scale as in inkling_kv_append
 * q, profiles, out, the pools and the workspace are 16-byte aligned, the rest 4.
 * The result of a request does not depend on where its pages are; it depends, in the
 * rounding of its sums alone, on the lengths in its batch. Equal calls give equal bits.
 * Limits (INKLING_ERR_UNSUPPORTED): N < 2^24, M * page_size, R and W < 2^30,
 * N * Hq * M * page_size < 2^40.
 */
typedef struct {
    int64_t requests, heads_q, rel_extent, window, max_pages;
    double scale;
} inkling_rel_attn_decode_dims;

/* Bytes of device workspace of inkling_rel_attn_decode; its contents need not be
 * set and mean nothing afterwards. Calls that follow each other may share one (two
 * captured graphs too, replayed one after the other), calls that can overlap on the
 * GPU need one each. 0 when the sizes are malformed. */
size_t inkling_rel_attn_decode_workspace_size(const inkling_kv_cache_desc* cache,
                                              const inkling_rel_attn_decode_dims* dims);

inkling_status inkling_rel_attn_decode(const inkling_kv_cache_desc* cache, const inkling_rel_attn_decode_dims* dims,
                                       const uint16_t* q, const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale, const uint16_t* profiles,
                                       const float* sink, const int32_t* block_table, const int32_t* lens, float* out,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INKLING_PAGED_ATTN_H */
