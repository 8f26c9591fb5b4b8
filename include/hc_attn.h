/*
 * hc_attn.h -- C ABI of the attention between the projections of a layer
 * (include/hc_proj.h) on AMD Instinct MI355X (gfx950), for batches that mix
 * single decoded tokens, verify windows and prefill chunks of many requests,
 * whose keys and values lie in a paged cache.
 *
 *   hc_rotate_heads   y = turn(norm(x) * weight, position) for every head of
 *                     every token
 *   hc_append_heads   the same for the queries and the keys of a batch; keys
 *                     and values go to the cache on the way
 *   hc_attend         out = sum_j softmax_j(score(t, h, j)) v[j] over the
 *                     positions j that the token sees
 *   hc_attend_shared  the same for requests that begin with prefixes which they
 *                     share, each prefix's part computed once for all of them
 *
 *   norm(x) = x / sqrt(mean x^2 + eps); turn: (a, b) -> (a cos - b sin, b cos +
 *   a sin) for the pairs of the first `rotated` columns, pair i by the angle
 *   position * frequencies[i]
 *   score = scale q[t,h] . k[j, h / (q_heads / heads)]; with a cap, cap * tanh(score /
 *   cap); with slopes, less slopes[h] * |p - j|, p the token's position
 *
 * Inference only.  Types: HC_BF16 or HC_FP16, one for all of a call's heads
 * and its cache.  Norms, angles' sines and cosines, scores, maxima, sums and
 * partial results are fp32 (angles themselves are reduced in fp64); outputs are
 * rounded once, to nearest even.  The softmax's numerators enter the matrix cores
 * in the 16-bit type: in two pieces, which keep twice its digits, where there are
 * no prefixes and up to 8 rows per request on average (heads of more than 128
 * columns: 32); else rounded once.
 *
 * Memory: every pointer is a DEVICE pointer, but for the descriptions hc_cache,
 * hc_batch and hc_prefix, which the call reads on the host.  Strides are in
 * elements; a head's `dim` columns are contiguous.  Heads start at multiples of
 * 16 bytes: strides are multiples of 8 and so is dim, up to HC_MAX_HEAD.
 * Everything else is aligned to its own type.  Outputs must not overlap inputs
 * or each other, but hc_rotate_heads and hc_append_heads may write the queries
 * where they read them (the same pointer and strides).  The caller owns all memory: nothing is
 * allocated, and a call's scratch (`work`) belongs to that call until the
 * stream has passed it.
 *
 * Execution: asynchronous on `stream` (a hipStream_t; NULL = the default
 * stream) of the current device, without host synchronization or allocation:
 * calls can be captured into graphs.  The same call gives the same bits (no
 * floating-point atomics).  A token's result does not depend on what other
 * requests hold, nor on what positions hold that it does not see (infinities
 * and NaN too); its last bits may differ with the sizes and the lengths of the
 * call, which choose how the work is split.
 *
 * Indices come from device memory and are not checked by the host.  The kernels
 * check them: offsets are clamped to [0, T], lengths to what the table's rows
 * hold, a page outside the cache reads as zeros and is not written.  Offsets and
 * starts that are not in order leave the call's results open, as many of them as
 * it writes; nothing but its outputs, its scratch and the pages of the table is
 * written.  A key or value of a position that a token sees should be a number of
 * its type; scores should be within 2^127, sums of a token's values and of a
 * head's squares numbers of fp32.
 *
 * Errors: status codes of hc.h; argument checks come before any launch.
 */
#ifndef HC_ATTN_H
#define HC_ATTN_H

#include "hc_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits. */
#define HC_MAX_HEAD 256        /* columns of a head */
#define HC_MAX_REQUESTS 2048   /* requests of one call, and prefixes */
#define HC_MAX_ROWS 262144     /* hc_attend: T * q_heads / heads */
#define HC_MIN_PAGE 16         /* positions of a page: a power of two from this */
#define HC_MAX_PAGE 65536      /* ... to this */
/* hc_attend, hc_attend_shared: a table's width * page_size (with prefixes, both
 * tables' in sum) is at most 2^31 - 65536. */

/*
 * A paged cache: position r of page g, head h at keys + g key_page + r key_row
 * + h key_head, and values likewise (in elements; row and head strides below
 * 2^23, page strides below 2^31 - 65536; up to 65536 heads, of queries too).
 */
typedef struct hc_cache {
    void* keys;
    void* values;
    int64_t pages, page_size, heads, dim;
    int64_t key_page, key_row, key_head;
    int64_t value_page, value_row, value_head;
    int64_t type; /* HC_BF16 or HC_FP16 */
} hc_cache;

/*
 * A batch: request b's new tokens are offsets[b] <= t < offsets[b+1], the last
 * ones of its lengths[b] positions; its position i lies in page
 * table[b][i / page_size].  Tokens of no request are left alone.
 */
typedef struct hc_batch {
    int64_t requests;
    const int32_t* offsets; /* [requests + 1], non-decreasing */
    const int32_t* lengths; /* [requests], the new tokens included */
    const int32_t* table;   /* [requests][width], row stride table_row */
    int64_t width, table_row;
} hc_batch;

/*
 * Prefixes: requests starts[g] <= b < starts[g+1] begin with the lengths[g]
 * positions whose pages are table[g]; the positions of their own (hc_batch)
 * follow.  Requests of no group have none.
 */
typedef struct hc_prefix {
    int64_t groups;
    const int32_t* starts;  /* [groups + 1], non-decreasing */
    const int32_t* lengths; /* [groups] */
    const int32_t* table;   /* [groups][width], row stride table_row */
    int64_t width, table_row;
} hc_prefix;

/*
 * hc_rotate_heads -- T tokens of `heads` heads.
 *
 *   x, out       [T][heads][dim], token and head strides in elements
 *   positions    int32 [T]; NULL without frequencies
 *   frequencies  float [rotated / 2], radians per position; NULL: no rotation
 *   rotated      columns that turn, a multiple of 8 up to dim; the rest pass
 *   interleaved  nonzero: pairs are columns (2i, 2i + 1); 0: (i, i + rotated / 2)
 *   weight       float [dim], or NULL: no norm
 */
HC_API int hc_rotate_heads(int64_t T, int64_t heads, int64_t dim, int type, const void* x, int64_t x_row,
                           int64_t x_head, const int32_t* positions, const float* frequencies, int64_t rotated,
                           int interleaved, const float* weight, float eps, void* out, int64_t out_row,
                           int64_t out_head, void* stream);

/*
 * hc_append_heads -- the new tokens of a batch: queries normed and turned to
 * `out`, keys normed and turned into the cache, values copied into it.
 *
 *   q, out       [T][q_heads][dim]; q_heads 0: no queries
 *   k, v         [T][cache heads][dim]
 *   positions    int32 [T]: what the angles go by; NULL: the position in the
 *                request's own sequence, which is where k and v are stored
 *   q_weight, k_weight  float [dim], or NULL: no norm
 *
 * A position outside the request's row of the table, or on a page outside the
 * cache, is not stored (its query is computed all the same).  Two tokens must
 * not be stored in one place.
 */
HC_API int hc_append_heads(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const void* k,
                           int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                           const hc_cache* cache, const hc_batch* batch, const int32_t* positions,
                           const float* frequencies, int64_t rotated, int interleaved, const float* q_weight,
                           const float* k_weight, float eps, void* out, int64_t out_row, int64_t out_head,
                           void* stream);

/*
 * hc_attend -- T tokens of a batch over their requests' positions.
 *
 *   q, out       [T][q_heads][dim]; q_heads is a multiple of the cache's heads
 *   scale        from -2^100 to 2^100
 *   cap          up to 2^100; 0: none
 *   slopes       float [q_heads], or NULL
 *   first, last  int32 [T], or NULL: token t sees positions first[t] <= j <
 *                last[t] of its request's sequence, by default 0 and p + 1.  A
 *                token that sees none gives zeros
 *   work         scratch of at least hc_attend_work(...) bytes
 */
HC_API int hc_attend(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const hc_cache* cache,
                     const hc_batch* batch, float scale, float cap, const float* slopes, const int32_t* first,
                     const int32_t* last, void* out, int64_t out_row, int64_t out_head, void* work,
                     int64_t work_bytes, void* stream);

/*
 * hc_attend_shared -- the same under prefixes.  Positions (p, j, first and last)
 * count from the prefix's first.  By default a token sees the whole prefix, and
 * of its request's own positions those up to its own.  Every row leaves two partial
 * results in `work`: for hundreds of new tokens per request, hc_attend with the
 * prefix's pages in every request's row of the table is faster and needs less.
 */
HC_API int hc_attend_shared(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head,
                            const hc_cache* cache, const hc_batch* batch, const hc_prefix* prefix, float scale,
                            float cap, const float* slopes, const int32_t* first, const int32_t* last, void* out,
                            int64_t out_row, int64_t out_head, void* work, int64_t work_bytes, void* stream);

/* Scratch bytes of hc_attend (groups 0) and hc_attend_shared for exactly these
 * sizes; 0: sizes that they refuse. */
HC_API int64_t hc_attend_work(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t requests,
                              int64_t groups);

/* Text for a status code of these calls (static storage; never NULL). */
HC_API const char* hc_attn_status_string(int status);

/* The hipError_t behind the last HC_ERR_LAUNCH / HC_ERR_DEVICE of these calls
 * on this host thread (0 if none). */
HC_API int hc_attn_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* HC_ATTN_H */
