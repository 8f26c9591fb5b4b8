/*
 * hc_proj.h -- C ABI of the projections around the hyper-connection read on
 * AMD Instinct MI355X (gfx950): what a layer computes on the read's 16-bit
 * images (include/hc.h), for batches that mix single decoded tokens, verify
 * windows and prefill chunks of many requests.
 *
 *   hc_project         y[t] = W x[t] + scale[a] * B[a] (A[a] x[t]), a = adapter[t]:
 *                      one shared projection and, beside it, the low-rank
 *                      adapter of each token's request
 *   hc_route           each token's k best experts of E, their weights, and
 *                      the token rows sorted by expert
 *   hc_expert_project  y[i] = W[e] x[rows[i]] for offsets[e] <= i < offsets[e+1],
 *                      or, gated, silu(Wg[e] x) * (Wu[e] x)
 *   hc_expert_combine  out[t] = sum_s weights[t][s] * y[pos[t][s]]
 *
 * Types: HC_BF16 and HC_FP16 operands with HC_FP32 accumulation on the matrix
 * cores; x, W, A and B of one call have one type.  Outputs are rounded once,
 * to nearest even, to the 16-bit type of the operands, or stored in fp32.  The
 * adapter's inner product A x stays in fp32 (B's product takes it as an exact
 * sum of three bf16 pieces); the gate's activation is computed in fp32.  A finite
 * scale may multiply A x before B does, in fp32, and their product should be a
 * number of fp32; an infinity or NaN multiplies B (A x).
 *
 * Memory: every pointer is a DEVICE pointer.  Weights are row-major
 * [outputs][inputs] and contiguous; x, out, y and logits have a row stride in
 * elements (ld*), and their rows are contiguous.  x, W, A, B and work are
 * 16-byte aligned, K and ldx are multiples of 8 and rank is a multiple of 8;
 * everything else is aligned to its own type.  N, C, E, T and the row counts
 * are any numbers below 2^31 - 65536 (experts' products: N up to half of that),
 * K up to 2^28; a call that needs 2^32 or more threads of one kernel is refused
 * (HC_ERR_SIZE).  Outputs must not overlap inputs or each other.  The caller
 * owns all memory: nothing is allocated, and a call's scratch (`work`) belongs
 * to that call until the stream has passed it, so graphs and streams share
 * scratch only if their caller makes them.
 *
 * Execution: asynchronous on `stream` (a hipStream_t; NULL = the default
 * stream) of the current device, without host synchronization or allocation:
 * calls can be captured into graphs.  Results do not depend on the order in
 * which workgroups run (no floating-point atomics).  While short-window reads
 * (hc.h) run, these kernels hold CUs like any other work on the device.
 *
 * Indices come from device memory and are not checked by the host.  The
 * kernels check them: an adapter outside [0, adapters) means no adapter, a row
 * outside x reads as zeros, a position outside y adds nothing, and offsets are
 * clamped to [0, R].  A token's result depends on its own row and its own
 * adapter or expert alone, whatever the others hold (infinities and NaN too); its
 * last bits may differ with the sizes of the call, which choose the kernel.
 *
 * Errors: status codes of hc.h; argument checks come before any launch.
 */
#ifndef HC_PROJ_H
#define HC_PROJ_H

#include "hc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define HC_BF16 0
#define HC_FP16 1
#define HC_FP32 2

/* Limits. */
#define HC_MAX_RANK 128    /* adapter rank */
#define HC_MAX_EXPERTS 512 /* experts of one router */
#define HC_MAX_TOPK 32     /* experts per token */

/*
 * hc_project -- one projection of T tokens with the adapters of their requests.
 *
 *   T, K, N    tokens, inputs (multiple of 8), outputs
 *   type       HC_BF16 or HC_FP16: type of x, W, A and B
 *   x          [T][K], row stride ldx
 *   W          [N][K]
 *   adapter    int32 [T]: each token's adapter; outside [0, adapters) none.
 *              NULL (or adapters == 0): no adapters at all; A, B, scale and
 *              rank are then ignored
 *   adapters   adapters stored
 *   rank       their rank, a multiple of 8 up to HC_MAX_RANK (adapters of
 *              smaller rank are stored with zero rows in A)
 *   A          [adapters][rank][K]
 *   B          [adapters][N][rank]
 *   scale      float [adapters], or NULL for 1
 *   out        [T][N], row stride ldo, of out_type (`type` or HC_FP32)
 *   work       scratch of at least hc_project_work(...) bytes; NULL if that is 0
 *
 * Returns HC_OK or an HC_ERR_* code (HC_ERR_SIZE: a size outside its limits,
 * or work_bytes too small).
 */
HC_API int hc_project(int64_t T, int64_t K, int64_t N, int type, const void* x, int64_t ldx, const void* W,
                      const int32_t* adapter, int64_t adapters, int64_t rank, const void* A, const void* B,
                      const float* scale, void* out, int64_t ldo, int out_type, void* work, int64_t work_bytes,
                      void* stream);

/* Scratch bytes of hc_project for exactly these sizes (pass rank 0 without
 * adapters); 0: none, as for one token of most sizes, or sizes that hc_project
 * refuses.  Fewer tokens or a smaller rank may need more: a caller with one
 * scratch for many sizes takes the most over the T that it will use, of its rank
 * and, where calls go without adapters, of rank 0.  (No more than 8 splits' sums
 * and A x: 32 T N + 16 T (rank + 8) bytes.) */
HC_API int64_t hc_project_work(int64_t T, int64_t K, int64_t N, int64_t rank);

/*
 * hc_route -- the k largest of E logits per token, and the sort by expert.
 *
 *   logits     [T][E], row stride ldl, of type HC_FP32, HC_BF16 or HC_FP16.
 *              Equal logits go to the lower expert.  -inf and NaN mask an
 *              expert out; +inf counts as the largest finite value
 *   renorm     nonzero: weights are the softmax over the token's k chosen
 *              experts; 0: over all its unmasked experts
 *   ids        int32 [T][k], best first; -1 where fewer than k are unmasked
 *   weights    float [T][k]; 0 where ids is -1
 *   offsets    int32 [E+1]: expert e's rows are offsets[e] <= i < offsets[e+1]
 *   rows       int32 [T*k]: the token of row i; tokens ascend inside an expert.
 *              -1 from offsets[E] on
 *   pos        int32 [T][k]: the row of (token, slot), -1 where ids is -1
 *   work       scratch of at least hc_route_work(...) bytes; NULL if that is 0
 *
 * 1 <= k <= min(E, HC_MAX_TOPK), E <= HC_MAX_EXPERTS, T * k < 2^31.
 */
HC_API int hc_route(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ldl, int type, int renorm,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* work,
                    int64_t work_bytes, void* stream);

/* Scratch bytes of hc_route for exactly these sizes; 0: none (short batches), or
 * sizes that hc_route refuses.  Fewer tokens may need more; none more than 2048 E. */
HC_API int64_t hc_route_work(int64_t T, int64_t E, int64_t k);

/*
 * hc_expert_project -- R rows in E ragged groups, each through its expert's
 * weights.
 *
 *   R          rows of out (T * k after hc_route)
 *   x          [x_rows][K], row stride ldx
 *   rows       int32 [R]: the row of x that row i reads, or NULL for row i itself
 *   W          [E][N][K]; gated: [E][2 N][K], the gate's N rows first
 *   offsets    int32 [E+1], non-decreasing: group e is offsets[e] <= i <
 *              offsets[e+1]; groups may be empty.  Rows of `out` in no group
 *              are left as they were
 *   gate       nonzero: out = silu(gate product) * (up product), N wide
 *   out        [R][N], row stride ldo, of out_type (`type` or HC_FP32)
 */
HC_API int hc_expert_project(int64_t R, int64_t K, int64_t N, int64_t E, int type, const void* x, int64_t x_rows,
                             int64_t ldx, const int32_t* rows, const void* W, const int32_t* offsets, int gate,
                             void* out, int64_t ldo, int out_type, void* stream);

/*
 * hc_expert_combine -- each token's rows of y, weighted and summed in fp32 in
 * the order of its slots.
 *
 *   y          [y_rows][C], row stride ldy, of type HC_BF16, HC_FP16 or HC_FP32
 *   pos        int32 [T][k]; a position outside [0, y_rows) adds nothing,
 *              whatever its weight (a token without any position gives 0)
 *   weights    float [T][k]
 *   out        [T][C], row stride ldo, of out_type (any of the three)
 *
 * k up to 512, T * k < 2^31.
 */
HC_API int hc_expert_combine(int64_t T, int64_t k, int64_t C, const void* y, int64_t y_rows, int64_t ldy, int type,
                             const int32_t* pos, const float* weights, void* out, int64_t ldo, int out_type,
                             void* stream);

/* Text for a status code of these calls (static storage; never NULL). */
HC_API const char* hc_proj_status_string(int status);

/* The hipError_t behind the last HC_ERR_LAUNCH / HC_ERR_DEVICE of these calls
 * on this host thread (0 if none). */
HC_API int hc_proj_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* HC_PROJ_H */
