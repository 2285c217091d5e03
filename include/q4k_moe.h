/*
 * q4k_moe.h -- mixture-of-experts layers over packed Q4_K weights (libq4k.so).
 *
 * A GGUF mixture-of-experts checkpoint keeps the experts' matrices of one
 * projection as one Q4_K tensor [E, N, K] (expert, output feature, input
 * feature).  The functions here are what such a layer needs next to
 * q4k_matmul (q4k.h): the router's choice and grouping, the products of every
 * expert with its own ragged set of rows, the gate/up pair with its SwiGLU
 * epilogue, and the down projection with the weighted sum over a token's
 * experts.  (The mlx-rs pull request #356 page names the same step for its
 * quantized switch layers: gather_qmm and router_topk.)
 *
 * Pairs and groups.  With M tokens and top_k experts per token, pair
 * p = m * top_k + j is token m's j-th choice; there are P = M * top_k pairs.
 *   offsets  DEVICE int32 [E + 1], ascending from 0: group e (expert e's
 *            pairs) is rows[offsets[e] .. offsets[e + 1])
 *   rows     DEVICE int32 [P]: the pairs in expert order (ascending within an
 *            expert); entries at and after offsets[E] belong to no group
 * offsets and rows live on the device and are read by the kernels only: no
 * call here waits for them.  Group sizes are ragged: any group may be empty
 * or hold every pair.
 *
 * Conventions are those of q4k.h: device pointers on the current device, the
 * caller's stream, no host synchronization, the library's per-stream
 * workspace (make one eager call of each shape before a graph capture; host
 * threads that share a stream take turns, and so do the replays of graphs
 * captured on one stream, which share its workspace), the same status codes,
 * nothing enqueued on an error.  Empty sizes (M, P or N zero) are successful
 * no-ops.
 *
 * Workspace.  Grouped products, except those of few pairs (q4k_grouped_tile: 4
 * rows), keep x's staged form, 1056 bytes for 256 values (1.03 times x) and 16
 * a row; the weighted sum also keeps the pairs' products, 4 * M * top_k * N
 * bytes.  Both stay allocated to the stream.
 */
#ifndef Q4K_MOE_H
#define Q4K_MOE_H

#include "q4k.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q4K_MAX_EXPERTS 1024
#define Q4K_MAX_TOP_K 64

enum q4k_route_flags {
    Q4K_ROUTE_SIGMOID = 1,  /* scores are sigmoid(logit); without it, the softmax over the experts */
    Q4K_ROUTE_NORMALIZE = 2 /* a token's weights are divided by their sum */
};

/* Top-k routing.  For each token m:
 *     s[e]   = softmax(logits[m, :])[e], or 1 / (1 + exp(-logits[m, e])),
 *     choice = the top_k experts with the largest s[e] + bias[e], best first,
 *              equal ones by the lower e (without a bias, the largest logits),
 *     expert[m, j] = choice j,  weight[m, j] = scale * s[choice j]
 *              (/ the sum of the chosen s with Q4K_ROUTE_NORMALIZE).
 * The bias takes part in the choice only.  An expert whose logit is NaN or
 * -inf takes no part in the softmax and is never chosen, nor is one whose
 * s + bias is NaN or -inf; where fewer than top_k are left the remaining
 * choices have expert -1 and weight 0.  A logit of +inf outweighs every
 * finite one (equal shares among several).  A chosen sum of 0 gives weights 0.
 *   logits: DEVICE float32 [M, E].  bias: DEVICE float32 [E] or NULL.
 *   expert: DEVICE int32 [M, top_k].  weight: DEVICE float32 [M, top_k].
 *   offsets, rows: the groups of these pairs, as above; entries of rows
 *   behind the last group are set to -1.  Pairs with expert -1 are in no group.
 *   With a bias the compared scores are computed in double, so that close
 *   scores are told apart by their values, not by how they were rounded.
 *   The weights' sigmoids are computed in double with or without a bias: they
 *   are 0, and equal, only from logits of about -745 on.
 *   Errors: M < 0, E outside [1, Q4K_MAX_EXPERTS], top_k outside
 *   [1, min(E, Q4K_MAX_TOP_K)], M * top_k > INT_MAX or unknown flags:
 *   Q4K_ERR_BAD_DIM; a NULL pointer (bias excepted): Q4K_ERR_NULL; a pointer
 *   not 4-byte aligned: Q4K_ERR_ALIGN.  M == 0 writes offsets (all 0). */
int q4k_moe_route(const float *logits, const float *bias, int M, int E, int top_k, int flags, float scale,
                  int *expert, float *weight, int *offsets, int *rows, hipStream_t stream);

/* The groups of an existing table of choices: expert DEVICE int32 [P] (a
 * value outside [0, E) puts the pair in no group).  Outputs and errors as for
 * q4k_moe_route. */
int q4k_moe_group(const int *expert, int P, int E, int *offsets, int *rows, hipStream_t stream);

/* Products grouped by expert: for every pair p = rows[i] of group e
 *     y[p, :] = x[p / x_div, :] . dequant(W[e])^T.
 * x_div = top_k reads one row of x per token (a projection's input), x_div = 1
 * one row per pair (the down projection's).
 *   w_packed: DEVICE, [E][N][K/256*144] bytes.  x: DEVICE float32,
 *   [ceil(P / x_div), K].  y: DEVICE float32 [P, N]; rows of pairs in no group
 *   are left as they were.  rows == NULL means rows[i] = i (pairs already in
 *   expert order).  w_packed, x, y 16-byte aligned, offsets and rows 4-byte.
 *   y must not overlap the inputs, and a pair must not be named twice.
 *   Entries of rows outside [0, P) are skipped, and offsets are read as if
 *   clamped to [0, P]; a pair of offsets that descends is an empty group.
 *   Numerics: x is split into two binary16 values scaled by a power of two per
 *   row or per 256 values of a row (about 22 significant bits of each value, or
 *   2^-39 of the largest magnitude there where that is more), and so is each sum
 *   of 32 values, which the min term takes (2^-33 of that magnitude where that is
 *   more); the quants times their 6-bit scales are exact integers, sums and
 *   scales are fp32: beside those, rounding of the order of
 *   1e-6 * sum_k |x_k| (|d sc q| + |dmin m|).  A NaN or infinity in a row of x
 *   gives NaN or infinities in that row of y only.
 *   Errors: negative sizes, E outside [1, Q4K_MAX_EXPERTS], x_div < 1, K not a
 *   positive multiple of 256 or above 2^26: Q4K_ERR_BAD_DIM; NULL (rows excepted):
 *   Q4K_ERR_NULL; alignment: Q4K_ERR_ALIGN; Q4K_ERR_ALLOC; Q4K_ERR_LAUNCH. */
int q4k_matmul_grouped(const void *w_packed, const float *x, int x_div, const int *offsets, const int *rows,
                       float *y, int E, int P, int N, int K, hipStream_t stream);

/* Gate and up projections of the experts with the SwiGLU epilogue: for every
 * pair p of group e
 *     out[p, :] = silu(x[p / x_div] . dequant(W_gate[e])^T) * (x[p / x_div] . dequant(W_up[e])^T),
 * silu and its rounding as for q4k_matmul_swiglu.  Both matrices [E][N][K/256*144]
 * bytes; everything else as for q4k_matmul_grouped. */
int q4k_matmul_grouped_swiglu(const void *w_gate, const void *w_up, const float *x, int x_div,
                              const int *offsets, const int *rows, float *out, int E, int P, int N, int K,
                              hipStream_t stream);

/* Down projections of the experts and the weighted sum over each token's
 * choices:
 *     out[m, :] = sum_j weight[m, j] * (x[m * top_k + j, :] . dequant(W[e])^T),
 * e = expert[m, j], the terms added in ascending j (a result never depends on
 * the order in which workgroups finish).  A choice whose expert is outside
 * [0, E) adds nothing; a token without any has a row of zeros.
 *   x: DEVICE float32 [M * top_k, K].  expert, weight, offsets, rows: as
 *   q4k_moe_route gives them; expert and the groups must agree (a pair whose
 *   expert is valid has to be in a group).  out: DEVICE float32 [M, N], 16-byte
 *   aligned, not overlapping the inputs.  The products go through the
 *   library's workspace ([M * top_k, N] float32).
 *   Errors: as for q4k_matmul_grouped, and top_k < 1 or M * top_k > INT_MAX:
 *   Q4K_ERR_BAD_DIM. */
int q4k_matmul_grouped_combine(const void *w_packed, const float *x, const int *expert, const float *weight,
                               const int *offsets, const int *rows, float *out, int E, int M, int top_k, int N,
                               int K, hipStream_t stream);

/* The kernel that a grouped product of these sizes runs, for tests and
 * benchmarks (as q4k_select_path is for q4k_matmul): the rows of its tiles, 4,
 * 16, 32 or 48, and in *parts (HOST, may be NULL) the parts into which a
 * workgroup splits K, one for each of its waves (4 rows: 4 or 8) or of its groups
 * of four waves (16 rows: 1, 2 or 4; otherwise 1).  swiglu != 0: the gate/up
 * form.  The weighted sum's product is the plain one of P = M * top_k pairs.
 * Tiles of 4 rows stage x themselves; the others use workspace slot 0.  Returns 0
 * (and 0 parts) where P or N is zero, Q4K_ERR_BAD_DIM as q4k_matmul_grouped
 * does.  No device is needed. */
int q4k_grouped_tile(int E, int P, int N, int K, int swiglu, int *parts);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_MOE_H */
