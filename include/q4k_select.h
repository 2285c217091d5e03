/*
 * q4k_select.h -- penalties, biases and grammar masks on logits, and the
 * greedy choice under them (libq4k.so).
 *
 * The pages' decode loop runs penalty -> pick on the host after every token
 * (nx_f32_llm_run_v3 source page: _frn3_apply_penalty over a window of recent
 * tokens, then _frn3_pick), and the rlx-llama32 crate page keeps a host-greedy
 * lm_head for its logit adjustment.  Here both steps run on the device, beside
 * q4k_matmul_argmax (q4k.h), whose plain maximum they extend.
 *
 * For row m (one sequence) and token n, with c the number of times n occurs
 * in history[m, :], in float32 and in this order:
 *     z = logits[m, n]
 *     if c > 0:  z = z > 0 ? z / repetition[m] : z * repetition[m]
 *     z = z - frequency[m] * c - presence[m]          (c > 0)
 *     z = z + b,  b = the sum of bias_value[m, i] over all i with
 *                 bias_id[m, i] == n, added in ascending i
 *     z = -inf where the mask's bit of n is clear (whatever z was, NaN too)
 *
 * Conventions are those of q4k.h (device pointers, the caller's stream, no
 * host synchronization, per-stream workspace, status codes).  The workspace of
 * a choice is 8 bytes for every 1024 or 4096 logits; behind the lm_head it also
 * holds the logits, 4 * M * N bytes, which stay allocated to the stream.
 */
#ifndef Q4K_SELECT_H
#define Q4K_SELECT_H

#include "q4k.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What is applied.  A HOST struct of DEVICE pointers, read during the call
 * only.  Every part is optional: a NULL pointer (or zero length) leaves that
 * step out.  All arrays are contiguous and 4-byte aligned. */
typedef struct q4k_adjustment {
    const int *history;      /* int32 [M, history_len]: each sequence's recent tokens; entries outside
                                [0, N) (padding) count for nothing */
    const float *repetition; /* float32 [M], or NULL: 1 */
    const float *frequency;  /* float32 [M], or NULL: 0 */
    const float *presence;   /* float32 [M], or NULL: 0 */
    const int *bias_id;      /* int32 [M, bias_len]; entries outside [0, N) are skipped */
    const float *bias_value; /* float32 [M, bias_len] */
    const unsigned *mask;    /* uint32 [M, ceil(N / 32)]: bit n % 32 of word n / 32 set = token n allowed */
    int history_len;
    int bias_len;
} q4k_adjustment;

/* out[m, n] = the adjusted logit.  logits and out: DEVICE float32 [M, N],
 * 4-byte aligned; out may be logits itself (any other overlap is not allowed).
 *   Errors: M, N, history_len or bias_len negative, or one of the last two
 *   above 2^30: Q4K_ERR_BAD_DIM; logits,
 *   out or the struct NULL, history NULL with history_len > 0, bias_id or
 *   bias_value NULL with bias_len > 0: Q4K_ERR_NULL; Q4K_ERR_ALIGN; M above
 *   65535: Q4K_ERR_LAUNCH.  M == 0 or N == 0 is a no-op. */
int q4k_logits_adjust(const float *logits, float *out, const q4k_adjustment *adjustment, int M, int N,
                      hipStream_t stream);

/* index[m] = the lowest allowed n with the largest adjusted logit, value[m] =
 * that logit.  NaN logits and masked tokens never win; a row in which nothing
 * is left (every token masked or NaN) gives index -1 and value -inf.  (A row of
 * NaN without a mask too, where q4k_matmul_argmax, which has no masks, gives index
 * 0 and value NaN.)
 *   index: DEVICE int32 [M].  value: DEVICE float32 [M] or NULL.
 *   Errors: as for q4k_logits_adjust, and N == 0 (no maximum):
 *   Q4K_ERR_BAD_DIM. */
int q4k_logits_argmax(const float *logits, const q4k_adjustment *adjustment, int M, int N, int *index,
                      float *value, hipStream_t stream);

/* q4k_matmul_argmax under an adjustment: the logits are x . dequant(W)^T, as
 * q4k_matmul computes them, and stay in the library's workspace.  Arguments
 * and errors as for q4k_matmul_argmax and q4k_logits_argmax. */
int q4k_matmul_argmax_adjusted(const void *w_packed, const float *x, const q4k_adjustment *adjustment, int M,
                               int N, int K, int *index, float *value, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_SELECT_H */
