/*
 * q4k_layer.h -- what stands between the packed products of a decoder layer
 * (libq4k.so): the norm with the residual's addition, the rotation of queries
 * and keys and the paged cache, and the attention that reads it.
 *
 * The pages' models run these steps around every DequantMatMul: the Llama-3.2
 * and Qwen3 layers named there have an RMS norm in front of q/k/v and of
 * gate/up, QK norm (Qwen3), RoPE, grouped heads and a KV cache that stays on
 * the device (Orpheus/Metal page, "resident decode"; rlx-qwen3 crate page;
 * mlx-rs pull request #356, KVCache).  Here a layer is
 *     q4k_rms_norm -> q4k_matmul_batched (q, k, v) -> q4k_kv_append ->
 *     q4k_attention -> q4k_matmul (o) -> q4k_rms_norm (residual) ->
 *     q4k_matmul_swiglu -> q4k_matmul (down).
 *
 * Sequences.  A call has T tokens of `count` sequences, packed: sequence b's
 * new tokens are rows offsets[b] .. offsets[b + 1) of q, k, v and out.  With
 * its n_b = offsets[b + 1] - offsets[b] new tokens sequence b has lengths[b]
 * tokens, so that its new token i has index j = lengths[b] - n_b + i in it.
 * Index j is kept in page pages[b, j / page_size] of the cache, place
 * j % page_size.  A whole prompt is n_b = lengths[b], a decoded token n_b = 1.
 * Rows of q, k, v at and after offsets[count] belong to no sequence: they are
 * not stored, and their rows of q_out and out are left as they were.
 * All three arrays live on the device and are read by the kernels only.
 *   - offsets have to ascend from 0.  Where they do not, rows hold unspecified
 *     values (nothing outside the arrays is read or written: they are read as
 *     if clamped to [0, T]).
 *   - An index that has no page (below 0, or at or behind
 *     max_pages * page_size, or a page number outside [0, cache->pages)) is
 *     not stored, and read as if masked: it takes no part in any softmax.
 *   - Sequences may share pages (a common prefix).  Where two new tokens of one
 *     call have the same place it holds values of either.
 *
 * Conventions are those of q4k.h: device pointers on the current device, the
 * caller's stream, no host synchronization, the library's per-stream
 * workspace, the same status codes, nothing enqueued on an error.  T == 0 or
 * count == 0 (M or N zero) is a successful no-op.  The arrays are not to be
 * changed while a call that reads them runs.
 *
 * Workspace.  Attention over few row tiles (fewer than 512 over all key heads,
 * 256 for the kernels that have a CU to themselves: single tokens of a batch,
 * chunks, trees, short prompts), or over contexts of very different lengths, is
 * split along the keys and keeps its parts there, for each part
 * 4 * (head_dim + 2) bytes a row of its tile (16 to 128 rows), at most 4 * 512
 * parts, and 8 KB of counters that every call leaves at zero.  So make one eager
 * call of each shape before a graph capture (an attention call that counts,
 * captured on a stream that has no counters yet, is Q4K_ERR_ALLOC); and host
 * threads that share a stream take turns, and so do the replays of graphs
 * captured on one stream.  Where they do not, the rows of those calls hold
 * unspecified values; later calls are right.
 */
#ifndef Q4K_LAYER_H
#define Q4K_LAYER_H

#include "q4k.h"

#ifdef __cplusplus
extern "C" {
#endif

enum q4k_kv_type {
    Q4K_KV_F16 = 0,
    Q4K_KV_BF16 = 1,
    Q4K_KV_E4M3 = 2 /* OCP 8-bit floating point: 4 exponent bits, 3 of mantissa, no infinities, at most 448 */
};

/* The cache.  A HOST struct of DEVICE pointers, read during the call only.
 * k and v: [pages][kv_heads][page_size][head_dim] of the type, contiguous,
 * 16-byte aligned; element values are stored * k_scale and stored * v_scale. */
typedef struct q4k_kv_cache {
    void *k;
    void *v;
    int type;      /* q4k_kv_type */
    int pages;     /* pages in the pool; 64-bit offsets, any number */
    int kv_heads;  /* 1 .. 1024 */
    int page_size; /* a power of two, 1 .. 65536 */
    int head_dim;  /* a multiple of 16, 16 .. 256 */
    float k_scale; /* positive and finite, and so is 1 / k_scale (above 2^-128); 1 keeps the values as they are */
    float v_scale;
} q4k_kv_cache;

/* A HOST struct of DEVICE pointers, read during the call only. */
typedef struct q4k_sequences {
    const int *offsets; /* int32 [count + 1] */
    const int *lengths; /* int32 [count] */
    const int *pages;   /* int32 [count, max_pages] */
    int count;          /* 0 .. 65535 */
    int max_pages;      /* max_pages * page_size <= 2^30 */
} q4k_sequences;

/* What is done to q and k before they are used.  A HOST struct of DEVICE
 * pointers, read during the call only; every part is optional. */
typedef struct q4k_rotation {
    const float *q_norm;   /* float32 [head_dim] or NULL: x = x * rsqrt(mean(x^2) + eps) * q_norm, each head by itself */
    const float *k_norm;   /* the same for k */
    const float *inv_freq; /* float32 [rotary / 2] or NULL: no rotation */
    const int *positions;  /* int32 [T] or NULL: the token's index in its sequence */
    float eps;
    int rotary;            /* leading dimensions that are rotated: a multiple of 8, up to head_dim */
    int interleaved;       /* 0: pairs (i, i + rotary / 2); 1: pairs (2 i, 2 i + 1) */
} q4k_rotation;

/* total = x + residual and y = total * rsqrt(mean(total^2) + eps) * weight,
 * row by row; without a residual total is x.
 *   x, residual, total, y: DEVICE float32 [M, N], 4-byte aligned; residual and
 *   total may be NULL.  weight: DEVICE float32 [N].  total may be x or residual
 *   and y may be x or residual (any other overlap is not allowed).
 *   The sum of squares is held in double.
 *   Errors: M or N negative, N above 2^30: Q4K_ERR_BAD_DIM; x, weight or y NULL:
 *   Q4K_ERR_NULL; Q4K_ERR_ALIGN; M of 2^24 or more: Q4K_ERR_LAUNCH. */
int q4k_rms_norm(const float *x, const float *residual, const float *weight, float eps, float *total, float *y,
                 int M, int N, hipStream_t stream);

/* Stores the new tokens' keys and values, and gives the queries: k is normed
 * (k_norm) and rotated by the angles position * inv_freq[i], multiplied by
 * 1 / k_scale and rounded to the cache's type; v is multiplied by 1 / v_scale
 * and rounded; q_out is q normed (q_norm) and rotated.
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * Angles are reduced in double (a position of 2^31 - 1 loses nothing), the
 * norms' sums of squares are held in double (heads of every float32 size), the
 * rest is float32 with one rounding to the cache's type: to the nearest, ties
 * to even; e4m3 saturates at +-448 (infinities too), NaN stays NaN.
 *   q: DEVICE float32 [T, q_heads, head_dim] or NULL (then q_out is NULL
 *   too); q_out may be q itself (any other overlap is not allowed).  k, v: DEVICE float32 [T, kv_heads,
 *   head_dim].  16-byte aligned, the int arrays and weights 4-byte.
 *   rotation may be NULL: q_out is a copy of q, k is stored as it is.
 *   A token without a place in the cache still has its q_out.
 *   Errors: a negative or unsupported size (the structs', T * q_heads or
 *   T * kv_heads above 2^30, q_heads not a positive multiple of kv_heads
 *   where q is given), a scale that is not positive and finite or whose
 *   reciprocal is not:
 *   Q4K_ERR_BAD_DIM; a NULL array or struct (the optional ones excepted):
 *   Q4K_ERR_NULL; Q4K_ERR_ALIGN; more than 2^26 tokens: Q4K_ERR_LAUNCH. */
int q4k_kv_append(const float *q, const float *k, const float *v, const q4k_kv_cache *cache,
                  const q4k_sequences *sequences, const q4k_rotation *rotation, float *q_out, int T, int q_heads,
                  hipStream_t stream);

/* Causal attention over the cache, with grouped heads (query head h reads key
 * and value head h / (q_heads / kv_heads)).  Token i of sequence b sees the
 * indexes j <= lengths[b] - n_b + i that have a page:
 *     s[j] = scale * (q . k[j]),  out = sum_j softmax(s)[j] v[j].
 * A token that sees nothing (or only scores of -inf) has a row of zeros.
 *   q, out: DEVICE float32 [T, q_heads, head_dim], 16-byte aligned; out must
 *   not overlap the inputs.
 *   Numerics: the query times scale, and the softmax's unnormalised weights,
 *   are split into two binary16 values (scaled by powers of two; three bfloat16
 *   values over a bfloat16 cache), so that each product with the stored values
 *   is good to about 2^-22 of its size; a weight below 2^-38 of its row's
 *   largest is dropped; products, maxima, sums and outputs are float32.
 *   What a token does not see never reaches its row, NaN and infinities
 *   included (keys and values behind a sequence's end may hold anything).  A
 *   NaN or infinity that it sees gives NaN or infinities there.  So may, over a
 *   bfloat16 cache, finite values above 2^138 / (keys that the row sees): 2^121
 *   with 131072 keys; up to 1024 keys every finite value is kept.
 *   Results do not depend on the order in which workgroups finish.
 *   Errors: as for q4k_kv_append, and Q4K_ERR_ALLOC; Q4K_ERR_LAUNCH also for more
 *   than 2^24 row tiles. */
int q4k_attention(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences, float scale, float *out,
                  int T, int q_heads, hipStream_t stream);

/* The same for drafted tokens that need not follow each other: the new tokens
 * of a sequence see every index j < lengths[b] - n_b, and among themselves
 * what mask says: token t (a row of q) sees the new token i of its sequence
 * where bit i % 32 of mask[t, i / 32] is set (its own bit included: a token
 * does not see itself otherwise).  New tokens i >= 32 * mask_words are not
 * seen.  Rotate such tokens by their depth (q4k_rotation.positions), and
 * append the accepted ones again at the places that they take.
 *   mask: DEVICE uint32 [T, mask_words], mask_words >= 1.
 *   Everything else as for q4k_attention. */
int q4k_attention_tree(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences,
                       const unsigned *mask, int mask_words, float scale, float *out, int T, int q_heads,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_LAYER_H */
