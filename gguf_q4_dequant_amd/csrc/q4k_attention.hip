// Attention over the paged cache (include/q4k_layer.h).
//
// One wave per query and head: 64 keys at a time, a lane each, with the
// running maximum and sum of the softmax; then every lane sums its part of the
// output's dimensions over the 64 values.
#include <math.h>

#include "q4k_cache.h"

namespace q4k {
namespace {

struct Attend {
    Paged p;
    const float *q;
    float *out;
    const unsigned *mask;  // null: causal
    int words;
    int q_heads;
    int group;  // query heads of a key head
    float scale;
};

template <int kType>
__device__ __forceinline__ float value_at(const uint8_t *base, int64_t at) {
    if constexpr (kType == Q4K_KV_F16) return static_cast<float>(*reinterpret_cast<const _Float16 *>(base + 2 * at));
    else if constexpr (kType == Q4K_KV_BF16) return static_cast<float>(*reinterpret_cast<const __bf16 *>(base + 2 * at));
    else return __builtin_amdgcn_cvt_f32_fp8(base[at], 0);
}

template <int kType>
__global__ __launch_bounds__(64) void attend_kernel(const Attend a) {
    const Paged &p = a.p;
    const int lane = threadIdx.x, t = blockIdx.x, h = blockIdx.y, kh = h / a.group, D = p.head_dim;
    __shared__ float q[256];
    __shared__ float weight[64];
    __shared__ int64_t place[64];
    const int b = last_started(p.count, t, [&](int i) { return offset_of(p, i); });
    const int first = offset_of(p, b), end = offset_of(p, b + 1);
    if (t < first || t >= end) return;
    const int length = p.lengths[b];
    const int64_t before = static_cast<int64_t>(length) - (end - first);
    const int64_t stop = a.mask ? length : before + (t - first) + 1;
    const float *row = a.q + (static_cast<size_t>(t) * a.q_heads + h) * D;
    for (int d = lane; d < D; d += 64) q[d] = row[d] * a.scale * p.k_scale;
    __syncthreads();
    float m = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t j0 = 0; j0 < stop && j0 < (static_cast<int64_t>(p.max_pages) << p.shift); j0 += 64) {
        const int64_t j = j0 + lane;
        int64_t at = j < stop ? place_of(p, b, j, kh) : -1;
        if (a.mask && j >= before) {
            const int64_t i = j - before;
            if (i >= static_cast<int64_t>(a.words) * 32 || !((a.mask[static_cast<size_t>(t) * a.words + (i >> 5)] >> (i & 31)) & 1u)) at = -1;
        }
        float s = -INFINITY;
        if (at >= 0) {
            s = 0.f;
            for (int d = 0; d < D; ++d) s = fmaf(q[d], value_at<kType>(p.k, at + d), s);
        }
        float top = s;
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        top = fmaxf(m, top);
        const float base = top == -INFINITY ? 0.f : top;
        const float w = at >= 0 ? expf(s - base) : 0.f, fade = expf(m - base);
        float ws = w;
        for (int o = 32; o > 0; o >>= 1) ws += __shfl_xor(ws, o);
        sum = sum * fade + ws;
        m = top;
        weight[lane] = w;
        place[lane] = at;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= fade;
        for (int k = 0; k < 64; ++k) {
            if (place[k] < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < D) acc[i] = fmaf(weight[k], value_at<kType>(p.v, place[k] + lane + 64 * i), acc[i]);
        }
        __syncthreads();
    }
    float *o = a.out + (static_cast<size_t>(t) * a.q_heads + h) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < D) o[lane + 64 * i] = sum == 0.f ? 0.f : acc[i] / sum * p.v_scale;
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool misaligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int attend(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences, const unsigned *mask, int words,
           float scale, float *out, int T, int q_heads, hipStream_t stream) {
    Attend a = {};
    if (q_heads < 1) return Q4K_ERR_BAD_DIM;
    int rc = check_paged(cache, sequences, T, q_heads, &a.p);
    if (rc != Q4K_OK || T == 0 || sequences->count == 0) return rc;
    if (!q || !out) return Q4K_ERR_NULL;
    if (misaligned16(q) || misaligned16(out) || misaligned4(mask)) return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    a.q = q;
    a.out = out;
    a.mask = mask;
    a.words = words;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale = scale;
    const dim3 grid(T, q_heads);
    if (cache->type == Q4K_KV_F16) hipLaunchKernelGGL((attend_kernel<Q4K_KV_F16>), grid, dim3(64), 0, stream, a);
    else if (cache->type == Q4K_KV_BF16) hipLaunchKernelGGL((attend_kernel<Q4K_KV_BF16>), grid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL((attend_kernel<Q4K_KV_E4M3>), grid, dim3(64), 0, stream, a);
    return hipGetLastError() == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_attention(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences, float scale,
                             float *out, int T, int q_heads, hipStream_t stream) {
    return q4k::attend(q, cache, sequences, nullptr, 0, scale, out, T, q_heads, stream);
}

extern "C" int q4k_attention_tree(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences,
                                  const unsigned *mask, int mask_words, float scale, float *out, int T, int q_heads,
                                  hipStream_t stream) {
    if (mask_words < 1) return Q4K_ERR_BAD_DIM;
    if (T > 0 && sequences && sequences->count > 0 && !mask) return Q4K_ERR_NULL;
    return q4k::attend(q, cache, sequences, mask, mask_words, scale, out, T, q_heads, stream);
}
