// New tokens' keys and values into the paged cache, with the norm of each head
// and the rotation on the way (include/q4k_layer.h).
//
// A lane has eight values of one head: with pairs (i, i + rotary / 2) four of
// each half, so that both partners of a rotation are in its registers, else
// eight neighbours.  A head is spread over a power of two of lanes (16 for 128
// values), which sum its squares among themselves.  The angles depend on the
// token and on the lane's place in its head only: they are taken once for all
// heads that a wave goes through.  Everything is read once and written once, so
// memory bounds it: packed prompts of 5.2k tokens, 32 query and 8 key heads of 128,
// e4m3: 281 MB in 57 us, 4.9 TB/s; one token 3 us, a launch's own time.
#include <math.h>

#include "q4k_cache.h"
#include "q4k_factor.h"

namespace q4k {

namespace {
bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool misaligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
}  // namespace

int check_paged(const q4k_kv_cache *cache, const q4k_sequences *sequences, int T, int q_heads, Paged *p) {
    if (!cache || !sequences) return Q4K_ERR_NULL;
    const q4k_kv_cache &c = *cache;
    const q4k_sequences &s = *sequences;
    if (T < 0 || q_heads < 0 || s.count < 0 || s.count > 65535 || s.max_pages < 0 || c.pages < 0) return Q4K_ERR_BAD_DIM;
    if (c.type != Q4K_KV_F16 && c.type != Q4K_KV_BF16 && c.type != Q4K_KV_E4M3) return Q4K_ERR_BAD_DIM;
    if (c.kv_heads < 1 || c.kv_heads > 1024) return Q4K_ERR_BAD_DIM;
    if (c.page_size < 1 || c.page_size > 65536 || (c.page_size & (c.page_size - 1)) != 0) return Q4K_ERR_BAD_DIM;
    if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16 != 0) return Q4K_ERR_BAD_DIM;
    if (static_cast<int64_t>(s.max_pages) * c.page_size > (1 << 30)) return Q4K_ERR_BAD_DIM;
    if (static_cast<int64_t>(T) * c.kv_heads > (1 << 30) || static_cast<int64_t>(T) * q_heads > (1 << 30)) return Q4K_ERR_BAD_DIM;
    if (q_heads % c.kv_heads != 0) return Q4K_ERR_BAD_DIM;
    // (the append multiplies by the reciprocals)
    for (const float scale : {c.k_scale, c.v_scale})
        if (!(scale > 0.f) || isinf(scale) || isinf(1.f / scale)) return Q4K_ERR_BAD_DIM;
    if (T == 0 || s.count == 0) return Q4K_OK;
    if (((!c.k || !c.v) && c.pages > 0) || !s.offsets || !s.lengths || (!s.pages && s.max_pages > 0)) return Q4K_ERR_NULL;
    if (misaligned16(c.k) || misaligned16(c.v) || misaligned4(s.offsets) || misaligned4(s.lengths) || misaligned4(s.pages))
        return Q4K_ERR_ALIGN;
    p->k = static_cast<uint8_t *>(c.k);
    p->v = static_cast<uint8_t *>(c.v);
    p->offsets = s.offsets;
    p->lengths = s.lengths;
    p->table = s.pages;
    p->count = s.count;
    p->max_pages = s.max_pages;
    p->pages = c.pages;
    p->shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
    p->kv_heads = c.kv_heads;
    p->head_dim = c.head_dim;
    p->tokens = T;
    p->k_scale = c.k_scale;
    p->v_scale = c.v_scale;
    return Q4K_OK;
}

namespace {

constexpr int kThreads = 256;

// Lanes that a head of D values is spread over, eight values a lane.
__host__ __device__ inline int lanes_of(int D) { return D <= 16 ? 2 : D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

struct Append {
    Paged p;
    const float *q, *k, *v;
    float *q_out;
    const float *q_norm, *k_norm, *inv_freq;
    const int *positions;
    float eps;
    float k_factor, v_factor;  // 1 / scale
    int rotary;
    int q_heads;  // 0: no queries
    int parts;  // waves that share a token's heads
};

// cos and sin of position * f.  The product has up to 55 bits and is taken in two
// parts, exactly; turns are taken from it with 1 / (2 pi) in two parts, so that what
// is left of it, in [-1/2, 1/2] turns, is good to 2^-100 of the product's size in
// turns before it is rounded to float32.  (No contraction: hi - rint(hi) would become
// a fused product that has hi's rounding in it, which lo holds too.)
__device__ __forceinline__ void turned(int position, float f, float &c, float &s) {
#pragma clang fp contract(off)
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
    const double a = static_cast<double>(position) * static_cast<double>(f);
    const double hi = a * kHi;
    const double rest = fma(static_cast<double>(position), static_cast<double>(f), -a);
    const double lo = fma(rest, kHi, fma(a, kLo, fma(a, kHi, -hi)));
    const float r = static_cast<float>((hi - rint(hi)) + lo);
    sincospif(2.f * r, &s, &c);
}

// Four values rounded to the cache's type at element `at`.
template <int kType>
__device__ __forceinline__ void store_rounded(uint8_t *base, int64_t at, const float *x) {
    if constexpr (kType == Q4K_KV_E4M3) {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = x[i] != x[i] ? x[i] : fminf(fmaxf(x[i], -448.f), 448.f);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], w, true);
        *reinterpret_cast<int *>(base + at) = w;
    } else if constexpr (kType == Q4K_KV_F16) {
        half4v h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = static_cast<_Float16>(x[i]);
        *reinterpret_cast<half4v *>(base + 2 * at) = h;
    } else {
        bf4v h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = static_cast<__bf16>(x[i]);
        *reinterpret_cast<bf4v *>(base + 2 * at) = h;
    }
}

template <int kType, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void append_kernel(const Append a) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 63;
    const int D = p.head_dim, eighths = D / 8;
    const int spread = lanes_of(D);
    const int together = 64 / spread;                                                 // heads of a wave's pass
    const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    const int t = unit / a.parts, part = unit % a.parts;
    if (t >= p.tokens) return;
    const int b = last_started(p.count, t, [&](int i) { return offset_of(p, i); });
    const int first = offset_of(p, b), end = offset_of(p, b + 1);
    if (t < first || t >= end) return;
    const int64_t index = static_cast<int64_t>(p.lengths[b]) - end + t;
    const int64_t place = place_of(p, b, index, 0);
    const int position = a.positions ? a.positions[t] : static_cast<int>(index);
    const int e = lane & (spread - 1);  // which eight values of the head
    const bool here = e < eighths;
    // first dimensions of the lane's two fours
    int d0 = 8 * e, d1 = 8 * e + 4;
    const bool rotated = a.inv_freq && here && 8 * e < a.rotary;
    if (!kInterleaved && rotated) {
        d0 = 4 * e;
        d1 = 4 * e + a.rotary / 2;
    }
    float c[4], s[4];
    if (rotated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turned(position, a.inv_freq[4 * e + i], c[i], s[i]);
    }
    const int q_heads = a.q_heads, heads = q_heads + 2 * p.kv_heads;
    for (int g = part; g * together < heads; g += a.parts) {
        const int head = g * together + lane / spread;
        if (head >= heads) continue;
        const int what = head < q_heads ? 0 : head < q_heads + p.kv_heads ? 1 : 2;
        const int h = what == 0 ? head : what == 1 ? head - q_heads : head - q_heads - p.kv_heads;
        if (what != 0 && place < 0) continue;
        const int of = what == 0 ? q_heads : p.kv_heads;
        const float *src = (what == 0 ? a.q : what == 1 ? a.k : a.v) + (static_cast<size_t>(t) * of + h) * D;
        // the values of v are not rotated: their lane's fours may be any two
        float x[8];
        if (here) {
            *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(src + d0);
            *reinterpret_cast<float4 *>(x + 4) = *reinterpret_cast<const float4 *>(src + d1);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
        }
        const float *norm = what == 0 ? a.q_norm : what == 1 ? a.k_norm : nullptr;
        if (norm) {
            double sum = 0.;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
            for (int o = spread / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
            const Factor f(sum / D, a.eps);
            if (here) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = f.times(x[i]) * norm[d0 + i];
                    x[4 + i] = f.times(x[4 + i]) * norm[d1 + i];
                }
            }
        }
        if (!here) continue;
        if (what != 2 && rotated) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &u = kInterleaved ? x[2 * i] : x[i], &w = kInterleaved ? x[2 * i + 1] : x[4 + i];
                const float u1 = u * c[i] - w * s[i], w1 = w * c[i] + u * s[i];
                u = u1;
                w = w1;
            }
        }
        if (what == 0) {
            float *dst = a.q_out + (static_cast<size_t>(t) * q_heads + h) * D;
            *reinterpret_cast<float4 *>(dst + d0) = *reinterpret_cast<float4 *>(x);
            *reinterpret_cast<float4 *>(dst + d1) = *reinterpret_cast<float4 *>(x + 4);
        } else {
            const float scale = what == 1 ? a.k_factor : a.v_factor;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= scale;
            uint8_t *base = what == 1 ? p.k : p.v;
            const int64_t at = place + ((static_cast<int64_t>(h) * D) << p.shift);
            store_rounded<kType>(base, at + d0, x);
            store_rounded<kType>(base, at + d1, x + 4);
        }
    }
}

template <int kType>
hipError_t launch_append(const Append &a, bool interleaved, hipStream_t stream) {
    const int64_t waves = static_cast<int64_t>(a.p.tokens) * a.parts;
    const dim3 grid(static_cast<unsigned>((waves + kThreads / 64 - 1) / (kThreads / 64)));
    if (interleaved)
        hipLaunchKernelGGL((append_kernel<kType, true>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((append_kernel<kType, false>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_kv_append(const float *q, const float *k, const float *v, const q4k_kv_cache *cache,
                             const q4k_sequences *sequences, const q4k_rotation *rotation, float *q_out, int T,
                             int q_heads, hipStream_t stream) {
    using namespace q4k;
    Append a = {};
    if (q && q_heads < 1) return Q4K_ERR_BAD_DIM;
    if (!q) q_heads = 0;  // (not looked at)
    int rc = check_paged(cache, sequences, T, q_heads, &a.p);
    if (rc != Q4K_OK) return rc;
    if (rotation) {
        if (rotation->inv_freq && (rotation->rotary < 0 || rotation->rotary % 8 != 0 || rotation->rotary > cache->head_dim ||
                                   (rotation->interleaved != 0 && rotation->interleaved != 1)))
            return Q4K_ERR_BAD_DIM;
    }
    if (T == 0 || sequences->count == 0) return Q4K_OK;
    if (!k || !v || (q == nullptr) != (q_out == nullptr)) return Q4K_ERR_NULL;
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(q_out)) return Q4K_ERR_ALIGN;
    bool interleaved = false;
    if (rotation) {
        const q4k_rotation &r = *rotation;
        if (misaligned4(r.q_norm) || misaligned4(r.k_norm) || misaligned4(r.inv_freq) || misaligned4(r.positions))
            return Q4K_ERR_ALIGN;
        a.q_norm = r.q_norm;
        a.k_norm = r.k_norm;
        a.inv_freq = r.rotary > 0 ? r.inv_freq : nullptr;
        a.positions = r.positions;
        a.eps = r.eps;
        a.rotary = r.rotary;
        interleaved = r.interleaved != 0;
    }
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_heads = q_heads;
    a.k_factor = 1.f / cache->k_scale;
    a.v_factor = 1.f / cache->v_scale;
    // Waves for a token's heads: one for each pass over them while there are few
    // tokens; 8192 in all keep the memory busy (5200 tokens of 32 + 16 heads of 128 values:
    // 63 us with one wave a token, 57 with two), more only take the angles more often.
    const int spread = lanes_of(cache->head_dim);
    const int passes = (q_heads + 2 * cache->kv_heads + 64 / spread - 1) / (64 / spread);
    const int64_t parts = (8192 + static_cast<int64_t>(T) - 1) / T;
    a.parts = static_cast<int>(parts < passes ? parts : passes);
    if (static_cast<int64_t>(T) * a.parts * 64 + kThreads > UINT32_MAX) return Q4K_ERR_LAUNCH;
    hipError_t err;
    if (cache->type == Q4K_KV_F16) err = launch_append<Q4K_KV_F16>(a, interleaved, stream);
    else if (cache->type == Q4K_KV_BF16) err = launch_append<Q4K_KV_BF16>(a, interleaved, stream);
    else err = launch_append<Q4K_KV_E4M3>(a, interleaved, stream);
    return err == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}
