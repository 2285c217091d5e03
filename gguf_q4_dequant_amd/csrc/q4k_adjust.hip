// Penalties for repeated tokens, biases and grammar masks on logits, and the
// greedy choice under them (include/q4k_select.h).
//
// One workgroup per chunk of one row.  The chunk's counts of history tokens
// are gathered in LDS, its biases in an ordered LDS list, both from the row's
// two short lists (every workgroup of a row reads them whole; they stay in the
// L2), so the logits are read once and written once and no [M, N] table of
// counts or biases ever exists.  The kernel is bound by that one pass over the
// logits: 96 x 128256 under a history of 4096, 64 biases and a mask 23.5 us,
// 102 MB at 4.3 TB/s; the choice over 32 x 151936 (history 1024, 16 biases,
// mask; 20 MB) 9 us and 2 us for the second launch, which joins the chunks; one
// row of 128256 6 us.  (One workgroup per row and no second launch: 24 us for
// that row, since one CU streams only about 25 GB/s.)  Counts are integers (LDS
// atomics in any order give the same); the biases of a token named more than
// once are added in list order by the thread that holds its logit.
#include <limits.h>
#include <math.h>

#include "../../include/q4k_select.h"
#include "q4k_internal.h"

namespace q4k {
namespace {

constexpr int kThreads = 256;
constexpr int kBiases = 512;  // biases looked through at a time
constexpr int kMaxList = 1 << 30;  // places in a list and one step behind its end stay in an int

typedef int int4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));  // rows of odd N start anywhere

__device__ __forceinline__ void take_better(float &v, int &i, float v2, int i2) {
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

__device__ __forceinline__ void wave_best(float &v, int &i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float v2 = __shfl_xor(v, o);
        const int i2 = __shfl_xor(i, o);
        take_better(v, i, v2, i2);
    }
}

// The definition's operations with a rounding each (no fused multiply-add),
// so that the result is the one the header states, bit for bit.
__device__ __forceinline__ float penalised(float z, float count, float rep, float freq, float pres) {
#pragma clang fp contract(off)
    const float t = z > 0.f ? z / rep : z * rep;
    const float f = freq * count;
    return (t - f) - pres;
}

// kPer logits per thread: chunks of kThreads * kPer.  kSelect: the chunk's
// best (value, index) pair goes to part, else the adjusted logits to out.
// out may be logits itself: every logit is read and written by one thread.
template <int kPer, bool kSelect>
__global__ __launch_bounds__(kThreads) void adjust_kernel(const float *logits, float *out, q4k_adjustment a, int N,
                                                          int chunks, float *part) {
    constexpr int kChunk = kThreads * kPer;
    __shared__ __align__(16) int counts[kChunk];
    __shared__ float2 list[kBiases];  // (place in the chunk, value)
    __shared__ int listed;
    const int tid = threadIdx.x, c = blockIdx.x;
    const size_t m = blockIdx.y;
    const int n0 = c * kChunk, n_here = min(kChunk, N - n0);
    const float *row = logits + m * N + n0;
    float z[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
        const int i = (j * kThreads / 4 + tid) * 4;
        if (i + 4 <= n_here) {
            const float4u v = *reinterpret_cast<const float4u *>(row + i);
            z[j] = v.x;
            z[j + 1] = v.y;
            z[j + 2] = v.z;
            z[j + 3] = v.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) z[j + k] = i + k < n_here ? row[i + k] : 0.f;
        }
    }
    if (a.history_len > 0) {
#pragma unroll
        for (int j = 0; j < kPer; j += 4) *reinterpret_cast<int4 *>(&counts[(j * kThreads / 4 + tid) * 4]) = int4{0, 0, 0, 0};
        __syncthreads();
        const int *ids = a.history + m * a.history_len;
        const auto count = [&](int id) {
            // negative ids wrap to far above any chunk
            const unsigned at = static_cast<unsigned>(id) - static_cast<unsigned>(n0);
            if (at < static_cast<unsigned>(n_here)) atomicAdd(&counts[at], 1);
        };
        const int fours = a.history_len / 4;
        for (int i = tid; i < fours; i += kThreads) {
            const int4u v = *reinterpret_cast<const int4u *>(ids + 4 * i);
            count(v.x);
            count(v.y);
            count(v.z);
            count(v.w);
        }
        if (tid < a.history_len - 4 * fours) count(ids[4 * fours + tid]);
        __syncthreads();
        const float rep = a.repetition ? a.repetition[m] : 1.f;
        const float freq = a.frequency ? a.frequency[m] : 0.f;
        const float pres = a.presence ? a.presence[m] : 0.f;
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            const int4 c4 = *reinterpret_cast<const int4 *>(&counts[(j * kThreads / 4 + tid) * 4]);
            const int n[4] = {c4.x, c4.y, c4.z, c4.w};
            if ((c4.x | c4.y | c4.z | c4.w) != 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n[k] > 0) z[j + k] = penalised(z[j + k], static_cast<float>(n[k]), rep, freq, pres);
            }
        }
    }
    if (a.bias_len > 0) {
        const int *bid = a.bias_id + m * a.bias_len;
        const float *bval = a.bias_value + m * a.bias_len;
        float sum[kPer];
        uint32_t named = 0;  // bit j: logit j of this thread has a bias
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = 0.f;
        for (int first = 0; first < a.bias_len; first += kBiases) {
            __syncthreads();  // the list of the round before has been read
            if (tid < 64) {   // one wave packs the chunk's entries in list order
                int found = 0;
                const int end = min(a.bias_len, first + kBiases);
                for (int i = first; i < end; i += 64) {
                    const int id = i + tid < end ? bid[i + tid] : -1;
                    const unsigned at = static_cast<unsigned>(id) - static_cast<unsigned>(n0);
                    const bool here = at < static_cast<unsigned>(n_here);
                    const uint64_t with = __ballot(here);
                    if (here) list[found + __builtin_popcountll(with & ((1ull << tid) - 1))] = float2{__uint_as_float(at), bval[i + tid]};
                    found += __builtin_popcountll(with);
                }
                if (tid == 0) listed = found;
            }
            __syncthreads();
            for (int h = 0; h < listed; ++h) {
                const unsigned at = __float_as_uint(list[h].x);
                if (((at >> 2) & (kThreads - 1)) != static_cast<unsigned>(tid)) continue;
                const float value = list[h].y;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (at == static_cast<unsigned>(((j & ~3) * kThreads / 4 + tid) * 4 + (j & 3))) {
                        sum[j] += value;
                        named |= 1u << j;
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if ((named >> j) & 1u) z[j] += sum[j];
    }
    uint32_t allowed = 0xFFFFFFFFu;  // bit j: logit j of this thread
    if (a.mask) {
        const unsigned *mask = a.mask + m * ((static_cast<size_t>(N) + 31) / 32) + n0 / 32;
        allowed = 0;
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            const int i = (j * kThreads / 4 + tid) * 4;
            const uint32_t word = i < n_here ? mask[i >> 5] : 0u;
            allowed |= ((word >> (i & 31)) & 15u) << j;
        }
    }
    if constexpr (!kSelect) {
        float *o = out + m * N + n0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (!((allowed >> j) & 1u)) z[j] = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            const int i = (j * kThreads / 4 + tid) * 4;
            if (i + 4 <= n_here) {
                *reinterpret_cast<float4u *>(o + i) = float4u{z[j], z[j + 1], z[j + 2], z[j + 3]};
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k < n_here) o[i + k] = z[j + k];
            }
        }
    } else {
        __shared__ float sv[kThreads / 64];
        __shared__ int si[kThreads / 64];
        float v = -INFINITY;
        int best = INT_MAX;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = ((j & ~3) * kThreads / 4 + tid) * 4 + (j & 3);
            if (((allowed >> j) & 1u) && i < n_here) take_better(v, best, z[j], n0 + i);
        }
        wave_best(v, best);
        if ((tid & 63) == 0) {
            sv[tid >> 6] = v;
            si[tid >> 6] = best;
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kThreads / 64; ++w) take_better(v, best, sv[w], si[w]);
            float *o = part + (m * chunks + c) * 2;
            o[0] = v;
            o[1] = __int_as_float(best);
        }
    }
}

__global__ __launch_bounds__(64) void select_rows(const float *part, int chunks, int *index, float *value) {
    const size_t m = blockIdx.x;
    float v = -INFINITY;
    int i = INT_MAX;
    for (int c = threadIdx.x; c < chunks; c += 64) {
        const float *p = part + (m * chunks + c) * 2;
        take_better(v, i, p[0], __float_as_int(p[1]));
    }
    wave_best(v, i);
    if (threadIdx.x == 0) {
        index[m] = i == INT_MAX ? -1 : i;
        if (value) value[m] = v;
    }
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

int check_adjustment(const q4k_adjustment *a, int M, int N) {
    if (M < 0 || N < 0) return Q4K_ERR_BAD_DIM;
    if (!a) return Q4K_ERR_NULL;
    if (a->history_len < 0 || a->bias_len < 0 || a->history_len > kMaxList || a->bias_len > kMaxList)
        return Q4K_ERR_BAD_DIM;
    if ((a->history_len > 0 && !a->history) || (a->bias_len > 0 && (!a->bias_id || !a->bias_value))) return Q4K_ERR_NULL;
    if (misaligned4(a->history) || misaligned4(a->repetition) || misaligned4(a->frequency) ||
        misaligned4(a->presence) || misaligned4(a->bias_id) || misaligned4(a->bias_value) || misaligned4(a->mask))
        return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

constexpr int kSmallPer = 4, kLargePer = 16;

// Chunks of 1024 logits give one row enough workgroups; with many rows the
// larger ones read the lists less often.
int per_thread(int M, int N) { return static_cast<int64_t>(M) * N <= (1 << 20) ? kSmallPer : kLargePer; }

template <bool kSelect>
hipError_t launch_adjust(const float *logits, float *out, const q4k_adjustment &a, int M, int N, float *part,
                         hipStream_t stream) {
    const int per = per_thread(M, N), chunk = kThreads * per, chunks = (N - 1) / chunk + 1;
    const dim3 grid(chunks, M);
    if (per == kSmallPer)
        hipLaunchKernelGGL((adjust_kernel<kSmallPer, kSelect>), grid, dim3(kThreads), 0, stream, logits, out, a, N,
                           chunks, part);
    else
        hipLaunchKernelGGL((adjust_kernel<kLargePer, kSelect>), grid, dim3(kThreads), 0, stream, logits, out, a, N,
                           chunks, part);
    return hipGetLastError();
}

size_t select_partials(int M, int N) {
    return static_cast<size_t>(M) * ((N - 1) / (kThreads * per_thread(M, N)) + 1);
}

// The choice over logits already in memory; part has room for select_partials pairs.
int run_select(const float *logits, const q4k_adjustment &a, int M, int N, float *part, int *index, float *value,
               hipStream_t stream) {
    if (launch_adjust<true>(logits, nullptr, a, M, N, part, stream) != hipSuccess) return Q4K_ERR_LAUNCH;
    const int chunks = static_cast<int>(select_partials(M, N) / M);
    hipLaunchKernelGGL(select_rows, dim3(M), dim3(64), 0, stream, part, chunks, index, value);
    return hipGetLastError() == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_logits_adjust(const float *logits, float *out, const q4k_adjustment *adjustment, int M, int N,
                                 hipStream_t stream) {
    using namespace q4k;
    int rc = check_adjustment(adjustment, M, N);
    if (rc != Q4K_OK || M == 0 || N == 0) return rc;
    if (!logits || !out) return Q4K_ERR_NULL;
    if (misaligned4(logits) || misaligned4(out)) return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    if (M > 65535) return Q4K_ERR_LAUNCH;
    return launch_adjust<false>(logits, out, *adjustment, M, N, nullptr, stream) == hipSuccess ? Q4K_OK
                                                                                               : Q4K_ERR_LAUNCH;
}

extern "C" int q4k_logits_argmax(const float *logits, const q4k_adjustment *adjustment, int M, int N, int *index,
                                 float *value, hipStream_t stream) {
    using namespace q4k;
    int rc = check_adjustment(adjustment, M, N);
    if (rc != Q4K_OK || M == 0) return rc;
    if (N == 0) return Q4K_ERR_BAD_DIM;
    if (!logits || !index) return Q4K_ERR_NULL;
    if (misaligned4(logits) || misaligned4(index) || misaligned4(value)) return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    if (M > 65535) return Q4K_ERR_LAUNCH;
    float *part = nullptr;
    if (workspace(stream, select_partials(M, N) * 2 * sizeof(float), &part, 1) != hipSuccess) return Q4K_ERR_ALLOC;
    return run_select(logits, *adjustment, M, N, part, index, value, stream);
}

extern "C" int q4k_matmul_argmax_adjusted(const void *w_packed, const float *x, const q4k_adjustment *adjustment,
                                          int M, int N, int K, int *index, float *value, hipStream_t stream) {
    using namespace q4k;
    int rc = check_adjustment(adjustment, M, N);
    if (rc != Q4K_OK) return rc;
    if (K < 0) return Q4K_ERR_BAD_DIM;
    if (M == 0) return Q4K_OK;
    if (N == 0 || K == 0 || K % kBlockWeights != 0) return Q4K_ERR_BAD_DIM;
    if (!w_packed || !x || !index) return Q4K_ERR_NULL;
    if (((reinterpret_cast<uintptr_t>(w_packed) | reinterpret_cast<uintptr_t>(x)) & 15u) != 0 || misaligned4(index) ||
        misaligned4(value))
        return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    if (M > 65535) return Q4K_ERR_LAUNCH;
    // Logits, then the (value, index) pairs, in workspace slot 1 (the product uses slot 0).
    const size_t logits = (static_cast<size_t>(M) * N + 3) & ~static_cast<size_t>(3);
    float *ws = nullptr;
    if (workspace(stream, (logits + 2 * select_partials(M, N)) * sizeof(float), &ws, 1) != hipSuccess)
        return Q4K_ERR_ALLOC;
    rc = q4k_matmul(w_packed, x, ws, M, N, K, stream);
    if (rc != Q4K_OK) return rc;
    return run_select(ws, *adjustment, M, N, ws + logits, index, value, stream);
}
