// Residual addition and root-mean-square norm (include/q4k_layer.h).
//
// One workgroup per row: its first kThreads * kHold * 4 = 4096 values are read once
// and kept in registers, the sum of squares is taken in double, and the row is
// written once.  What a longer row has behind them is read a second time (of 5120
// values the last 1024, from the L2).  Memory bounds it: 4096 rows of 5120 (336 MB)
// 67.5 us, 5.0 TB/s; one row of 2048 2.9 us, a launch's own time.
#include <math.h>

#include "../../include/q4k_layer.h"
#include "q4k_factor.h"
#include "q4k_internal.h"

namespace q4k {
namespace {

typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));  // rows of odd N start anywhere

constexpr int kHold = 4;  // vectors of four that a thread keeps

// The four values at i of a row of N, zero behind its end.
__device__ __forceinline__ float4u load4(const float *row, int i, int N) {
    if (i + 4 <= N) return *reinterpret_cast<const float4u *>(row + i);
    float4u v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < N) v[k] = row[i + k];
    return v;
}

__device__ __forceinline__ void store4(float *row, int i, int N, float4u v) {
    if (i + 4 <= N) {
        *reinterpret_cast<float4u *>(row + i) = v;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < N) row[i + k] = v[k];
}

__device__ __forceinline__ double squares(float4u v) {
    double s = 0.;
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fma(static_cast<double>(v[k]), static_cast<double>(v[k]), s);
    return s;
}

// total may be x or residual and y may be x or residual: every value is read
// by the thread that writes it, before it does.
template <int kThreads>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(const float *x, const float *residual, const float *weight,
                                                            float eps, float *total, float *y, int N) {
    __shared__ double sums[kThreads / 64];
    const size_t at = static_cast<size_t>(blockIdx.x) * N;
    const float *xr = x + at, *rr = residual ? residual + at : nullptr;
    float *tr = total ? total + at : nullptr, *yr = y + at;
    const int first = threadIdx.x * 4;
    constexpr int kStep = kThreads * 4;
    float4u h[kHold];
    double sum = 0.;
#pragma unroll
    for (int j = 0; j < kHold; ++j) h[j] = load4(xr, first + j * kStep, N);
    if (rr) {
#pragma unroll
        for (int j = 0; j < kHold; ++j) h[j] += load4(rr, first + j * kStep, N);
    }
#pragma unroll
    for (int j = 0; j < kHold; ++j) sum += squares(h[j]);
    for (int64_t i = first + static_cast<int64_t>(kHold) * kStep; i < N; i += kStep) {
        float4u v = load4(xr, static_cast<int>(i), N);
        if (rr) v += load4(rr, static_cast<int>(i), N);
        sum += squares(v);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (kThreads > 64) {
        if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0.;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) sum += sums[w];
    }
    const Factor f(sum / N, eps);
    const auto finish = [&](int i, float4u v) {
        if (tr) store4(tr, i, N, v);
        const float4u w = load4(weight, i, N);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = f.times(v[k]);
        store4(yr, i, N, v * w);
    };
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (first + j * kStep < N) finish(first + j * kStep, h[j]);
    for (int64_t i = first + static_cast<int64_t>(kHold) * kStep; i < N; i += kStep) {
        float4u v = load4(xr, static_cast<int>(i), N);
        if (rr) v += load4(rr, static_cast<int>(i), N);
        finish(static_cast<int>(i), v);
    }
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace
}  // namespace q4k

extern "C" int q4k_rms_norm(const float *x, const float *residual, const float *weight, float eps, float *total,
                            float *y, int M, int N, hipStream_t stream) {
    using namespace q4k;
    if (M < 0 || N < 0 || N > 1 << 30) return Q4K_ERR_BAD_DIM;
    if (M == 0 || N == 0) return Q4K_OK;
    if (!x || !weight || !y) return Q4K_ERR_NULL;
    if (misaligned4(x) || misaligned4(residual) || misaligned4(weight) || misaligned4(total) || misaligned4(y))
        return Q4K_ERR_ALIGN;
    const int rc = check_device();
    if (rc != Q4K_OK) return rc;
    if (M >= 1 << 24) return Q4K_ERR_LAUNCH;
    hipLaunchKernelGGL((rms_norm_kernel<256>), dim3(M), dim3(256), 0, stream, x, residual, weight, eps, total, y, N);
    return hipGetLastError() == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}
