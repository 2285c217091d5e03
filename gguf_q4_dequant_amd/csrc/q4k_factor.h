// What a root-mean-square norm multiplies by, shared by the norm of rows and that of heads.
#pragma once

#include <hip/hip_runtime.h>

namespace q4k {

// 1 / sqrt(mean + eps) of a mean of squares, from double, as a fraction and a power of two:
// by itself it is beyond float32 for values below 2^-128 (without an eps) and a subnormal
// number for values above 2^126.
struct Factor {
    float fraction;
    int exponent;
    __device__ __forceinline__ Factor(double mean, float eps) {
        const double f = 1. / sqrt(mean + static_cast<double>(eps));
        exponent = __builtin_amdgcn_frexp_exp(f);
        fraction = static_cast<float>(__builtin_amdgcn_frexp_mant(f));
    }
    __device__ __forceinline__ float times(float x) const { return ldexpf(x, exponent) * fraction; }
};

}  // namespace q4k
