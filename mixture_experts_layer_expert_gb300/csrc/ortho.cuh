// ortho.cuh -- what the two forms of the orthogonalised update share: the gradient's
// operand, its norm, and fp16 helpers.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace fs {
namespace ortho {

// Instruction descriptor, kind::f16: fp32 accumulator, A and B fp16 (formats 0), B MN-major if b_mn.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

struct Source {
    const void* g;
    long long row, mat;        // strides in elements
    int m, n, f32, vec;        // vec: every row can be read in 16-byte vectors
};

inline Source source(const OrthoArgs& o, const void* g) {
    const size_t es = o.f32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(g) & 15u) == 0 && o.g_row * es % 16 == 0 && o.g_mat * es % 16 == 0 &&
                     o.n * es % 16 == 0;
    return Source{g, o.g_row, o.g_mat, o.m, o.n, o.f32, vec};
}

__device__ __forceinline__ float at(const Source& s, const void* base, long long i) {
    return s.f32 ? static_cast<const float*>(base)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

// Sums of squares over fp32's whole range: three partial sums, of values above 2^40 (scaled by
// 2^-88), below 2^-50 (by 2^100) and between, none of which can overflow or vanish.
struct Squares {
    float big = 0.f, mid = 0.f, small = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float a = fabsf(x);
        if (a > 0x1p40f) big += (x * 0x1p-88f) * (x * 0x1p-88f);
        else if (a < 0x1p-50f) small += (x * 0x1p100f) * (x * 0x1p100f);
        else mid += x * x;                     // a NaN lands here
    }
    // Several at once: squared as they are where none can overflow or matters below 2^-63, else range by range.
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N]) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
        if ((top >= 0x1p-40f && top <= 0x1p40f) || top == 0.0f) {
#pragma unroll
            for (int i = 0; i < N; ++i) mid += x[i] * x[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) add(x[i]);
        }
    }
};

// xscale / (norm + eps) as two fp32 factors, the first a power of two: no product with them leaves
// fp32's range on the way.  A matrix of zeros stays zero, one with a NaN or infinity becomes NaN.
__device__ __forceinline__ void norm_factors(double big, double mid, double small, double eps, float xscale, float* f1,
                                             float* f2) {
    // the usual case, without the slow 64-bit functions: 2^28 values below 2^-50 add at most 2^-72, 2^-28 of it
    if (big == 0.0 && mid > 0x1p-44 && mid < 0x1p80) {
        const float n = sqrtf(static_cast<float>(mid)) + static_cast<float>(eps);
        *f1 = 1.0f;
        *f2 = xscale / n;
        return;
    }
    const double norm = sqrt(big * 0x1p176 + mid + small * 0x1p-200) + eps;
    int e = 0;
    frexp(norm, &e);
    int k = -e;
    k = k < -126 ? -126 : (k > 127 ? 127 : k);
    const bool fine = norm > 0.0 && norm < INFINITY;
    *f1 = fine ? static_cast<float>(ldexp(1.0, k)) : (norm == 0.0 ? 0.0f : NAN);
    *f2 = fine ? static_cast<float>(xscale / (norm * ldexp(1.0, k))) : 1.0f;
}

}  // namespace ortho
}  // namespace fs
