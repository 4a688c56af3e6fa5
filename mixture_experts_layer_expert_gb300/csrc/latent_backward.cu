// latent_backward.cu -- the gradient of expanded latent attention over packed sequences:
//   s_ij = scale (q_n,i . k_n,j + q_r,i . k_r,j),  out_i = sum_j softmax(s_i)_j v_j,  lse_i = log sum_j exp(s_ij)
//   p = exp(s - lse), dp = d_out . v, ds = scale p (dp - <d_out, out>)
//   dq = sum_j ds k, dk_n = sum_i ds q_n, dk_r = sum_heads sum_i ds q_r, dv = sum_i p d_out
#include <math_constants.h>

#include "kernels.h"
#include "latent.cuh"

namespace fs {

// Sequence of packed row t: cu[b] <= t < cu[b + 1]; -1 past the last one.
__device__ __forceinline__ int seq_of(const int32_t* cu, int B, int t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

struct Seq { int q0, q1, k0, k1; bool ok; };
__device__ __forceinline__ Seq seq_at(const LatentPrefillArgs& a, int b) {
    Seq s{a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1], true};
    s.ok = s.q0 >= 0 && s.q1 >= s.q0 && s.q1 <= a.Tq && s.k0 >= 0 && s.k1 >= s.k0 && s.k1 <= a.Tk;
    if (!s.ok) set_dev_error(a.err, DEV_ERR_OFFSETS);
    return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
template <int N>
__device__ __forceinline__ void ld_bf16(float (&v)[N], const __nv_bfloat16* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __bfloat162float(p[i]);
}
template <int N>
__device__ __forceinline__ float dot(const float (&x)[N], const float (&y)[N]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += x[i] * y[i];
    return s;
}
template <int N>
__device__ __forceinline__ void st_bf16(__nv_bfloat16* p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __float2bfloat16(v[i]);
}

// One warp per (query, head): out and lse (BWD = false) or dq (BWD = true).
// Lane l holds elements 4 l .. 4 l + 3 of the unrotated part and of v, 2 l and 2 l + 1 of the rotary part.
template <bool BWD>
__global__ void __launch_bounds__(128) prefill_query_kernel(LatentPrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (w >= static_cast<long long>(a.Tq) * a.H) return;
    const int t = static_cast<int>(w / a.H), h = static_cast<int>(w % a.H);
    const int b = seq_of(a.cu_q, a.B, t);
    if (b < 0) return;
    const Seq s = seq_at(a, b);
    if (!s.ok) return;
    const int end = a.causal ? min(s.k1, s.k1 - (s.q1 - t) + 1) : s.k1;
    float qn[4], qr[2], acc[4] = {}, accr[2] = {}, dO[4] = {};
    const __nv_bfloat16* q = a.q + t * a.q_row + h * a.q_head;
    ld_bf16(qn, q + 4 * lane);
    ld_bf16(qr, q + kNope + 2 * lane);
    float m = -CUDART_INF_F, z = 0.f, lse = 0.f, delta = 0.f;
    if constexpr (BWD) {
        float o[4];
        ld_bf16(dO, a.d_out + t * a.do_row + h * a.do_head + 4 * lane);
        ld_bf16(o, a.out + t * a.o_row + h * a.o_head + 4 * lane);
        delta = warp_sum(dot(dO, o));
        lse = a.lse[static_cast<long long>(h) * a.Tq + t];
    }
    for (int j = s.k0; j < end; ++j) {
        float kn[4], kr[2], v[4];
        ld_bf16(kn, a.kn + j * a.kn_row + h * a.kn_head + 4 * lane);
        ld_bf16(kr, a.kr + j * a.kr_row + 2 * lane);
        ld_bf16(v, a.v + j * a.v_row + h * a.v_head + 4 * lane);
        const float x = warp_sum(dot(qn, kn) + dot(qr, kr)) * a.scale;
        if constexpr (BWD) {
            const float ds = __expf(x - lse) * (warp_sum(dot(dO, v)) - delta) * a.scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += ds * kn[i];
#pragma unroll
            for (int i = 0; i < 2; ++i) accr[i] += ds * kr[i];
        } else {
            const float mn = fmaxf(m, x);
            if (mn == -CUDART_INF_F) continue;
            const float al = __expf(m - mn), p = __expf(x - mn);
            z = z * al + p;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = acc[i] * al + p * v[i];
            m = mn;
        }
    }
    if constexpr (BWD) {
        __nv_bfloat16* d = a.dq + t * a.dq_row + h * a.dq_head;
        st_bf16(d + 4 * lane, acc);
        st_bf16(d + kNope + 2 * lane, accr);
    } else {
        const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= inv;
        st_bf16(a.out_w + t * a.o_row + h * a.o_head + 4 * lane, acc);
        if (lane == 0) a.lse_w[static_cast<long long>(h) * a.Tq + t] = m + logf(z);
    }
}

// One warp per key: for every head, dk_n and dv; dk_r summed over the heads in order.
__global__ void __launch_bounds__(128) prefill_key_kernel(LatentPrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const long long j = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (j >= a.Tk) return;
    const int b = seq_of(a.cu_k, a.B, static_cast<int>(j));
    if (b < 0) return;
    const Seq s = seq_at(a, b);
    if (!s.ok) return;
    float kr[2], dkr[2] = {};
    ld_bf16(kr, a.kr + j * a.kr_row + 2 * lane);
    const int first = a.causal ? max(s.q0, s.q1 - (s.k1 - static_cast<int>(j))) : s.q0;
    for (int h = 0; h < a.H; ++h) {
        float kn[4], v[4], dkn[4] = {}, dv[4] = {};
        ld_bf16(kn, a.kn + j * a.kn_row + h * a.kn_head + 4 * lane);
        ld_bf16(v, a.v + j * a.v_row + h * a.v_head + 4 * lane);
        for (int t = first; t < s.q1; ++t) {
            float qn[4], qr[2], dO[4], o[4];
            const __nv_bfloat16* q = a.q + t * a.q_row + h * a.q_head;
            ld_bf16(qn, q + 4 * lane);
            ld_bf16(qr, q + kNope + 2 * lane);
            ld_bf16(dO, a.d_out + t * a.do_row + h * a.do_head + 4 * lane);
            ld_bf16(o, a.out + t * a.o_row + h * a.o_head + 4 * lane);
            const float x = warp_sum(dot(qn, kn) + dot(qr, kr)) * a.scale;
            const float p = __expf(x - a.lse[static_cast<long long>(h) * a.Tq + t]);
            const float ds = p * (warp_sum(dot(dO, v)) - warp_sum(dot(dO, o))) * a.scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) { dkn[i] += ds * qn[i]; dv[i] += p * dO[i]; }
#pragma unroll
            for (int i = 0; i < 2; ++i) dkr[i] += ds * qr[i];
        }
        st_bf16(a.dkn + j * a.dkn_row + h * a.dkn_head + 4 * lane, dkn);
        st_bf16(a.dv + j * a.dv_row + h * a.dv_head + 4 * lane, dv);
    }
    st_bf16(a.dkr + j * a.dkr_row + 2 * lane, dkr);
}

size_t latent_backward_ws_bytes(int, int, int) { return 256; }

cudaError_t launch_latent_backward(const LatentPrefillArgs& a, void*, cudaStream_t st) {
    const long long warps = static_cast<long long>(a.Tq) * a.H;
    prefill_query_kernel<true><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(a);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    prefill_key_kernel<<<static_cast<unsigned>((static_cast<long long>(a.Tk) + 3) / 4), 128, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
