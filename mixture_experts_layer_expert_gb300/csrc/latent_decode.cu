// latent_decode.cu -- absorbed latent attention of the newest tokens of each
// sequence over the paged latent cache:
//   s_i = scale (q_l . c_i + q_r . k_i),  out = sum_i softmax(s)_i c_i,  lse = log sum_i exp(s_i)
#include <math_constants.h>

#include "kernels.h"
#include "latent.cuh"

namespace fs {

// One warp per (query row, head), one pass over the sequence with the running
// maximum and sum; lane l holds latent elements [16 l, 16 l + 16) and rotary
// elements 2 l, 2 l + 1.
template <bool FP8>
__global__ void __launch_bounds__(128)
latent_decode_kernel(LatentDecodeArgs a) {
    const int lane = threadIdx.x & 31;
    const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const long long rows = static_cast<long long>(a.B) * a.n_q;
    if (w >= rows * a.H) return;
    const long long r = w / a.H;
    const int h = static_cast<int>(w - r * a.H);
    const int b = static_cast<int>(r / a.n_q), j = static_cast<int>(r - static_cast<long long>(b) * a.n_q);
    long long len = a.seq_lens[b];
    if (len < 0 || len > static_cast<long long>(a.max_pages) * a.page_size) {
        if (lane == 0) set_dev_error(a.err, DEV_ERR_PAGE);
        len = 0;
    }
    const int end = static_cast<int>(len) - (a.n_q - 1 - j);
    float q[16], qr[2], o[16];
    const __nv_bfloat16* ql = a.ql + r * a.ql_row + h * a.ql_head + 16 * lane;
    const __nv_bfloat16* qp = a.qr + r * a.qr_row + h * a.qr_head + 2 * lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) { q[i] = __bfloat162float(ql[i]); o[i] = 0.f; }
    qr[0] = __bfloat162float(qp[0]); qr[1] = __bfloat162float(qp[1]);
    float m = -CUDART_INF_F, z = 0.f;
    for (int i = 0; i < end; ++i) {
        const int page = a.table[b * a.table_row + i / a.page_size];
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) set_dev_error(a.err, DEV_ERR_PAGE);
            continue;
        }
        const uint8_t* rec = a.cache + (static_cast<long long>(page) * a.page_size + i % a.page_size) *
                                           (FP8 ? kRecFp8 : kRecBf16);
        float c[16], k[2], s = 0.f;
        if constexpr (FP8) {
            const float sc = *reinterpret_cast<const float*>(rec + kFp8ScaleOff);
            const uint4 v = *(reinterpret_cast<const uint4*>(rec) + lane);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = e4m3x2_to_bf16x2((u[e / 2] >> (16 * (e & 1))) & 0xffffu, sc);
                c[2 * e] = bf16lo(x); c[2 * e + 1] = bf16hi(x);
            }
        } else {
            const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(rec) + 16 * lane;
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = __bfloat162float(p[e]);
        }
        const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(rec + (FP8 ? kFp8RopeOff : 2 * kLatent)) + 2 * lane;
        k[0] = __bfloat162float(kp[0]); k[1] = __bfloat162float(kp[1]);
#pragma unroll
        for (int e = 0; e < 16; ++e) s += q[e] * c[e];
        s += qr[0] * k[0] + qr[1] * k[1];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        if (mn == -CUDART_INF_F) continue;
        const float al = __expf(m - mn), p = __expf(s - mn);
        z = z * al + p;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = o[e] * al + p * c[e];
        m = mn;
    }
    const float inv = z > 0.f ? 1.f / z : 0.f;
    __nv_bfloat16* op = a.out + r * a.o_row + h * a.o_head + 16 * lane;
#pragma unroll
    for (int e = 0; e < 16; ++e) op[e] = __float2bfloat16(o[e] * inv);
    if (a.lse && lane == 0) a.lse[r * a.H + h] = m + logf(z);
}

size_t latent_decode_ws_bytes(int, int, int) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void*, cudaStream_t st) {
    const long long warps = static_cast<long long>(a.B) * a.n_q * a.H;
    const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
    if (fp8) latent_decode_kernel<true><<<blocks, 128, 0, st>>>(a);
    else latent_decode_kernel<false><<<blocks, 128, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
