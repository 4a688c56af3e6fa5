// rope.cu -- rotary positions: y_a = a cos - b sin, y_b = a sin + b cos for
// every pair (a, b) of the rotated part of a head, angle = position * inverse
// frequency of the pair; the inverse rotation is the gradient.
//
// Memory bound: x is read and y written once.  A thread owns one 16-byte vector
// (interleaved layout) or one vector of each half (half layout) of a token, has
// the vector's cos and sin computed once, and walks over up to 8 heads with it,
// so the sine costs an eighth of a per-element evaluation (fewer heads a thread, for
// more threads, cost 12.3 us instead of 10.6 for 1,024 tokens x 128 heads x 64); neighbouring threads
// cover neighbouring vectors, then neighbouring heads, so every warp access is
// whole 128-byte lines when the heads are contiguous.  Measured: 65,536 tokens x 32
// heads x 128, bf16, 170 us (6.3 TB/s, 0.93 of a copy's rate).  x and y may be the same,
// so a thread's next load stays behind its last store: its eight heads are eight round
// trips in turn.  Where all threads fit the SMs at once (the 1,024 tokens above: 131,072
// threads, 2.1 MB in flight) these latencies, not the traffic's 5 us, are most of the time.
#include "kernels.h"
#include "latent.cuh"

namespace fs {

template <typename T>
struct Vec16 {      // 16 bytes of bf16 or fp32 as floats
    static constexpr int N = 16 / sizeof(T);
    float v[N];
    __device__ __forceinline__ void load(const T* p) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                v[2 * i] = bf16lo(u[i]);
                v[2 * i + 1] = bf16hi(u[i]);
            } else {
                v[i] = __uint_as_float(u[i]);
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            else u[i] = __float_as_uint(v[i]);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

constexpr int kRopeHeads = 8;    // heads a thread walks over

template <typename T, bool HALF>
__global__ void __launch_bounds__(256)
rope_kernel(const __grid_constant__ RopeTab tab, long long n, int groups, int hchunks, int H,
            const int32_t* __restrict__ pos, const T* x, long long x_row, long long x_head, T* y, long long y_row,
            long long y_head) {
    constexpr int N = Vec16<T>::N;
    const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (id >= n) return;
    const long long r = id / groups;
    const int g = static_cast<int>(id - r * groups);
    const long long t = r / hchunks;
    const int h0 = static_cast<int>(r - t * hchunks);
    const int p = __ldg(pos + t);
    constexpr int NF = HALF ? N : N / 2;         // pairs per thread
    float2 cs[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) cs[i] = rope_cs(tab.frac[g * NF + i], tab.mscale, tab.inverse, p);
    const T* xt = x + t * x_row + g * N;
    T* yt = y + t * y_row + g * N;
    const int half = tab.d_rot / 2;
#pragma unroll 4
    for (int h = h0; h < H; h += hchunks) {
        Vec16<T> a, b;
        a.load(xt + h * x_head);
        if constexpr (HALF) {
            b.load(xt + h * x_head + half);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float u = a.v[i], w = b.v[i];
                a.v[i] = u * cs[i].x - w * cs[i].y;
                b.v[i] = u * cs[i].y + w * cs[i].x;
            }
            b.store(yt + h * y_head + half);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float u = a.v[2 * i], w = a.v[2 * i + 1];
                a.v[2 * i] = u * cs[i].x - w * cs[i].y;
                a.v[2 * i + 1] = u * cs[i].y + w * cs[i].x;
            }
        }
        a.store(yt + h * y_head);
    }
}

cudaError_t launch_rope(const RopeTab& tab, bool f32, long long T, int H, const int32_t* pos, const void* x,
                        long long x_row, long long x_head, void* y, long long y_row, long long y_head,
                        cudaStream_t st) {
    const int N = f32 ? 4 : 8;
    const int groups = tab.d_rot / (tab.half ? 2 * N : N);
    const int hchunks = (H + kRopeHeads - 1) / kRopeHeads;
    const long long n = T * hchunks * groups;
    const long long blocks = (n + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
#define FS_ROPE(TY, HF)                                                                                             \
    rope_kernel<TY, HF><<<static_cast<unsigned>(blocks), 256, 0, st>>>(                                             \
        tab, n, groups, hchunks, H, pos, static_cast<const TY*>(x), x_row, x_head, static_cast<TY*>(y), y_row, y_head)
    if (f32) {
        if (tab.half) FS_ROPE(float, true); else FS_ROPE(float, false);
    } else {
        if (tab.half) FS_ROPE(__nv_bfloat16, true); else FS_ROPE(__nv_bfloat16, false);
    }
#undef FS_ROPE
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
