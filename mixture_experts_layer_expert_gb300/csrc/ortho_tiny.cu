// ortho_tiny.cu -- orthogonalised updates of matrices whose shorter side is at
// most 16, in fp32 on the CUDA cores: all steps of a matrix in one launch.
//
// The mathematics is ortho.cu's.  With few rows a rounding of X X^T or of B to fp16 does not average
// out: it moves the few singular values themselves, and a result could be 0.6% off where bf16's own
// rounding leaves 0.17.  So nothing is rounded below fp32 here, and a matrix unit would be mostly idle.
// A cluster of C blocks holds a matrix, a thread one or two columns of X in registers.  Per step
//   every thread's 136 products x_i x_j, summed over a warp by halving (each exchange hands over half of the sums
//   that a lane still holds: 155 shuffles instead of 680), over the block's warps and then the blocks in rank order
//   A, then M = a 1 + b A + c A A, one element a thread;  X = M X, M's rows read as broadcasts.
// Bound by latency: some 2,000 instructions a warp and step and one exchange between blocks
// (16 x 4,000 23 us; with the 64-row tensor tiles of ortho_small.cu 38).
#include "common.cuh"
#include "kernels.h"
#include "ortho.cuh"

namespace fs {
namespace ortho {
namespace tiny {

constexpr int R = 16;
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int PAIRS = 160;                     // 136 pairs (i <= j), padded to five a lane
constexpr int MAX_CLUSTER = 16;

struct Args {
    Source src;
    __nv_bfloat16* out;
    long long out_row, out_mat;
    int r, q, tall, steps, batch;
    float scale, eps;
    float coefs[48];
};

__host__ __device__ constexpr int pair(int i, int j) { return i * R - i * (i - 1) / 2 + j - i; }

__device__ __forceinline__ void st_cluster_f32(const float* local, int cta, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_cta(smem_u32(local), cta)), "f"(v) : "memory");
}

// v[0 .. 2 H) of the lanes that differ in bit `o`: each keeps the sums of one half, the upper one if its bit is set.
template <int H>
__device__ __forceinline__ void halve(float (&v)[PAIRS], int lane, int o) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const float give = upper ? v[i] : v[i + H], keep = upper ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
}

template <int J>
__global__ void __launch_bounds__(THREADS, 1) tiny_kernel(const __grid_constant__ Args a) {
    __shared__ float sums[2][MAX_CLUSTER][PAIRS];      // by step's parity and rank: written by every block of the cluster
    __shared__ float norms[MAX_CLUSTER][4];
    __shared__ float part[WARPS][PAIRS];
    __shared__ float A[R][R + 1];
    __shared__ __align__(16) float M[R][R];
    __shared__ float factors[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t size;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
    const int C = static_cast<int>(size), rank = static_cast<int>(cluster_ctarank());
    const int ti = threadIdx.x / R, tj = threadIdx.x % R, my_pair = ti < tj ? pair(ti, tj) : pair(tj, ti);
    cudaGridDependencySynchronize();
    cluster_sync();                            // every block of the cluster runs before its memory is written

#pragma unroll 1
    for (int z = blockIdx.x / C; z < a.batch; z += gridDim.x / C) {
        float x[J][R];
        const size_t es = a.src.f32 ? 4 : 2;
        const uint8_t* g = static_cast<const uint8_t*>(a.src.g) + z * a.src.mat * es;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (rank * J + j) * THREADS + threadIdx.x;
            const long long first = a.tall ? c * a.src.row : c, step = a.tall ? 1 : a.src.row;
#pragma unroll
            for (int i = 0; i < R; ++i) x[j][i] = c < a.q && i < a.r ? at(a.src, g, first + i * step) : 0.0f;
        }
        {
            Squares sq;
#pragma unroll
            for (int j = 0; j < J; ++j) sq.add(x[j]);
            float v[3] = {sq.big, sq.mid, sq.small};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            }
            if (lane == 0) part[warp][0] = v[0], part[warp][1] = v[1], part[warp][2] = v[2];
            __syncthreads();
            if (threadIdx.x < 3) {
                float t = 0.0f;
                for (int w = 0; w < WARPS; ++w) t += part[w][threadIdx.x];
                for (int c = 0; c < C; ++c) st_cluster_f32(&norms[rank][threadIdx.x], c, t);
            }
            cluster_sync();
            if (threadIdx.x == 0) {
                double s[3] = {0.0, 0.0, 0.0};
                for (int c = 0; c < C; ++c)
                    for (int k = 0; k < 3; ++k) s[k] += norms[c][k];
                norm_factors(s[0], s[1], s[2], a.eps, 1.0f, &factors[0], &factors[1]);
            }
            __syncthreads();
        }
        const float n1 = factors[0], n2 = factors[1];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < R; ++i) x[j][i] = x[j][i] * n1 * n2;

#pragma unroll 1
        for (int k = 0; k < a.steps; ++k) {
            {
                float v[PAIRS];
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int l = i; l < R; ++l) {
                        float s = x[0][i] * x[0][l];
#pragma unroll
                        for (int j = 1; j < J; ++j) s += x[j][i] * x[j][l];
                        v[pair(i, l)] = s;
                    }
#pragma unroll
                for (int i = R * (R + 1) / 2; i < PAIRS; ++i) v[i] = 0.0f;
                halve<80>(v, lane, 16);
                halve<40>(v, lane, 8);
                halve<20>(v, lane, 4);
                halve<10>(v, lane, 2);
                halve<5>(v, lane, 1);          // lane l has the sums of pairs 5 l to 5 l + 4
#pragma unroll
                for (int i = 0; i < 5; ++i) part[warp][5 * lane + i] = v[i];
            }
            __syncthreads();
            float(*const mine)[PAIRS] = sums[k & 1];
            if (threadIdx.x < PAIRS) {
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) t += part[w][threadIdx.x];
                if (C == 1) mine[0][threadIdx.x] = t;
                else
                    for (int c = 0; c < C; ++c) st_cluster_f32(&mine[rank][threadIdx.x], c, t);
            }
            if (C == 1) __syncthreads();
            else cluster_sync();
            float s = 0.0f;
            for (int c = 0; c < C; ++c) s += mine[c][my_pair];
            A[ti][tj] = s;
            __syncthreads();
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) ss += A[ti][i] * A[tj][i];
            M[ti][tj] = a.coefs[3 * k + 1] * s + a.coefs[3 * k + 2] * ss + (ti == tj ? a.coefs[3 * k] : 0.0f);
            __syncthreads();
            float y[J][R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int j = 0; j < J; ++j) y[j][i] = 0.0f;
#pragma unroll
                for (int l = 0; l < R; l += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(&M[i][l]);
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        y[j][i] += m.x * x[j][l] + m.y * x[j][l + 1] + (m.z * x[j][l + 2] + m.w * x[j][l + 3]);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < R; ++i) x[j][i] = y[j][i];
        }
        uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + z * a.out_mat;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (rank * J + j) * THREADS + threadIdx.x;
            const long long first = a.tall ? c * a.out_row : c, step = a.tall ? 1 : a.out_row;
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (c < a.q && i < a.r) o[first + i * step] = static_cast<uint16_t>(pack_bf16x2(a.scale * x[j][i], 0.0f));
        }
        __syncthreads();                       // `part` and `factors` are the next matrix's
    }
    cluster_sync();                            // no block leaves while another may write its memory
}

}  // namespace tiny
}  // namespace ortho

// Columns a thread and blocks of a cluster for q columns; no blocks if the matrix is another kernel's.
static int tiny_cluster(int r, int q, int* per) {
    using namespace ortho::tiny;
    *per = q <= THREADS ? 1 : 2;
    if (r > R) return 0;
    int c = 1;
    while (c * *per * THREADS < q) c *= 2;
    return c <= MAX_CLUSTER ? c : 0;
}

bool ortho_tiny_fits(int m, int n) {
    int per;
    return tiny_cluster(m < n ? m : n, m < n ? n : m, &per) > 0;
}

template <int J>
static cudaError_t launch_tiny(const ortho::tiny::Args& a, int C, cudaStream_t st) {
    static bool wide[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && !wide[dev]) {
        e = cudaFuncSetAttribute(ortho::tiny::tiny_kernel<J>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        wide[dev] = true;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch < 152 / C ? a.batch : 152 / C) * C);
    cfg.blockDim = dim3(ortho::tiny::THREADS);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, ortho::tiny::tiny_kernel<J>, a);
    count_launch();
    return e;
}

cudaError_t launch_ortho_tiny(const OrthoArgs& o, cudaStream_t st) {
    ortho::tiny::Args a{};
    a.src = ortho::source(o, o.g);
    a.out = o.out;
    a.out_row = o.out_row;
    a.out_mat = o.out_mat;
    a.tall = o.m > o.n;
    a.r = a.tall ? o.n : o.m;
    a.q = a.tall ? o.m : o.n;
    a.steps = o.steps;
    a.batch = o.batch;
    a.scale = o.scale;
    a.eps = static_cast<float>(o.eps);
    for (int i = 0; i < 3 * o.steps; ++i) a.coefs[i] = o.coefs[i];
    int per = 0;
    const int C = tiny_cluster(a.r, a.q, &per);
    return per == 1 ? launch_tiny<1>(a, C, st) : launch_tiny<2>(a, C, st);
}

}  // namespace fs
