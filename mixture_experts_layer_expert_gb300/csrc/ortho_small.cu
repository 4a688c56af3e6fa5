// ortho_small.cu -- orthogonalised updates of matrices whose shorter side is at
// most 128: all steps of a matrix in one launch.
//
// The mathematics is ortho.cu's.  A cluster of C thread blocks holds one matrix: block c a
// slice of up to 256 columns of X, in fp32 registers (a row and 64 columns a thread) and as the
// fp16 operand H in shared memory.  Per step
//   the block's share of X X^T (tensor cores) -> summed over the cluster in rank order, each block
//   a band of rows -> A (fp16) in every block
//   B = b A + c A A in every block (the same bits), its diagonal kept apart in fp32
//   X = a X + B H for the block's columns.
// H serves both products where it lies: K-major for X X^T, MN-major for B H.  X never leaves the
// block, so it is carried in full fp32.  The shares go through the workspace, that is L2:
// distributed shared memory moves about 14 bytes a cycle and SM, and the exchange of a 128 x 128
// share took 11,000 cycles of a step that way.
// Bound by latency: three products of 900 to 1,400 cycles behind each other, the conversions between them
// (H 800, A 900, B 1,700, X 1,600 cycles of 128 x 256) and two cluster barriers a step; the gradient's way in takes
// 7,000 to 12,000 cycles.  8 of 256 x 128 34 us, 64 x 2,048 35 us, 128 x 4,096 56 us.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "ortho.cuh"

namespace fs {
namespace ortho {
namespace small {

constexpr int R = 128;                         // rows held (r <= R; the rest are zero)
constexpr int W = 256;                         // columns a block can hold
constexpr int THREADS = 512;                   // (256 threads with 128 columns each: 8 of 256 x 128 took 35 us, not 32)
constexpr int WARPS = THREADS / 32;
constexpr int XC = W / (WARPS / 4);            // columns of X a thread holds
constexpr int BLOCK = R * 64 * 2;              // 64 columns of fp16: the 128-byte-swizzle tile, 16 KB
constexpr int H_OFF = 0;
constexpr int A_OFF = H_OFF + (W / 64) * BLOCK;
constexpr int B_OFF = A_OFF + 2 * BLOCK;
constexpr int P_OFF = B_OFF + 2 * BLOCK;
constexpr int P_ROW = R + 4;                   // floats: 16-byte accesses of 8 rows fall into different banks
constexpr int SHARE = 2 * R * R * 4;           // bytes of a block's shares of X X^T in the workspace, two steps' in turn
constexpr int D_OFF = P_OFF + R * P_ROW * 4;   // fp32: B's diagonal
constexpr int N_OFF = D_OFF + R * 4;           // sums of squares of the cluster's blocks, 16 x 4 floats at most
constexpr int S_OFF = N_OFF + 16 * 16;         // of this block's warps, 4 floats each, then the two factors
constexpr int BAR_OFF = S_OFF + WARPS * 16 + 16;
constexpr size_t SMEM_BYTES = 1024 + BAR_OFF + 32;
constexpr int D_A = 0, D_AA = 128, D_X = 256;  // TMEM columns
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(H_OFF + R * P_ROW * 4 <= P_OFF, "the operands' room holds 128 columns of G");

struct Args {
    Source src;
    __nv_bfloat16* out;
    long long out_row, out_mat;
    int out_vec;
    int r, q, tall, steps, width;              // width: columns per block, a multiple of 64
    int rr, batch;                             // rr: r rounded up to 64
    uint8_t* ws;                               // per block a share, then per cluster A [rr][rr] fp16
    float scale, eps;
    OrthoScales sc;
    float fa, fb, fc, fx;                      // storage scales of A and its products: X to A, A to B, A A to B, B X to X
    float coefs[48];
    int* err;
};

// Element (row, col) of a [128][64 n] operand in swizzled tiles of 64 columns; `col` a multiple of 8: its 16-byte chunk.
__device__ __forceinline__ uint32_t chunk(int row, int col) {
    return (col >> 6) * BLOCK + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint4 v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ int cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return static_cast<int>(n);
}

__global__ void __launch_bounds__(THREADS, 1) small_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* dvec = reinterpret_cast<float*>(smem + D_OFF);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3, group = warp >> 2;
    const int row = quarter * 32 + lane;
    const int C = cluster_size(), rank = static_cast<int>(cluster_ctarank());
    const int cluster = blockIdx.x / C, clusters = gridDim.x / C;
    const int rr = a.rr, cols_a = rr / 4;                           // columns of A and B that a thread takes: 16 or 32
    float* share = reinterpret_cast<float*>(a.ws + static_cast<size_t>(blockIdx.x) * SHARE);
    const float* shares = reinterpret_cast<const float*>(a.ws + static_cast<size_t>(cluster) * C * SHARE);
    uint8_t* a_out = a.ws + static_cast<size_t>(gridDim.x) * SHARE + static_cast<size_t>(cluster) * (R * R * 2);
    const int col_first = rank * a.width + group * XC;              // this thread's first column of X
    const int ncol = min(XC, a.width - group * XC);                 // and how many it holds (64, or none: <= 0)

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(bar), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                          // every block of the cluster runs before its memory is written
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t idesc_sq = idesc_f16(R, rr, 0);
    const uint32_t idesc_x = idesc_f16(R, a.width, 1);
    uint32_t phase = 0;
    bool ok = true;          // after a wait that gave up the phases go on (the cluster's barriers have to match), unwaited
    auto finish_mma = [&]() {
        if (ok) ok = mbar_wait(smem_u32(bar), phase, abort_flag, a.err);
        phase ^= 1u;
        tc_fence_after();
    };

    // Line l of the block's part of G or of the result: 128 elements along a row of G, which is a row of X (two lines a row
    // if the block has more columns) or, of tall matrices, a column.
    float* P = reinterpret_cast<float*>(smem + P_OFF);
    float* P2 = reinterpret_cast<float*>(smem + H_OFF);
    struct Line {
        float* buf;
        long long row;
        int col;
    };
    const int per = a.tall ? 128 : rr, lines = a.tall ? a.width : rr * ((a.width + 127) >> 7);
    const auto line = [&](int l) {
        const int second = l >= per ? 1 : 0, i = l - second * per;
        const int c0 = rank * a.width;
        return Line{(second ? P2 : P) + i * P_ROW, a.tall ? c0 + l : i, a.tall ? 0 : c0 + 128 * second};
    };
    float* mine = (group < 2 ? P : P2) + (a.tall ? (group & 1) * XC * P_ROW + row : row * P_ROW + (group & 1) * XC);

#pragma unroll 1
    for (int z = cluster; z < a.batch; z += clusters) {
    // ---- the block's slice of G through two buffers of 128 columns (the share's and, before there are operands, theirs),
    // and the norm.  (Loops of a few instructions that read along G's rows: as straight code, each thread its own
    // columns, this took 7,000 cycles, most of them fetching instructions.)
    float x[XC];
#pragma unroll
    for (int c = 0; c < XC; ++c) x[c] = 0.0f;
    if (!a.tall && a.src.vec) {              // q is a multiple of a vector, so of 4
        const int c0 = rank * a.width;
        const size_t es = a.src.f32 ? 4 : 2;
        const uint8_t* g = static_cast<const uint8_t*>(a.src.g) + (z * a.src.mat + c0) * es;
        constexpr int U = 8;                 // loads in flight before the first store
#pragma unroll 1
        for (int l0 = warp; l0 < lines; l0 += U * WARPS) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int l = l0 + u * WARPS, r = l < rr ? l : l - rr, c = l < rr ? 0 : 128;
                const uint8_t* at_r = g + (static_cast<long long>(r) * a.src.row + c) * es;
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (l < lines && c0 + c + 4 * lane < a.q && r < a.r) {
                    if (a.src.f32) {
                        v[u] = reinterpret_cast<const float4*>(at_r)[lane];
                    } else {
                        const uint2 x = reinterpret_cast<const uint2*>(at_r)[lane];
                        v[u] = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int l = l0 + u * WARPS;
                if (l < lines) *reinterpret_cast<float4*>((l < rr ? P + l * P_ROW : P2 + (l - rr) * P_ROW) + 4 * lane) = v[u];
            }
        }
    } else
#pragma unroll 4
    for (int l = warp; l < lines; l += WARPS) {
        const Line ln = line(l);
        const int have = ln.row < (a.tall ? a.q : a.r) ? (a.tall ? a.r : a.q) - ln.col : 0;       // of 128 elements, G has
        const size_t es = a.src.f32 ? 4 : 2;
        const uint8_t* g = static_cast<const uint8_t*>(a.src.g) + (z * a.src.mat + ln.row * a.src.row + ln.col) * es;
        if (a.src.vec) {                     // `have` is a multiple of a vector, so of 4
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * lane < have) {
                if (a.src.f32) {
                    v = reinterpret_cast<const float4*>(g)[lane];
                } else {
                    const uint2 u = reinterpret_cast<const uint2*>(g)[lane];
                    v = make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
                }
            }
            *reinterpret_cast<float4*>(ln.buf + 4 * lane) = v;
        } else {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = lane + 32 * k < have ? at(a.src, g, lane + 32 * k) : 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) ln.buf[lane + 32 * k] = v[k];
        }
    }
    __syncthreads();
    if (ncol > 0 && row < rr) {
        if (a.tall) {
#pragma unroll
            for (int c = 0; c < XC; ++c) x[c] = mine[c * P_ROW];
        } else {
#pragma unroll
            for (int c = 0; c < XC; c += 4) {
                const float4 v = *reinterpret_cast<const float4*>(mine + c);
                x[c] = v.x; x[c + 1] = v.y; x[c + 2] = v.z; x[c + 3] = v.w;
            }
        }
    }
    Squares sq;
    sq.add(x);
    float* factors = reinterpret_cast<float*>(smem + S_OFF + WARPS * 16);
    {
        float v[3] = {sq.big, sq.mid, sq.small};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        }
        if (lane == 0) *reinterpret_cast<float4*>(smem + S_OFF + warp * 16) = make_float4(v[0], v[1], v[2], 0.f);
        __syncthreads();
        if (warp == 0) {                     // the block's sums to every block of the cluster, a lane each
            const float4 u = *reinterpret_cast<const float4*>(smem + S_OFF + (lane & 15) * 16);
            v[0] = u.x; v[1] = u.y; v[2] = u.z;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            }
            if (lane < C)
                st_cluster(map_to_cta(base + N_OFF + rank * 16, lane),
                           make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), 0u));
            __syncwarp();
        }
        cluster_sync();
        if (warp == 0) {
            const float4 u = lane < C ? *reinterpret_cast<const float4*>(smem + N_OFF + lane * 16) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = u.x; v[1] = u.y; v[2] = u.z;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            }
            if (lane == 0) norm_factors(v[0], v[1], v[2], a.eps, a.sc.x, &factors[0], &factors[1]);
        }
        __syncthreads();
    }
    {
        const float f1 = factors[0], f2 = factors[1];
#pragma unroll
        for (int c = 0; c < XC; ++c) x[c] = x[c] * f1 * f2;
    }

#pragma unroll 1
    for (int k = 0; k < a.steps; ++k) {
        const float ca = a.coefs[3 * k], cb = a.coefs[3 * k + 1], cc = a.coefs[3 * k + 2];
        // ---- H
#pragma unroll
        for (int c = 0; c < XC; c += 8) {
            if (c < ncol)
                *reinterpret_cast<uint4*>(smem + H_OFF + chunk(row, group * XC + c)) =
                    make_uint4(pack_half2(x[c], x[c + 1]), pack_half2(x[c + 2], x[c + 3]), pack_half2(x[c + 4], x[c + 5]),
                               pack_half2(x[c + 6], x[c + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        // ---- this block's share of X X^T.  (The products' loops are unrolled, with descriptors made outside the
        // election: of a loop left rolled, the second operand of B H lost the upper half of its descriptor.)
        if (warp == 0) {
            tc_fence_after();
            const uint64_t dh = smem_desc_sw128(base + H_OFF);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < W / 16; ++kk) {
                    const uint64_t d = dh + static_cast<uint64_t>((kk >> 2) * (BLOCK / 16) + 2 * (kk & 3));
                    if (16 * kk < a.width) tc_mma_bf16(tmem + D_A, d, d, idesc_sq, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(bar));
            }
            __syncwarp();
        }
        finish_mma();
        const float fa = a.fa;
        if (C == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (16 * h >= cols_a || row >= rr) break;
                uint32_t v[16];
                const int c0 = group * cols_a + h * 16;
                tmem_ld16_sync(taddr + D_A + c0, v);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t p[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        p[w] = pack_half2(fa * __uint_as_float(v[8 * q + 2 * w]), fa * __uint_as_float(v[8 * q + 2 * w + 1]));
                    *reinterpret_cast<uint4*>(smem + A_OFF + chunk(row, c0 + 8 * q)) = make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
        } else {
            float* prow = P + row * P_ROW;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (16 * h >= cols_a || row >= rr) break;
                uint32_t v[16];
                const int c0 = group * cols_a + h * 16;
                tmem_ld16_sync(taddr + D_A + c0, v);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4*>(prow + c0 + 4 * q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
            __syncthreads();
            // this step's half of the shares: a block may write its next one while another still reads
            const int turn = (k & 1) * R * R;
            const int vr = rr / 4, lg = rr == 64 ? 4 : 5;           // float4 per row, and its logarithm
            for (int i = threadIdx.x; i < rr * vr; i += THREADS)
                __stcg(reinterpret_cast<float4*>(share + turn) + i,
                       *reinterpret_cast<const float4*>(P + (i >> lg) * P_ROW + (i & (vr - 1)) * 4));
            cluster_sync();
            if (rr == 64 && C <= 8) {
                // small shares: every block sums them whole, without a second exchange (64 x 512 35 us, not 38; of
                // 128 rows 128 x 1,024 would take 76, not 59)
                for (int i = threadIdx.x; i < rr * vr; i += THREADS) {
                    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = 0; c < C; ++c) {
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(shares + turn + c * (SHARE / 4)) + i);
                        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
                    }
                    const int r = i >> lg, c0 = (i & (vr - 1)) * 4;
                    *reinterpret_cast<uint2*>(smem + A_OFF + chunk(r, c0 & ~7) + (c0 & 4) * 2) =
                        make_uint2(pack_half2(fa * t.x, fa * t.y), pack_half2(fa * t.z, fa * t.w));
                }
            } else {
                // rows [rank rr / C, ..) of A, four columns a thread, summed in rank order
                const int first = rank * (rr / C) * vr;
                for (int i = threadIdx.x; i < rr / C * vr; i += THREADS) {
                    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = 0; c < C; ++c) {
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(shares + turn + c * (SHARE / 4)) + first + i);
                        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
                    }
                    __stcg(reinterpret_cast<uint2*>(a_out) + first + i,
                           make_uint2(pack_half2(fa * t.x, fa * t.y), pack_half2(fa * t.z, fa * t.w)));
                }
                cluster_sync();
                for (int i = threadIdx.x; i < rr * rr / 8; i += THREADS) {
                    const int r = i >> (lg - 1), c0 = (i & (vr / 2 - 1)) * 8;
                    *reinterpret_cast<uint4*>(smem + A_OFF + chunk(r, c0)) = __ldcg(reinterpret_cast<const uint4*>(a_out) + i);
                }
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        // ---- B = b A + c A A
        if (warp == 0) {
            tc_fence_after();
            const uint64_t da = smem_desc_sw128(base + A_OFF);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < R / 16; ++kk) {
                    const uint64_t d = da + static_cast<uint64_t>((kk >> 2) * (BLOCK / 16) + 2 * (kk & 3));
                    if (16 * kk < rr) tc_mma_bf16(tmem + D_AA, d, d, idesc_sq, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(bar));
            }
            __syncwarp();
        }
        finish_mma();
        const float f1 = cb * a.fb, f2 = cc * a.fc;
        const auto make_b = [&](auto& v, auto load) {
            constexpr int N = sizeof(v) / 4;
            const int c0 = group * N;
            load(taddr + D_AA + c0, v);
            float on = 0.0f;
#pragma unroll
            for (int q = 0; q < N / 8; ++q) {
                const uint4 av = *reinterpret_cast<const uint4*>(smem + A_OFF + chunk(row, c0 + 8 * q));
                const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
                uint32_t p[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int c = 8 * q + 2 * w;
                    const float2 b = fma2(make_float2(f2, f2), make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                          mul2(make_float2(f1, f1), unpack_half2(aw[w])));
                    p[w] = pack_half2(b.x, b.y);
                    v[c] = __float_as_uint(b.x);
                    v[c + 1] = __float_as_uint(b.y);
                }
                *reinterpret_cast<uint4*>(smem + B_OFF + chunk(row, c0 + 8 * q)) = make_uint4(p[0], p[1], p[2], p[3]);
            }
            if ((c0 >> 5) == quarter) {          // the diagonal: in fp32 elsewhere, and zero in the product's operand
                const int diag = row - c0;
#pragma unroll
                for (int c = 0; c < N; ++c) on = c == diag ? __uint_as_float(v[c]) : on;
                if (diag >= 0 && diag < N) {
                    dvec[row] = on;
                    *reinterpret_cast<uint16_t*>(smem + B_OFF + chunk(row, row & ~7) + (row & 7) * 2) = 0;
                }
            }
        };
        if (rr == R) {
            uint32_t v[32];
            make_b(v, [](uint32_t t, uint32_t (&r)[32]) { tmem_ld32_sync(t, r); });
        } else if (row < rr) {
            uint32_t v[16];
            make_b(v, [](uint32_t t, uint32_t (&r)[16]) { tmem_ld16_sync(t, r); });
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        // ---- X = a X + B H
        if (warp == 0) {
            tc_fence_after();
            const uint64_t db = smem_desc_sw128(base + B_OFF), dh = smem_desc_sw128_mn(base + H_OFF, BLOCK);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < R / 16; ++kk) {
                    const uint64_t d = db + static_cast<uint64_t>((kk >> 2) * (BLOCK / 16) + 2 * (kk & 3));
                    if (16 * kk < rr) tc_mma_bf16(tmem + D_X, d, dh + 128ull * kk, idesc_x, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(bar));
            }
            __syncwarp();
        }
        const float d = row < rr ? dvec[row] : 0.0f, fx = a.fx;
        finish_mma();
#pragma unroll
        for (int c = 0; c < XC; c += 32) {
            if (c < ncol && quarter * 32 < rr) {
                uint32_t v[32];
                tmem_ld32_sync(taddr + D_X + group * XC + c, v);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 h = unpack_half2(pack_half2(x[c + j], x[c + j + 1]));
                    const float2 t = fma2(make_float2(d, d), h, make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
                    const float2 n = fma2(make_float2(fx, fx), t, mul2(make_float2(ca, ca), make_float2(x[c + j], x[c + j + 1])));
                    x[c + j] = n.x;
                    x[c + j + 1] = n.y;
                }
            }
        }
    }
    // ---- the result, by the same way back
    const float f = a.scale / a.sc.x;
    if (ncol > 0 && row < rr) {
        if (a.tall) {
#pragma unroll
            for (int c = 0; c < XC; ++c) mine[c * P_ROW] = f * x[c];
        } else {
#pragma unroll
            for (int c = 0; c < XC; c += 4)
                *reinterpret_cast<float4*>(mine + c) = make_float4(f * x[c], f * x[c + 1], f * x[c + 2], f * x[c + 3]);
        }
    }
    __syncthreads();
    if (!a.tall && a.out_vec && a.q % 4 == 0) {
        const int c0 = rank * a.width;
        uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + z * a.out_mat + c0;
#pragma unroll 4
        for (int l = warp; l < lines; l += WARPS) {
            const int r = l < rr ? l : l - rr, c = (l < rr ? 0 : 128) + 4 * lane;
            const float4 v = *reinterpret_cast<const float4*>((l < rr ? P : P2) + r * P_ROW + 4 * lane);
            if (r < a.r && c < a.width && c0 + c < a.q)
                *reinterpret_cast<uint2*>(o + static_cast<long long>(r) * a.out_row + c) =
                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
    } else
#pragma unroll 2
    for (int l = warp; l < lines; l += WARPS) {
        const Line ln = line(l);
        const int cols = a.tall ? a.r : min(a.width - (l < rr ? 0 : 128), a.q - ln.col);
        const int have = ln.row < (a.tall ? a.q : a.r) ? cols : 0;
        uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + z * a.out_mat + ln.row * a.out_row + ln.col;
        if (a.out_vec && 4 * lane + 4 <= have) {
            const float4 v = *reinterpret_cast<const float4*>(ln.buf + 4 * lane);
            *reinterpret_cast<uint2*>(o + 4 * lane) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        } else {
            const int step = a.out_vec ? 1 : 32;
#pragma unroll 1
            for (int c = a.out_vec ? 4 * lane : lane, n = 0; n < 4 && c < have; ++n, c += step)
                o[c] = static_cast<uint16_t>(pack_bf16x2(ln.buf[c], 0.0f));
        }
    }
    __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                          // no block leaves while another may read its memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace small
}  // namespace ortho

// Blocks of a cluster for q columns, 0 if the matrix does not fit one.
static int small_cluster(int r, int q) {
    if (r > ortho::small::R) return 0;
    int c = 1;
    while (c * ortho::small::W < q) c *= 2;
    return c <= 16 ? c : 0;                  // (16 blocks: more than the portable 8, asked for below)
}

bool ortho_small_fits(int m, int n) { return small_cluster(m < n ? m : n, m < n ? n : m) > 0; }

// Clusters in flight: as many as 152 SMs hold.
static int small_clusters(int batch, int C) { return batch < 152 / C ? batch : 152 / C; }

size_t ortho_small_ws_bytes(int batch, int m, int n) {
    const int C = small_cluster(m < n ? m : n, m < n ? n : m);
    if (C == 1) return 256;
    return static_cast<size_t>(small_clusters(batch, C)) * (C * ortho::small::SHARE + ortho::small::R * ortho::small::R * 2);
}

cudaError_t launch_ortho_small(const OrthoArgs& o, void* ws, cudaStream_t st) {
    using namespace ortho::small;
    using ortho::source;
    static bool set[kMaxDevices];
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(small_kernel), SMEM_BYTES, set);
    if (e != cudaSuccess) return e;
    static bool wide[kMaxDevices];
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && !wide[dev]) {
        e = cudaFuncSetAttribute(small_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        wide[dev] = true;
    }
    Args a{};
    a.src = source(o, o.g);
    a.out = o.out;
    a.out_row = o.out_row;
    a.out_mat = o.out_mat;
    a.out_vec = (reinterpret_cast<uintptr_t>(o.out) & 15u) == 0 && o.out_row % 8 == 0 && o.out_mat % 8 == 0;
    a.tall = o.m > o.n;
    a.r = a.tall ? o.n : o.m;
    a.q = a.tall ? o.m : o.n;
    a.steps = o.steps;
    a.scale = o.scale;
    a.eps = static_cast<float>(o.eps);
    a.sc = o.scales;
    a.fa = a.sc.a / (a.sc.x * a.sc.x);
    a.fb = a.sc.b / a.sc.a;
    a.fc = a.sc.b / (a.sc.a * a.sc.a);
    a.fx = 1.0f / a.sc.b;
    for (int i = 0; i < 3 * o.steps; ++i) a.coefs[i] = o.coefs[i];
    a.err = dev_error_ptr();
    a.ws = static_cast<uint8_t*>(ws);
    a.batch = o.batch;
    a.rr = (a.r + 63) / 64 * 64;
    const int C = small_cluster(a.r, a.q);
    a.width = ((a.q + C - 1) / C + 63) / 64 * 64;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(small_clusters(o.batch, C)) * C);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, small_kernel, a);
    count_launch();
    return e;
}

}  // namespace fs
