// gemm_mx.cuh -- what the single-CTA and the CTA-pair GEMM on block-scaled operands
// share: arguments, tile order, scale copies and the epilogues.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace fs {
namespace mx {

constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int PIECE_BYTES = 2048;
constexpr int kGroupM = 16;

struct Args {
    const int* plan;          // E4M3: [2 (G + 1)]: m-tile prefix, row starts (multiples of 128)
    const int* offsets;       // E2M1: [G + 1] row starts on the device, or null: one group of `rows` rows
    int G, rows, N, K, n_tiles, max_mtiles;
    const uint8_t* a_sf;      // A scale chunks [rows128 / 128][K / 128][512]
    const uint8_t* b_sf;      // B scale chunks [G][n_tiles][K / 128][1024]
    void* out;
    long long ldo;            // output row stride (elements)
    int out_cols;
    uint8_t* h_sf;            // EPI_SWIGLU: scale chunks of the MX hidden out (codes at out, row stride ldo bytes)
    int tma_out;
    int* err;
};

// Instruction descriptor: B scale byte (bits 4-5), A and B formats (bits 7-9,
// 10-12: 0 = E4M3 of kind::mxf8f6f4, 1 = E2M1 of kind::mxf4), K-major, N >> 3
// (17-22), UE8M0 scales (bit 23), M >> 4 (24-28), A scale byte (29-30).
template <bool F4>
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, int sf_id) {
    return (static_cast<uint32_t>(sf_id) << 4) | (F4 ? (1u << 7) | (1u << 10) : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) |
           (static_cast<uint32_t>(sf_id) << 29);
}

// SiLU(g) u of two columns as bf16, in some ten instructions a value: this epilogue's code is run
// once a tile, and with few rows by one warp, at the rate at which instructions are fetched (with
// silu_f's division and exponential the 64 values of a thread took 24,000 cycles then, and the gate/up
// product of 61 tokens over 64 experts 86 us instead of 36).
// g / (1 + 2^(-g log2 e)) with the approximate exponential and reciprocal (2 units of 2^-23 each).
__device__ __forceinline__ float swiglu_fast(uint32_t gate, uint32_t up) {
    const float g = __uint_as_float(gate);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * __uint_as_float(up);
}
__device__ __forceinline__ uint32_t swiglu_pair(uint32_t g0, uint32_t u0, uint32_t g1, uint32_t u1) {
    return pack_bf16x2(swiglu_fast(g0, u0), swiglu_fast(g1, u1));
}

struct Tile {
    int g, m, n, a_row, rows_valid;
};

template <int BM>
__device__ __forceinline__ Tile decode(int t, const int* mt_start, const int* row_start, int G, int n_tiles) {
    const int q = t / n_tiles;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (mt_start[mid] <= q) lo = mid; else hi = mid;
    }
    Tile r;
    r.g = lo;
    const int mtiles = mt_start[lo + 1] - mt_start[lo];
    const int local = t - mt_start[lo] * n_tiles;
    const int GM = mtiles <= 2 * kGroupM ? mtiles : kGroupM;
    const int blk = local / (GM * n_tiles);
    const int gm = min(GM, mtiles - blk * GM);
    const int rr = local - blk * GM * n_tiles;
    r.n = rr / gm;
    r.m = blk * GM + (rr - r.n * gm);
    r.a_row = row_start[lo] + r.m * BM;
    const int rem = row_start[lo + 1] - r.a_row;
    r.rows_valid = rem < BM ? rem : BM;
    return r;
}

// E2M1: m-tile prefix and row starts of the groups in shared memory, from their offsets, by all threads of a block (its
// own plan a block, instead of a launch before the products).  Offsets that are not increasing inside [0, rows] give no tiles.
template <int BM>
__device__ __forceinline__ void make_plan(const Args& args, int* mt_start, int* row_start) {
    __shared__ int sums[THREADS / 32];
    constexpr int PER = 2;                     // groups a thread: 640 of kMaxExperts
    static_assert(THREADS * PER >= kMaxExperts, "groups");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = args.G;
    int tiles[PER], bad = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = threadIdx.x * PER + i;
        tiles[i] = 0;
        if (g < G) {
            const int a = args.offsets ? args.offsets[g] : 0, b = args.offsets ? args.offsets[g + 1] : args.rows;
            bad |= a < 0 || b < a || b > args.rows;
            row_start[g] = a;
            if (g == G - 1) row_start[G] = b;
            tiles[i] = bad ? 0 : (b - a + BM - 1) / BM;
        }
    }
    int run = tiles[0] + tiles[1];
    const int mine = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += n;
    }
    if (lane == 31) sums[warp] = run;
    bad = __syncthreads_or(bad);
    int before = run - mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = threadIdx.x * PER + i;
        if (g < G) mt_start[g] = bad ? 0 : before;
        before += tiles[i];
        if (g == G - 1) mt_start[G] = bad ? 0 : before;
    }
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_dev_error(args.err, DEV_ERR_OFFSETS);
}

// One piece of 32 rows x 64 bytes (32 bf16 or 16 fp32 columns) through the warp's staging buffer and a TMA store.
__device__ __forceinline__ void store_piece(const CUtensorMap* tmo, uint8_t* piece, const uint32_t* pk, int lane, int x,
                                            int y) {
    if (lane == 0) bulk_wait_read0();
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int sw = q ^ ((lane >> 1) & 3);
        *reinterpret_cast<uint4*>(piece + lane * 64 + sw * 16) =
            make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(tmo, smem_u32(piece), x, y);
        bulk_commit();
    }
}

// The epilogue of a warp's 32 rows (this thread's: row r of the tile's rows from a_row on) and HALF columns of column
// tile n, from the accumulator copied to v.
template <int EPI, bool F4, int HALF>
__device__ __forceinline__ void epilogue(const uint32_t (&v)[HALF], const Args& args, const CUtensorMap* tmO, int n, int half,
                                         int a_row, int rows_valid, int r, uint8_t* piece) {
    const bool row_ok = r < rows_valid;
    const long long orow = static_cast<long long>(a_row) + r;
    const int lanew = r & 31, q32 = r & ~31;
    const bool piece_ok = args.tma_out && q32 + 32 <= rows_valid;
    if constexpr (EPI == EPI_SWIGLU) {
        // packed columns of this half: gate 64 | up 64 -> hidden columns
        // 128 n + 64 half + [0, 64), two blocks of 32
        const int hc0 = n * 128 + half * 64;
        if (row_ok && hc0 < args.out_cols) {
            uint8_t* H = static_cast<uint8_t*>(args.out) + orow * args.ldo;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if constexpr (F4) {
                    uint32_t h[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        h[j] = swiglu_pair(v[32 * b + 2 * j], v[64 + 32 * b + 2 * j], v[32 * b + 2 * j + 1],
                                           v[64 + 32 * b + 2 * j + 1]);
                    const Mx4Quant m = mx4_scale(absmax_bits(h));
                    *reinterpret_cast<uint4*>(H + (hc0 + 32 * b) / 2) =
                        make_uint4(mx4_codes8(h[0], h[1], h[2], h[3], m.mult), mx4_codes8(h[4], h[5], h[6], h[7], m.mult),
                                   mx4_codes8(h[8], h[9], h[10], h[11], m.mult),
                                   mx4_codes8(h[12], h[13], h[14], h[15], m.mult));
                    args.h_sf[mx_sf_byte(orow, (hc0 + 32 * b) / 32, args.out_cols)] = m.ue8m0;
                } else {
                    float h[32];
                    float amax = 0.0f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float g = __uint_as_float(v[32 * b + j]), u = __uint_as_float(v[64 + 32 * b + j]);
                        // the stored hidden: bf16 rounding of SiLU(g) u
                        h[j] = __bfloat162float(__float2bfloat16_rn(silu_f(g) * u));
                        amax = fmaxf(amax, fabsf(h[j]));
                    }
                    const MxQuant m = mx_quant(amax);
                    uint32_t c[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a0, a1, a2, a3;
                        if (!m.q.wide) {
                            a0 = h[4 * j] * m.q.mult; a1 = h[4 * j + 1] * m.q.mult;
                            a2 = h[4 * j + 2] * m.q.mult; a3 = h[4 * j + 3] * m.q.mult;
                        } else {
                            a0 = scaled_wide(h[4 * j], m.q.e); a1 = scaled_wide(h[4 * j + 1], m.q.e);
                            a2 = scaled_wide(h[4 * j + 2], m.q.e); a3 = scaled_wide(h[4 * j + 3], m.q.e);
                        }
                        c[j] = cvt_e4m3x2(a0, a1) | (cvt_e4m3x2(a2, a3) << 16);
                    }
                    uint4* dst = reinterpret_cast<uint4*>(H + hc0 + 32 * b);
                    dst[0] = make_uint4(c[0], c[1], c[2], c[3]);
                    dst[1] = make_uint4(c[4], c[5], c[6], c[7]);
                    args.h_sf[mx_sf_byte(orow, (hc0 + 32 * b) / 32, args.out_cols)] = m.ue8m0;
                }
            }
        }
    } else if constexpr (EPI == EPI_BF16) {
        const int c_base = n * 2 * HALF + half * HALF;
        __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(args.out);
#pragma unroll
        for (int c0 = 0; c0 < HALF; c0 += 32) {
            if (c_base + c0 >= args.out_cols) break;
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q)
                pk[q] = pack_bf16x2(__uint_as_float(v[c0 + 2 * q]), __uint_as_float(v[c0 + 2 * q + 1]));
            if (piece_ok) {
                store_piece(tmO, piece, pk, lanew, c_base + c0, a_row + q32);
            } else if (row_ok) {
                uint4* dst = reinterpret_cast<uint4*>(Y + orow * args.ldo + c_base + c0);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (c_base + c0 + 8 * w < args.out_cols) dst[w] = make_uint4(pk[4 * w], pk[4 * w + 1], pk[4 * w + 2], pk[4 * w + 3]);
            }
        }
    } else {   // EPI_F32
        const int c_base = n * 2 * HALF + half * HALF;
        float* Z = static_cast<float*>(args.out);
        if (piece_ok) {
#pragma unroll
            for (int c0 = 0; c0 < HALF; c0 += 16) {
                if (c_base + c0 >= args.out_cols) break;
                store_piece(tmO, piece, &v[c0], lanew, c_base + c0, a_row + q32);
            }
        } else if (row_ok) {
#pragma unroll
            for (int c0 = 0; c0 < HALF; c0 += 4) {
                if (c_base + c0 >= args.out_cols) break;
                *reinterpret_cast<uint4*>(Z + orow * args.ldo + c_base + c0) =
                    make_uint4(v[c0], v[c0 + 1], v[c0 + 2], v[c0 + 3]);
            }
        }
    }
}

// gemm_mx.cu
cudaError_t out_map(CUtensorMap* m, int epi, void* out, long long rows, int cols, long long ldo, int* tma_out);

}  // namespace mx
}  // namespace fs
