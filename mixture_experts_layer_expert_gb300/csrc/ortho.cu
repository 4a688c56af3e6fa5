// ortho.cu -- orthogonalised updates: Newton-Schulz steps on a batch of matrices
// (the expert weights' gradients).
//
//   X = G / (|G|_F + eps);  per step  A = X X^T,  B = b A + c A A,  X = a X + B X
// with X [r, q], r <= q (a tall G works as its transpose).  2 r^2 q + r^3 of the
// multiply-adds are the symmetric products' halves.
//
// Rounding.  The steps multiply small singular values by a each time (3.4445^5 =
// 485 for the usual coefficients), and with them any error in directions that G
// does not have: gradients of experts with fewer tokens than rows have many.  X
// rounded to bf16 between the steps is 10 to 30% off for such G, in fp16 1 to 4%.
// So X is a pair, H in fp16 and L a byte in 254ths of H's step (19 bits), as long as the steps to come can
// multiply by more than four, and the products read H only: an error of H enters through
// B H, whose left side has no component outside G's own directions, and the term a X is
// exact to 19 bits.  (L in fp16 was no more exact in the result and cost 1.6 GB of traffic more for 128 x 768 x
// 2,048, mostly in the first scaling: 230 us, not 200.)  A and B are fp16, B's diagonal (its largest part once the rows are
// nearly orthonormal) fp32 and applied to H in the epilogue.  What remains is 0.06 to 0.15%,
// below the rounding of a bf16 result (without the diagonal 0.2%; with L until the last
// step no better, with L only while the steps multiply by more than 16 0.25%).  All three
// carry powers of two that keep the largest values the coefficients allow below 2^14 (see
// OrthoScales); sums fp32.
//
// One GEMM serves the three products: CTA pairs (2-SM MMA) on 256 x 256 tiles, operands
// by TMA in five stages of 64 along K, two accumulators in TMEM.  X X^T and A A compute
// the tiles on and above the diagonal and store each 32 x 32 piece and its transpose; their
// tiles are 256 x 128 where few tiles leave clusters idle (five matrices of 333 rows: 15 tiles or 20;
// a half tile takes 0.7 of a whole one's time, its MMAs being bound by the operand reads), and in a last round of
// few tiles (3 x 2,048 rows: 108 tiles on 76 pairs, 77 to 70 us).
// B X reads X as the MN-major operand, where it lies.  The epilogue's own inputs (the piece
// of A, of H and L) come and go by TMA through two 4 KB buffers per warp.
// Measured, 3 x 2,048 x 7,168: X X^T 70 us and B X 122 us (1.45 PFLOP/s each; bound by the reads of operands from shared
// memory, 620 cycles a stage for 512 of MMAs); 128 x 768 x 2,048: B X 295 us, 4.3 TB/s of DRAM and some 60% of what
// L2 hands an SM (a tile's operands and pieces 585 KB in 13,700 cycles), X X^T 145 us.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "ortho.cuh"

namespace fs {
namespace ortho {

constexpr int BT = 256;                       // tile rows of a pair (and columns: BN)
constexpr int BK = 64;
constexpr int STAGES = 5;
constexpr int A_STAGE = 128 * BK * 2;         // this CTA's 128 rows of the first operand
constexpr int B_STAGE = 128 * BK * 2;         // room for its BN / 2 rows (or columns) of the second
constexpr int STAGE_BYTES = A_STAGE + B_STAGE;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int NACC = 2;
constexpr int TMEM_COLS = 512;
constexpr int PIECE = 32 * 32 * 2;            // 32 x 32 fp16
constexpr int LOW = 32 * 32;                  // of L
constexpr int BUF = 2 * PIECE;
constexpr int EPI_OFF = STAGES * STAGE_BYTES;
constexpr int BAR_OFF = EPI_OFF + EPI_WARPS * 2 * BUF;
constexpr size_t SMEM_BYTES = 1024 + BAR_OFF + 512;
static_assert(SMEM_BYTES <= 232448, "shared memory");

// GRAM: A = X X^T;  POLY: B = b A + c A A;  STEP: X = a X + B X;  LAST: the same, as the bf16 result
enum { GRAM = 0, POLY = 1, STEP = 2, LAST = 3 };

struct Args {
    int R, C, batch, kb;          // tiles of rows and columns, matrices, stages along K
    int whole, units;             // tiles that are worked on whole, and units in all: the others are two each
    int rows, cols;               // extents of the output (cols padded to 64)
    float alpha, beta;            // out = alpha in + beta acc (+ beta diag H)
    int low_in, low_out;          // X comes and goes as a pair
    float* diag;                  // [batch][rows] B's diagonal, times its power of two
    __nv_bfloat16* out;           // LAST: result [m, n]
    long long out_row, out_mat;
    int m, n, tall, tma_out;
    int* err;
};

struct Tile {
    int z, i, j;
    int col, cols;                // first column and how many
};

// Tiles of a matrix: R x C, or of R x C those that reach the diagonal or lie above it.
template <bool SYM, int BN>
__host__ __device__ __forceinline__ int tiles_per_matrix(int R, int C) {
    if (!SYM) return R * C;
    if (BN == BT) return R * (R + 1) / 2;
    const int m = C / 2;                   // columns 2m and 2m + 1 of tiles have m + 1 each
    return (m + 1) * (m + (C & 1));
}

template <bool SYM, int BN>
__device__ __forceinline__ Tile decode(int t, const Args& a, int per) {
    Tile r;
    int part = -1;                     // half of a tile, of those behind a.whole
    if (SYM && BN == BT && t >= a.whole) {
        part = (t - a.whole) & 1;
        t = a.whole + (t - a.whole) / 2;
    }
    r.z = t / per;
    const int x = t - r.z * per;
    if constexpr (SYM && BN == BT) {   // column by column of the upper triangle: tile (i, j), i <= j, is j (j + 1) / 2 + i
        int j = static_cast<int>((sqrtf(8.0f * static_cast<float>(x) + 1.0f) - 1.0f) * 0.5f);
        while (j * (j + 1) / 2 > x) --j;
        while ((j + 1) * (j + 2) / 2 <= x) ++j;
        r.j = j;
        r.i = x - j * (j + 1) / 2;
    } else if constexpr (SYM) {        // the first tile of column 2m is m (m + 1)
        int m = static_cast<int>((sqrtf(4.0f * static_cast<float>(x) + 1.0f) - 1.0f) * 0.5f);
        while (m * (m + 1) > x) --m;
        while ((m + 1) * (m + 2) <= x) ++m;
        const int rem = x - m * (m + 1);
        r.j = 2 * m + rem / (m + 1);
        r.i = rem % (m + 1);
    } else {
        r.j = x / a.R;
        r.i = x - r.j * a.R;
    }
    r.col = r.j * BN + (part > 0 ? BN / 2 : 0);
    r.cols = part < 0 ? BN : BN / 2;
    return r;
}

__device__ __forceinline__ void store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    tc_mma_bf16_pair(d, adesc, bdesc, idesc, acc);      // kind::f16; the descriptor says fp16
}

// 16-byte chunk q of row `row` in a 32 x 32 piece with the 64-byte swizzle.
__device__ __forceinline__ int chunk_at(int row, int q) { return row * 64 + ((q ^ ((row >> 1) & 3)) << 4); }
// Element (row, col) of it.
__device__ __forceinline__ int elem_at(int row, int col) { return chunk_at(row, col >> 3) + (col & 7) * 2; }

// L: what H leaves of X, one byte each: 128 + 254 (x - h) / ulp(h), so 1 to 255, and off by
// ulp(h) / 508 at most.  For h = +-1.f 2^(E - 15), p = 2^(E - 15) stands in h's own exponent bits, ulp(h) is 2^-10 p; of a
// subnormal h p reads 0 and L is dropped (2^-25 at most, 2^-38 of the largest X).
__device__ __forceinline__ uint32_t low_codes2(uint32_t h, float x0, float x1) {
    const float2 v = unpack_half2(h), inv = unpack_half2(0x78007800u - (h & 0x7C007C00u));       // 1 / p
    constexpr float S = 254.0f * 1024.0f, M = 12582912.0f + 128.0f;      // 1.5 2^23: the integer lands in the low bits
    const float a = fmaf((x0 - v.x) * inv.x, S, M), b = fmaf((x1 - v.y) * inv.y, S, M);
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040) & 0xffffu;
}
__device__ __forceinline__ float low_byte(uint32_t word, int k) {        // 2^23 + its byte k, less 2^23 + 128
    return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u + k)) - (8388608.0f + 128.0f);
}
__device__ __forceinline__ float2 with_low(uint32_t h, uint32_t word, int k) {
    constexpr float U = 1.0f / (254.0f * 1024.0f);
    const float2 v = unpack_half2(h), p = unpack_half2(h & 0x7C007C00u);
    return make_float2(fmaf(low_byte(word, k), p.x * U, v.x), fmaf(low_byte(word, k + 1), p.y * U, v.y));
}

template <int MODE, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmIn, const __grid_constant__ CUtensorMap tmInL,
            const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmOutL, const Args args) {
    constexpr bool SYM = MODE == GRAM || MODE == POLY;
    constexpr bool B_MN = !SYM;
    constexpr bool LOADS = MODE != GRAM;
    static_assert(BN == BT || SYM, "the MN-major operand comes in boxes of 64 columns, two a CTA");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint64_t* full = bars;
    uint64_t* empty = bars + STAGES;
    uint64_t* tfull = bars + 2 * STAGES;
    uint64_t* tempty = tfull + NACC;
    uint64_t* fin = tempty + NACC;
    uint64_t* ebar = fin + 1;                      // [EPI_WARPS][2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ebar + 2 * EPI_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < NACC; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 2 * EPI_WARPS);
        }
        mbar_init(smem_u32(fin), 1);
        for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(smem_u32(&ebar[i]), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    cudaGridDependencySynchronize();
    const int per = tiles_per_matrix<SYM, BN>(args.R, args.C);
    const int total = args.units;
    const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(nclusters_x());

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += ncl) {
                const Tile tl = decode<SYM, BN>(t, args, per);
                const int a_row = tl.i * BT + static_cast<int>(rank) * 128;
                const int b_rows = tl.cols / 2, b_row = tl.col + static_cast<int>(rank) * b_rows;
                for (int kb = 0; kb < args.kb; ++kb) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.err)) { ok = false; break; }
                    const uint32_t fb_local = smem_u32(&full[stage]);
                    if (leader) mbar_arrive_expect_tx(fb_local, 2 * (A_STAGE + b_rows * BK * 2));
                    const uint32_t fb = map_to_cta(fb_local, 0);
                    const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_STAGE;
                    tma_load_3d_pair(sa, &tmA, fb, kb * BK, a_row, tl.z);
                    if constexpr (B_MN) {          // two boxes of 64 K rows x 64 columns
                        tma_load_3d_pair(sb, &tmB, fb, b_row, kb * BK, tl.z);
                        tma_load_3d_pair(sb + 8192, &tmB, fb, b_row + 64, kb * BK, tl.z);
                    } else {               // (of half a tile in boxes of half the rows)
                        tma_load_3d_pair(sb, tl.cols == BN ? &tmB : &tmInL, fb, kb * BK, b_row, tl.z);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (leader) {       // the loads of both CTAs complete on this CTA's barriers
                const int pending = issued < STAGES ? issued : STAGES;
                for (int j = 1; j <= pending; ++j) {
                    int s = stage - j;
                    uint32_t ph = phase;
                    if (s < 0) { s += STAGES; ph ^= 1u; }
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(smem_u32(&full[s]), ph)) {
                        if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMA
        if (leader) {
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += ncl, ++it) {
                const int acc = it & 1;
                const uint32_t use = static_cast<uint32_t>(it >> 1);
                if (!mbar_wait(smem_u32(&tempty[acc]), (use & 1u) ^ 1u, abort_flag, args.err)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                const uint32_t idesc = SYM && BN == BT && t >= args.whole ? idesc_f16(BT, BN / 2, B_MN) : idesc_f16(BT, BN, B_MN);
                for (int kb = 0; kb < args.kb; ++kb) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, args.err)) { ok = false; break; }
                    tc_fence_after();
                    __syncwarp();
                    if (elect_one()) {
                        const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                        const uint64_t adesc = smem_desc_sw128(sa);
                        const uint64_t bdesc = B_MN ? smem_desc_sw128_mn(sa + A_STAGE, 8192) : smem_desc_sw128(sa + A_STAGE);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)        // 16 of K: 32 bytes of a row, or 16 rows of 128 bytes
                            mma_f16_pair(d_tmem, adesc + 2ull * kk, bdesc + (B_MN ? 128ull : 2ull) * kk, idesc,
                                         (kb > 0 || kk > 0) ? 1u : 0u);
                        tc_commit_pair_multicast(smem_u32(&empty[stage]), 0x3);
                        if (kb == args.kb - 1) tc_commit_pair_multicast(smem_u32(&tfull[acc]), 0x3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            __syncwarp();
            if (elect_one()) tc_commit_pair_multicast(smem_u32(fin), 0x3);
            __syncwarp();
        }
        // both CTAs: every MMA writing this CTA's TMEM has completed
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(fin), 0)) {
            if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
        uint8_t* buf0 = smem + EPI_OFF + ew * 2 * BUF;
        int it = 0;
        uint32_t asked = 0, used = 0;              // pieces whose inputs were asked for, and taken
        [[maybe_unused]] uint32_t stored = 0;
        for (int t = cid; t < total; t += ncl, ++it) {
            const Tile tl = decode<SYM, BN>(t, args, per);
            const int row0 = tl.i * BT + static_cast<int>(rank) * 128 + quarter * 32;
            const int mine = tl.cols / 2, col0 = tl.col + half * mine;
            // this warp's pieces [first, last) along its columns
            int last = row0 < args.rows ? min(mine / 32, (args.cols - col0 + 31) / 32) : 0;
            int first = SYM && col0 < row0 ? (row0 - col0) / 32 : 0;
            if (last < first) last = first;
            const int acc = it & 1;
            const uint32_t use = static_cast<uint32_t>(it >> 1);
            auto ask = [&](int c) {
                const uint32_t b = asked & 1u;
                if (lane == 0) {
                    bulk_wait_read0();              // the buffer's last store has read it
                    const uint32_t bar = smem_u32(&ebar[2 * ew + b]), dst = smem_u32(buf0 + b * BUF);
                    const bool low = !SYM && args.low_in;
                    mbar_arrive_expect_tx(bar, low ? PIECE + LOW : PIECE);
                    tma_load_3d(dst, &tmIn, bar, col0 + 32 * c, row0, tl.z);
                    if (low) tma_load_3d(dst + PIECE, &tmInL, bar, col0 + 32 * c, row0, tl.z);
                }
                ++asked;
            };
            if (LOADS && first < last) {
                __syncwarp();
                ask(first);
            }
            float* drow = nullptr;                 // this lane's row of B's diagonal
            if (MODE != GRAM && row0 + lane < args.rows) drow = args.diag + static_cast<long long>(tl.z) * args.rows + row0 + lane;
            const float d = !SYM && drow ? *drow : 0.0f;
            if (!mbar_wait(smem_u32(&tfull[acc]), use & 1u, abort_flag, args.err)) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * BN + half * mine);
            bool ok = true;
#pragma unroll 1
            for (int c = first; c < last; ++c) {
                uint32_t v[32];
                tmem_ld32_sync(tbase + 32 * c, v);
                const uint32_t b = LOADS ? used & 1u : stored++ & 1u;
                uint8_t* buf = buf0 + b * BUF;
                const int x = col0 + 32 * c;
                if constexpr (LOADS) {
                    if (c + 1 < last) ask(c + 1);
                    if (!mbar_wait(smem_u32(&ebar[2 * ew + b]), (used >> 1) & 1u, abort_flag, args.err)) { ok = false; break; }
                    ++used;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 h = *reinterpret_cast<const uint4*>(buf + chunk_at(lane, q));
                        const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
                        uint32_t lw[2] = {0x80808080u, 0x80808080u};
                        if (!SYM && args.low_in) {
                            const uint2 l = *reinterpret_cast<const uint2*>(buf + PIECE + lane * 32 + 8 * q);
                            lw[0] = l.x; lw[1] = l.y;
                        }
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            float2 in = unpack_half2(hw[w]);
                            uint32_t& v0 = v[8 * q + 2 * w];
                            uint32_t& v1 = v[8 * q + 2 * w + 1];
                            float a0 = __uint_as_float(v0), a1 = __uint_as_float(v1);
                            if constexpr (!SYM) {
                                a0 += d * in.x;
                                a1 += d * in.y;
                                if (args.low_in) in = with_low(hw[w], lw[w >> 1], 2 * (w & 1));
                            }
                            v0 = __float_as_uint(args.alpha * in.x + args.beta * a0);
                            v1 = __float_as_uint(args.alpha * in.y + args.beta * a1);
                        }
                    }
                    __syncwarp();
                } else {
                    // the store before the last one has read this buffer
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(args.beta * __uint_as_float(v[j]));
                }
                if (MODE == POLY && x == row0) {
                    uint32_t on = 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        on = j == lane ? v[j] : on;
                        v[j] = j == lane ? 0u : v[j];
                    }
                    if (drow) *drow = __uint_as_float(on);
                }
                if constexpr (MODE == LAST) {
                    // the result's piece, transposed for a tall matrix
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t p[4];
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            p[w] = pack_bf16x2(__uint_as_float(v[8 * q + 2 * w]), __uint_as_float(v[8 * q + 2 * w + 1]));
                        if (!args.tall) {
                            *reinterpret_cast<uint4*>(buf + chunk_at(lane, q)) = make_uint4(p[0], p[1], p[2], p[3]);
                        } else {
#pragma unroll
                            for (int w = 0; w < 8; ++w)
                                *reinterpret_cast<uint16_t*>(buf + elem_at(8 * q + w, lane)) =
                                    static_cast<uint16_t>(p[w >> 1] >> (16 * (w & 1)));
                        }
                    }
                    const int oy = args.tall ? x : row0, ox = args.tall ? row0 : x;      // piece's corner in the result
                    if (args.tma_out) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            store_3d(&tmOut, smem_u32(buf), ox, oy, tl.z);
                            bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        uint16_t* o = reinterpret_cast<uint16_t*>(args.out) + tl.z * args.out_mat;
                        const bool in = ox + lane < args.n;
                        o += oy * args.out_row + ox + lane;
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (in && oy + y < args.m)
                                o[y * args.out_row] = *reinterpret_cast<const uint16_t*>(buf + elem_at(y, lane));
                        fence_proxy_async_smem();      // the buffer's next content comes by TMA, over what was written here
                        __syncwarp();
                    }
                } else {
                    uint32_t p[16];
#pragma unroll
                    for (int w = 0; w < 16; ++w)
                        p[w] = pack_half2(__uint_as_float(v[2 * w]), __uint_as_float(v[2 * w + 1]));
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(buf + chunk_at(lane, q)) =
                            make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
                    if constexpr (SYM) {
                        if (x > row0) {
#pragma unroll
                            for (int w = 0; w < 32; ++w)
                                *reinterpret_cast<uint16_t*>(buf + PIECE + elem_at(w, lane)) =
                                    static_cast<uint16_t>(p[w >> 1] >> (16 * (w & 1)));
                        }
                    } else if (args.low_out) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t l[4];
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint32_t* x = &v[16 * q + 4 * w];
                                l[w] = low_codes2(p[8 * q + 2 * w], __uint_as_float(x[0]), __uint_as_float(x[1])) |
                                       low_codes2(p[8 * q + 2 * w + 1], __uint_as_float(x[2]), __uint_as_float(x[3])) << 16;
                            }
                            *reinterpret_cast<uint4*>(buf + PIECE + lane * 32 + 16 * q) = make_uint4(l[0], l[1], l[2], l[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        store_3d(&tmOut, smem_u32(buf), x, row0, tl.z);
                        if constexpr (SYM) {
                            if (x > row0) store_3d(&tmOut, smem_u32(buf + PIECE), row0, x, tl.z);
                        } else if (args.low_out) {
                            store_3d(&tmOutL, smem_u32(buf + PIECE), x, row0, tl.z);
                        }
                        bulk_commit();
                    }
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_tmem(map_to_cta(smem_u32(&tempty[acc]), 0));
        }
        if (lane == 0) {
            while (used != asked) {                // a wait gave up: this warp's loads end before its buffers do
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(smem_u32(&ebar[2 * ew + (used & 1u)]), (used >> 1) & 1u)) {
                    if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
                }
                ++used;
            }
            bulk_wait0();
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------- preparation
constexpr int NORM_BLOCKS = 256;              // at most, per matrix

__global__ void __launch_bounds__(256) norm_kernel(const Source s, float* part) {
    __shared__ float sh[8][3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t es = s.f32 ? 4 : 2;
    const int per = s.f32 ? 4 : 8;
    const uint8_t* g = static_cast<const uint8_t*>(s.g) + static_cast<long long>(blockIdx.y) * s.mat * es;
    Squares q;
    cudaGridDependencySynchronize();
    for (int i = blockIdx.x * 8 + warp; i < s.m; i += gridDim.x * 8) {
        const uint8_t* row = g + i * s.row * es;
        // a lane adds the elements of whole vectors, also where they are read one by one: the sum, and with it the result's
        // last bits, depend on neither alignment nor strides
        const int nv = (s.n + per - 1) / per;
        for (int v0 = lane; v0 < nv; v0 += 128) {
            float f[32];
            if (s.vec) {
                uint4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = v0 + 32 * k < nv ? reinterpret_cast<const uint4*>(row)[v0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        f[8 * k + 2 * h] = s.f32 ? __uint_as_float(w[h]) : bf16lo(w[h]);
                        f[8 * k + 2 * h + 1] = s.f32 ? 0.0f : bf16hi(w[h]);
                    }
                }
            } else if (s.f32) {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int j = 4 * (v0 + 32 * (k >> 3)) + ((k & 7) >> 1);
                    f[k] = !(k & 1) && j < s.n ? reinterpret_cast<const float*>(row)[j] : 0.0f;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int j = 8 * (v0 + 32 * (k >> 3)) + (k & 7);
                    f[k] = j < s.n ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[j]) : 0.0f;
                }
            }
            q.add(f);
        }
    }
    float v[3] = {q.big, q.mid, q.small};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (lane == 0) sh[warp][k] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float t = 0.f;
        for (int w = 0; w < 8; ++w) t += sh[w][threadIdx.x];
        part[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = t;
    }
}

// The two factors that scale matrix z, from its blocks' sums; all threads of a block call it.
__device__ __forceinline__ void block_factors(const float* part, int nb, int z, double eps, float xscale, float* f1, float* f2) {
    __shared__ float f[2];
    if (threadIdx.x < 32) {
        double big = 0, mid = 0, small = 0;
        for (int i = threadIdx.x; i < nb; i += 32) {
            const float* p = part + (static_cast<long long>(z) * nb + i) * 3;
            big += p[0];
            mid += p[1];
            small += p[2];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            big += __shfl_xor_sync(0xffffffffu, big, o);
            mid += __shfl_xor_sync(0xffffffffu, mid, o);
            small += __shfl_xor_sync(0xffffffffu, small, o);
        }
        if (threadIdx.x == 0) norm_factors(big, mid, small, eps, xscale, &f[0], &f[1]);
    }
    __syncthreads();
    *f1 = f[0];
    *f2 = f[1];
}

// Eight values as H and L (16 and 8 bytes).
__device__ __forceinline__ void split8(const float (&x)[8], uint4* h, uint2* l) {
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        hw[w] = pack_half2(x[2 * w], x[2 * w + 1]);
        lw[w] = low_codes2(hw[w], x[2 * w], x[2 * w + 1]);
    }
    *h = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *l = make_uint2(lw[0] | lw[1] << 16, lw[2] | lw[3] << 16);
}

// X = G / (|G| + eps) as H and L times its power of two, rows where they are: a warp a row, eight
// columns a lane, four such in flight.  Columns past q up to the padded width are zero.
__global__ void __launch_bounds__(256)
scale_rows_kernel(const Source s, const float* part, int nb, double eps, float xscale, __half* H, uint8_t* L, int qp) {
    const int lane = threadIdx.x & 31, z = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5);
    cudaGridDependencySynchronize();
    float f1, f2;
    block_factors(part, nb, z, eps, xscale, &f1, &f2);
    if (i >= s.m) return;
    const size_t es = s.f32 ? 4 : 2;
    const uint8_t* row = static_cast<const uint8_t*>(s.g) + (static_cast<long long>(z) * s.mat + static_cast<long long>(i) * s.row) * es;
    const long long at_ = (static_cast<long long>(z) * s.m + i) * qp;
    for (int c0 = 8 * lane; c0 < qp; c0 += 4 * 256) {
        float x[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + 256 * u;
            if (s.vec && c + 8 <= s.n) {
                if (s.f32) {
                    const float4 a = reinterpret_cast<const float4*>(row)[c / 4], b = reinterpret_cast<const float4*>(row)[c / 4 + 1];
                    x[u][0] = a.x; x[u][1] = a.y; x[u][2] = a.z; x[u][3] = a.w;
                    x[u][4] = b.x; x[u][5] = b.y; x[u][6] = b.z; x[u][7] = b.w;
                } else {
                    const uint4 a = reinterpret_cast<const uint4*>(row)[c / 8];
                    x[u][0] = bf16lo(a.x); x[u][1] = bf16hi(a.x); x[u][2] = bf16lo(a.y); x[u][3] = bf16hi(a.y);
                    x[u][4] = bf16lo(a.z); x[u][5] = bf16hi(a.z); x[u][6] = bf16lo(a.w); x[u][7] = bf16hi(a.w);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[u][k] = c + k < s.n ? at(s, row, c + k) : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + 256 * u;
            if (c >= qp) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[u][k] = x[u][k] * f1 * f2;
            split8(x[u], reinterpret_cast<uint4*>(H + at_ + c), reinterpret_cast<uint2*>(L + at_ + c));
        }
    }
}

// The same for a tall G, transposed: a 64 x 64 tile per block.
__global__ void __launch_bounds__(256)
scale_tall_kernel(const Source s, const float* part, int nb, double eps, float xscale, int tiles, int tiles_n, __half* H, uint8_t* L,
                  int r, int qp) {
    __shared__ float tile[64][65];
    const int z = blockIdx.y;
    cudaGridDependencySynchronize();
    const size_t es = s.f32 ? 4 : 2;
    const uint8_t* g = static_cast<const uint8_t*>(s.g) + static_cast<long long>(z) * s.mat * es;
    // 16 lanes a row of the tile, 8 lanes a row of its transpose: whole lines either way (four lanes of 64 bytes each
    // moved 890 MB through L2 for 3 x 7,168 x 2,048, not 360, and took 97 us, not 58), and the next tile's loads
    // are on their way while this one is written
    float4 in[4];
    const auto fetch = [&](int t) {
        const int ti = t / tiles_n, j = (t - ti * tiles_n) * 64 + (threadIdx.x & 15) * 4;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = ti * 64 + (threadIdx.x >> 4) + 16 * u;
            const uint8_t* row = g + static_cast<long long>(i) * s.row * es;
            if (s.vec && i < s.m && j + 4 <= s.n) {
                if (s.f32) {
                    in[u] = reinterpret_cast<const float4*>(row)[j / 4];
                } else {
                    const uint2 x = reinterpret_cast<const uint2*>(row)[j / 4];
                    in[u] = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
                }
            } else {
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = i < s.m && j + k < s.n ? at(s, row, j + k) : 0.0f;
                in[u] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    };
    fetch(blockIdx.x);
    float f1, f2;
    block_factors(part, nb, z, eps, xscale, &f1, &f2);
#pragma unroll 1
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float* to = &tile[(threadIdx.x >> 4) + 16 * u][(threadIdx.x & 15) * 4];
            to[0] = in[u].x * f1 * f2; to[1] = in[u].y * f1 * f2; to[2] = in[u].z * f1 * f2; to[3] = in[u].w * f1 * f2;
        }
        __syncthreads();
        if (t + static_cast<int>(gridDim.x) < tiles) fetch(t + gridDim.x);
        const int ti = t / tiles_n, tj = t - ti * tiles_n;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int lr = (threadIdx.x >> 3) + 32 * u, c = (threadIdx.x & 7) * 8, xr = tj * 64 + lr;
            if (xr < r) {
                const long long at_ = (static_cast<long long>(z) * r + xr) * qp + ti * 64 + c;
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = tile[c + k][lr];
                split8(x, reinterpret_cast<uint4*>(H + at_), reinterpret_cast<uint2*>(L + at_));
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host
struct Shape {
    int r, q, rp, qp;
    bool tall;
};
Shape shape(int m, int n) {
    Shape s;
    s.tall = m > n;
    s.r = s.tall ? n : m;
    s.q = s.tall ? m : n;
    s.rp = (s.r + 63) / 64 * 64;
    s.qp = (s.q + 63) / 64 * 64;
    return s;
}

struct Layout {
    int group;                       // matrices in flight
    size_t h[2], l, a, b, diag, part, end;
};
size_t up(size_t x) { return (x + 1023) / 1024 * 1024; }
// Matrices are worked on in groups whose buffers stay within 2 GiB (one matrix at least).
Layout layout(int batch, int m, int n) {
    const Shape s = shape(m, n);
    const size_t x = static_cast<size_t>(s.r) * s.qp * 2, sq = static_cast<size_t>(s.r) * s.rp * 2;
    const size_t each = 5 * x / 2 + 2 * sq + static_cast<size_t>(s.r) * 4 + NORM_BLOCKS * 12;
    size_t g = (size_t(2) << 30) / each;
    g = g < 1 ? 1 : (g > 16384 ? 16384 : g);
    if (g > static_cast<size_t>(batch)) g = batch;
    const size_t rounds = (batch + g - 1) / g;
    g = (batch + rounds - 1) / rounds;            // rounds of equal size
    Layout l;
    l.group = static_cast<int>(g);
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at_ = o; o = up(o + bytes); return at_; };
    l.h[0] = take(g * x);
    l.h[1] = take(g * x);
    l.l = take(g * (x / 2));
    l.a = take(g * sq);
    l.b = take(g * sq);
    l.diag = take(g * s.r * 4);
    l.part = take(g * NORM_BLOCKS * 12);
    l.end = o;
    return l;
}

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, void* base, long long cols, long long rows, long long mats,
                   long long row_bytes, long long mat_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(mat_bytes)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    return encode_map(map, type, 3, base, dims, strides, box, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// fp16 [mats, rows, cols] contiguous: boxes of 64 columns for the products, pieces of 32 x 32 for the epilogue.
cudaError_t operand(CUtensorMap* map, void* base, int cols, int rows, int mats, int box_rows) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols, rows, mats, cols * 2LL,
                  static_cast<long long>(rows) * cols * 2, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
cudaError_t pieces(CUtensorMap* map, void* base, int cols, int rows, int mats) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols, rows, mats, cols * 2LL,
                  static_cast<long long>(rows) * cols * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaError_t low_pieces(CUtensorMap* map, void* base, int cols, int rows, int mats) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, cols, rows, mats, cols, static_cast<long long>(rows) * cols, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Tiles of the last round of clusters, if there are few enough of them to be worked on in halves (0.7 of a tile's time).
int last_round(int tiles, int clusters) {
    const int rest = tiles % clusters;
    return tiles > clusters && 2 * rest <= clusters ? rest : 0;
}

template <int MODE, int BN>
cudaError_t launch_tiles(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& in, const CUtensorMap& in_l,
                         const CUtensorMap& out, const CUtensorMap& out_l, Args args, int sms, cudaStream_t st) {
    static bool set[kMaxDevices];
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(gemm_kernel<MODE, BN>), SMEM_BYTES, set);
    if (e != cudaSuccess) return e;
    args.C = (args.cols + BN - 1) / BN;
    const int tiles = tiles_per_matrix<MODE <= POLY, BN>(args.R, args.C) * args.batch;
    const int clusters = tiles < sms / 2 ? tiles : sms / 2;
    const int rest = MODE <= POLY && BN == BT ? last_round(tiles, clusters) : 0;
    args.whole = tiles - rest;
    args.units = tiles + rest;
    count_launch();
    return launch_after(gemm_kernel<MODE, BN>, dim3(2 * clusters), dim3(THREADS), SMEM_BYTES, st, a, b, in, in_l, out, out_l, args);
}

// The symmetric products: a is the map of boxes of 128 rows, b_half of 64.  The tile width whose rounds of
// clusters take less time: measured 37 and 27 us for a tile of K = 7,168, 14 and 9 us for K = 2,048.
template <int MODE>
cudaError_t launch_square(const CUtensorMap& a, const CUtensorMap& b_half, const CUtensorMap& in, const CUtensorMap& out,
                          const Args& args, int sms, cudaStream_t st) {
    const int most = sms / 2, c = (args.cols + 127) / 128;
    const long long tiles = static_cast<long long>(tiles_per_matrix<true, BT>(args.R, args.R)) * args.batch;
    const long long narrow = static_cast<long long>(tiles_per_matrix<true, 128>(args.R, c)) * args.batch;
    if (narrow > 0x3fffffff) return cudaErrorInvalidValue;
    const long long whole = 10 * ((tiles + most - 1) / most) - (last_round(static_cast<int>(tiles), most) ? 3 : 0);
    return 7 * ((narrow + most - 1) / most) < whole ? launch_tiles<MODE, 128>(a, b_half, in, b_half, out, out, args, sms, st)
                                                    : launch_tiles<MODE, BT>(a, a, in, b_half, out, out, args, sms, st);
}

}  // namespace ortho

size_t ortho_ws_bytes(int batch, int m, int n) {
    if (ortho_tiny_fits(m, n)) return 256;
    return ortho_small_fits(m, n) ? ortho_small_ws_bytes(batch, m, n) : ortho::layout(batch, m, n).end;
}

cudaError_t launch_orthogonalize(const OrthoArgs& o, void* ws, cudaStream_t st) {
    using namespace ortho;
    if (ortho_tiny_fits(o.m, o.n)) return launch_ortho_tiny(o, st);
    if (ortho_small_fits(o.m, o.n)) return launch_ortho_small(o, ws, st);
    const Shape s = shape(o.m, o.n);
    const Layout l = layout(o.batch, o.m, o.n);
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e != cudaSuccess) return e;
    uint8_t* w = static_cast<uint8_t*>(ws);
    const size_t es = o.f32 ? 4 : 2;
    const bool tma_out = (reinterpret_cast<uintptr_t>(o.out) & 15u) == 0 && o.out_row % 8 == 0 && o.out_mat % 8 == 0;
    for (int z0 = 0; z0 < o.batch; z0 += l.group) {
        const int nb = o.batch - z0 < l.group ? o.batch - z0 : l.group;
        const Source src = source(o, static_cast<const uint8_t*>(o.g) + z0 * o.g_mat * static_cast<long long>(es));
        float* part = reinterpret_cast<float*>(w + l.part);
        // a row per warp; the split depends on the matrix alone, so that a matrix's result does not depend on its batch
        int blocks = (o.m + 7) / 8;
        blocks = blocks > NORM_BLOCKS ? NORM_BLOCKS : blocks;
        count_launch();
        if ((e = launch_after(norm_kernel, dim3(blocks, nb), dim3(256), 0, st, src, part)) != cudaSuccess) return e;
        __half* H[2] = {reinterpret_cast<__half*>(w + l.h[0]), reinterpret_cast<__half*>(w + l.h[1])};
        uint8_t* L = w + l.l;
        if (s.tall) {                          // tiles of G; for X's padded width the last ones reach past it
            const int tm = s.qp / 64, tn = s.rp / 64;
            const int most = (6 * sms + nb - 1) / nb;
            e = launch_after(scale_tall_kernel, dim3(tm * tn < most ? tm * tn : most, nb), dim3(256), 0, st, src, part, blocks,
                             o.eps, o.scales.x, tm * tn, tn, H[0], L, s.r, s.qp);
        } else {
            e = launch_after(scale_rows_kernel, dim3((s.r + 7) / 8, nb), dim3(256), 0, st, src, part, blocks, o.eps, o.scales.x,
                             H[0], L, s.qp);
        }
        count_launch();
        if (e != cudaSuccess) return e;

        CUtensorMap xk[2], xn[2], xp[2], lp, ak, an, ap, bk, bp, op;
        void *A = w + l.a, *B = w + l.b;
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            e = operand(&xk[i], H[i], s.qp, s.r, nb, 128);
            if (e == cudaSuccess) e = operand(&xn[i], H[i], s.qp, s.r, nb, 64);
            if (e == cudaSuccess) e = pieces(&xp[i], H[i], s.qp, s.r, nb);
        }
        if (e == cudaSuccess) e = low_pieces(&lp, L, s.qp, s.r, nb);
        if (e == cudaSuccess) e = operand(&ak, A, s.rp, s.r, nb, 128);
        if (e == cudaSuccess) e = operand(&an, A, s.rp, s.r, nb, 64);
        if (e == cudaSuccess) e = pieces(&ap, A, s.rp, s.r, nb);
        if (e == cudaSuccess) e = operand(&bk, B, s.rp, s.r, nb, 128);
        if (e == cudaSuccess) e = pieces(&bp, B, s.rp, s.r, nb);
        __nv_bfloat16* out = o.out + z0 * o.out_mat;
        op = xp[0];
        if (e == cudaSuccess && tma_out)
            e = encode(&op, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, o.n, o.m, nb, o.out_row * 2, o.out_mat * 2, 32, 32,
                       CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;

        Args g{};
        g.R = (s.r + BT - 1) / BT;
        g.batch = nb;
        g.rows = s.r;
        g.m = o.m;
        g.n = o.n;
        g.tall = s.tall;
        g.out = out;
        g.out_row = o.out_row;
        g.out_mat = o.out_mat;
        g.tma_out = tma_out;
        g.err = dev_error_ptr();
        g.diag = reinterpret_cast<float*>(w + l.diag);
        const OrthoScales& sc = o.scales;
        // X stays a pair while the steps from here on can multiply by more than four
        bool low[kMaxOrthoSteps + 1] = {};
        double grow = 1.0;
        for (int k = o.steps - 1; k >= 0; --k) {
            grow *= fabs(o.coefs[3 * k]) > 1.0f ? fabs(o.coefs[3 * k]) : 1.0;
            low[k] = grow > 4.0;
        }
        int cur = 0;
        for (int k = 0; k < o.steps; ++k, cur ^= 1) {
            const float ca = o.coefs[3 * k], cb = o.coefs[3 * k + 1], cc = o.coefs[3 * k + 2];
            const bool last = k == o.steps - 1;
            Args a = g;
            a.cols = s.rp;
            a.kb = s.qp / BK;
            a.beta = sc.a / (sc.x * sc.x);
            e = launch_square<GRAM>(xk[cur], xn[cur], ap, ap, a, sms, st);
            if (e != cudaSuccess) return e;
            a.kb = s.rp / BK;
            a.alpha = cb * (sc.b / sc.a);
            a.beta = cc * (sc.b / (sc.a * sc.a));
            e = launch_square<POLY>(ak, an, ap, bp, a, sms, st);
            if (e != cudaSuccess) return e;
            a.cols = s.qp;
            a.low_in = low[k];
            a.low_out = low[k + 1];
            a.alpha = ca;
            a.beta = 1.0f / sc.b;
            if (!last) {
                e = launch_tiles<STEP, BT>(bk, xn[cur], xp[cur], lp, xp[cur ^ 1], lp, a, sms, st);
            } else {
                a.alpha *= o.scale / sc.x;
                a.beta *= o.scale / sc.x;
                e = launch_tiles<LAST, BT>(bk, xn[cur], xp[cur], lp, op, op, a, sms, st);
            }
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace fs
