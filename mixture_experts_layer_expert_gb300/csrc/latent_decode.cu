// latent_decode.cu -- absorbed latent attention of the newest tokens of each
// sequence over the paged latent cache:
//   s_i = scale (q_l . c_i + q_r . k_i),  out = sum_i softmax(s)_i c_i,  lse = log sum_i exp(s_i)
//
// All heads (and the n_q new tokens) of a sequence read the same records, so a
// block takes up to 64 query rows (row = new token * heads + head; more rows go to
// CTA pairs, latent_decode_pair.cu) against tiles of 64 records, staged once in shared memory as bf16 and used twice as the A
// operand of transposed products:
//   S^T = K Q^T      64 records x rows x 576, the tile read K-major
//   O^T += C^T P     512 (4 x 128) x rows x 64 records, the same tile read MN-major
// so the MMAs' N is the number of rows (rounded to 16, 32 or 64) and a few heads
// cost little; an MMA costs a fixed 28 (M = 64) or 43 (M = 128) cycles beside N/2.
// A thread holds one record's scores for all rows.  Against a running maximum per
// row that is only raised when a score exceeds it by 2^8, no thread needs the
// others' scores: the sum of p stays per record until the end, and the maximum,
// the rescaling of O^T and the shuffles they need run in a sequence's first tile
// and on the rare tiles that raise it (one barrier with an OR decides).
//
// Bound: the records' bytes while the MMAs of a block of rows fit under them: 64
// records are 73.7 KB (bf16) or 42 KB (FP8), 3,150 or 1,790 cycles of one SM's
// share of the memory bandwidth; the MMAs take 36 x 36 + 16 x 52 = 2,130 cycles for 16
// rows, 36 x 60 + 16 x 75 = 3,360 for 64.  Measured: 256 sequences of up to 8,191 tokens
// x 16 heads on an FP8 cache 223 us (3.2 TB/s; 3,400 cycles a tile, the chain of
// conversion, scores, softmax and P C over the 2.25 tiles that the ring holds: faster
// conversion, an earlier release of the raw stages or one wait for all four stages did
// not shorten it); one sequence of 4,097 tokens x 16 heads, join included, 26.6 us.
//
// The records of all sequences form one list of tiles which is cut into equal
// ranges, one per block, whatever the lengths.  A
// sequence inside one range is finished there; one that is cut leaves fp32
// partials (normalised O and lse) which a second kernel joins in range order.
//
// Warps 0-3: softmax, rescaling, output; warp 4: Q of each sequence and the MMAs of the
// scores; warp 5: the MMAs of P C; warp 6: page lookup, three tiles ahead; warp 7: TMA (a
// tile of consecutive records as two boxes per stage, else gathers of four records) into
// ring stages of 64 records x 128 latent columns (16 KB).  FP8: raw codes come into a ring of
// their own, warps 8 .. turn them into bf16 stages unscaled; a record's scale multiplies its
// latent scores (the rotary part has TMEM columns of its own) and its p.
#include "kernels.h"
#include "latent_decode.cuh"

namespace fs {
namespace dc {

constexpr int TT = 64;                        // records per tile
constexpr int ROWS = 64;                      // query rows per block
constexpr int MAXP = 11;                      // ring stages: 11, 10, 7 with 16, 32, 64 query rows; FP8: 9, 8, 5
constexpr int MAXRAW = 4;                     // FP8: raw stages (64 records x 128 codes, 8 KB)
constexpr int CTRL = 6144;
struct Shared {
    uint64_t full[MAXP], empty[MAXP], raw_full[MAXRAW], raw_empty[MAXRAW], r_full[2], r_empty[2], info_full[kInfo], tile_full[2], tile_empty[2];
    uint64_t q_empty, s_full[2], s_free[2], p_full, pv_done, o_empty, fin[2];
    uint32_t tmem;
    int abort_flag;
    int b0, tile0, left;                      // first piece of this block's range
    uint32_t live[kInfo][2];                  // records of a tile that count
    alignas(16) float m[ROWS], f[ROWS];       // running maximum (log2 units), rescaling factor or 1 / l
    int lag[ROWS];                            // a row sees positions [0, length - lag)
    float red[4][ROWS];                       // the warps' maxima or sums
    float scale[kInfo][TT];                   // FP8: the records' scales
    TileRecs<TT> recs[2];
};
static_assert(sizeof(Shared) <= CTRL, "control area");

// FP8: warps that turn codes into bf16 (four where 64 rows need the registers; their 384 threads leave 168
// a thread, and 456 bytes are spilled).
template <bool FP8, int RN> constexpr int kConv = FP8 ? (RN == 64 ? 4 : 8) : 0;
template <bool FP8, int RN> constexpr int kThreads = 32 * (8 + kConv<FP8, RN>);

template <bool FP8, int RN>
__global__ void __launch_bounds__(kThreads<FP8, RN>, 1)
decode_kernel(const __grid_constant__ CUtensorMap tmTile, const __grid_constant__ CUtensorMap tmRun, const __grid_constant__ CUtensorMap tmRow,
              const LatentDecodeArgs a, const int ranges, float* __restrict__ part, float* __restrict__ part_lse,
              Meta* __restrict__ meta) {
    // all of the SM's shared memory and no static part: the block's memory starts on a 1 KB boundary
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) set_dev_error(a.err, DEV_ERR_LIMIT);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int range = blockIdx.x, rows = a.n_q * a.H;
    // Q (9 chunks of RN rows), P (64 records x 64 rows, 128 bytes a record), rope ring, stage ring, control
    constexpr int QC = RN * 128, CW = kConv<FP8, RN>;
    constexpr int raws = FP8 ? 4 : 0;
    constexpr int stages = (RN == 16 ? 11 : (RN == 32 ? 10 : 7)) - raws / 2;
    uint8_t* sq = smem;
    uint8_t* sp = smem + 9 * QC;
    uint8_t* srope = sp + CH;
    uint8_t* sraw = srope + 2 * CH;                // FP8: codes as they lie in the cache
    uint8_t* sring = sraw + raws * CH;
    static_assert(9 * QC + (3 + raws) * CH + stages * PAIR + CTRL <= SMEM && raws <= MAXRAW, "shared memory");
    Shared& sh = *reinterpret_cast<Shared*>(smem + (SMEM - CTRL));
    volatile int* abort_flag = &sh.abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAXP; ++i) { mbar_init(smem_u32(&sh.full[i]), FP8 ? CW / 4 : 1); mbar_init(smem_u32(&sh.empty[i]), 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.r_full[i]), 1);
            mbar_init(smem_u32(&sh.r_empty[i]), 1);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.s_free[i]), 4);
            mbar_init(smem_u32(&sh.fin[i]), 1);
        }
        for (int i = 0; i < MAXRAW; ++i) { mbar_init(smem_u32(&sh.raw_full[i]), 1); mbar_init(smem_u32(&sh.raw_empty[i]), FP8 ? CW / 4 : 1); }
        for (int i = 0; i < kInfo; ++i) mbar_init(smem_u32(&sh.info_full[i]), 1);
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&sh.tile_full[i]), 1); mbar_init(smem_u32(&sh.tile_empty[i]), 1); }
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.p_full), 128);
        mbar_init(smem_u32(&sh.pv_done), 1);
        mbar_init(smem_u32(&sh.o_empty), 128);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    if (threadIdx.x < ROWS) sh.lag[threadIdx.x] = a.n_q - 1 - min(static_cast<int>(threadIdx.x) / a.H, a.n_q - 1);
    if (warp == 0) find_range(a, range, ranges, TT, true, meta, &sh.b0, &sh.tile0, &sh.left);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // S^T twice, FP8: the rotary part of S^T twice (not scaled by the record), O^T
    const uint32_t tm_s = sh.tmem, tm_r = sh.tmem + 128, tm_o = sh.tmem + 256;
    int b = sh.b0, tile = sh.tile0, left = sh.left;
    Piece p;

    if (warp >= 8) {
        // ------------------------------------------- FP8 codes to bf16 stages
        if constexpr (FP8) {
            // a quarter of the warps per stage of a tile, so that four stages are under way at once
            constexpr int NT = 8 * CW, NU = TT * 8 / NT;            // threads, 16-byte units a thread takes of a stage
            const int t = (threadIdx.x - 256) % NT, c = (threadIdx.x - 256) / NT;
            uint32_t u = c;
            bool ok = true;
            while (ok && next_piece(a, b, tile, left, &p, TT)) {
                for (int n = p.t1 - p.t0; n > 0; --n, u += 4) {
                    const uint32_t rs = u % raws, s = u % stages;
                    if (!warp_wait(smem_u32(&sh.raw_full[rs]), (u / raws) & 1, abort_flag, a.err) ||
                        !warp_wait(smem_u32(&sh.empty[s]), ((u / stages) & 1) ^ 1, abort_flag, a.err)) { ok = false; break; }
#pragma unroll 1
                    for (int e0 = 0; e0 < NU; e0 += 4) {
                        uint4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = t + NT * (e0 + e), r = i >> 3, x = i & 7;
                            v[e] = *reinterpret_cast<const uint4*>(sraw + rs * CH + r * 128 + ((x ^ (r & 7)) << 4));
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = t + NT * (e0 + e), r = i >> 3, x = i & 7;
                            put_codes(v[e], smem_u32(sring) + s * PAIR + (x >> 2) * CH + r * 128, 2 * (x & 3), r);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&sh.raw_empty[rs]));
                        mbar_arrive(smem_u32(&sh.full[s]));
                    }
                }
            }
        }
    } else if (warp == 7) {
        // -------------------------------------------------------------- loads
        if (lane == 0) { tma_prefetch_desc(&tmTile); tma_prefetch_desc(&tmRun); tma_prefetch_desc(&tmRow); }
        // bf16: stages of 2 boxes for the MMAs; FP8: raw stages of 1 box for the converters
        constexpr int depth = FP8 ? raws : stages, chunks = FP8 ? 1 : 2, step = FP8 ? 128 : 64;
        uint64_t* full = FP8 ? sh.raw_full : sh.full;
        uint64_t* empty = FP8 ? sh.raw_empty : sh.empty;
        const uint32_t dst = smem_u32(FP8 ? sraw : sring), rope = smem_u32(srope);
        uint32_t u = 0, g = 0, nr = 0;                 // stages, tiles and rope loads so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            for (int ti = p.t0; ti < p.t1; ++ti, ++g) {
                if (!wait(&sh.tile_full[g & 1], (g >> 1) & 1)) break;
                const Half hf = read_half(sh.recs[g & 1], 0, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.tile_empty[g & 1]));
#pragma unroll 1
                for (int c = 0; c < 4; ++c, ++u) {
                    const uint32_t s = u % depth;
                    if (!wait(&empty[s], ((u / depth) & 1) ^ 1)) break;
                    load_half<false>(&tmTile, &tmRun, &tmRow, hf, dst + s * (FP8 ? CH : PAIR), smem_u32(&full[s]), smem_u32(&full[s]), chunks * CH,
                                     128 * c, step, chunks, lane);
                }
                if (!ok || !wait(&sh.r_empty[g & 1], ((g >> 1) & 1) ^ 1)) break;
                load_half<false>(&tmTile, &tmRun, &tmRow, hf, rope + (g & 1) * CH, smem_u32(&sh.r_full[g & 1]), smem_u32(&sh.r_full[g & 1]), CH,
                                 kLatent, step, 1, lane);
                ++nr;
            }
        }
        if (lane == 0) {                                // nothing is in flight when the block ends
            for (uint32_t e = 1; e <= static_cast<uint32_t>(depth) && e <= u; ++e) drain_bar(&full[(u - e) % depth], ((u - e) / depth) & 1, a.err);
            for (uint32_t e = 1; e <= 2 && e <= nr; ++e) drain_bar(&sh.r_full[(nr - e) & 1], ((nr - e) >> 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 6) {
        lookup_tiles<FP8, TT>(a, b, tile, left, 0, 0, sh.recs, sh.tile_full, sh.tile_empty, sh.live, sh.scale, sh.info_full,
                              abort_flag);
    } else if (warp == 4) {
        // ---------------------- Q of each sequence, scores: S^T of every tile as it arrives
        constexpr uint32_t id_s = idesc_bf16_f32(TT, RN);
        uint32_t u = 0, g = 0, np = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            if (!wait(&sh.q_empty, (np & 1) ^ 1)) break;      // the scores of the piece before are complete
            load_q<RN>(a, p.b, 0, rows, smem_u32(sq), lane);
            __syncwarp();
            ++np;
            for (int n = p.t1 - p.t0; n > 0; --n, ++g) {
                if (!wait(&sh.s_free[g & 1], ((g >> 1) & 1) ^ 1)) break;
                const uint32_t d = tm_s + 64 * (g & 1);
#pragma unroll 1
                for (int c = 0; c < 4; ++c, ++u) {
                    const uint32_t s = u % stages;
                    if (!wait(&sh.full[s], (u / stages) & 1)) break;
                    if (elect_one()) {
                        tc_fence_after();
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint64_t bd = smem_desc_sw128(smem_u32(sq + (2 * c + e) * QC));
                            const uint64_t ad = smem_desc_sw128(smem_u32(sring + s * PAIR + e * CH));
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_bf16(d, ad + 2ull * kk, bd + 2ull * kk, id_s, c > 0 || e > 0 || kk > 0);
                        }
                    }
                    __syncwarp();
                }
                if (!ok || !wait(&sh.r_full[g & 1], (g >> 1) & 1)) break;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t bd = smem_desc_sw128(smem_u32(sq + 8 * QC));
                    const uint64_t ad = smem_desc_sw128(smem_u32(srope + (g & 1) * CH));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16(FP8 ? tm_r + 64 * (g & 1) : d, ad + 2ull * kk, bd + 2ull * kk, id_s, !FP8 || kk > 0);
                    tc_commit(smem_u32(&sh.r_empty[g & 1]));
                    tc_commit(smem_u32(&sh.s_full[g & 1]));
                    if (n == 1) tc_commit(smem_u32(&sh.q_empty));
                }
                __syncwarp();
            }
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin[0]));
            drain_bar(&sh.fin[0], 0, a.err);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------- O^T += C^T P
        constexpr uint32_t id_o = idesc_bf16_f32_t(128, RN, 1, 1);
        uint32_t u = 0, g = 0, np = 0;
        bool ok = true;
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            for (int i = 0; i < p.t1 - p.t0; ++i, ++g) {
                if (i == 0) ok = warp_wait(smem_u32(&sh.o_empty), (np++ & 1) ^ 1, abort_flag, a.err);
                if (!ok || !(ok = warp_wait(smem_u32(&sh.p_full), g & 1, abort_flag, a.err))) break;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t bd = smem_desc_sw128_mn(smem_u32(sp), CH);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t st = (u + q) % stages;
                        const uint64_t ad = smem_desc_sw128_mn(smem_u32(sring + st * PAIR), CH);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_bf16(tm_o + q * RN, ad + 128ull * kk, bd + 128ull * kk, id_o, i > 0 || kk > 0);
                        tc_commit(smem_u32(&sh.empty[st]));
                    }
                    tc_commit(smem_u32(&sh.pv_done));
                }
                __syncwarp();
                u += 4;
            }
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin[1]));
            drain_bar(&sh.fin[1], 0, a.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------- softmax, rescaling and output
        // (a wait that gives up does not leave the loops: the four warps meet at barriers)
        // S^T rows (records) 16 w .. 16 w + 15 lie in the first 16 lanes of warp w's TMEM quarter
        const int rec = 16 * warp + (lane & 15);
        const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
        const float c = a.scale * kLog2e;
        uint32_t g = 0;
        // sequences without records: zero rows, spread over the ranges
        for (int e = range; e < a.B; e += ranges) {
            if (seq_len(a, e) != 0) continue;
            for (int i = threadIdx.x; i < rows * 64; i += 128) {
                const int q = i >> 6, jj = q / a.H, hh = q - jj * a.H;
                const long long row = static_cast<long long>(e) * a.n_q + jj;
                reinterpret_cast<uint4*>(a.out + row * a.o_row + hh * a.o_head)[i & 63] = make_uint4(0, 0, 0, 0);
                if (a.lse && (i & 63) == 0) a.lse[row * a.H + hh] = -CUDART_INF_F;
            }
        }
        while (next_piece(a, b, tile, left, &p, TT)) {
            float l[RN];
#pragma unroll
            for (int i = 0; i < RN; ++i) l[i] = 0.f;
            for (int ti = p.t0; ti < p.t1; ++ti, ++g) {
                wait_bar(smem_u32(&sh.info_full[g % kInfo]), (g / kInfo) & 1, abort_flag, a.err);
                wait_bar(smem_u32(&sh.s_full[g & 1]), (g >> 1) & 1, abort_flag, a.err);
                tc_fence_after();
                uint32_t s[RN];
#pragma unroll
                for (int q = 0; q < RN / 16; ++q) {
                    uint32_t (&part16)[16] = *reinterpret_cast<uint32_t (*)[16]>(&s[16 * q]);
                    tmem_ld16(tm_s + 64 * (g & 1) + 16 * q + lane_base, part16);
                }
                if constexpr (FP8) {
                    const float sc = sh.scale[g % kInfo][rec];
                    constexpr int W = RN == 16 ? 16 : 32;        // columns of the rotary part at a time
#pragma unroll
                    for (int q = 0; q < RN; q += W) {
                        uint32_t kr[W];
                        if constexpr (W == 16) tmem_ld16(tm_r + 64 * (g & 1) + q + lane_base, kr);
                        else tmem_ld32(tm_r + 64 * (g & 1) + q + lane_base, kr);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            s[q + i] = __float_as_uint(fmaf(__uint_as_float(s[q + i]), sc, __uint_as_float(kr[i])));
                    }
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.s_free[g & 1]));
                const bool live = lane < 16 && ((sh.live[g % kInfo][rec >> 5] >> (rec & 31)) & 1u);
                const int pos = ti * TT + rec;
                // rows of earlier new tokens see fewer positions: query j sees [0, len - (n_q - 1 - j))
                const bool edge = a.n_q > 1 && ti * TT + TT > p.len - a.n_q + 1;
                if (edge) {
#pragma unroll
                    for (int i = 0; i < RN; ++i)
                        if (pos >= p.len - sh.lag[i]) s[i] = 0xff800000u;
                }
                float over = -CUDART_INF_F;                     // the largest excess over the running maxima
                if (ti > p.t0) {
                    const float4* m4 = reinterpret_cast<const float4*>(sh.m);
#pragma unroll
                    for (int q = 0; q < RN / 4; ++q) {
                        const float4 m = m4[q];
                        over = fmaxf(over, fmaxf(fmaxf(fmaf(__uint_as_float(s[4 * q]), c, -m.x), fmaf(__uint_as_float(s[4 * q + 1]), c, -m.y)),
                                                 fmaxf(fmaf(__uint_as_float(s[4 * q + 2]), c, -m.z), fmaf(__uint_as_float(s[4 * q + 3]), c, -m.w))));
                    }
                }
                if (bar_any(1, 128, ti == p.t0 || (live && over > kRescale))) {
                    // new maxima: over the warp's records by shuffles, over the warps through shared memory
                    for (int i0 = 0; i0 < RN; i0 += 16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float v = -CUDART_INF_F;
#pragma unroll
                            for (int q = 0; q < RN / 16; ++q)
                                if (i0 == 16 * q) v = __uint_as_float(s[16 * q + i]) * c;
                            if (!live) v = -CUDART_INF_F;
#pragma unroll
                            for (int d = 8; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                            if (lane == 0) sh.red[warp][i0 + i] = v;
                        }
                    }
                    bar_sync(1, 128);
                    if (threadIdx.x < RN) {
                        const int i = threadIdx.x;
                        const float old = ti == p.t0 ? -CUDART_INF_F : sh.m[i];
                        // a row that has seen nothing yet keeps a harmless maximum of -1e30 (its p are 2^-inf = 0)
                        const float top = fmaxf(fmaxf(fmaxf(sh.red[0][i], sh.red[1][i]), fmaxf(sh.red[2][i], sh.red[3][i])), -1e30f);
                        const float nm = top > old + kRescale ? top : fmaxf(old, -1e30f);
                        sh.f[i] = exp2_fast(old - nm);
                        sh.m[i] = nm;
                    }
                    bar_sync(1, 128);
                    if (ti > p.t0) {
#pragma unroll
                        for (int i = 0; i < RN; ++i) l[i] *= sh.f[i];
                        // O^T is complete up to the tile before
                        wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < 4 * RN; cc += 16) {
                            uint32_t o[16];
                            tmem_ld16(tm_o + cc + lane_base, o);
                            tmem_ld_wait();
                            const float4* f4 = reinterpret_cast<const float4*>(&sh.f[cc % RN]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 f = f4[e];
                                o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) * f.x);
                                o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) * f.y);
                                o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) * f.z);
                                o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) * f.w);
                            }
                            tmem_st16(tm_o + cc + lane_base, o);
                        }
                        tmem_st_wait();
                    }
                }
                // P is free once the product of the tile before is done
                if (g > 0) wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
                const float4* m4 = reinterpret_cast<const float4*>(sh.m);
                const uint32_t prow = smem_u32(sp) + rec * 128;
                const float vs = FP8 ? sh.scale[g % kInfo][rec] : 1.f;      // V's rows are codes
#pragma unroll
                for (int q = 0; q < RN / 8; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 m = m4[2 * q + e];
                        const int i = 8 * q + 4 * e;
                        float x0 = exp2_fast(fmaf(__uint_as_float(s[i]), c, -m.x)), x1 = exp2_fast(fmaf(__uint_as_float(s[i + 1]), c, -m.y));
                        float x2 = exp2_fast(fmaf(__uint_as_float(s[i + 2]), c, -m.z)), x3 = exp2_fast(fmaf(__uint_as_float(s[i + 3]), c, -m.w));
                        if (!live) x0 = x1 = x2 = x3 = 0.f;
                        l[i] += x0; l[i + 1] += x1; l[i + 2] += x2; l[i + 3] += x3;
                        if constexpr (FP8) { x0 *= vs; x1 *= vs; x2 *= vs; x3 *= vs; }
                        w[2 * e] = pack_bf16x2(x0, x1);
                        w[2 * e + 1] = pack_bf16x2(x2, x3);
                    }
                    if (lane < 16) sts16(prow + ((q ^ (rec & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full));
            }
            // l over the records
#pragma unroll
            for (int i = 0; i < RN; ++i) {
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
                if (lane == 0) sh.red[warp][i] = l[i];
            }
            bar_sync(1, 128);
            const bool whole = p.t0 == 0 && p.t1 == p.n;
            const long long slot = static_cast<long long>(range) * 2 + (p.b == sh.b0 ? 0 : 1);
            if (threadIdx.x < RN) {
                const int i = threadIdx.x;
                const float z = (sh.red[0][i] + sh.red[1][i]) + (sh.red[2][i] + sh.red[3][i]);
                sh.f[i] = z != 0.f ? 1.f / z : 0.f;
                if (i < rows) {
                    const float lse = z != 0.f ? sh.m[i] + log2f(z) : -CUDART_INF_F;       // log2 units
                    const int j = i / a.H, h = i - j * a.H;
                    if (!whole) part_lse[slot * ROWS + i] = lse;
                    else if (a.lse) a.lse[(static_cast<long long>(p.b) * a.n_q + j) * a.H + h] = lse * kLn2;
                }
            }
            bar_sync(1, 128);
            wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
            tc_fence_after();
            // O^T: lane = latent element, column = row
#pragma unroll 1
            for (int cc = 0; cc < 4 * RN; cc += 16) {
                uint32_t o[16];
                tmem_ld16(tm_o + cc + lane_base, o);
                tmem_ld_wait();
                const int d = (cc / RN) * 128 + 32 * warp + lane, r0 = cc % RN;
                int qq = r0, jj = qq / a.H, hh = qq - jj * a.H;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (r0 + e < rows) {
                        const float f = sh.f[r0 + e];
                        const float v = f != 0.f ? __uint_as_float(o[e]) * f : 0.f;
                        if (whole)
                            a.out[(static_cast<long long>(p.b) * a.n_q + jj) * a.o_row + hh * a.o_head + d] = __float2bfloat16(v);
                        else
                            part[(slot * ROWS + r0 + e) * kLatent + d] = v;
                    }
                    if (++hh == a.H) { hh = 0; ++jj; }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.o_empty));
            bar_sync(1, 128);                     // every warp has read 1 / l
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

constexpr int kRanges = 152;                  // ranges at most: a block per SM of the full part

// Joins the partials of the sequences that range boundaries cut, in range order, a row on 8 / RB warps.  Block
// (boundary, RB rows, row block): of the boundaries inside a sequence, the one before range s, the first joins; with
// RB = 1 (sequence, row, row block), which looks for its s.  RB = 8 for batches (a block per row spent its time on the search for the pieces, 2 us of dependent
// loads in four waves of blocks: 64 sequences x 128 rows 15.9 us, now 9.2); RB = 1 where a sequence has more than 8
// pieces on average (one sequence of 65 pieces x 16 rows: 16 us more with a warp per row).
constexpr int kJoinWarps = 8;
static_assert(32 * kJoinWarps >= kRanges, "a thread a range");
template <int RB>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_kernel(const LatentDecodeArgs a, const int rb_count, const int ranges, const int block_rows, const float* __restrict__ part,
            const float* __restrict__ part_lse, const Meta* __restrict__ all_meta) {
    constexpr int W = kJoinWarps / RB;
    __shared__ float sums[W > 1 ? W : 1][W > 1 ? kLatent : 1];
    __shared__ int slots[kRanges];
    __shared__ float weight[kJoinWarps][kRanges];
    __shared__ int count;
    __shared__ Meta meta[kRanges];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < ranges) meta[threadIdx.x] = all_meta[threadIdx.x];      // one latency for the whole search
    __syncthreads();
    const int r = blockIdx.y * RB + warp / W, rb = blockIdx.z, q = rb * block_rows + r;
    int s = blockIdx.x + 1;
    Meta m{static_cast<int>(blockIdx.x), 1, 1, 0};
    if constexpr (RB > 1) {
        m = meta[s];
        if (m.b >= a.B || m.tiles == 0 || m.off == 0) return; // no tiles, or the sequence starts here
    }
    if (warp == 0) {
        if constexpr (RB == 1) {
            s = 0;
            for (int k0 = 0; k0 < ranges && s == 0; k0 += 32) {
                Meta mk{-1, 0, 0, 0};
                if (k0 + lane < ranges) mk = meta[k0 + lane];
                const unsigned inside = __ballot_sync(0xffffffffu, mk.b == m.b && mk.tiles > 0 && mk.off > 0);
                if (inside) s = k0 + __ffs(inside) - 1;       // (range 0 starts with a sequence)
            }
        }
        // the range before (empty ones, where there are fewer tiles than ranges, aside) holds the piece before
        int first = s - 1;
        for (; first >= 0; first -= 32) {
            const int k = first - lane;
            const unsigned some = __ballot_sync(0xffffffffu, k >= 0 && meta[k < 0 ? 0 : k].tiles > 0);
            if (some) { first -= __ffs(some) - 1; break; }
        }
        int n = 0;
        const Meta mf = meta[first < 0 ? 0 : first];
        if (s > 0 && first >= 0 && !(mf.b == m.b && mf.off > 0)) {     // else an earlier boundary is inside the sequence too
            for (int k0 = first; k0 < ranges; k0 += 32) {
                const int k = k0 + lane;
                Meta mk{-1, 0, 0, 0};
                if (k < ranges) mk = meta[k];
                const bool in = mk.tiles > 0 && (mk.b == m.b || k == first);
                const unsigned mask = __ballot_sync(0xffffffffu, in);
                if (in) slots[n + __popc(mask & ((1u << lane) - 1u))] = (k * rb_count + rb) * 2 + (mk.b == m.b ? 0 : 1);
                n += __popc(mask);
                if (__any_sync(0xffffffffu, mk.tiles > 0 && mk.b > m.b)) break;      // a later sequence's range
            }
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    if (n == 0 || r >= block_rows || q >= a.n_q * a.H) return;      // (with RB = 1 the whole block)
    float* wt = weight[warp];
    float top = -CUDART_INF_F;
    for (int k = lane; k < n; k += 32) {
        wt[k] = __ldg(part_lse + static_cast<long long>(slots[k]) * block_rows + r);
        top = fmaxf(top, wt[k]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float z = 0.f;
    for (int k = lane; k < n; k += 32) {
        wt[k] = exp2_fast(wt[k] - ref);
        z += wt[k];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    __syncwarp();
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = warp % W; k < n; k += W) {
        const float w = wt[k];
        const float4* src = reinterpret_cast<const float4*>(part + (static_cast<long long>(slots[k]) * block_rows + r) * kLatent) + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(src + 32 * i);
            acc[i].x += w * v.x; acc[i].y += w * v.y; acc[i].z += w * v.z; acc[i].w += w * v.w;
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(sums[warp])[lane + 32 * i] = acc[i];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = reinterpret_cast<const float4*>(sums[w])[lane + 32 * i];
                acc[i].x += v.x; acc[i].y += v.y; acc[i].z += v.z; acc[i].w += v.w;
            }
    }
    const float inv = z != 0.f ? 1.f / z : 0.f;
    const int j = q / a.H, h = q - j * a.H;
    const long long row = static_cast<long long>(m.b) * a.n_q + j;
    uint2* dst = reinterpret_cast<uint2*>(a.out + row * a.o_row + h * a.o_head) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        dst[32 * i] = make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (a.lse && lane == 0) a.lse[row * a.H + h] = z != 0.f ? (ref + log2f(z)) * kLn2 : -CUDART_INF_F;
}

// Up to 64 query rows: one block per range; more: CTA pairs, 128 rows each, as many ranges as there are pairs left.
// A block takes an SM's whole shared memory and ranges are of equal length, so blocks beyond the device's `sms`
// would be a second wave as long as the first.
struct Shape { int rb, ranges, block_rows; };
Shape shape(int H, int n_q, int sms) {
    sms = sms < kRanges ? sms : kRanges;
    if (H * n_q <= ROWS) return Shape{1, sms, ROWS};
    const int rb = (H * n_q + 2 * ROWS - 1) / (2 * ROWS), ranges = sms / 2 / rb;
    return Shape{rb, ranges > 0 ? ranges : 1, 2 * ROWS};
}

}  // namespace dc

// Partials of at most two cut pieces per range and row block, their lse, the ranges' descriptions; enough for any device.
size_t latent_decode_ws_bytes(int H, int, int n_q) {
    const dc::Shape s = dc::shape(H, n_q, dc::kRanges);
    const size_t slots = static_cast<size_t>(s.rb) * s.ranges * 2;
    return slots * s.block_rows * (kLatent + 1) * 4 + (s.ranges * sizeof(dc::Meta) + 255) / 256 * 256;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void* ws, cudaStream_t st) {
    static bool attr[2][3][kMaxDevices] = {{{false}}};
    using Fn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, LatentDecodeArgs, int, float*, float*, dc::Meta*);
    static const Fn fns[2][3] = {{dc::decode_kernel<false, 16>, dc::decode_kernel<false, 32>, dc::decode_kernel<false, 64>},
                                 {dc::decode_kernel<true, 16>, dc::decode_kernel<true, 32>, dc::decode_kernel<true, 64>}};
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e != cudaSuccess) return e;
    const dc::Shape sp = dc::shape(a.H, a.n_q, sms);
    const int all = a.H * a.n_q, rows = all < sp.block_rows ? all : sp.block_rows;
    CUtensorMap tile, run, row;
    const long long records = a.n_pages * a.page_size;
    const int cols = fp8 ? kRecFp8 : kLatent + kRope;          // elements of a record (FP8: bytes)
    e = make_map(&tile, a.cache, records, cols, dc::TT, fp8);
    if (e == cudaSuccess) e = make_map(&run, a.cache, records, cols, 16, fp8);
    if (e == cudaSuccess) e = make_map(&row, a.cache, records, cols, 1, fp8);
    if (e != cudaSuccess) return e;
    const size_t slots = static_cast<size_t>(sp.rb) * sp.ranges * 2;
    float* part = static_cast<float*>(ws);
    float* part_lse = part + slots * sp.block_rows * kLatent;
    dc::Meta* meta = reinterpret_cast<dc::Meta*>(part_lse + slots * sp.block_rows);
    if (sp.block_rows > dc::ROWS) {
        e = launch_decode_pair(tile, run, row, a, fp8, sp.rb, sp.ranges, part, part_lse, meta, st);
    } else {
        const int v = rows <= 16 ? 0 : (rows <= 32 ? 1 : 2);
        const Fn fn = fns[fp8][v];
        e = smem_attr_once(reinterpret_cast<const void*>(fn), dc::SMEM, attr[fp8][v]);
        if (e != cudaSuccess) return e;
        fn<<<static_cast<unsigned>(sp.ranges), 32 * (8 + (!fp8 ? 0 : (v == 2 ? 4 : 8))), dc::SMEM, st>>>(
            tile, run, row, a, sp.ranges, part, part_lse, meta);
        count_launch();
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || sp.ranges == 1) return e;
    if (a.B <= sp.ranges / 8)
        dc::join_kernel<1><<<dim3(a.B, rows, sp.rb), 32 * dc::kJoinWarps, 0, st>>>(a, sp.rb, sp.ranges, sp.block_rows, part, part_lse, meta);
    else
        dc::join_kernel<8><<<dim3(sp.ranges - 1, (rows + 7) / 8, sp.rb), 32 * dc::kJoinWarps, 0, st>>>(a, sp.rb, sp.ranges, sp.block_rows, part, part_lse, meta);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
