// latent_decode_pair.cu -- absorbed latent attention for more than 64 query rows (new tokens x heads)
// a sequence, on CTA pairs:
//   S = Q K^T   128 rows x 128 records x 576,   O += P C   128 rows x 512 x 128 records
// The pair's 2-SM MMAs (M = 128) give each CTA 64 rows: its Q (73.7 KB) stays in shared memory and its
// accumulators take 64 columns of S and 256 of O (an accumulator's first half of columns lies in
// lanes 0-63, the second in 64-127), so 128 rows meet in one pass over the records what one CTA's TMEM
// could not hold.  An M = 128 pair MMA costs 73 cycles at N = 128 and 105 at N = 256 where two CTAs of 64
// rows would spend 2 x 60 and 4 x 75: 4,308 cycles for 128 records instead of 6,720.
//
// The B operands split over the pair: for S each CTA holds its 64 records x 576, for P C all 128
// records x half of the 512 columns.  Both come as stages of 64 records x 128 columns through one ring in
// the order of their use, K(0) K(1) V(0) K(2) V(1) ..., so a stage is held only from its arrival to its
// MMAs and seven loads are always under way; V's second read hits L2 (a stage read twice costs 32 of
// the 40 bytes a cycle that L2 gives an SM, measured).  S(i+1) runs while the softmax of tile i does.
//
// Bound: with 128 rows a record's 139 k multiply-adds meet its 1,152 bytes at about the balance of tensor
// rate and memory; here the MMAs' fixed costs decide.  Measured: 64 sequences of 2,000 to 14,000 tokens x 128
// heads, bf16 cache, 164 us (890 TFLOP/s, 3.8 TB/s; on blocks of 64 rows it was 388 us); 32 sequences x
// 128 heads x 2 new tokens, FP8 cache, 149 us (its 512 threads leave 128 registers: 20 bytes are spilled).
//
// Per CTA: warps 0-3 softmax, rescaling and output (thread = row of the lane and half of the records);
// warp 4 MMA issue in the even CTA, in the odd one it tells the even CTA which stages have
// arrived; warp 5 Q; warp 6 page lookup; warp 7 TMA; FP8: warps 8-15 turn raw codes into bf16 stages.
#include "kernels.h"
#include "latent_decode.cuh"

namespace fs {
namespace dp {
using namespace dc;

constexpr int TT = 128;                       // records per tile
constexpr int ROWS = 64;                      // query rows per CTA
constexpr int MAXP = 7, MAXRAW = 4;
constexpr int CTRL = 7168;
template <bool FP8> constexpr int kThreads = FP8 ? 512 : 256;

struct Shared {
    uint64_t full[MAXP], empty[MAXP], peer[MAXP], raw_full[MAXRAW], raw_empty[MAXRAW], r_full[2], r_empty[2], info_full[kInfo], tile_full[2], tile_empty[2];
    uint64_t q_full, q_empty, s_full[2], p_full, pv_done, o_empty, fin;
    uint32_t tmem;
    int abort_flag;
    int b0, tile0, left;
    uint32_t live[kInfo][4];                  // records of a tile that count
    // What the two warps of a row hand each other: its maximum over their halves of a tile's records, and its sum of p.
    // Arrays of their own: a maximum is read behind the barrier that follows its write, but from there to a piece's
    // end, where the sums are written, no barrier need follow (the piece's last tile may have raised the maximum).
    // Each array's next write lies behind a barrier that its readers reach after reading: the next tile's bar_any, the
    // barrier at the piece's end.
    float red[2][ROWS], sum[2][ROWS];
    alignas(16) float scale[kInfo][TT];       // FP8: the records' scales
    TileRecs<TT> recs[2];
};
static_assert(sizeof(Shared) <= CTRL, "control area");

// Arrive on a barrier of the pair's even CTA (shared::cluster address).  What the arrival publishes is shared
// memory that only the tensor cores of its own SM read, made visible to them by fence.proxy.async before;
// with a cluster-scope release, which it does not need, an arrival costs about 1,000 cycles.
__device__ __forceinline__ void arrive_even(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

template <bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<FP8>, 1)
decode_pair_kernel(const __grid_constant__ CUtensorMap tmTile, const __grid_constant__ CUtensorMap tmRun, const __grid_constant__ CUtensorMap tmRow,
                   const LatentDecodeArgs a, const int rb_count, const int ranges, float* __restrict__ part,
                   float* __restrict__ part_lse, Meta* __restrict__ meta) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int cid = static_cast<int>(blockIdx.x >> 1), rb = cid % rb_count, range = cid / rb_count;
    const int row0 = rb * 2 * ROWS + rank * ROWS;                     // first query row of this CTA
    const int rows = max(0, min(ROWS, a.n_q * a.H - row0));
    constexpr int QC = ROWS * 128, raws = FP8 ? 4 : 0, stages = FP8 ? 5 : 7;
    uint8_t* sq = smem;                            // Q: 9 chunks of 64 rows x 64 columns
    uint8_t* sp = smem + 9 * QC;                   // P: 2 chunks of 64 rows x 64 records
    uint8_t* srope = sp + 2 * CH;                  // rotary keys of this CTA's 64 records, twice
    uint8_t* sraw = srope + 2 * CH;
    uint8_t* sring = sraw + raws * CH;
    static_assert(9 * QC + (4 + raws) * CH + stages * PAIR + CTRL <= SMEM && stages <= MAXP && raws <= MAXRAW, "shared memory");
    Shared& sh = *reinterpret_cast<Shared*>(smem + (SMEM - CTRL));
    volatile int* abort_flag = &sh.abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAXP; ++i) {
            mbar_init(smem_u32(&sh.full[i]), FP8 ? 2 : 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            mbar_init(smem_u32(&sh.peer[i]), 1);
        }
        for (int i = 0; i < MAXRAW; ++i) { mbar_init(smem_u32(&sh.raw_full[i]), 1); mbar_init(smem_u32(&sh.raw_empty[i]), 2); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.r_full[i]), 1);
            mbar_init(smem_u32(&sh.r_empty[i]), 1);
        }
        for (int i = 0; i < kInfo; ++i) mbar_init(smem_u32(&sh.info_full[i]), 1);
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&sh.tile_full[i]), 1); mbar_init(smem_u32(&sh.tile_empty[i]), 1); }
        mbar_init(smem_u32(&sh.q_full), 2);        // a warp of each CTA
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.s_full[0]), 1);
        mbar_init(smem_u32(&sh.s_full[1]), 1);
        mbar_init(smem_u32(&sh.p_full), 8);        // four warps of each CTA
        mbar_init(smem_u32(&sh.pv_done), 1);
        mbar_init(smem_u32(&sh.o_empty), 8);
        mbar_init(smem_u32(&sh.fin), 1);
        sh.abort_flag = 0;
        fence_mbar_init();
        if (smem_u32(smem) & 1023u) set_dev_error(a.err, DEV_ERR_LIMIT);
    }
    if (warp == 4) {
        tmem_alloc_pair(smem_u32(&sh.tmem), 512);
        tmem_relinquish_pair();
    }
    if (warp == 0) find_range(a, range, ranges, TT, rb == 0 && rank == 0, meta, &sh.b0, &sh.tile0, &sh.left);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                // both CTAs' barriers exist before either signals them
    tc_fence_after();
    // S twice (64 columns each), FP8: its rotary part twice, O (2 x 128)
    const uint32_t tm_s = sh.tmem, tm_r = sh.tmem + 128, tm_o = sh.tmem + 256;
    int b = sh.b0, tile = sh.tile0, left = (smem_u32(smem) & 1023u) ? 0 : sh.left;
    Piece p;
    // the even CTA's copy of a barrier
    auto leader_bar = [&](uint64_t* bar) { return map_to_cta(smem_u32(bar), 0); };

    if (warp >= 8) {
        // ------------------------------------------- FP8 codes to bf16 stages
        if constexpr (FP8) {
            // two warps per stage, four stages at once
            const int t = threadIdx.x & 63, c = (threadIdx.x - 256) >> 6;
            uint32_t u = c;
            bool ok = true;
            while (ok && next_piece(a, b, tile, left, &p, TT)) {
                for (int n = 2 * (p.t1 - p.t0); n > 0; --n, u += 4) {
                    const uint32_t rs = u % MAXRAW, s = u % stages;
                    if (!warp_wait(smem_u32(&sh.raw_full[rs]), (u / MAXRAW) & 1, abort_flag, a.err) ||
                        !warp_wait(smem_u32(&sh.empty[s]), ((u / stages) & 1) ^ 1, abort_flag, a.err)) { ok = false; break; }
#pragma unroll
                    for (int e0 = 0; e0 < 8; e0 += 4) {
                        uint4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = t + 64 * (e0 + e), r = i >> 3, x = i & 7;
                            v[e] = *reinterpret_cast<const uint4*>(sraw + rs * CH + r * 128 + ((x ^ (r & 7)) << 4));
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = t + 64 * (e0 + e), r = i >> 3, x = i & 7;
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
        constexpr int depth = FP8 ? MAXRAW : stages, chunks = FP8 ? 1 : 2, step = FP8 ? 128 : 64;
        uint64_t* full = FP8 ? sh.raw_full : sh.full;
        uint64_t* empty = FP8 ? sh.raw_empty : sh.empty;
        const uint32_t dst = smem_u32(FP8 ? sraw : sring);
        uint32_t u = 0, g = 0;                          // stages and tiles so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        auto stage = [&](const Half& gr, int col) {
            const uint32_t s = u % depth;
            if (!wait(&empty[s], ((u / depth) & 1) ^ 1)) return false;
            const uint32_t lb = smem_u32(&full[s]);
            // bf16: both CTAs' loads complete on the even CTA's barrier, which expects the bytes of both
            if constexpr (FP8)
                load_half<false>(&tmTile, &tmRun, &tmRow, gr, dst + s * CH, lb, lb, CH, col, step, chunks, lane);
            else
                load_half<true>(&tmTile, &tmRun, &tmRow, gr, dst + s * PAIR, map_to_cta(lb, 0), lb, rank ? 0 : 2 * PAIR, col, step, chunks, lane);
            ++u;
            return true;
        };
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            Half cur[2], nxt[2];
            // K of tile ti (its halves into nxt), then V of tile ti - 1 (cur)
            for (int ti = p.t0; ti <= p.t1 && ok; ++ti) {
                if (ti < p.t1) {
                    if (!wait(&sh.tile_full[g & 1], (g >> 1) & 1)) break;
                    nxt[0] = read_half(sh.recs[g & 1], 0, lane);
                    nxt[1] = read_half(sh.recs[g & 1], 1, lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.tile_empty[g & 1]));
                    const Half own = rank ? nxt[1] : nxt[0];
                    for (int c = 0; c < 4 && ok; ++c) stage(own, 128 * c);
                    if (!ok || !wait(&sh.r_empty[g & 1], ((g >> 1) & 1) ^ 1)) break;
                    load_half<true>(&tmTile, &tmRun, &tmRow, own, smem_u32(srope) + (g & 1) * CH, leader_bar(&sh.r_full[g & 1]),
                                    smem_u32(&sh.r_full[g & 1]), rank ? 0 : 2 * CH, kLatent, step, 1, lane);
                    ++g;
                }
                if (ti > p.t0)                          // V: column halves j, record halves h
                    for (int c = 0; c < 4 && ok; ++c) stage(c & 1 ? cur[1] : cur[0], 256 * (c >> 1) + 128 * rank);
                cur[0] = nxt[0];
                cur[1] = nxt[1];
            }
        }
        if (lane == 0) {                                // nothing is in flight when the block ends
            // (the even CTA waits for both CTAs' loads; the pair leaves together)
            if (FP8 || rank == 0)
                for (uint32_t e = 1; e <= static_cast<uint32_t>(depth) && e <= u; ++e) drain_bar(&full[(u - e) % depth], ((u - e) / depth) & 1, a.err);
            if (rank == 0)
                for (uint32_t e = 1; e <= 2 && e <= g; ++e) drain_bar(&sh.r_full[(g - e) & 1], ((g - e) >> 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 6) {
        lookup_tiles<FP8, TT>(a, b, tile, left, rank, rank, sh.recs, sh.tile_full, sh.tile_empty, sh.live, sh.scale,
                              sh.info_full, abort_flag);
    } else if (warp == 5) {
        // ------------------------------------------------ Q of each sequence
        uint32_t np = 0;
        while (next_piece(a, b, tile, left, &p, TT)) {
            if (!warp_wait(smem_u32(&sh.q_empty), (np & 1) ^ 1, abort_flag, a.err)) break;
            load_q<ROWS>(a, p.b, row0, rows, smem_u32(sq), lane);
            __syncwarp();
            if (lane == 0) arrive_even(leader_bar(&sh.q_full));
            ++np;
        }
    } else if (warp == 4 && rank == 1) {
        // ------------- FP8: the even CTA learns which stages are converted here
        uint32_t u = 0;
        bool ok = FP8;
        auto pass = [&](uint64_t* bar, uint64_t* peer, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            if (ok && lane == 0) arrive_even(leader_bar(peer));
            __syncwarp();
        };
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            for (int ti = p.t0; ti <= p.t1 && ok; ++ti) {
                if (ti < p.t1) {
                    for (int c = 0; c < 4 && ok; ++c, ++u) pass(&sh.full[u % stages], &sh.peer[u % stages], (u / stages) & 1);
                }
                if (ti > p.t0)
                    for (int c = 0; c < 4 && ok; ++c, ++u) pass(&sh.full[u % stages], &sh.peer[u % stages], (u / stages) & 1);
            }
        }
    } else if (warp == 4) {
        // ---------------------------------------------------------------- MMA
        constexpr uint32_t id_s = idesc_bf16_f32(2 * ROWS, TT), id_o = idesc_bf16_f32_t(2 * ROWS, 256, 0, 1);
        uint32_t u = 0, g = 0, np = 0, gp = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        auto wait_stage = [&](uint32_t uu) {
            const uint32_t s = uu % stages, par = (uu / stages) & 1;
            if (lane == 0)
                ok = wait_bar(smem_u32(&sh.full[s]), par, abort_flag, a.err) &&
                     (!FP8 || wait_bar(smem_u32(&sh.peer[s]), par, abort_flag, a.err));
            ok = __shfl_sync(0xffffffffu, ok, 0);
            return ok;
        };
        auto ring = [&](uint32_t uu) { return smem_u32(sring + (uu % stages) * PAIR); };
        auto score = [&]() {                              // S of tile g
            const uint32_t d = tm_s + 64 * (g & 1);
            for (int c = 0; c < 4; ++c, ++u) {
                if (!wait_stage(u)) return;
                if (elect_one()) {
                    tc_fence_after();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t ad = smem_desc_sw128(smem_u32(sq + (2 * c + e) * QC)), bd = smem_desc_sw128(ring(u) + e * CH);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_bf16_pair(d, ad + 2ull * kk, bd + 2ull * kk, id_s, c > 0 || e > 0 || kk > 0);
                    }
                    tc_commit_pair_multicast(smem_u32(&sh.empty[u % stages]), 3);
                }
                __syncwarp();
            }
            if (!wait(&sh.r_full[g & 1], (g >> 1) & 1)) return;
            if (elect_one()) {
                tc_fence_after();
                const uint64_t ad = smem_desc_sw128(smem_u32(sq + 8 * QC)), bd = smem_desc_sw128(smem_u32(srope) + (g & 1) * CH);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_bf16_pair(FP8 ? tm_r + 64 * (g & 1) : d, ad + 2ull * kk, bd + 2ull * kk, id_s, !FP8 || kk > 0);
                tc_commit_pair_multicast(smem_u32(&sh.r_empty[g & 1]), 3);
                tc_commit_pair_multicast(smem_u32(&sh.s_full[g & 1]), 3);
            }
            __syncwarp();
            ++g;
        };
        while (ok && next_piece(a, b, tile, left, &p, TT)) {
            if (!wait(&sh.q_full, np & 1)) break;
            const int n = p.t1 - p.t0;
            score();
            for (int i = 0; ok && i < n; ++i, ++gp) {
                if (i + 1 < n) score();
                if (!ok) break;
                if (i + 2 >= n && (i + 2 == n || n == 1) && elect_one()) tc_commit_pair_multicast(smem_u32(&sh.q_empty), 3);
                __syncwarp();
                if (i == 0 && !wait(&sh.o_empty, (np & 1) ^ 1)) break;
                if (!wait(&sh.p_full, gp & 1)) break;
                for (int c = 0; c < 4; ++c, ++u) {        // column half j = c / 2, record half h = c % 2
                    if (!wait_stage(u)) break;
                    if (elect_one()) {
                        tc_fence_after();
                        const uint64_t ad = smem_desc_sw128(smem_u32(sp + (c & 1) * CH)), bd = smem_desc_sw128_mn(ring(u), CH);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_bf16_pair(tm_o + 128 * (c >> 1), ad + 2ull * kk, bd + 128ull * kk, id_o,
                                             i > 0 || (c & 1) || kk > 0);
                        tc_commit_pair_multicast(smem_u32(&sh.empty[u % stages]), 3);
                        if (c == 3) tc_commit_pair_multicast(smem_u32(&sh.pv_done), 3);
                    }
                    __syncwarp();
                }
            }
            ++np;
        }
        if (elect_one()) {
            tc_commit_pair_multicast(smem_u32(&sh.fin), 1);
            drain_bar(&sh.fin, 0, a.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------- softmax, rescaling and output
        // (a wait that gives up does not leave the loops: the four warps meet at barriers)
        const int th = warp >> 1, hr = 32 * (warp & 1) + lane;         // half of the records, row of the CTA
        const bool mine = hr < rows;
        const int qrow = row0 + (mine ? hr : 0), j = min(qrow / a.H, a.n_q - 1), h = qrow - j * a.H;
        const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
        const float c = a.scale * kLog2e;
        uint32_t g = 0;
        for (int e = range; e < a.B; e += ranges) {                    // sequences without records: zero rows
            if (seq_len(a, e) != 0) continue;
            for (int i = threadIdx.x; i < rows * 64; i += 128) {
                const int q = row0 + (i >> 6), jj = q / a.H, hh = q - jj * a.H;
                const long long row = static_cast<long long>(e) * a.n_q + jj;
                reinterpret_cast<uint4*>(a.out + row * a.o_row + hh * a.o_head)[i & 63] = make_uint4(0, 0, 0, 0);
                if (a.lse && (i & 63) == 0) a.lse[row * a.H + hh] = -CUDART_INF_F;
            }
        }
        while (next_piece(a, b, tile, left, &p, TT)) {
            const int end = mine ? p.len - (a.n_q - 1 - j) : 0;        // this row sees positions [0, end)
            float m = -CUDART_INF_F, l = 0.f;
            for (int ti = p.t0; ti < p.t1; ++ti, ++g) {
                wait_bar(smem_u32(&sh.info_full[g % kInfo]), (g / kInfo) & 1, abort_flag, a.err);
                wait_bar(smem_u32(&sh.s_full[g & 1]), (g >> 1) & 1, abort_flag, a.err);
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(tm_s + 64 * (g & 1) + lane_base, s[0]);
                tmem_ld32(tm_s + 64 * (g & 1) + 32 + lane_base, s[1]);
                tmem_ld_wait();
                const float4* sc4 = reinterpret_cast<const float4*>(&sh.scale[g % kInfo][64 * th]);
                if constexpr (FP8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t kr[16];
                        tmem_ld16(tm_r + 64 * (g & 1) + 16 * q + lane_base, kr);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 f = sc4[4 * q + e];
                            const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                uint32_t& v = s[q >> 1][16 * (q & 1) + 4 * e + z];
                                v = __float_as_uint(fmaf(__uint_as_float(v), fs[z], __uint_as_float(kr[4 * e + z])));
                            }
                        }
                    }
                }
                const int lim = end - ti * TT - 64 * th;
                uint32_t live[2] = {sh.live[g % kInfo][2 * th], sh.live[g % kInfo][2 * th + 1]};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int k = lim - 32 * q;
                    live[q] &= k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
                }
                if (__any_sync(0xffffffffu, (live[0] & live[1]) != 0xffffffffu)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((live[q] >> e) & 1u)) s[q][e] = 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = __uint_as_float(s[q >> 1][16 * (q & 1)]);
#pragma unroll
                    for (int e = 1; e < 16; ++e) mx[q] = fmaxf(mx[q], __uint_as_float(s[q >> 1][16 * (q & 1) + e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool first = ti == p.t0;
                if (bar_any(1, 128, first || top > m + kRescale)) {
                    // the row's other half of the records, in the other warp
                    sh.red[th][hr] = top;
                    bar_sync(1, 128);
                    const float t = fmaxf(fmaxf(top, sh.red[th ^ 1][hr]), -1e30f);    // -1e30: nothing seen yet
                    const float nm = first || t > m + kRescale ? t : m;
                    const float f = exp2_fast(m - nm);
                    m = nm;
                    l *= f;
                    if (!first) {
                        wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < 256; cc += 32) {
                            uint32_t o[32];
                            tmem_ld32(tm_o + cc + lane_base, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(tm_o + cc + lane_base, o);
                        }
                        tmem_st_wait();
                    }
                }
                // p, then P once the product of the tile before has read it
                float sum[2] = {0.f, 0.f};
                uint32_t w[32];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = exp2_fast(fmaf(__uint_as_float(s[q >> 3][4 * (q & 7) + e]), c, -m));
                    sum[0] += x[0] + x[2];
                    sum[1] += x[1] + x[3];
                    if constexpr (FP8) {                               // V's rows are codes
                        const float4 f = sc4[q];
                        x[0] *= f.x; x[1] *= f.y; x[2] *= f.z; x[3] *= f.w;
                    }
                    w[2 * q] = pack_bf16x2(x[0], x[1]);
                    w[2 * q + 1] = pack_bf16x2(x[2], x[3]);
                }
                l += sum[0] + sum[1];
                if (g > 0) wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
                const uint32_t prow = smem_u32(sp) + th * CH + hr * 128;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    sts16(prow + ((q ^ (hr & 7)) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_even(leader_bar(&sh.p_full));
            }
            sh.sum[th][hr] = l;
            bar_sync(1, 128);
            const float z = l + sh.sum[th ^ 1][hr];
            const float inv = z != 0.f ? 1.f / z : 0.f;
            const bool whole = p.t0 == 0 && p.t1 == p.n;
            const long long slot = (static_cast<long long>(range) * rb_count + rb) * 2 + (p.b == sh.b0 ? 0 : 1);
            const long long prow = slot * 2 * ROWS + rank * ROWS + hr;
            const long long orow = static_cast<long long>(p.b) * a.n_q + j;
            if (mine && th == 0) {
                const float lse = z != 0.f ? m + log2f(z) : -CUDART_INF_F;     // log2 units
                if (!whole) part_lse[prow] = lse;
                else if (a.lse) a.lse[orow * a.H + h] = lse * kLn2;
            }
            wait_bar(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err);
            tc_fence_after();
            // O: TMEM column 128 j + i of lanes 64 th .. is output element 256 j + 128 th + i
#pragma unroll 1
            for (int cc = 0; cc < 256; cc += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(tm_o + cc + lane_base, o);
                tmem_ld_wait();
                if (!mine) continue;
                const int d = 256 * (cc >> 7) + 128 * th + (cc & 127);
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = inv != 0.f ? __uint_as_float(o[e]) * inv : 0.f;
                if (whole) {
                    uint4* dst = reinterpret_cast<uint4*>(a.out + orow * a.o_row + h * a.o_head + d);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        dst[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                            pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + prow * kLatent + d);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(leader_bar(&sh.o_empty));
            bar_sync(1, 128);                     // every warp has read the other half's sum
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                               // no CTA leaves while the other may still signal it
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc_pair(sh.tmem, 512);
    }
}

}  // namespace dp

cudaError_t launch_decode_pair(const CUtensorMap& tile, const CUtensorMap& run, const CUtensorMap& row, const LatentDecodeArgs& a, bool fp8,
                               int rb, int ranges, float* part, float* part_lse, void* meta, cudaStream_t st) {
    static bool attr[2][kMaxDevices] = {{false}};
    auto fn = fp8 ? dp::decode_pair_kernel<true> : dp::decode_pair_kernel<false>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), dc::SMEM, attr[fp8]);
    if (e != cudaSuccess) return e;
    fn<<<static_cast<unsigned>(2 * rb * ranges), fp8 ? 512 : 256, dc::SMEM, st>>>(tile, run, row, a, rb, ranges, part, part_lse,
                                                                                  static_cast<dc::Meta*>(meta));
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
