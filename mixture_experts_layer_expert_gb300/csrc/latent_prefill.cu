// latent_prefill.cu -- expanded latent attention over packed sequences:
//   s_ij = scale (q_n,i . k_n,j + q_r,i . k_r,j),  out_i = sum_j softmax(s_i)_j v_j,  lse_i = log sum_j exp(s_ij)
//
// One pass over the keys with a running maximum M and sum l per query row, on
// the tensor cores.  A work item is 256 query rows of one head, as two tiles of
// 128 (t = 0, 1); keys come in tiles of 128:
//   S_t = Q_t K^T     128 x 128 x 192, operands in shared memory, S in TMEM
//   P_t = 2^(S_t scale log2 e - M), bf16, back into S_t's TMEM columns
//   O_t += P_t V      128 x 128 x 128, P from TMEM, V read MN-major where TMA left it
// TMEM: S_0, S_1, O_0, O_1, 128 columns each.  While one tile's softmax runs on
// its four warps, the other tile's MMAs run, so the tensor cores see a stream
// of S_0(i+1), PV_1(i), S_1(i+1), PV_0(i+1), ...: MMAs of one thread execute in
// issue order, so S_t(i+1) may overwrite P_t(i) right behind PV_t(i).
// O is rescaled only when a row's maximum grows by more than 8 (a factor 2^8):
// P then stays below 2^8, which costs no precision in bf16 or fp32, and the
// TMEM round trip of O is rare after a sequence's first tiles.
//
// Bound: 2 x 128 x 128 x 320 flops per key tile and query tile; q, k, v and out
// are a few bytes per thousand flops.  Exponentials, 128 x 128 per tile, take
// less issue time than the tile's MMAs: 12 x 107 + 8 x 75 = 1,884 cycles (an MMA
// with both operands in shared memory costs 43 cycles beside N / 2).  Measured: 4 x
// 2,048 tokens x 128 heads, causal, 620 us, 1.11 PFLOP/s of the pairs that count; the
// tiles on the diagonal do 1/17 more than those.
//
// Warps 0-3 / 4-7: softmax and output of tile 0 / 1 (thread = row = TMEM lane);
// warp 8: work distribution and TMA loads; warp 9: MMA issue.  K, V and the
// shared rotary key go through a ring of eight 16 KB units (128 rows x 64
// columns): three of K (two of k_n, one of k_r), two of V per key tile, one barrier
// for each three and two.
// Blocks take further items from the grid's not yet started blocks (cluster
// launch control), so the next item's loads overlap this item's last tiles, and
// items are numbered with the longest key range of each sequence first.
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "handover.h"
#include "kernels.h"
#include "latent.cuh"

namespace fs {
namespace pf {

constexpr int TQ = 128, TK = 128;
constexpr int UNIT = 128 * 64 * 2;              // 16 KB
constexpr int NU = 8;                           // ring units
constexpr int Q_UNITS = 6;                      // two tiles x 192 columns
constexpr int RING_OFF = Q_UNITS * UNIT;
constexpr int BAR_OFF = RING_OFF + NU * UNIT;
constexpr int THREADS = 320;
constexpr size_t SMEM = 1024 + BAR_OFF + 512;
constexpr float kRescale = 8.0f;                // log2 of the growth of the maximum that rescales O

struct Item {
    int valid;            // 1: work, 0: nothing to do for this number, -1: no more items
    int head, row0, rows; // first query row, rows of the item (1 .. 256)
    int k0, lk;           // first key row, keys
    int off;              // lk - lq + (first row's index in its sequence): row r sees keys < off + r + 1 (causal)
    int n[2];             // key tiles of each query tile
};

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, q_empty, s_full[2], p_full[2], pv_done[2], item_full[2], item_empty[2];
    uint64_t next_bar, fin;
    alignas(16) uint32_t next_resp[4];
    uint32_t tmem;
    int abort_flag;
    Item item[2];
};
static_assert(sizeof(Shared) <= 512, "barrier area");

__device__ __forceinline__ int row_limit(const Item& it, bool causal, int r) {
    return causal ? min(it.lk, it.off + r + 1) : it.lk;
}

// A warp's 32 rows x 64 bytes, a row a lane: four lanes exchange their 16-byte chunks, so that a store instruction covers
// eight rows' whole 64-byte runs instead of 32 rows' 16 bytes.
__device__ __forceinline__ void store_rows(int lane, const uint32_t* w, uint8_t* dst, long long row_bytes, int rows) {
    const int q = lane & 3;
    uint32_t got[4][4];                          // [s]: chunk q of the row of lane ^ s
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = (q ^ s) & 1 ? w[4 + e] : w[e], hi = (q ^ s) & 1 ? w[12 + e] : w[8 + e];
            got[s][e] = __shfl_xor_sync(0xffffffffu, (q ^ s) & 2 ? hi : lo, s);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = (lane & ~3) + j;           // this row came in round j ^ q
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = (j ^ q) & 1 ? got[1][e] : got[0][e], hi = (j ^ q) & 1 ? got[3][e] : got[2][e];
            v[e] = (j ^ q) & 2 ? hi : lo;
        }
        if (r < rows) *reinterpret_cast<uint4*>(dst + r * row_bytes + 16 * q) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

__global__ void __launch_bounds__(THREADS, 1)
prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKn,
               const __grid_constant__ CUtensorMap tmKr, const __grid_constant__ CUtensorMap tmV,
               const LatentPrefillArgs a, const int max_tiles) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& sh = *reinterpret_cast<Shared*>(smem + BAR_OFF);
    volatile int* abort_flag = &sh.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sh.k_full[t]), 1);
            mbar_init(smem_u32(&sh.k_empty[t]), 1);
            mbar_init(smem_u32(&sh.v_full[t]), 1);
            mbar_init(smem_u32(&sh.v_empty[t]), 1);
            mbar_init(smem_u32(&sh.s_full[t]), 1);
            mbar_init(smem_u32(&sh.p_full[t]), 128);
            mbar_init(smem_u32(&sh.pv_done[t]), 1);
            mbar_init(smem_u32(&sh.item_full[t]), 1);
            mbar_init(smem_u32(&sh.item_empty[t]), 9);
        }
        mbar_init(smem_u32(&sh.next_bar), 1);
        mbar_init(smem_u32(&sh.fin), 1);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm_s = sh.tmem, tm_o = sh.tmem + 256;      // S_t at 128 t, O_t at 256 + 128 t

    const uint32_t ring = smem_u32(smem + RING_OFF);
    if (warp == 8) {
        // ------------------------------------------------ items and loads
        if (lane == 0) {
            tma_prefetch_desc(&tmQ); tma_prefetch_desc(&tmKn); tma_prefetch_desc(&tmKr); tma_prefetch_desc(&tmV);
        }
        uint32_t j = 0, u = 0;        // key tiles loaded so far, the ring unit the next one starts at
        uint32_t nq = 0, nk = 0, nv = 0;      // loads of Q, K and V tiles so far
        int id = blockIdx.x;
        bool ok = true;
        HandOver ho;
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1, use = k >> 1;
            if (id >= 0) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_u32(&sh.next_bar), 16);
                    next_block_request(smem_u32(sh.next_resp), smem_u32(&sh.next_bar));
                }
                ho.ask();
            }
            Item it{};
            it.valid = id < 0 ? -1 : 0;
            if (id >= 0) {
                it.head = id / max_tiles;
                // counted from the back: the last tiles of a sequence have the longest key ranges
                PackedSeq s;
                const int tile = find_tile(a.cu_q, a.cu_k, a.B, a.Tq, a.Tk, 2 * TQ, false,
                                           max_tiles - 1 - (id - it.head * max_tiles), a.err, &s);
                if (tile >= 0) {
                    it.valid = 1;
                    it.row0 = s.q0 + tile * 2 * TQ;
                    it.rows = min(2 * TQ, s.lq - tile * 2 * TQ);
                    it.k0 = s.k0;
                    it.lk = s.lk;
                    it.off = s.lk - s.lq + tile * 2 * TQ;
                    for (int t = 0; t < 2; ++t) {
                        const int last = min(it.rows, TQ * (t + 1)) - 1;
                        it.n[t] = last < TQ * t ? 0 : (max(0, row_limit(it, a.causal, last)) + TK - 1) / TK;
                    }
                }
            }
            ok = warp_wait(smem_u32(&sh.item_empty[slot]), (use & 1) ^ 1, abort_flag, a.err);
            if (!ok) break;
            if (lane == 0) {
                sh.item[slot] = it;
                mbar_arrive(smem_u32(&sh.item_full[slot]));
            }
            if (id < 0) break;
            const int n = max(it.n[0], it.n[1]);
            if (it.valid == 1 && n > 0 && lane == 0) {
                ok = wait_bar(smem_u32(&sh.q_empty), (nq & 1) ^ 1, abort_flag, a.err);
                if (ok) {
                    ++nq;
                    const uint32_t fb = smem_u32(&sh.q_full);
                    const int tiles = it.rows > TQ ? 2 : 1;
                    mbar_arrive_expect_tx(fb, tiles * 3 * UNIT);
                    for (int t = 0; t < tiles; ++t)
                        for (int c = 0; c < 3; ++c)
                            tma_load_3d(smem_u32(smem + (3 * t + c) * UNIT), &tmQ, fb, 64 * c, it.head,
                                        it.row0 + TQ * t);
                }
                // K of tile j takes the units that V and the last of K of tile j - 2 held, V those of K of tile j - 1 ...
                // (units 5 j .. 5 j + 4 of a ring of 8): waits on whole K and V tiles, a barrier each
                for (int i = 0; ok && i < n; ++i, ++j, u = (u + 5) & 7) {
                    const int row = it.k0 + TK * i, par = j & 1;
                    const uint32_t ph = (j >> 1) & 1;
                    ok = wait_bar(smem_u32(&sh.v_empty[par]), ph ^ 1, abort_flag, a.err) &&
                         wait_bar(smem_u32(&sh.k_empty[par]), ph ^ 1, abort_flag, a.err);
                    if (!ok) break;
                    uint32_t fb = smem_u32(&sh.k_full[par]);
                    mbar_arrive_expect_tx(fb, 3 * UNIT);
                    tma_load_3d(ring + u * UNIT, &tmKn, fb, 0, it.head, row);
                    tma_load_3d(ring + ((u + 1) & 7) * UNIT, &tmKn, fb, 64, it.head, row);
                    tma_load_3d(ring + ((u + 2) & 7) * UNIT, &tmKr, fb, 0, 0, row);
                    ++nk;
                    if (j > 0) ok = wait_bar(smem_u32(&sh.k_empty[par ^ 1]), ((j - 1) >> 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    fb = smem_u32(&sh.v_full[par]);
                    mbar_arrive_expect_tx(fb, 2 * UNIT);
                    tma_load_3d(ring + ((u + 3) & 7) * UNIT, &tmV, fb, 0, it.head, row);
                    tma_load_3d(ring + ((u + 4) & 7) * UNIT, &tmV, fb, 64, it.head, row);
                    ++nv;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                ok = wait_bar(smem_u32(&sh.next_bar), ho.parity(), abort_flag, a.err);
                if (ok) id = next_block_answer(smem_u32(sh.next_resp));
                fence_proxy_async_smem();        // the answer is read before the next one may be written
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ho.answer();
            id = __shfl_sync(0xffffffffu, id, 0);
        }
        if (lane == 0) {
            // the loads in flight land before the block exits
            for (uint32_t e = 1; e <= 2 && e <= nk; ++e) drain_bar(&sh.k_full[(nk - e) & 1], ((nk - e) >> 1) & 1, a.err);
            for (uint32_t e = 1; e <= 2 && e <= nv; ++e) drain_bar(&sh.v_full[(nv - e) & 1], ((nv - e) >> 1) & 1, a.err);
            if (nq > 0) {
                drain_bar(&sh.q_full, (nq - 1) & 1, a.err);
            }
            if (ho.pending()) drain_bar(&sh.next_bar, ho.parity(), a.err);       // after a wait that gave up
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t id_s = idesc_bf16_f32(TQ, TK), id_o = idesc_bf16_f32_t(TQ, kDv, 0, 1), id_h = idesc_bf16_f32_t(TQ, 64, 0, 1);
        uint32_t j = 0, u = 0, nq = 0, np[2] = {0, 0};        // key tiles so far, ring unit of the current one
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        const uint64_t dq = smem_desc_sw128(smem_u32(smem)), dk = smem_desc_sw128(ring), dv = smem_desc_sw128_mn(ring, UNIT);
        auto score = [&](int t, uint32_t u0) {                // S_t = Q_t K^T, K at units u0 .. u0 + 2
            if (elect_one()) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const uint64_t ad = dq + static_cast<uint64_t>((3 * t + c) * (UNIT >> 4));
                    const uint64_t bd = dk + static_cast<uint64_t>(((u0 + c) & 7) * (UNIT >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16(tm_s + 128 * t, ad + 2ull * kk, bd + 2ull * kk, id_s, c > 0 || kk > 0);
                }
                tc_commit(smem_u32(&sh.s_full[t]));
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t* bar) {
            if (elect_one()) tc_commit(smem_u32(bar));
            __syncwarp();
        };
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1;
            if (!wait(&sh.item_full[slot], (k >> 1) & 1)) break;
            const int valid = sh.item[slot].valid, n0 = sh.item[slot].n[0], n1 = sh.item[slot].n[1], lk = sh.item[slot].lk;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[slot]));
            if (valid < 0) break;
            const int n = max(n0, n1);
            if (valid == 0 || n == 0) continue;
            if (!wait(&sh.q_full, nq++ & 1)) break;
            if (!wait(&sh.k_full[j & 1], (j >> 1) & 1)) break;
            if (n0 > 0) score(0, u);
            if (n1 > 0) score(1, u);
            commit(&sh.k_empty[j & 1]);
            // Q is free, and the next item's on its way, once the last scores are there
            if (n == 1) commit(&sh.q_empty);
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++j, u = (u + 5) & 7) {
                const uint32_t un = (u + 5) & 7;              // K of tile i + 1
                if (!wait(&sh.v_full[j & 1], (j >> 1) & 1)) break;
                // rows past the sequence's last key: p there is zero, but what lies in V's rows need not be finite
                const int keys = min(TK, lk - TK * i), steps = (keys + 15) >> 4, zrows = 16 * steps - keys;
                if (zrows > 0) {
                    for (int c = 0; c < 2; ++c) {
                        uint8_t* unit = smem + RING_OFF + ((u + 3 + c) & 7) * UNIT;
                        for (int z = lane; z < zrows * 8; z += 32)
                            *reinterpret_cast<uint4*>(unit + keys * 128 + z * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const int nt = t ? n1 : n0;
                    if (i < nt) {
                        if (!wait(&sh.p_full[t], np[t]++ & 1)) break;
                        if (elect_one()) {
                            tc_fence_after();
                            const uint32_t uv = (u + 3) & 7;
                            const uint64_t v0 = dv + static_cast<uint64_t>(uv * (UNIT >> 4));
                            const uint32_t d = tm_o + 128 * t, pa = tm_s + 128 * t;
                            if (uv != 7 && steps == 8) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    tc_mma_bf16_ts(d, pa + 8 * kk, v0 + 128ull * kk, id_o, i > 0 || kk > 0);
                            } else if (uv != 7) {
#pragma unroll 1
                                for (int kk = 0; kk < steps; ++kk)
                                    tc_mma_bf16_ts(d, pa + 8 * kk, v0 + 128ull * kk, id_o, i > 0 || kk > 0);
                            } else {                          // V's two halves lie at the ring's two ends
#pragma unroll 1
                                for (int kk = 0; kk < steps; ++kk) {
                                    tc_mma_bf16_ts(d, pa + 8 * kk, v0 + 128ull * kk, id_h, i > 0 || kk > 0);
                                    tc_mma_bf16_ts(d + 64, pa + 8 * kk, dv + 128ull * kk, id_h, i > 0 || kk > 0);
                                }
                            }
                            tc_commit(smem_u32(&sh.pv_done[t]));
                            if (t == 1) tc_commit(smem_u32(&sh.v_empty[j & 1]));
                        }
                        __syncwarp();
                    } else if (t == 1) {
                        commit(&sh.v_empty[j & 1]);
                    }
                    if (t == 0 && i + 1 < n && !wait(&sh.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1)) break;
                    if (i + 1 < nt) score(t, un);
                }
                if (!ok) break;
                if (i + 1 < n) commit(&sh.k_empty[(j + 1) & 1]);
                if (i + 2 == n) commit(&sh.q_empty);
            }
            if (!ok) break;
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin));          // every MMA completes before TMEM is released
            drain_bar(&sh.fin, 0, a.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------------- softmax and output of tile t
        const int t = warp >> 2;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tm_s + 128 * t + lane_base, to = tm_o + 128 * t + lane_base;
        const int r = 128 * t + 32 * (warp & 3) + lane;
        const float c = a.scale * 1.4426950408889634f;
        uint32_t ns = 0, npv = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const uint32_t slot = k & 1;
            if (!warp_wait(smem_u32(&sh.item_full[slot]), (k >> 1) & 1, abort_flag, a.err)) break;
            const Item it = sh.item[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[slot]));
            if (it.valid < 0) break;
            if (it.valid == 0 || 128 * t >= it.rows) continue;
            const int limit = row_limit(it, a.causal, r);
            float m = 0.f, l = 0.f;
            const int n = t ? it.n[1] : it.n[0];
            for (int i = 0; i < n; ++i) {
                if (!warp_wait(smem_u32(&sh.s_full[t]), ns++ & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                // two passes over the scores, 32 columns at a time: the loop bodies stay small and the registers few
                const int lim = limit - TK * i;
                const bool edge = __any_sync(0xffffffffu, lim < TK);
                float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
                for (int q = 0; q < TK; q += 32) {
                    uint32_t s[32];
                    tmem_ld32(ts + q, s);
                    tmem_ld_wait();
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (q + j >= lim) s[j] = 0xff800000u;      // -inf
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        mx[0] = fmaxf(mx[0], __uint_as_float(s[j]));
                        mx[1] = fmaxf(mx[1], __uint_as_float(s[j + 1]));
                    }
                }
                const float top = fmaxf(mx[0], mx[1]) * c;
                if (i == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
                    // O and l to the new maximum (a row without one so far, m = -inf, has nothing in them)
                    const float mn = fmaxf(m, top), al = mn == -CUDART_INF_F ? 1.f : exp2_fast(m - mn);
                    m = mn;
                    l *= al;
                    if (!warp_wait(smem_u32(&sh.pv_done[t]), (npv + i - 1) & 1, abort_flag, a.err)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tmem_ld32(to + 32 * q, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
                        tmem_st32(to + 32 * q, o);
                    }
                }
                const float me = m == -CUDART_INF_F ? 0.f : m;
                float sum[2] = {0.f, 0.f};
#pragma unroll 1
                for (int q = 0; q < TK; q += 32) {
                    uint32_t s[32], p[16];
                    tmem_ld32(ts + q, s);
                    tmem_ld_wait();
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (q + j >= lim) s[j] = 0xff800000u;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float x0 = exp2_fast(fmaf(__uint_as_float(s[2 * j]), c, -me));
                        const float x1 = exp2_fast(fmaf(__uint_as_float(s[2 * j + 1]), c, -me));
                        sum[0] += x0;
                        sum[1] += x1;
                        p[j] = pack_bf16x2(x0, x1);
                    }
                    tmem_st16(ts + q / 2, p);       // P's columns q / 2 .. hold scores that were read before
                }
                l += sum[0] + sum[1];
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[t]));
            }
            if (!ok) break;
            npv += n;
            if (n > 0) {
                if (!warp_wait(smem_u32(&sh.pv_done[t]), (npv - 1) & 1, abort_flag, a.err)) break;
                tc_fence_after();
            }
            const float inv = l != 0.f ? 1.f / l : 0.f;
            const bool mine = r < it.rows;
            __nv_bfloat16* dst = a.out_w + (static_cast<long long>(it.row0) + r - lane) * a.o_row +
                                 static_cast<long long>(it.head) * a.o_head;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(to + 32 * q, o);
                    tmem_ld_wait();
                }
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    w[j] = l != 0.f ? pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv) : 0u;
                store_rows(lane, w, reinterpret_cast<uint8_t*>(dst + 32 * q), 2 * a.o_row, it.rows - (r - lane));
            }
            if (mine)
                a.lse_w[static_cast<long long>(it.head) * a.Tq + it.row0 + r] =
                    l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -CUDART_INF_F;
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

}  // namespace pf

// A [rows, heads, width] bf16 operand with strides in elements (3D map: column,
// head, row), box 64 columns x 1 head x box_rows rows, 128-byte swizzle.  The
// stride of a dimension of extent 1 is never used and may be anything.
cudaError_t make_map_rows(CUtensorMap* m, const void* base, long long rows, int heads, int width, long long row,
                          long long head, int box_rows) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    cuuint64_t gdim[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t gstride[2] = {heads > 1 ? static_cast<cuuint64_t>(head) * 2 : static_cast<cuuint64_t>(width) * 2,
                             rows > 1 ? static_cast<cuuint64_t>(row) * 2 : static_cast<cuuint64_t>(width) * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t st) {
    static bool attr[kMaxDevices] = {false};
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(pf::prefill_kernel), pf::SMEM, attr);
    if (e != cudaSuccess) return e;
    CUtensorMap q, kn, kr, v;
    e = make_map_rows(&q, a.q, a.Tq, a.H, kDqk, a.q_row, a.q_head, 128);
    if (e == cudaSuccess) e = make_map_rows(&kn, a.kn, a.Tk, a.H, kNope, a.kn_row, a.kn_head, 128);
    if (e == cudaSuccess) e = make_map_rows(&kr, a.kr, a.Tk, 1, kRope, a.kr_row, 0, 128);
    if (e == cudaSuccess) e = make_map_rows(&v, a.v, a.Tk, a.H, kDv, a.v_row, a.v_head, 128);
    if (e != cudaSuccess) return e;
    const int tiles = a.Tq / (2 * pf::TQ) + a.B;             // at least the row tiles of any split into B sequences
    pf::prefill_kernel<<<static_cast<unsigned>(tiles) * a.H, pf::THREADS, pf::SMEM, st>>>(q, kn, kr, v, a, tiles);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
