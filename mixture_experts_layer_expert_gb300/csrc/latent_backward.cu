// latent_backward.cu -- the gradient of expanded latent attention over packed
// sequences, from the forward's out and lse:
//   s = scale (q_n . k_n + q_r . k_r), p = exp(s - lse), dp = d_out . v, D = <d_out, out>
//   ds = p (dp - D);  dv = sum_i p d_out, dk = scale sum_i ds q, dq = scale sum_j ds k,
//   and dk's rotary part summed over the heads that share it.
//
// Three passes, no atomics, every sum in a fixed order:
//   1. D of every (query, head), memory bound;
//   2. dk, dv: a work item is 128 keys of one head; queries come in tiles of 64;
//   3. dq: a work item is 128 queries of one head; keys come in tiles of 128.
// One pass over tile pairs with dq added into memory would need 832 instead of
// 1,152 multiply-adds per (query, key), but dq's 98 KB fp32 tile would cross L2
// twice for every 2.7 us of products, and in an order that changes results.
//
// Pass 2 works transposed (rows = keys = TMEM lanes), so that p and ds leave the
// registers as the A operand of the products that need them:
//   S^T = K Q^T (128 x 64 x 192), dP^T = V dO^T (128 x 64 x 128)
//   dV += P^T dO (128 x 128 x 64), dK += dS^T Q (128 x 192 x 64)
// TMEM: dV 128, dK 192, S^T 2 x 64 and dP^T 64 columns = 512; P^T and dS^T (bf16)
// overwrite the columns their own warps have read.  Order of the MMAs:
//   dV(j) | dK(j) | dP(j+1) | S(j+2)
// so the exponentials of tile j+1 and the ds of tile j run under MMAs.  Bound: the
// tensor cores, 24 x 75 + 4 x 107 = 2,230 cycles a tile of 64 queries (an MMA with both
// operands in shared memory costs 43 cycles beside N / 2, with A in TMEM 11; 1,280 would
// be the multiply-adds); 2,570 are measured.
//
// Pass 3: S = Q K^T, dP = dO V^T (128 x 128 each), dQ += dS K; TMEM: S 128, dP 128,
// dS 64, dQ 192 = 512 columns.  Order: dP(i+1) | S(i+1) | dQ(i), ds of tile i beside the
// first two.  Bound: 20 x 107 + 8 x 107 = 3,000 cycles a tile; what is left beside it is
// K's load, whose place of 48 KB is free only behind dQ(i-1) (a third place for K does
// not fit beside Q, dO and V).
//
// Measured, 4 x 2,048 tokens x 16 heads, causal: D 15.7 us (4.3 TB/s), dk and dv 190 us,
// the sum over the heads 8.4 us, dq 144 us; 617 TFLOP/s of the 832 multiply-adds over all.
#include <math_constants.h>

#include "handover.h"
#include "kernels.h"
#include "latent.cuh"

namespace fs {
namespace bw {

constexpr float kLog2e = 1.4426950408889634f;

// D = <d_out, out> of each query and head -> delta [H, Tq]; 16 lanes a row.
__global__ void __launch_bounds__(256) delta_kernel(LatentPrefillArgs a, float* __restrict__ delta) {
    const int lane = threadIdx.x & 15;
    const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
    const long long n = static_cast<long long>(a.Tq) * a.H;
    const long long t = (w < n ? w : 0) / a.H;
    const int h = static_cast<int>((w < n ? w : 0) - t * a.H);
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.d_out + t * a.do_row + h * a.do_head) + lane);
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(a.out + t * a.o_row + h * a.o_head) + lane);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += bf16lo(xs[i]) * bf16lo(ys[i]) + bf16hi(xs[i]) * bf16hi(ys[i]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0 && w < n) delta[static_cast<long long>(h) * a.Tq + t] = s;
}

// dk_rope[j] = sum over the heads, in order, of the fp32 partials [H][Tk][64].  A block takes 16 keys of a 128-key
// tile (blockIdx.y), a thread 4 columns of one: enough blocks to cover the loads' latency.
__global__ void __launch_bounds__(256) rope_sum_kernel(LatentPrefillArgs a, const float* __restrict__ part) {
    PackedSeq s;
    const int tile = find_tile(a.cu_q, a.cu_k, a.B, a.Tq, a.Tk, 128, true, blockIdx.x, nullptr, &s);
    if (tile < 0) return;
    const int r = 128 * tile + 16 * blockIdx.y + (threadIdx.x >> 4), c = (threadIdx.x & 15) * 4;
    if (r >= s.lk) return;
    const long long row = s.k0 + r;
    const float4* src = reinterpret_cast<const float4*>(part + row * kRope + c);
    const long long step = static_cast<long long>(a.Tk) * kRope / 4;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < a.H; ++h) {
        const float4 v = __ldg(src + h * step);
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    *reinterpret_cast<uint2*>(a.dkr + row * a.dkr_row + c) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
}

constexpr int THREADS = 320;                    // warps 0-7: elementwise and output, 8: loads, 9: MMA
constexpr int UNIT = 128 * 64 * 2;              // 128 rows x 64 columns

struct Item {
    int valid;            // 1: work, 0: nothing for this number, -1: no more items
    int head;
    int row0, rows;       // first resident row (keys in pass 2, queries in pass 3) and how many
    int other0;           // first streamed row of the first tile
    int n;                // streamed tiles
    int len;              // streamed rows of the sequence from other0 on
    int diag;             // pass 2: key row r is seen by streamed query c >= r + diag; pass 3: query row r sees keys <= r + diag
};

// Hand-over of work items: the load warp takes the block's own number first, then
// those of blocks that have not started.
struct Queue {
    uint64_t full[2], empty[2], next_bar;
    alignas(16) uint32_t next_resp[4];
    Item item[2];
};

// Zero rows [from, to) of `units` units of `unit` bytes (128-byte rows), by one warp.
__device__ __forceinline__ void zero_rows(uint8_t* base, int units, int unit, int from, int to, int lane) {
    const int n = (to - from) * 8;
    for (int c = 0; c < units; ++c)
        for (int z = lane; z < n; z += 32)
            *reinterpret_cast<uint4*>(base + c * unit + from * 128 + z * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// A warp's 32 rows x 64 bytes go out through shared memory (2 KB, the row's four 16-byte chunks rotated against bank
// conflicts): a store instruction then covers eight rows' whole 64-byte runs instead of 32 rows' 16 bytes.
__device__ __forceinline__ void store_rows(uint4* buf, int lane, const uint32_t* w, uint8_t* dst, long long row_bytes, int rows) {
#pragma unroll
    for (int v = 0; v < 4; ++v) buf[4 * lane + (v ^ ((lane >> 1) & 3))] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), v = lane & 3;
        if (r < rows) *reinterpret_cast<uint4*>(dst + r * row_bytes + 16 * v) = buf[4 * r + (v ^ ((r >> 1) & 3))];
    }
    __syncwarp();
}

// ------------------------------------------------------------------ pass 2
namespace kv {
constexpr int TQ = 64, STAGES = 3;
constexpr int QU = 64 * 64 * 2;                     // 64 rows x 64 columns, 8 KB
constexpr int STAGE = 5 * QU;                       // Q (3 units), dO (2 units)
constexpr int K_OFF = 0, V_OFF = 3 * UNIT, ST_OFF = 5 * UNIT, OUT_OFF = ST_OFF + STAGES * STAGE, BAR_OFF = OUT_OFF + 8 * 2048;
constexpr size_t SMEM = 1024 + BAR_OFF + 2560;

struct Shared {
    uint64_t full[STAGES], empty[STAGES], kv_full, kv_empty, s_full[2], p_full[2], dp_full, ds_full, acc_full, acc_empty, fin;
    uint32_t tmem;
    int abort_flag;
    Queue q;
    float lse[STAGES][TQ], delta[STAGES][TQ];       // log2 units; +inf where a query sees nothing or is past the end
};
static_assert(sizeof(Shared) <= 2560, "barrier area");

__global__ void __launch_bounds__(THREADS, 1)
dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKn,
           const __grid_constant__ CUtensorMap tmKr, const __grid_constant__ CUtensorMap tmV,
           const __grid_constant__ CUtensorMap tmDo, const LatentPrefillArgs a, const int max_tiles,
           const float* __restrict__ delta, float* __restrict__ rope_part) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& sh = *reinterpret_cast<Shared*>(smem + BAR_OFF);
    volatile int* abort_flag = &sh.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) { mbar_init(smem_u32(&sh.full[i]), 1); mbar_init(smem_u32(&sh.empty[i]), 1); }
        mbar_init(smem_u32(&sh.kv_full), 1);
        mbar_init(smem_u32(&sh.kv_empty), 1);
        mbar_init(smem_u32(&sh.s_full[0]), 1);
        mbar_init(smem_u32(&sh.s_full[1]), 1);
        mbar_init(smem_u32(&sh.p_full[0]), 256);
        mbar_init(smem_u32(&sh.p_full[1]), 256);
        mbar_init(smem_u32(&sh.dp_full), 1);
        mbar_init(smem_u32(&sh.ds_full), 256);
        mbar_init(smem_u32(&sh.acc_full), 1);
        mbar_init(smem_u32(&sh.acc_empty), 256);
        for (int t = 0; t < 2; ++t) { mbar_init(smem_u32(&sh.q.full[t]), 1); mbar_init(smem_u32(&sh.q.empty[t]), 9); }
        mbar_init(smem_u32(&sh.q.next_bar), 1);
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
    // dV, dK (128 + 64 columns), S^T twice, dP^T
    const uint32_t tm_dv = sh.tmem, tm_dk = sh.tmem + 128, tm_s = sh.tmem + 320, tm_dp = sh.tmem + 448;

    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch_desc(&tmQ); tma_prefetch_desc(&tmKn); tma_prefetch_desc(&tmKr); tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmDo);
        }
        uint32_t u = 0, nkv = 0;
        int id = blockIdx.x;
        bool ok = true;
        HandOver ho;
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1;
            if (id >= 0) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_u32(&sh.q.next_bar), 16);
                    next_block_request(smem_u32(sh.q.next_resp), smem_u32(&sh.q.next_bar));
                }
                ho.ask();
            }
            Item it{};
            it.valid = id < 0 ? -1 : 0;
            if (id >= 0) {
                it.head = id / max_tiles;
                PackedSeq s;
                // first tiles first: under a causal mask they are seen by the most queries
                const int tile = find_tile(a.cu_q, a.cu_k, a.B, a.Tq, a.Tk, 128, true, id - it.head * max_tiles, a.err, &s);
                if (tile >= 0) {
                    it.valid = 1;
                    it.row0 = s.k0 + 128 * tile;
                    it.rows = min(128, s.lk - 128 * tile);
                    // key 128 tile + r is seen by queries i >= 128 tile + r - (lk - lq)
                    const int first = a.causal ? 128 * tile - (s.lk - s.lq) : 0;
                    const int from = max(0, first) / TQ * TQ;
                    it.other0 = s.q0 + from;
                    it.len = s.lq - from;
                    it.n = it.len > 0 ? (it.len + TQ - 1) / TQ : 0;
                    it.diag = a.causal ? first - from : -(1 << 30);
                }
            }
            ok = warp_wait(smem_u32(&sh.q.empty[slot]), ((k >> 1) & 1) ^ 1, abort_flag, a.err);
            if (!ok) break;
            if (lane == 0) {
                sh.q.item[slot] = it;
                mbar_arrive(smem_u32(&sh.q.full[slot]));
            }
            if (id < 0) break;
            if (it.valid == 1 && it.n > 0) {
                if (lane == 0) {
                    ok = wait_bar(smem_u32(&sh.kv_empty), (nkv & 1) ^ 1, abort_flag, a.err);
                    if (ok) {
                        const uint32_t fb = smem_u32(&sh.kv_full);
                        mbar_arrive_expect_tx(fb, 5 * UNIT);
                        for (int c = 0; c < 2; ++c) {
                            tma_load_3d(smem_u32(smem + K_OFF + c * UNIT), &tmKn, fb, 64 * c, it.head, it.row0);
                            tma_load_3d(smem_u32(smem + V_OFF + c * UNIT), &tmV, fb, 64 * c, it.head, it.row0);
                        }
                        tma_load_3d(smem_u32(smem + K_OFF + 2 * UNIT), &tmKr, fb, 0, 0, it.row0);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                ++nkv;
                for (int j = 0; j < it.n; ++j, ++u) {
                    const uint32_t s = u % STAGES;
                    // the statistics' loads do not wait for the stage
                    float l2[2], dl[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = TQ * j + 32 * e + lane;
                        l2[e] = CUDART_INF_F;
                        dl[e] = 0.f;
                        if (c < it.len) {
                            const long long at = static_cast<long long>(it.head) * a.Tq + it.other0 + c;
                            const float l = __ldg(a.lse + at);
                            if (l != -CUDART_INF_F) l2[e] = l * kLog2e;
                            dl[e] = __ldg(delta + at);
                        }
                    }
                    ok = warp_wait(smem_u32(&sh.empty[s]), ((u / STAGES) & 1) ^ 1, abort_flag, a.err);
                    if (!ok) break;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sh.lse[s][32 * e + lane] = l2[e];
                        sh.delta[s][32 * e + lane] = dl[e];
                    }
                    __syncwarp();
                    if (lane == 0) {
                        const uint32_t fb = smem_u32(&sh.full[s]);
                        const uint32_t dst = smem_u32(smem + ST_OFF + s * STAGE);
                        const int row = it.other0 + TQ * j;
                        mbar_arrive_expect_tx(fb, STAGE);
                        for (int c = 0; c < 3; ++c) tma_load_3d(dst + c * QU, &tmQ, fb, 64 * c, it.head, row);
                        for (int c = 0; c < 2; ++c) tma_load_3d(dst + (3 + c) * QU, &tmDo, fb, 64 * c, it.head, row);
                    }
                }
            }
            if (!ok) break;
            if (lane == 0) {
                ok = wait_bar(smem_u32(&sh.q.next_bar), ho.parity(), abort_flag, a.err);
                if (ok) id = next_block_answer(smem_u32(sh.q.next_resp));
                fence_proxy_async_smem();
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ho.answer();
            id = __shfl_sync(0xffffffffu, id, 0);
        }
        if (lane == 0) {
            const uint32_t pend = u < STAGES ? u : STAGES;
            for (uint32_t j = 1; j <= pend; ++j) drain_bar(&sh.full[(u - j) % STAGES], ((u - j) / STAGES) & 1, a.err);
            if (nkv > 0) drain_bar(&sh.kv_full, (nkv - 1) & 1, a.err);
            if (ho.pending()) drain_bar(&sh.q.next_bar, ho.parity(), a.err);       // after a wait that gave up
        }
        __syncwarp();
    } else if (warp == 9) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, TQ);
        constexpr uint32_t id_v = idesc_bf16_f32_t(128, kDv, 0, 1), id_k = idesc_bf16_f32_t(128, kDqk, 0, 1);
        uint32_t u = 0, nkv = 0, nd = 0, nacc = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        const uint32_t sk = smem_u32(smem + K_OFF), sv = smem_u32(smem + V_OFF), sst = smem_u32(smem + ST_OFF);
        // a stage's tail rows (past the sequence's last query) become zeros before anything reads them
        auto stage_in = [&](uint32_t uu, int left) {
            const uint32_t s = uu % STAGES;
            if (!wait(&sh.full[s], (uu / STAGES) & 1)) return false;
            if (left < TQ) {
                if (wait_bar(smem_u32(&sh.full[s]), (uu / STAGES) & 1, abort_flag, a.err))
                    zero_rows(smem + ST_OFF + s * STAGE, 5, QU, left, TQ, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            return true;
        };
        // issued by one lane: S^T = K Q^T and dP^T = V dO^T of the queries in stage uu
        const uint64_t dk = smem_desc_sw128(sk), dvd = smem_desc_sw128(sv), dst = smem_desc_sw128(sst), dmn = smem_desc_sw128_mn(sst, QU);
        auto score = [&](uint32_t uu) {
            const uint64_t q = dst + static_cast<uint64_t>((uu % STAGES) * (STAGE >> 4));
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_bf16(tm_s + 64 * (uu & 1), dk + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk),
                                q + static_cast<uint64_t>(c * (QU >> 4) + 2 * kk), id_s, c > 0 || kk > 0);
            tc_commit(smem_u32(&sh.s_full[uu & 1]));
        };
        auto dprob = [&](uint32_t uu) {
            const uint64_t o = dst + static_cast<uint64_t>((uu % STAGES) * (STAGE >> 4) + 3 * (QU >> 4));
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_bf16(tm_dp, dvd + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk),
                                o + static_cast<uint64_t>(c * (QU >> 4) + 2 * kk), id_s, c > 0 || kk > 0);
            tc_commit(smem_u32(&sh.dp_full));
        };
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1;
            if (!wait(&sh.q.full[slot], (k >> 1) & 1)) break;
            const int valid = sh.q.item[slot].valid, n = sh.q.item[slot].n, len = sh.q.item[slot].len;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q.empty[slot]));
            if (valid < 0) break;
            if (valid == 0 || n == 0) continue;
            if (!wait(&sh.kv_full, nkv++ & 1)) break;
            if (!stage_in(u, len)) break;
            if (elect_one()) {
                tc_fence_after();
                score(u);
                dprob(u);
            }
            __syncwarp();
            if (n > 1) {
                if (!stage_in(u + 1, len - TQ)) break;
                if (elect_one()) {
                    tc_fence_after();
                    score(u + 1);
                }
                __syncwarp();
            }
            if (!wait(&sh.acc_empty, (nacc & 1) ^ 1)) break;
            // S runs two tiles ahead: its buffer was P^T of the tile whose dV has been issued
#pragma unroll 1
            for (int j = 0; j < n; ++j, ++u) {
                const uint32_t acc = j > 0, so = (u % STAGES) * (STAGE >> 4);
                const int steps = (min(TQ, len - TQ * j) + 15) >> 4;
                if (!wait(&sh.p_full[u & 1], (u >> 1) & 1)) break;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t o = dmn + static_cast<uint64_t>(so + 3 * (QU >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)        // P^T: queries 0-31 in columns 0-15, 32-63 in 32-47
                        if (kk < steps)
                            tc_mma_bf16_ts(tm_dv, tm_s + 64 * (u & 1) + 32 * (kk >> 1) + 8 * (kk & 1), o + 128ull * kk, id_v, acc | (kk > 0));
                }
                __syncwarp();
                if (!wait(&sh.ds_full, nd++ & 1)) break;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t q = dmn + static_cast<uint64_t>(so);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps)                   // 192 columns: the unrotated 128 and the rotary 64
                            tc_mma_bf16_ts(tm_dk, tm_dp + 32 * (kk >> 1) + 8 * (kk & 1), q + 128ull * kk, id_k, acc | (kk > 0));
                    tc_commit(smem_u32(&sh.empty[u % STAGES]));
                    if (j + 1 < n) dprob(u + 1);
                }
                __syncwarp();
                if (j + 2 < n) {
                    if (!stage_in(u + 2, len - TQ * (j + 2))) break;
                    if (elect_one()) {
                        tc_fence_after();
                        score(u + 2);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            ++nacc;
            if (elect_one()) {
                tc_commit(smem_u32(&sh.acc_full));
                tc_commit(smem_u32(&sh.kv_empty));
            }
            __syncwarp();
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin));
            drain_bar(&sh.fin, 0, a.err);
        }
        __syncwarp();
    } else {
        const int half = warp >> 2, r = 32 * (warp & 3) + lane;      // key row; columns [32 half, 32 half + 32)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = a.scale * kLog2e;
        uint32_t u = 0, ndp = 0, nacc = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const uint32_t slot = k & 1;
            if (!warp_wait(smem_u32(&sh.q.full[slot]), (k >> 1) & 1, abort_flag, a.err)) break;
            const Item it = sh.q.item[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q.empty[slot]));
            if (it.valid < 0) break;
            if (it.valid == 0) continue;
            for (int j = 0; j < it.n; ++j, ++u) {
                const uint32_t st = u % STAGES, buf = u & 1;
                const uint32_t ts = tm_s + 64 * buf + 32 * half + lane_base, td = tm_dp + 32 * half + lane_base;
                if (!warp_wait(smem_u32(&sh.s_full[buf]), (u >> 1) & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[32];
                tmem_ld32(ts, s);
                // the statistics were written before the stage's loads were issued (the wait returns at once)
                if (!warp_wait(smem_u32(&sh.full[st]), (u / STAGES) & 1, abort_flag, a.err)) { ok = false; break; }
                const float4* ls = reinterpret_cast<const float4*>(&sh.lse[st][32 * half]);
                const float4* dl = reinterpret_cast<const float4*>(&sh.delta[st][32 * half]);
                tmem_ld_wait();
                const int first = r + it.diag - TQ * j - 32 * half;       // first visible column of this row
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 l4 = ls[q];
                    const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[4 * q + e] = __float_as_uint(exp2_fast(fmaf(__uint_as_float(s[4 * q + e]), c, -l[e])));
                }
                if (__any_sync(0xffffffffu, first > 0)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < first) s[i] = 0u;
                }
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
                tmem_st16(ts, w);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[buf]));
                if (!warp_wait(smem_u32(&sh.dp_full), ndp++ & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                uint32_t d[32];
                tmem_ld32(td, d);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 d4 = dl[q];
                    const float e4[4] = {d4.x, d4.y, d4.z, d4.w};
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(s[4 * q + e]) * (__uint_as_float(d[4 * q + e]) - e4[e]);
                    w[2 * q] = pack_bf16x2(v[0], v[1]);
                    w[2 * q + 1] = pack_bf16x2(v[2], v[3]);
                }
                tmem_st16(td, w);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.ds_full));
            }
            if (!ok) break;
            if (it.n > 0) {
                if (!warp_wait(smem_u32(&sh.acc_full), nacc++ & 1, abort_flag, a.err)) break;
                tc_fence_after();
            }
            // half 0: dV, half 1: dK's unrotated part; the rotary part 32 columns each
            const int rows = it.rows - 32 * (warp & 3);
            const long long row = static_cast<long long>(it.row0) + 32 * (warp & 3);         // of the warp's first
            uint4* buf = reinterpret_cast<uint4*>(smem + OUT_OFF + 2048 * warp);
            __nv_bfloat16* dst = half == 0 ? a.dv + row * a.dv_row + it.head * a.dv_head
                                           : a.dkn + row * a.dkn_row + it.head * a.dkn_head;
            const long long dst_row = 2 * (half == 0 ? a.dv_row : a.dkn_row);
            const float mul = half == 0 ? 1.f : a.scale;
            const uint32_t acc = (half == 0 ? tm_dv : tm_dk) + lane_base;
            uint32_t o[32];
            const bool any = it.n > 0;
#pragma unroll 1
            for (int q = 0; q < 5; ++q) {
                if (any) {
                    tmem_ld32(q < 4 ? acc + 32 * q : tm_dk + 128 + 32 * half + lane_base, o);
                    tmem_ld_wait();
                }
                if (q == 4) break;
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = any ? pack_bf16x2(__uint_as_float(o[2 * e]) * mul, __uint_as_float(o[2 * e + 1]) * mul) : 0u;
                store_rows(buf, lane, w, reinterpret_cast<uint8_t*>(dst + 32 * q), dst_row, rows);
            }
            if (any) {
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.acc_empty));
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * a.scale) : 0u;
            uint8_t* part = reinterpret_cast<uint8_t*>(rope_part + (static_cast<long long>(it.head) * a.Tk + row) * kRope + 32 * half);
            store_rows(buf, lane, o, part, 4 * kRope, rows);
            store_rows(buf, lane, o + 16, part + 64, 4 * kRope, rows);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}
}  // namespace kv

// ------------------------------------------------------------------ pass 3
namespace dq {
// Q, dO resident; K twice (three units each), V once: K of a tile is held until its dQ product, V only until dP
constexpr int Q_OFF = 0, DO_OFF = 3 * UNIT, K_OFF = 5 * UNIT, V_OFF = 11 * UNIT, OUT_OFF = 13 * UNIT, BAR_OFF = OUT_OFF + 8 * 2048;
constexpr size_t SMEM = 1024 + BAR_OFF + 512;

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full, v_empty, q_full, q_empty, sp_full, sp_free, ds_full, acc_empty, fin;
    uint32_t tmem;
    int abort_flag;
    Queue q;
};
static_assert(sizeof(Shared) <= 512, "barrier area");

__global__ void __launch_bounds__(THREADS, 1)
dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKn,
          const __grid_constant__ CUtensorMap tmKr, const __grid_constant__ CUtensorMap tmV,
          const __grid_constant__ CUtensorMap tmDo, const LatentPrefillArgs a, const int max_tiles,
          const float* __restrict__ delta) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& sh = *reinterpret_cast<Shared*>(smem + BAR_OFF);
    volatile int* abort_flag = &sh.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&sh.k_full[i]), 1); mbar_init(smem_u32(&sh.k_empty[i]), 1); }
        mbar_init(smem_u32(&sh.v_full), 1);
        mbar_init(smem_u32(&sh.v_empty), 1);
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.sp_full), 1);
        mbar_init(smem_u32(&sh.sp_free), 256);
        mbar_init(smem_u32(&sh.ds_full), 256);
        mbar_init(smem_u32(&sh.acc_empty), 256);
        for (int t = 0; t < 2; ++t) { mbar_init(smem_u32(&sh.q.full[t]), 1); mbar_init(smem_u32(&sh.q.empty[t]), 9); }
        mbar_init(smem_u32(&sh.q.next_bar), 1);
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
    const uint32_t tm_s = sh.tmem, tm_dp = sh.tmem + 128, tm_ds = sh.tmem + 256, tm_dq = sh.tmem + 320;

    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch_desc(&tmQ); tma_prefetch_desc(&tmKn); tma_prefetch_desc(&tmKr); tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmDo);
        }
        uint32_t u = 0, nq = 0, nk = 0, nv = 0;
        int id = blockIdx.x;
        bool ok = true;
        HandOver ho;
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1;
            if (id >= 0) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_u32(&sh.q.next_bar), 16);
                    next_block_request(smem_u32(sh.q.next_resp), smem_u32(&sh.q.next_bar));
                }
                ho.ask();
            }
            Item it{};
            it.valid = id < 0 ? -1 : 0;
            if (id >= 0) {
                it.head = id / max_tiles;
                PackedSeq s;
                const int tile = find_tile(a.cu_q, a.cu_k, a.B, a.Tq, a.Tk, 128, false,
                                           max_tiles - 1 - (id - it.head * max_tiles), a.err, &s);
                if (tile >= 0) {
                    it.valid = 1;
                    it.row0 = s.q0 + 128 * tile;
                    it.rows = min(128, s.lq - 128 * tile);
                    it.other0 = s.k0;
                    it.len = s.lk;
                    it.diag = s.lk - s.lq + 128 * tile;
                    const int end = a.causal ? min(s.lk, it.diag + it.rows) : s.lk;       // keys the last query sees
                    it.n = max(0, end + 127) / 128;
                }
            }
            ok = warp_wait(smem_u32(&sh.q.empty[slot]), ((k >> 1) & 1) ^ 1, abort_flag, a.err);
            if (!ok) break;
            if (lane == 0) {
                sh.q.item[slot] = it;
                mbar_arrive(smem_u32(&sh.q.full[slot]));
            }
            if (id < 0) break;
            if (it.valid == 1 && it.n > 0 && lane == 0) {
                ok = wait_bar(smem_u32(&sh.q_empty), (nq & 1) ^ 1, abort_flag, a.err);
                if (ok) {
                    ++nq;
                    const uint32_t fb = smem_u32(&sh.q_full);
                    mbar_arrive_expect_tx(fb, 5 * UNIT);
                    for (int c = 0; c < 3; ++c)
                        tma_load_3d(smem_u32(smem + Q_OFF + c * UNIT), &tmQ, fb, 64 * c, it.head, it.row0);
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d(smem_u32(smem + DO_OFF + c * UNIT), &tmDo, fb, 64 * c, it.head, it.row0);
                }
                for (int i = 0; ok && i < it.n; ++i, ++u) {
                    const int row = it.other0 + 128 * i;
                    const uint32_t kd = smem_u32(smem + K_OFF) + (u & 1) * 3 * UNIT, vd = smem_u32(smem + V_OFF);
                    ok = wait_bar(smem_u32(&sh.v_empty), (u & 1) ^ 1, abort_flag, a.err);
                    if (!ok) break;
                    uint32_t fb = smem_u32(&sh.v_full);
                    mbar_arrive_expect_tx(fb, 2 * UNIT);
                    tma_load_3d(vd, &tmV, fb, 0, it.head, row);
                    tma_load_3d(vd + UNIT, &tmV, fb, 64, it.head, row);
                    ++nv;
                    ok = wait_bar(smem_u32(&sh.k_empty[u & 1]), ((u >> 1) & 1) ^ 1, abort_flag, a.err);
                    if (!ok) break;
                    fb = smem_u32(&sh.k_full[u & 1]);
                    mbar_arrive_expect_tx(fb, 3 * UNIT);
                    tma_load_3d(kd, &tmKn, fb, 0, it.head, row);
                    tma_load_3d(kd + UNIT, &tmKn, fb, 64, it.head, row);
                    tma_load_3d(kd + 2 * UNIT, &tmKr, fb, 0, 0, row);
                    ++nk;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                ok = wait_bar(smem_u32(&sh.q.next_bar), ho.parity(), abort_flag, a.err);
                if (ok) id = next_block_answer(smem_u32(sh.q.next_resp));
                fence_proxy_async_smem();
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ho.answer();
            id = __shfl_sync(0xffffffffu, id, 0);
        }
        if (lane == 0) {
            for (uint32_t e = 1; e <= 2 && e <= nk; ++e) drain_bar(&sh.k_full[(nk - e) & 1], ((nk - e) >> 1) & 1, a.err);
            if (nv > 0) drain_bar(&sh.v_full, (nv - 1) & 1, a.err);
            if (nq > 0) drain_bar(&sh.q_full, (nq - 1) & 1, a.err);
            if (ho.pending()) drain_bar(&sh.q.next_bar, ho.parity(), a.err);       // after a wait that gave up
        }
        __syncwarp();
    } else if (warp == 9) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128), id_q = idesc_bf16_f32_t(128, kDqk, 0, 1);
        uint32_t u = 0, nq = 0, nacc = 0;                     // key tiles so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(smem_u32(bar), parity, abort_flag, a.err);
            return ok;
        };
        const uint64_t dqd = smem_desc_sw128(smem_u32(smem + Q_OFF)), dod = smem_desc_sw128(smem_u32(smem + DO_OFF)),
                       dkd = smem_desc_sw128(smem_u32(smem + K_OFF)), dvd = smem_desc_sw128(smem_u32(smem + V_OFF)),
                       dkm = smem_desc_sw128_mn(smem_u32(smem + K_OFF), UNIT);
        // dP = dO V^T and S = Q K^T of key tile uu, which holds `keys` rows of the sequence; dP first: its V came long
        // ago, while K's place has only just been left by the dQ product before
        auto products = [&](uint32_t uu, int keys) {
            if (!wait(&sh.v_full, uu & 1)) return false;
            if (elect_one()) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16(tm_dp, dod + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk), dvd + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk),
                                    id_s, c > 0 || kk > 0);
                tc_commit(smem_u32(&sh.v_empty));
            }
            __syncwarp();
            if (!wait(&sh.k_full[uu & 1], (uu >> 1) & 1)) return false;
            if (keys < 128) {       // K's rows past the last key meet ds = 0, but need not be finite
                zero_rows(smem + K_OFF + (uu & 1) * 3 * UNIT, 3, UNIT, keys, (keys + 15) & ~15, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (elect_one()) {
                tc_fence_after();
                const uint64_t kd = dkd + static_cast<uint64_t>((uu & 1) * 3 * (UNIT >> 4));
#pragma unroll
                for (int c = 0; c < 3; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16(tm_s, dqd + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk), kd + static_cast<uint64_t>(c * (UNIT >> 4) + 2 * kk),
                                    id_s, c > 0 || kk > 0);
                tc_commit(smem_u32(&sh.sp_full));
            }
            __syncwarp();
            return true;
        };
        for (uint32_t k = 0;; ++k) {
            const uint32_t slot = k & 1;
            if (!wait(&sh.q.full[slot], (k >> 1) & 1)) break;
            const int valid = sh.q.item[slot].valid, n = sh.q.item[slot].n, len = sh.q.item[slot].len;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q.empty[slot]));
            if (valid < 0) break;
            if (valid == 0 || n == 0) continue;
            if (!wait(&sh.q_full, nq++ & 1)) break;
            // S and dP of the item before have been read (its last ds is complete)
            if (!products(u, min(128, len))) break;
            if (!wait(&sh.acc_empty, (nacc & 1) ^ 1)) break;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++u) {
                if (!wait(&sh.sp_free, u & 1)) break;
                if (i + 1 < n && !products(u + 1, min(128, len - 128 * (i + 1)))) break;
                if (!wait(&sh.ds_full, u & 1)) break;
                if (elect_one()) {
                    tc_fence_after();
                    const int steps = (min(128, len - 128 * i) + 15) >> 4;
                    const uint64_t kd = dkm + static_cast<uint64_t>((u & 1) * 3 * (UNIT >> 4));
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < steps) tc_mma_bf16_ts(tm_dq, tm_ds + 8 * kk, kd + 128ull * kk, id_q, i > 0 || kk > 0);
                    tc_commit(smem_u32(&sh.k_empty[u & 1]));
                }
                __syncwarp();
            }
            if (!ok) break;
            ++nacc;
            if (elect_one()) tc_commit(smem_u32(&sh.q_empty));
            __syncwarp();
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin));
            drain_bar(&sh.fin, 0, a.err);
        }
        __syncwarp();
    } else {
        const int half = warp >> 2, r = 32 * (warp & 3) + lane;      // query row; keys [64 half, 64 half + 64)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = a.scale * kLog2e;
        uint32_t n_sp = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const uint32_t slot = k & 1;
            if (!warp_wait(smem_u32(&sh.q.full[slot]), (k >> 1) & 1, abort_flag, a.err)) break;
            const Item it = sh.q.item[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q.empty[slot]));
            if (it.valid < 0) break;
            if (it.valid == 0) continue;
            const bool mine = r < it.rows;
            float l2 = CUDART_INF_F, dl = 0.f;
            if (mine) {
                const long long at = static_cast<long long>(it.head) * a.Tq + it.row0 + r;
                const float l = __ldg(a.lse + at);
                if (l != -CUDART_INF_F) l2 = l * kLog2e;
                dl = __ldg(delta + at);
            }
            // keys this row sees: [0, end)
            const int end = !mine ? 0 : (a.causal ? min(it.len, it.diag + r + 1) : it.len);
            for (int i = 0; i < it.n; ++i, ++n_sp) {
                if (!warp_wait(smem_u32(&sh.sp_full), n_sp & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[2][32], d[2][32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    tmem_ld32(tm_s + 64 * half + 32 * q + lane_base, s[q]);
                    tmem_ld32(tm_dp + 64 * half + 32 * q + lane_base, d[q]);
                }
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.sp_free));
                const int lim = end - 128 * i - 64 * half;
                const bool edge = __any_sync(0xffffffffu, lim < 64);
                uint32_t w[32];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float v[2];
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const int col = 2 * e + z;
                            const float p = exp2_fast(fmaf(__uint_as_float(s[q][col]), c, -l2));
                            v[z] = p * (__uint_as_float(d[q][col]) - dl);
                            if (edge && 32 * q + col >= lim) v[z] = 0.f;
                        }
                        w[16 * q + e] = pack_bf16x2(v[0], v[1]);
                    }
                // the dQ product of the tile before has read dS
                if (n_sp > 0 && !warp_wait(smem_u32(&sh.k_empty[(n_sp - 1) & 1]), ((n_sp - 1) >> 1) & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                tmem_st32(tm_ds + 32 * half + lane_base, w);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.ds_full));
            }
            if (!ok) break;
            if (it.n > 0) {
                if (!warp_wait(smem_u32(&sh.k_empty[(n_sp - 1) & 1]), ((n_sp - 1) >> 1) & 1, abort_flag, a.err)) break;
                tc_fence_after();
            }
            const bool any = it.n > 0;
            uint4* buf = reinterpret_cast<uint4*>(smem + OUT_OFF + 2048 * warp);
            __nv_bfloat16* dst = a.dq + (static_cast<long long>(it.row0) + 32 * (warp & 3)) * a.dq_row + it.head * a.dq_head + 96 * half;
#pragma unroll 1
            for (int q = 0; q < 3; ++q) {
                uint32_t o[32], w[16];
                if (any) {
                    tmem_ld32(tm_dq + 96 * half + 32 * q + lane_base, o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = any ? pack_bf16x2(__uint_as_float(o[2 * e]) * a.scale, __uint_as_float(o[2 * e + 1]) * a.scale) : 0u;
                store_rows(buf, lane, w, reinterpret_cast<uint8_t*>(dst + 32 * q), 2 * a.dq_row, it.rows - 32 * (warp & 3));
            }
            if (it.n > 0) {
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.acc_empty));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}
}  // namespace dq

size_t delta_bytes(int H, int Tq) { return (static_cast<size_t>(H) * Tq * 4 + 255) / 256 * 256; }

}  // namespace bw

size_t latent_backward_ws_bytes(int H, int Tq, int Tk) {
    return bw::delta_bytes(H, Tq) + static_cast<size_t>(H) * Tk * kRope * 4;
}

cudaError_t launch_latent_backward(const LatentPrefillArgs& a, void* ws, cudaStream_t st) {
    static bool attr_kv[kMaxDevices] = {false}, attr_dq[kMaxDevices] = {false};
    float* delta = static_cast<float*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + bw::delta_bytes(a.H, a.Tq));
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(bw::kv::dkv_kernel), bw::kv::SMEM, attr_kv);
    if (e == cudaSuccess) e = smem_attr_once(reinterpret_cast<const void*>(bw::dq::dq_kernel), bw::dq::SMEM, attr_dq);
    CUtensorMap q64, do64, q128, do128, kn, kr, v;
    auto map = [&](CUtensorMap* m, const void* p, int rows, int heads, int width, long long row, long long head, int box) {
        if (e == cudaSuccess) e = make_map_rows(m, p, rows, heads, width, row, head, box);
    };
    map(&q64, a.q, a.Tq, a.H, kDqk, a.q_row, a.q_head, 64);
    map(&do64, a.d_out, a.Tq, a.H, kDv, a.do_row, a.do_head, 64);
    map(&q128, a.q, a.Tq, a.H, kDqk, a.q_row, a.q_head, 128);
    map(&do128, a.d_out, a.Tq, a.H, kDv, a.do_row, a.do_head, 128);
    map(&kn, a.kn, a.Tk, a.H, kNope, a.kn_row, a.kn_head, 128);
    map(&kr, a.kr, a.Tk, 1, kRope, a.kr_row, 0, 128);
    map(&v, a.v, a.Tk, a.H, kDv, a.v_row, a.v_head, 128);
    if (e != cudaSuccess) return e;
    const long long pairs = static_cast<long long>(a.Tq) * a.H;
    bw::delta_kernel<<<static_cast<unsigned>((pairs + 15) / 16), 256, 0, st>>>(a, delta);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int ktiles = a.Tk / 128 + a.B, qtiles = a.Tq / 128 + a.B;
    bw::kv::dkv_kernel<<<static_cast<unsigned>(ktiles) * a.H, bw::THREADS, bw::kv::SMEM, st>>>(
        q64, kn, kr, v, do64, a, ktiles, delta, part);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    bw::rope_sum_kernel<<<dim3(ktiles, 8), 256, 0, st>>>(a, part);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    bw::dq::dq_kernel<<<static_cast<unsigned>(qtiles) * a.H, bw::THREADS, bw::dq::SMEM, st>>>(
        q128, kn, kr, v, do128, a, qtiles, delta);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
