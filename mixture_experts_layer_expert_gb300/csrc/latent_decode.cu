// latent_decode.cu -- absorbed latent attention of the newest tokens of each
// sequence over the paged latent cache:
//   s_i = scale (q_l . c_i + q_r . k_i),  out = sum_i softmax(s)_i c_i,  lse = log sum_i exp(s_i)
//
// All heads (and the n_q new tokens) of a sequence read the same records, so a
// block takes 64 query rows (row = new token * heads + head) against tiles of 64
// records, staged once in shared memory as bf16 and used twice:
//   S  = Q K^T      64 rows x 64 records x 576, both K-major
//   O^T += C^T P^T  512 (4 x 128) x rows x 64 records: the same tile read MN-major
//                   as the A operand, P (bf16, shared memory) as the B operand
// O^T keeps the 512-wide output in 4 x rows TMEM columns (rows rounded up to 16)
// and a few heads cost few columns; its rescaling by a row factor is rare, as in
// the expanded form (only when a maximum grows by 2^8).
//
// Bound: the records' bytes.  64 records are 73.7 KB (bf16) or 42 KB (FP8), 3,150 or
// 1,790 cycles of one SM's share of the memory bandwidth; 64 rows of MMAs take
// 1,152 + 768 cycles, 16 rows 1,152 + 576.
//
// The records of all sequences form one list of tiles which is cut into equal
// ranges, one per block (and per block of 64 rows), whatever the lengths.  A
// sequence inside one range is finished there; one that is cut leaves fp32
// partials (normalised O and lse) which a second kernel joins in range order.
//
// Warps 0-3: softmax, rescaling, output; warp 4: MMA issue; warps 5-12: page
// lookup and loads (cp.async for bf16; FP8 codes through registers, where code *
// scale is exact in bf16).  Ring stages of 64 records x 128 latent columns (16 KB).
#include <math_constants.h>

#include "kernels.h"
#include "latent.cuh"

namespace fs {
namespace dc {

constexpr int TT = 64;                        // records per tile
constexpr int ROWS = 64;                      // query rows per block
constexpr int CH = 64 * 128;                  // 64 records (or query rows) x 64 columns, 8 KB
constexpr int PAIR = 2 * CH;                  // ring stage: 128 latent columns
constexpr int MAXP = 11;                      // ring stages (8 with 64 query rows, 11 with 16)
constexpr int LOADERS = 256;
constexpr int THREADS = 160 + LOADERS;
constexpr int CTRL = 2048;
constexpr size_t SMEM = 232448;               // 227 KB
constexpr float kRescale = 8.0f;
constexpr uint32_t NONE = 0xffffffffu;        // (a cache of 2^32 - 1 records does not fit the memory)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Meta {                                 // of each range: the sequence of its first tile
    int b, off, tiles, pad;                   // off: tiles of the sequence before the range; tiles: of the range
};

struct Shared {
    uint64_t full[MAXP], empty[MAXP], r_full[2], r_empty[2], q_full, q_empty, s_full[2], p_full, pv_done, o_empty, fin;
    uint32_t tmem;
    int abort_flag;
    int b0, tile0, left;                      // first piece of this block's range
    uint32_t live[4][2];                      // records of a tile that count (4 tiles deep)
    int flag[2][4];
    float alpha[2][ROWS];                     // rescaling factors of a tile; 1 / l at the end of a piece
    uint32_t rec[2][TT];                      // each record's index, NONE: a zero row
    float scale[2][TT];
};
static_assert(sizeof(Shared) <= CTRL, "control area");

struct Piece {
    int b, t0, t1, n, len;                    // tiles [t0, t1) of the n of sequence b
};

__device__ __forceinline__ int seq_len(const LatentDecodeArgs& a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return n < 0 || n > static_cast<long long>(a.max_pages) * a.page_size ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return static_cast<int>((static_cast<unsigned>(len) + TT - 1) / TT); }

// Next piece of the range; b, tile, left advance.  False at the end.
__device__ __forceinline__ bool next_piece(const LatentDecodeArgs& a, int& b, int& tile, long long& left, Piece* p) {
    if (left <= 0) return false;
    int len = 0, n = 0;
    for (; b < a.B; ++b, tile = 0) {
        len = seq_len(a, b);
        n = tiles_of(len);
        if (tile < n) break;
    }
    if (b >= a.B) return false;
    p->b = b; p->len = len; p->n = n; p->t0 = tile;
    p->t1 = static_cast<int>(min(static_cast<long long>(n), tile + left));
    left -= p->t1 - p->t0;
    ++b;
    tile = 0;
    return true;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? 16 : 0;                // 0: sixteen zero bytes, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// The barrier receives this thread's arrival when its earlier cp.async copies are done.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

template <bool FP8>
__global__ void __launch_bounds__(THREADS, 1)
decode_kernel(const LatentDecodeArgs a, const int rb_count, const int ranges, float* __restrict__ part,
              float* __restrict__ part_lse, Meta* __restrict__ meta) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rb = blockIdx.x % rb_count, range = blockIdx.x / rb_count;
    const int rows = min(ROWS, a.n_q * a.H - rb * ROWS), rn = (rows + 15) & ~15;
    // Q chunks of rn rows (the MMA's 64 rows run on into what follows: rows nobody reads), P, rope ring, stage ring, control
    const int q_chunk = rn * 128, stages = rn <= 16 ? 11 : (rn <= 32 ? 10 : (rn <= 48 ? 9 : 8));
    uint8_t* sq = smem;
    uint8_t* sp = smem + 9 * q_chunk;
    uint8_t* srope = sp + CH;
    uint8_t* sring = srope + 2 * CH;
    Shared& sh = *reinterpret_cast<Shared*>(smem + (SMEM - 1024 - CTRL));
    volatile int* abort_flag = &sh.abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAXP; ++i) { mbar_init(smem_u32(&sh.full[i]), LOADERS); mbar_init(smem_u32(&sh.empty[i]), 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.r_full[i]), LOADERS + 2);
            mbar_init(smem_u32(&sh.r_empty[i]), 1);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
        }
        mbar_init(smem_u32(&sh.q_full), LOADERS);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.p_full), 128);
        mbar_init(smem_u32(&sh.pv_done), 1);
        mbar_init(smem_u32(&sh.o_empty), 128);
        mbar_init(smem_u32(&sh.fin), 1);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    if (warp == 0) {
        // this block's range of the list of tiles, and where it starts
        long long total = 0;
        for (int b = lane; b < a.B; b += 32) {
            const int n = __ldg(a.seq_lens + b);
            if (n < 0 || n > static_cast<long long>(a.max_pages) * a.page_size) set_dev_error(a.err, DEV_ERR_PAGE);
            total += tiles_of(seq_len(a, b));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        const long long g0 = total * range / ranges, g1 = total * (range + 1) / ranges;
        long long before = 0;
        int found_b = a.B, found_t = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int n = b0 + lane < a.B ? tiles_of(seq_len(a, b0 + lane)) : 0;
            long long end = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, end, d);
                if (lane >= d) end += v;
            }
            end += before;
            const unsigned past = __ballot_sync(0xffffffffu, end > g0);
            if (past) {
                const int l = __ffs(past) - 1;
                found_b = b0 + l;
                found_t = static_cast<int>(g0 - __shfl_sync(0xffffffffu, end - n, l));
                break;
            }
            before = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) {
            sh.b0 = found_b;
            sh.tile0 = found_t;
            sh.left = static_cast<int>(g1 - g0);
            if (rb == 0) meta[range] = Meta{found_b, found_t, static_cast<int>(g1 - g0), 0};
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm_s = sh.tmem, tm_o = sh.tmem + 128;
    int b = sh.b0, tile = sh.tile0;
    long long left = sh.left;
    Piece p;

    if (warp >= 5) {
        // -------------------------------------------------------------- loads
        const int t = threadIdx.x - 160;
        constexpr int REC = FP8 ? kRecFp8 : kRecBf16;
        uint32_t u = 0, g = 0, np = 0;                 // ring stages, tiles, pieces so far
        bool ok = true;
        auto offset = [&](uint32_t rec) { return rec == NONE ? -1LL : static_cast<long long>(rec) * REC; };
        const uint32_t ring = smem_u32(sring), rope = smem_u32(srope), qs = smem_u32(sq);
        while (ok && next_piece(a, b, tile, left, &p)) {
            // Q of the piece's sequence: rn rows x 72 sixteen-byte units; rows past the last are zeros
            if (!mbar_wait(smem_u32(&sh.q_empty), (np & 1) ^ 1, abort_flag, a.err)) break;
            for (int i = t; i < rn * 72; i += LOADERS) {
                const int r = i / 72, x = i - r * 72, c = x >> 3, qr = rb * ROWS + r;
                const int j = qr / a.H, h = qr - j * a.H;
                const long long row = static_cast<long long>(p.b) * a.n_q + j;
                const bool in = r < rows;
                const __nv_bfloat16* src = !in ? a.ql : (c < 8 ? a.ql + row * a.ql_row + h * a.ql_head + 8 * x
                                                               : a.qr + row * a.qr_row + h * a.qr_head + 8 * (x - 64));
                cp16(qs + c * q_chunk + r * 128 + (((x & 7) ^ (r & 7)) << 4), src, in);
            }
            cp_arrive(smem_u32(&sh.q_full));
            ++np;
            for (int ti = p.t0; ti < p.t1; ++ti, ++g) {
                const int par = g & 1;
                if (t < TT) {
                    const int pos = ti * TT + t;
                    uint32_t rec = NONE;
                    float sc = 0.f;
                    if (pos < p.len) {
                        const int pg = pos / a.page_size;
                        const int page = __ldg(a.table + p.b * a.table_row + pg);
                        if (page < 0 || page >= a.n_pages)
                            set_dev_error(a.err, DEV_ERR_PAGE);
                        else
                            rec = static_cast<uint32_t>(page) * static_cast<uint32_t>(a.page_size) + static_cast<uint32_t>(pos - pg * a.page_size);
                    }
                    sh.rec[par][t] = rec;
                    if constexpr (FP8) {
                        if (rec != NONE) sc = *reinterpret_cast<const float*>(a.cache + static_cast<long long>(rec) * REC + kFp8ScaleOff);
                        sh.scale[par][t] = sc;
                    }
                    const uint32_t live = __ballot_sync(0xffffffffu, rec != NONE);
                    if (lane == 0) sh.live[g & 3][t >> 5] = live;
                }
                bar_sync(2, LOADERS);
                // rotary keys: 64 records x 8 units
                if (!mbar_wait(smem_u32(&sh.r_empty[par]), ((g >> 1) & 1) ^ 1, abort_flag, a.err)) { ok = false; break; }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = (t >> 3) + 32 * e, x = t & 7;
                    const long long off = offset(sh.rec[par][r]);
                    cp16(rope + par * CH + r * 128 + ((x ^ (r & 7)) << 4),
                         a.cache + (off < 0 ? 0 : off) + (FP8 ? kFp8RopeOff : 2 * kLatent) + 16 * x, off >= 0);
                }
                cp_arrive(smem_u32(&sh.r_full[par]));
                if (t < TT && lane == 0) mbar_arrive(smem_u32(&sh.r_full[par]));      // live is written
                if constexpr (!FP8) {
                    for (int c = 0; c < 4; ++c, ++u) {
                        const uint32_t s = u % stages;
                        if (!mbar_wait(smem_u32(&sh.empty[s]), ((u / stages) & 1) ^ 1, abort_flag, a.err)) { ok = false; break; }
                        const int x = t & 15, r0 = t >> 4;             // unit of the 256 bytes, row
                        const uint32_t dst = ring + s * PAIR + (x >> 3) * CH + (((x & 7) ^ (r0 & 7)) << 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = r0 + 16 * e;
                            const long long off = offset(sh.rec[par][r]);
                            cp16(dst + r * 128, a.cache + (off < 0 ? 0 : off) + 256 * c + 16 * x, off >= 0);
                        }
                        cp_arrive(smem_u32(&sh.full[s]));
                    }
                } else {
                    // a thread takes 16 codes of a record in each stage: all loads of the tile first
                    const int x = t & 7, r0 = t >> 3;
                    uint4 v[4][2];
                    float sc[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const long long off = offset(sh.rec[par][r0 + 32 * e]);
                        sc[e] = sh.scale[par][r0 + 32 * e];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            v[c][e] = off < 0 ? make_uint4(0, 0, 0, 0)
                                              : __ldg(reinterpret_cast<const uint4*>(a.cache + off + 128 * c + 16 * x));
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c, ++u) {
                        const uint32_t s = u % stages;
                        if (!mbar_wait(smem_u32(&sh.empty[s]), ((u / stages) & 1) ^ 1, abort_flag, a.err)) { ok = false; break; }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = r0 + 32 * e;
                            const uint32_t w[4] = {v[c][e].x, v[c][e].y, v[c][e].z, v[c][e].w};
                            uint32_t o[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[2 * i] = e4m3x2_to_bf16x2(w[i] & 0xffffu, sc[e]);
                                o[2 * i + 1] = e4m3x2_to_bf16x2(w[i] >> 16, sc[e]);
                            }
                            const uint32_t base = ring + s * PAIR + (x >> 2) * CH + r * 128;
                            const int y = 2 * (x & 3);
                            sts16(base + ((y ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
                            sts16(base + (((y + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
                        }
                        fence_proxy_async_smem();
                        mbar_arrive(smem_u32(&sh.full[s]));
                    }
                }
                if (!ok) break;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");       // nothing is in flight when the block ends
    } else if (warp == 4) {
        // ---------------------------------------------------------------- MMA
        const uint32_t id_s = idesc_bf16_f32(ROWS, TT), id_o = idesc_bf16_f32_t(128, rn, 1, 0);
        uint32_t u = 0, g = 0, np = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (lane == 0) ok = mbar_wait(smem_u32(bar), parity, abort_flag, a.err);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            return ok;
        };
        // S of tile gg whose first ring stage is uu
        auto score = [&](uint32_t gg, uint32_t uu) {
            if (!wait(&sh.r_full[gg & 1], (gg >> 1) & 1)) return false;
            const uint32_t d = tm_s + 64 * (gg & 1);
            if (elect_one()) {
                fence_proxy_async_smem();              // the copies' writes, before the tensor cores read them
                tc_fence_after();
                const uint64_t ad = smem_desc_sw128(smem_u32(sq + 8 * q_chunk));
                const uint64_t bd = smem_desc_sw128(smem_u32(srope + (gg & 1) * CH));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) tc_mma_bf16(d, ad + 2ull * kk, bd + 2ull * kk, id_s, kk > 0);
                tc_commit(smem_u32(&sh.r_empty[gg & 1]));
            }
            __syncwarp();
            for (int c = 0; c < 4; ++c) {
                const uint32_t s = (uu + c) % stages;
                if (!wait(&sh.full[s], ((uu + c) / stages) & 1)) return false;
                if (elect_one()) {
                    fence_proxy_async_smem();
                    tc_fence_after();
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t ad = smem_desc_sw128(smem_u32(sq + (2 * c + e) * q_chunk));
                        const uint64_t bd = smem_desc_sw128(smem_u32(sring + s * PAIR + e * CH));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) tc_mma_bf16(d, ad + 2ull * kk, bd + 2ull * kk, id_s, 1);
                    }
                }
                __syncwarp();
            }
            if (elect_one()) tc_commit(smem_u32(&sh.s_full[gg & 1]));
            __syncwarp();
            return true;
        };
        while (ok && next_piece(a, b, tile, left, &p)) {
            if (!wait(&sh.q_full, np & 1)) break;
            if (!score(g, u)) break;
            const int n = p.t1 - p.t0;
            if (n == 1 && elect_one()) tc_commit(smem_u32(&sh.q_empty));
            for (int i = 0; i < n; ++i, ++g, u += 4) {
                if (i + 1 < n) {
                    if (!score(g + 1, u + 4)) break;
                    if (i + 2 == n && elect_one()) tc_commit(smem_u32(&sh.q_empty));
                }
                if (i == 0 && !wait(&sh.o_empty, (np & 1) ^ 1)) break;
                if (!wait(&sh.p_full, g & 1)) break;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t bd = smem_desc_sw128(smem_u32(sp));
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t s = (u + c) % stages;
                        const uint32_t v = smem_u32(sring + s * PAIR);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_bf16(tm_o + c * rn, smem_desc_sw128_mn(v + 2048 * kk, CH), bd + 2ull * kk, id_o,
                                        i > 0 || kk > 0);
                        tc_commit(smem_u32(&sh.empty[s]));
                    }
                    tc_commit(smem_u32(&sh.pv_done));
                }
                __syncwarp();
            }
            ++np;
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.fin));
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&sh.fin), 0))
                if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(a.err, DEV_ERR_TIMEOUT); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------------- softmax, rescaling and output
        // S rows 16 w .. 16 w + 15 lie in the first 16 lanes of warp w's TMEM quarter
        const int r = 16 * warp + (lane & 15);
        const bool mine = lane < 16 && r < rows;
        const int qrow = rb * ROWS + min(r, rows - 1), j = qrow / a.H, h = qrow - j * a.H;
        const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
        const float c = a.scale * kLog2e;
        uint32_t g = 0;
        bool ok = true;
        // sequences without records: zero rows, spread over the ranges
        for (int e = range; e < a.B; e += ranges) {
            if (seq_len(a, e) != 0) continue;
            for (int i = threadIdx.x; i < rows * 64; i += 128) {
                const int q = rb * ROWS + (i >> 6), jj = q / a.H, hh = q - jj * a.H;
                const long long row = static_cast<long long>(e) * a.n_q + jj;
                reinterpret_cast<uint4*>(a.out + row * a.o_row + hh * a.o_head)[i & 63] = make_uint4(0, 0, 0, 0);
                if (a.lse && (i & 63) == 0) a.lse[row * a.H + hh] = -CUDART_INF_F;
            }
        }
        while (ok && next_piece(a, b, tile, left, &p)) {
            const int end = p.len - (a.n_q - 1 - j);           // this row sees positions [0, end)
            float m = -CUDART_INF_F, l = 0.f;
            for (int ti = p.t0; ti < p.t1; ++ti, ++g) {
                if (!mbar_wait(smem_u32(&sh.s_full[g & 1]), (g >> 1) & 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(tm_s + 64 * (g & 1) + lane_base, s[0]);
                tmem_ld32(tm_s + 64 * (g & 1) + 32 + lane_base, s[1]);
                tmem_ld_wait();
                const int lim = mine ? end - ti * TT : 0;
                uint32_t live[2] = {sh.live[g & 3][0], sh.live[g & 3][1]};
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
                float al = 1.f;
                bool grow = false;
                if (ti == p.t0) {
                    m = top;
                } else if (top > m + kRescale) {               // also the first record a row sees (m = -inf)
                    grow = true;
                    al = exp2_fast(m - top);
                    m = top;
                    l *= al;
                }
                const bool any = __any_sync(0xffffffffu, grow);
                if (lane < 16) sh.alpha[g & 1][r] = al;
                if (lane == 0) sh.flag[g & 1][warp] = any;
                bar_sync(1, 128);
                // P and O are free once the product of the tile before is done
                if (g > 0 && !mbar_wait(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err)) { ok = false; break; }
                const int* fl = sh.flag[g & 1];
                if (fl[0] | fl[1] | fl[2] | fl[3]) {
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < 4 * rn; cc += 16) {
                        uint32_t o[16];
                        tmem_ld16(tm_o + cc + lane_base, o);
                        tmem_ld_wait();
                        const float4* f4 = reinterpret_cast<const float4*>(&sh.alpha[g & 1][cc % rn]);
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
                const float me = m == -CUDART_INF_F ? 0.f : m;
                float sum[2] = {0.f, 0.f};
                const uint32_t prow = smem_u32(sp) + r * 128;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = exp2_fast(fmaf(__uint_as_float(s[q >> 2][8 * (q & 3) + 2 * e]), c, -me));
                        const float x1 = exp2_fast(fmaf(__uint_as_float(s[q >> 2][8 * (q & 3) + 2 * e + 1]), c, -me));
                        sum[0] += x0;
                        sum[1] += x1;
                        w[e] = pack_bf16x2(x0, x1);
                    }
                    if (lane < 16 && r < rn) sts16(prow + ((q ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                l += sum[0] + sum[1];
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full));
            }
            if (!ok) break;
            if (!mbar_wait(smem_u32(&sh.pv_done), (g - 1) & 1, abort_flag, a.err)) break;
            tc_fence_after();
            const bool whole = p.t0 == 0 && p.t1 == p.n;
            const long long slot = (static_cast<long long>(range) * rb_count + rb) * 2 + (p.b == sh.b0 ? 0 : 1);
            if (lane < 16) sh.alpha[g & 1][r] = l > 0.f ? 1.f / l : 0.f;
            if (mine) {
                const float lse = l > 0.f ? m + log2f(l) : -CUDART_INF_F;      // log2 units
                if (!whole) part_lse[slot * ROWS + r] = lse;
                else if (a.lse) a.lse[(static_cast<long long>(p.b) * a.n_q + j) * a.H + h] = lse * kLn2;
            }
            bar_sync(1, 128);
            // O^T: lane = latent element, column = row
#pragma unroll 1
            for (int cc = 0; cc < 4 * rn; cc += 16) {
                uint32_t o[16];
                tmem_ld16(tm_o + cc + lane_base, o);
                tmem_ld_wait();
                const int d = (cc / rn) * 128 + 32 * warp + lane, r0 = cc % rn;
                int qq = rb * ROWS + r0, jj = qq / a.H, hh = qq - jj * a.H;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (r0 + e < rows) {
                        const float f = sh.alpha[g & 1][r0 + e];
                        const float v = f > 0.f ? __uint_as_float(o[e]) * f : 0.f;
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

constexpr int kRanges = 152;                  // one block per SM

// Joins the partials of the sequences that range boundaries cut.  Block (boundary, row, row block): the boundary
// before range s; the first boundary inside a sequence joins all its pieces, in range order.
__global__ void __launch_bounds__(128)
join_kernel(const LatentDecodeArgs a, const int rb_count, const int ranges, const float* __restrict__ part,
            const float* __restrict__ part_lse, const Meta* __restrict__ meta) {
    __shared__ int slots[kRanges];
    __shared__ float weight[kRanges];
    __shared__ int count;
    __shared__ float z_ref[2];
    const int s = blockIdx.x + 1, r = blockIdx.y, rb = blockIdx.z;
    const int q = rb * ROWS + r;
    if (q >= a.n_q * a.H) return;
    const Meta m = meta[s];
    if (m.b >= a.B || m.tiles == 0 || m.off == 0) return;     // no tiles, or the sequence starts here
    if (threadIdx.x < 32) {
        // the range before (empty ones, where there are fewer tiles than ranges, aside) holds the piece before
        const int lane = threadIdx.x;
        int first = s - 1;
        for (;; first -= 32) {
            const int k = first - lane;
            const unsigned some = __ballot_sync(0xffffffffu, k >= 0 && meta[k < 0 ? 0 : k].tiles > 0);
            if (some) { first -= __ffs(some) - 1; break; }
            if (first < 32) break;                            // (cannot be: m.off > 0)
        }
        int n = 0;
        float top = -CUDART_INF_F;
        const Meta mf = meta[first < 0 ? 0 : first];
        if (first >= 0 && !(mf.b == m.b && mf.off > 0)) {     // else an earlier boundary is inside the sequence too
            for (int k0 = first; k0 < ranges; k0 += 32) {
                const int k = k0 + lane;
                Meta mk{-1, 0, 0, 0};
                if (k < ranges) mk = meta[k];
                const bool in = mk.tiles > 0 && (mk.b == m.b || k == first);
                const unsigned mask = __ballot_sync(0xffffffffu, in);
                if (in) {
                    const int at = n + __popc(mask & ((1u << lane) - 1u));
                    slots[at] = (k * rb_count + rb) * 2 + (mk.b == m.b ? 0 : 1);
                    weight[at] = part_lse[static_cast<long long>(slots[at]) * ROWS + r];
                    top = fmaxf(top, weight[at]);
                }
                n += __popc(mask);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            __syncwarp();
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            float z = 0.f;
            for (int k = lane; k < n; k += 32) {
                weight[k] = exp2_fast(weight[k] - ref);
                z += weight[k];
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            if (lane == 0) { z_ref[0] = z; z_ref[1] = ref; }
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    if (n == 0) return;
    const float z = z_ref[0];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
        const float w = weight[k];
        const float4 v = __ldg(reinterpret_cast<const float4*>(part + (static_cast<long long>(slots[k]) * ROWS + r) * kLatent) + threadIdx.x);
        acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
    const float inv = z > 0.f ? 1.f / z : 0.f;
    const int j = q / a.H, h = q - j * a.H;
    const long long row = static_cast<long long>(m.b) * a.n_q + j;
    reinterpret_cast<uint2*>(a.out + row * a.o_row + h * a.o_head)[threadIdx.x] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse && threadIdx.x == 0) a.lse[row * a.H + h] = z > 0.f ? (z_ref[1] + log2f(z)) * kLn2 : -CUDART_INF_F;
}


void shape(int H, int n_q, int* rb, int* ranges) {
    *rb = (H * n_q + ROWS - 1) / ROWS;
    *ranges = kRanges / *rb > 0 ? kRanges / *rb : 1;
}

}  // namespace dc

// Partials of at most two cut pieces per range and row block, their lse, the ranges' descriptions.
size_t latent_decode_ws_bytes(int H, int, int n_q) {
    int rb, ranges;
    dc::shape(H, n_q, &rb, &ranges);
    const size_t slots = static_cast<size_t>(rb) * ranges * 2;
    return slots * dc::ROWS * (kLatent + 1) * 4 + (ranges * sizeof(dc::Meta) + 255) / 256 * 256;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void* ws, cudaStream_t st) {
    static bool attr[2][kMaxDevices] = {{false}};
    auto fn = fp8 ? dc::decode_kernel<true> : dc::decode_kernel<false>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), dc::SMEM, attr[fp8]);
    if (e != cudaSuccess) return e;
    int rb, ranges;
    dc::shape(a.H, a.n_q, &rb, &ranges);
    const size_t slots = static_cast<size_t>(rb) * ranges * 2;
    float* part = static_cast<float*>(ws);
    float* part_lse = part + slots * dc::ROWS * kLatent;
    dc::Meta* meta = reinterpret_cast<dc::Meta*>(part_lse + slots * dc::ROWS);
    fn<<<static_cast<unsigned>(rb * ranges), dc::THREADS, dc::SMEM, st>>>(a, rb, ranges, part, part_lse, meta);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess || ranges == 1) return e;
    const int rows = a.H * a.n_q < dc::ROWS ? a.H * a.n_q : dc::ROWS;
    dc::join_kernel<<<dim3(ranges - 1, rows, rb), 128, 0, st>>>(a, rb, ranges, part, part_lse, meta);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
