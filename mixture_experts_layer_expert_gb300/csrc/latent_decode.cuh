// latent_decode.cuh -- what the two kernels of absorbed latent attention share: the list of tiles of
// all sequences and its ranges, page lookup, loads of 64 records, FP8 codes to bf16.
#pragma once

#include <math_constants.h>

#include "kernels.h"
#include "latent.cuh"

namespace fs {
namespace dc {

constexpr int CH = 64 * 128;                  // 64 records (or query rows) x 128 bytes, 8 KB
constexpr int PAIR = 2 * CH;                  // ring stage: 64 records x 128 latent columns in bf16
constexpr size_t SMEM = 232448;               // 227 KB
constexpr float kRescale = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t NONE = 0xffffffffu;        // no record

struct Meta {                                 // of each range: the sequence of its first tile
    int b, off, tiles, pad;                   // off: tiles of the sequence before the range; tiles: of the range
};

struct Piece {
    int b, t0, t1, n, len;                    // tiles [t0, t1) of the n of sequence b
};

// Whether a sequence's length is one that its table can hold (and whose last tile's positions fit an int).
__device__ __forceinline__ bool good_len(const LatentDecodeArgs& a, int n) {
    return n >= 0 && n <= 0x7fffffff - 256 && n <= static_cast<long long>(a.max_pages) * a.page_size;
}
__device__ __forceinline__ int seq_len(const LatentDecodeArgs& a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return good_len(a, n) ? n : 0;
}
// Next piece of the range (tiles of tt records); b, tile, left advance.  False at the end.
__device__ __forceinline__ bool next_piece(const LatentDecodeArgs& a, int& b, int& tile, int& left, Piece* p, int tt) {
    if (left <= 0) return false;
    int len = 0, n = 0;
    for (; b < a.B; ++b, tile = 0) {
        len = seq_len(a, b);
        n = static_cast<int>((static_cast<unsigned>(len) + tt - 1) / tt);
        if (tile < n) break;
    }
    if (b >= a.B) return false;
    p->b = b; p->len = len; p->n = n; p->t0 = tile;
    p->t1 = tile + min(n - tile, left);
    left -= p->t1 - p->t0;
    ++b;
    tile = 0;
    return true;
}

// A tile's records as the loader needs them, for TT / 64 halves of 64 consecutive positions.
template <int TT>
struct TileRecs {
    alignas(16) int rec[TT];    // record of each position; one that does not count: a copy of one that does (its p is 0)
    int start[TT / 64];         // first record of a half that is one box: 64 consecutive records, or none at all (start
    int box[TT / 64];           //   past the cache's end: zeros); else four records at a time are gathered
};
constexpr int kInfo = 8;        // depth of what the lookup leaves for the softmax (see lookup_tiles)

// The lookup warp: for every tile of the block's range, its records (two tiles ahead of the loads at most),
// which of them count and (FP8) their scales, and its halves own0 .. own1 asked into L2.  Three tiles are under
// way: the table's entries of one, the scales of the tile before, the publication of the tile before that, so no
// load is waited for in the iteration that issues it.  Tile g is published once the loads of tile g - 3 are all
// issued; the last of them needed its place in the ring, which holds 11 stages at most (with FP8 that of the raw
// stage four before it, converted into a ring of 9 at most), and that place was left by the product P C of tile
// g - 5 (g - 6) or a later one: the softmax is past that tile, so kInfo slots are enough.
template <bool FP8, int TT>
__device__ __forceinline__ void lookup_tiles(const LatentDecodeArgs& a, int b, int tile, int left, int own0, int own1,
                                             TileRecs<TT>* recs, uint64_t* tile_full, uint64_t* tile_empty,
                                             uint32_t (*live)[TT / 32], float (*scale)[TT], uint64_t* info_full,
                                             volatile int* abort_flag) {
    constexpr int NE = TT / 32, REC = FP8 ? kRecFp8 : kRecBf16;
    const int lane = threadIdx.x & 31;
    const int records = static_cast<int>(a.n_pages * a.page_size);
    const int step_pages = TT / a.page_size, step_off = TT % a.page_size;
    Piece p;
    uint32_t g = 0;
    while (next_piece(a, b, tile, left, &p, TT)) {
        const int32_t* table = a.table + p.b * a.table_row;
        int pi[NE], off[NE], page[NE], poff[NE];     // page index and offset of the next tile's positions 32 e + lane
        uint32_t r[NE];                              // records (and scales) of the tile to publish next
        float sc[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int pos = p.t0 * TT + 32 * e + lane;
            pi[e] = pos / a.page_size;
            off[e] = pos - pi[e] * a.page_size;
            page[e] = poff[e] = 0;
            r[e] = NONE;
            sc[e] = 0.f;
        }
#pragma unroll 1
        for (int ti = p.t0; ti < p.t1 + 2; ++ti) {
            if (ti >= p.t0 + 2) {                    // publish tile ti - 2
                if (!warp_wait(smem_u32(&tile_empty[g & 1]), ((g >> 1) & 1) ^ 1, abort_flag, a.err)) return;
                TileRecs<TT>& t = recs[g & 1];
                const uint32_t k = g % kInfo;
#pragma unroll
                for (int h = 0; h < TT / 64; ++h) {
                    const uint32_t r0 = r[2 * h], r1 = r[2 * h + 1];
                    const uint32_t l0 = __ballot_sync(0xffffffffu, r0 != NONE), l1 = __ballot_sync(0xffffffffu, r1 != NONE);
                    const uint32_t start = __shfl_sync(0xffffffffu, r0, 0);
                    const bool none = (l0 | l1) == 0;
                    const bool box = none || __all_sync(0xffffffffu, r0 == start + lane && r1 == start + 32 + lane && r1 != NONE);
                    const uint32_t s0 = __shfl_sync(0xffffffffu, r0, l0 ? __ffs(l0) - 1 : 0);
                    const uint32_t s1 = __shfl_sync(0xffffffffu, r1, l1 ? __ffs(l1) - 1 : 0);
                    const uint32_t some = l0 ? s0 : s1;
                    t.rec[64 * h + lane] = static_cast<int>(r0 == NONE ? some : r0);
                    t.rec[64 * h + 32 + lane] = static_cast<int>(r1 == NONE ? some : r1);
                    if (FP8) {
                        scale[k][64 * h + lane] = sc[2 * h];
                        scale[k][64 * h + 32 + lane] = sc[2 * h + 1];
                    }
                    if (lane == 0) {
                        t.start[h] = none ? records : static_cast<int>(start);
                        t.box[h] = box;
                        live[k][2 * h] = l0;
                        live[k][2 * h + 1] = l1;
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&tile_full[g & 1]));
                    mbar_arrive(smem_u32(&info_full[k]));
                }
                ++g;
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                // records of tile ti - 1 from its pages; a page outside the cache is recorded and its positions left out
                r[e] = NONE;
                sc[e] = 0.f;
                if (ti > p.t0 && (ti - 1) * TT + 32 * e + lane < p.len) {
                    if (page[e] < 0 || page[e] >= a.n_pages) {
                        set_dev_error(a.err, DEV_ERR_PAGE);
                    } else {
                        r[e] = static_cast<uint32_t>(page[e]) * static_cast<uint32_t>(a.page_size) + static_cast<uint32_t>(poff[e]);
                        const uint8_t* rec = a.cache + static_cast<long long>(r[e]) * REC;
                        if (FP8) sc[e] = *reinterpret_cast<const float*>(rec + kFp8ScaleOff);
                        if (e / 2 >= own0 && e / 2 <= own1) {
#pragma unroll 1
                            for (int q = 0; q < REC; q += 128) prefetch_l2(rec + q);
                        }
                    }
                }
                // the table's entry of tile ti
                poff[e] = off[e];
                if (ti < p.t1 && ti * TT + 32 * e + lane < p.len) page[e] = __ldg(table + pi[e]);
                pi[e] += step_pages;
                off[e] += step_off;
                if (off[e] >= a.page_size) { off[e] -= a.page_size; ++pi[e]; }
            }
        }
    }
}

// One half of a tile in the loader's registers.
struct Half {
    int start;
    bool box;
    bool run;                   // the sixteen records of lane group lane / 4 follow one another
    int4 y;                     // the four records of gather group lane & 15
};
template <int TT>
__device__ __forceinline__ Half read_half(const TileRecs<TT>& t, int h, int lane) {
    const int4 y = *reinterpret_cast<const int4*>(&t.rec[64 * h + 4 * (lane & 15)]);
    const int first = __shfl_sync(0xffffffffu, y.x, lane & 28) + 4 * (lane & 3);
    const unsigned next = __ballot_sync(0xffffffffu, y.x == first && y.y == first + 1 && y.z == first + 2 && y.w == first + 3);
    return Half{t.start[h], t.box[h] != 0, ((next >> (lane & 28)) & 15u) == 15u, y};
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Whole warp: `chunks` boxes of 64 records x 128 bytes (columns from col on, col_step elements apart) to dst, each
// 8 KB; records that do not follow one another come in boxes of sixteen where those do (pages of a multiple of 16),
// else by gathers of four, which take the TMA unit about 100 cycles each (48-token pages, FP8, 256 query rows: 230 us
// with gathers alone, 162 so).  expect: the barrier's one arrival with this many bytes (0: another CTA makes it).  PAIR_BAR: bar is a
// shared::cluster address.
template <bool PAIR_BAR>
__device__ __forceinline__ void load_half(const CUtensorMap* tile, const CUtensorMap* run, const CUtensorMap* row, const Half& g, uint32_t dst,
                                          uint32_t bar, uint32_t local_bar, uint32_t expect, int col, int col_step, int chunks,
                                          int lane) {
    if (g.box) {
        if (elect_one()) {
            if (expect) mbar_arrive_expect_tx(local_bar, expect);
            for (int c = 0; c < chunks; ++c) {
                if constexpr (PAIR_BAR) tma_load_2d_pair(dst + c * CH, tile, bar, col + c * col_step, g.start);
                else tma_load_2d(dst + c * CH, tile, bar, col + c * col_step, g.start);
            }
        }
    } else {
        if (expect && lane == 0) mbar_arrive_expect_tx(local_bar, expect);
        __syncwarp();
        const int c = lane >> 4;
        const uint32_t to = dst + c * CH + (lane & 15) * 512;
        if (c < chunks && g.run) {
            if ((lane & 3) == 0) {
                if constexpr (PAIR_BAR) tma_load_2d_pair(to, run, bar, col + c * col_step, g.y.x);
                else tma_load_2d(to, run, bar, col + c * col_step, g.y.x);
            }
        } else if (c < chunks) {
            if constexpr (PAIR_BAR) tma_gather4_pair(to, row, bar, col + c * col_step, g.y.x, g.y.y, g.y.z, g.y.w);
            else tma_gather4(to, row, bar, col + c * col_step, g.y.x, g.y.y, g.y.z, g.y.w);
        }
    }
    __syncwarp();
}
// One warp: R query rows from row0 on of sequence b (rows of them real, the others zeros) into R-row chunks of 64
// columns at dst.  All copies are in flight together, then visible to the tensor cores.
template <int R>
__device__ __forceinline__ void load_q(const LatentDecodeArgs& a, int b, int row0, int rows, uint32_t dst, int lane) {
    constexpr int PER = R < 32 ? 32 / R : 1;    // threads per row
#pragma unroll
    for (int r = lane / PER; r < R; r += 32 / PER) {
        // a row past the last: sixteen zero bytes from an address inside the operand (row0 itself lies behind the last
        // row in a pair's second CTA that has none)
        const int qr = r < rows ? row0 + r : 0, j = qr / a.H, h = qr - j * a.H;
        const long long row = static_cast<long long>(b) * a.n_q + j;
        const __nv_bfloat16* ql = a.ql + row * a.ql_row + h * a.ql_head;
        const __nv_bfloat16* qr64 = a.qr + row * a.qr_row + h * a.qr_head;
        const int n = r < rows ? 16 : 0;        // 0: sixteen zero bytes, nothing is read
#pragma unroll 8
        for (int x = lane % PER; x < 72; x += PER) {
            const __nv_bfloat16* src = x < 64 ? ql + 8 * x : qr64 + 8 * (x - 64);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (x >> 3) * (R * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4)),
                         "l"(src), "r"(n)
                         : "memory");
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
}
// 16 E4M3 codes -> 32 bytes of bf16 at units y, y + 1 of the 128-byte row at base (swizzled by row r).
__device__ __forceinline__ void put_codes(const uint4& v, uint32_t base, int y, int r) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = e4m3x2_to_bf16x2(w[i] & 0xffffu);
        o[2 * i + 1] = e4m3x2_to_bf16x2(w[i] >> 16);
    }
    sts16(base + ((y ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
    sts16(base + (((y + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// Barrier of n threads that also tells whether any of them brought `v`.
__device__ __forceinline__ bool bar_any(int id, int n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// One warp: the range's first sequence and tile (of tt records), and its length, for the block and (write) for the join.
__device__ __forceinline__ void find_range(const LatentDecodeArgs& a, int range, int ranges, int tt, bool write, Meta* meta,
                                           int* b0, int* tile0, int* left) {
    const int lane = threadIdx.x & 31;
    auto tiles = [&](int b) { return static_cast<int>((static_cast<unsigned>(seq_len(a, b)) + tt - 1) / tt); };
    long long total = 0;
    for (int b = lane; b < a.B; b += 32) {
        const int n = __ldg(a.seq_lens + b);
        if (!good_len(a, n)) set_dev_error(a.err, DEV_ERR_PAGE);
        total += tiles(b);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    const long long g0 = total * range / ranges, g1 = total * (range + 1) / ranges;
    long long before = 0;
    int found_b = a.B, found_t = 0;
    for (int c0 = 0; c0 < a.B; c0 += 32) {
        const int n = c0 + lane < a.B ? tiles(c0 + lane) : 0;
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
            found_b = c0 + l;
            found_t = static_cast<int>(g0 - __shfl_sync(0xffffffffu, end - n, l));
            break;
        }
        before = __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) {
        *b0 = found_b;
        *tile0 = found_t;
        *left = static_cast<int>(g1 - g0);
        if (write) meta[range] = Meta{found_b, found_t, static_cast<int>(g1 - g0), 0};
    }
}

}  // namespace dc
}  // namespace fs
