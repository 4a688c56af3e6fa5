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

__device__ __forceinline__ int seq_len(const LatentDecodeArgs& a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return n < 0 || n > static_cast<long long>(a.max_pages) * a.page_size ? 0 : n;
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

// The table's entry for position pos of sequence b (0 past the end): only the load, so that it can be issued a
// tile ahead of its use.
__device__ __forceinline__ int page_at(const LatentDecodeArgs& a, int b, int len, int pos) {
    return pos < len ? __ldg(a.table + b * a.table_row + pos / a.page_size) : 0;
}
// Record of position pos on that page, or NONE (past the end, or a page outside the cache, which is recorded).
__device__ __forceinline__ uint32_t record_of(const LatentDecodeArgs& a, int len, int pos, int page) {
    if (pos >= len) return NONE;
    if (page < 0 || page >= a.n_pages) {
        set_dev_error(a.err, DEV_ERR_PAGE);
        return NONE;
    }
    return static_cast<uint32_t>(page) * static_cast<uint32_t>(a.page_size) + static_cast<uint32_t>(pos % a.page_size);
}

// 64 consecutive positions of a sequence as one load: lane l brings the records of positions l and 32 + l.
struct Group {
    uint32_t live0, live1;      // which count
    int start;                  // first record
    bool box;                   // 64 consecutive records, or none at all (start: past the cache's end)
    int y[4];                   // the four records of gather group lane & 15
};
__device__ __forceinline__ Group make_group(uint32_t r0, uint32_t r1, int records, int lane) {
    Group g;
    g.live0 = __ballot_sync(0xffffffffu, r0 != NONE);
    g.live1 = __ballot_sync(0xffffffffu, r1 != NONE);
    const uint32_t start = __shfl_sync(0xffffffffu, r0, 0);
    const bool none = (g.live0 | g.live1) == 0;
    g.start = none ? records : static_cast<int>(start);
    g.box = none || __all_sync(0xffffffffu, r0 == start + lane && r1 == start + 32 + lane && r1 != NONE);
    // a record that does not count is read as a copy of one that does: its p is 0
    const uint32_t a = __shfl_sync(0xffffffffu, r0, g.live0 ? __ffs(g.live0) - 1 : 0);
    const uint32_t b = __shfl_sync(0xffffffffu, r1, g.live1 ? __ffs(g.live1) - 1 : 0);
    const uint32_t some = g.live0 ? a : b;
    if (r0 == NONE) r0 = some;
    if (r1 == NONE) r1 = some;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int src = 4 * (lane & 7) + e;
        const uint32_t lo = __shfl_sync(0xffffffffu, r0, src), hi = __shfl_sync(0xffffffffu, r1, src);
        g.y[e] = static_cast<int>((lane & 8) ? hi : lo);
    }
    return g;
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Whole warp: `chunks` boxes of 64 records x 128 bytes (columns from col on, col_step elements apart) to dst, each
// 8 KB.  expect: the barrier's one arrival with this many bytes (0: another CTA makes it).  A group without
// records is a box past the cache's end: zeros.  PAIR_BAR: bar is a shared::cluster address.
template <bool PAIR_BAR>
__device__ __forceinline__ void load_group(const CUtensorMap* tile, const CUtensorMap* row, const Group& g, uint32_t dst,
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
        if (c < chunks) {
            if constexpr (PAIR_BAR) tma_gather4_pair(to, row, bar, col + c * col_step, g.y[0], g.y[1], g.y[2], g.y[3]);
            else tma_gather4(to, row, bar, col + c * col_step, g.y[0], g.y[1], g.y[2], g.y[3]);
        }
    }
    __syncwarp();
}
// 64 threads (t): R query rows from row0 on of sequence b (rows of them real, the others zeros) into R-row chunks of
// 64 columns at dst.  All copies are in flight together, then visible to the tensor cores.
template <int R>
__device__ __forceinline__ void load_q(const LatentDecodeArgs& a, int b, int row0, int rows, uint32_t dst, int t) {
    constexpr int PER = 64 / R;                 // threads per row
    const int r = t / PER, x0 = t % PER, qr = row0 + (r < rows ? r : 0), j = qr / a.H, h = qr - j * a.H;
    const long long row = static_cast<long long>(b) * a.n_q + j;
    const __nv_bfloat16* ql = a.ql + row * a.ql_row + h * a.ql_head;
    const __nv_bfloat16* qr64 = a.qr + row * a.qr_row + h * a.qr_head;
    const int n = r < rows ? 16 : 0;            // 0: sixteen zero bytes, nothing is read
#pragma unroll 8
    for (int x = x0; x < 72; x += PER) {
        const __nv_bfloat16* src = x < 64 ? ql + 8 * x : qr64 + 8 * (x - 64);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (x >> 3) * (R * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4)),
                     "l"(src), "r"(n)
                     : "memory");
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
// Bounded wait without regard to the abort flag, for loads in flight at the block's end.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, int* err) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(bar), parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(err, DEV_ERR_TIMEOUT); break; }
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
        if (n < 0 || n > static_cast<long long>(a.max_pages) * a.page_size) set_dev_error(a.err, DEV_ERR_PAGE);
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
