// latent.cuh -- shared definitions of the latent-attention operators: head
// sizes, the paged cache's token records, the rotary table.
//
// One token's keys and values come from one latent vector c (512) and one
// rotary key (64) shared by all heads.  A cache record holds both:
//   bf16: 512 bf16 latent, 64 bf16 rotary key                         (1152 bytes)
//   FP8 : 512 E4M3 codes, 64 bf16 rotary key, fp32 scale, 12 zero bytes (656 bytes)
// The FP8 latent is quantised as an FP8 row (fp8.cuh): one power-of-two scale
// per token, so code * scale is exact in bf16 and only the E4M3 conversion
// rounds.  The rotary key stays bf16: it carries the position, and it is 11% of
// the bf16 record.
#pragma once

#include <cuda_fp16.h>

#include "fp8.cuh"

namespace fs {

constexpr int kLatent = 512;     // latent vector c
constexpr int kRope = 64;        // rotary key shared by the heads
constexpr int kNope = 128;       // unrotated part of an expanded key
constexpr int kDv = 128;         // expanded value
constexpr int kDqk = kNope + kRope;
constexpr int kRecBf16 = 2 * (kLatent + kRope);
constexpr int kRecFp8 = kLatent + 2 * kRope + 16;
constexpr int kFp8RopeOff = kLatent;                 // byte offsets inside an FP8 record
constexpr int kFp8ScaleOff = kLatent + 2 * kRope;
constexpr int kMaxRot = 256;     // largest rotated width

// Rotary frequencies in turns per position as 64-bit fractions: position *
// frac mod 2^64 is the angle's fraction of a turn, exact for any int32 position
// (fp32 products lose the angle once position * frequency passes 2^24 ulps).
struct RopeTab {
    uint64_t frac[kMaxRot / 2];
    float mscale;                // multiplies cos and sin
    int d_rot;
    int half;                    // 0: pairs (2i, 2i+1); 1: pairs (i, i + d_rot/2)
    int inverse;                 // rotate by minus the angle (the gradient)
};

// cos and sin (times mscale) of a pair with frequency frac at position pos.
__device__ __forceinline__ float2 rope_cs(uint64_t frac, float mscale, int inverse, int pos) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * frac;
    // signed fraction of a turn in [-1/2, 1/2), rounded once to fp32; the angle is pi * (2 * fraction)
    const float h = __ll2float_rn(static_cast<int64_t>(turns)) * 0x1p-63f;
    float s, c;
    sincospif(h, &s, &c);
    s *= mscale;
    return make_float2(c * mscale, inverse ? -s : s);
}

// Two E4M3 codes (low byte first) times the row's power-of-two scale, as packed
// bf16: exact (3 mantissa bits) in the normal range; below it too for a row that
// was bf16 (its values are multiples of 2^-133, bf16's smallest step, and rounding
// to fewer bits leaves them so).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes16, float scale) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(codes16)));
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h2));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

// Two E4M3 codes as packed bf16, unscaled (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes16) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(codes16)));
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h2));
    return pack_bf16x2(f.x, f.y);
}

// One packed sequence: query rows [q0, q0 + lq), key rows [k0, k0 + lk).
struct PackedSeq {
    int q0, lq, k0, lk;
};

// Whole warp: the sequence and the tile inside it of row tile `tile` (tiles of
// `rows` rows; by_key: of the key rows, else of the query rows), sequences in
// order.  Returns the tile's index in its sequence, or -1 past the last tile.
// Inconsistent offsets (decreasing, or outside [0, Tq] / [0, Tk]) record an
// error and count as an empty sequence.
__device__ __forceinline__ int find_tile(const int32_t* cu_q, const int32_t* cu_k, int B, int Tq, int Tk, int rows,
                                         bool by_key, int tile, int* err, PackedSeq* out) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        PackedSeq s{0, 0, 0, 0};
        if (b < B) {
            const int qa = __ldg(cu_q + b), qb = __ldg(cu_q + b + 1), ka = __ldg(cu_k + b), kb = __ldg(cu_k + b + 1);
            if (qa < 0 || qb < qa || qb > Tq || ka < 0 || kb < ka || kb > Tk)
                set_dev_error(err, DEV_ERR_OFFSETS);
            else
                s = PackedSeq{qa, qb - qa, ka, kb - ka};
        }
        const int n = ((by_key ? s.lk : s.lq) + rows - 1) / rows;
        int end = n;                                         // inclusive prefix sum over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end += v;
        }
        end += before;
        const unsigned past = __ballot_sync(0xffffffffu, end > tile);
        if (past) {
            const int l = __ffs(past) - 1;
            out->q0 = __shfl_sync(0xffffffffu, s.q0, l);
            out->lq = __shfl_sync(0xffffffffu, s.lq, l);
            out->k0 = __shfl_sync(0xffffffffu, s.k0, l);
            out->lk = __shfl_sync(0xffffffffu, s.lk, l);
            return tile - __shfl_sync(0xffffffffu, end - n, l);
        }
        before = __shfl_sync(0xffffffffu, end, 31);
    }
    return -1;
}

// mbar_wait (common.cuh) with its loop out of line.  These kernels run six or more different loops at once on an
// SM, each with several waits: inlined, the loops outgrow the instruction caches (no-instruction stalls were a
// quarter of all warp cycles).
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                set_dev_error(err, DEV_ERR_TIMEOUT);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, err);
}
// For loads in flight at a block's end: bounded, without regard to the abort flag.
static __device__ __noinline__ void drain_bar(uint64_t* bar, uint32_t parity, int* err) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(bar), parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(err, DEV_ERR_TIMEOUT); break; }
}

// wait_bar by a whole warp with one answer for all its lanes: what follows a
// failed wait must not split a warp that goes on to warp-wide operations.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, err));
}

// 2^x (x <= 0 here up to rounding): one hardware operation, relative error about 2^-22.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace fs
