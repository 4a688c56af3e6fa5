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

// cos and sin (times mscale) of pair i at position pos.
__device__ __forceinline__ float2 rope_cs(const RopeTab& tab, int i, int pos) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * tab.frac[i];
    // signed fraction of a turn in [-1/2, 1/2), rounded once to fp32; the angle is pi * (2 * fraction)
    const float h = __ll2float_rn(static_cast<int64_t>(turns)) * 0x1p-63f;
    float s, c;
    sincospif(h, &s, &c);
    s *= tab.mscale;
    return make_float2(c * tab.mscale, tab.inverse ? -s : s);
}

// Two E4M3 codes (low byte first) times the row's power-of-two scale, as packed
// bf16: exact (3 mantissa bits) while the products stay normal bf16 numbers.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes16, float scale) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(codes16)));
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h2));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

}  // namespace fs
