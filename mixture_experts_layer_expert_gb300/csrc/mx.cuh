// mx.cuh -- block-scaled (MX) operand layouts of the MX expert paths: 8-bit E4M3
// and 4-bit E2M1 codes.
//
// Every operand row of an expert GEMM is cut, along the contraction, into
// blocks of 32 elements; each block is E4M3 codes times its own power-of-two
// scale 2^e (e the smallest integer with max |x_i| 2^-e <= 448, clamped to the
// UE8M0 range [-127, 127]), stored as the UE8M0 byte e + 127.  The tensor
// cores apply both operands' block scales inside the contraction
// (tcgen05.mma kind::mxf8f6f4.block_scale, scale factors in TMEM).
//
// Scale-factor bytes are kept in the arrangement the scale-factor copy into
// TMEM (tcgen05.cp 32x128b.warpx4) takes: for a group of 128 rows and one
// 128-element stage of the contraction (4 blocks), a 512-byte chunk whose byte
// (m % 32) * 16 + (m / 32) * 4 + b holds row m's scale of block b.
//   MX matrix [rows, cols] (activations): codes [rows128][cols] row-major
//     (rows128 = rows rounded up to 128), then from a 256-byte boundary the
//     chunks [rows128 / 128][cols / 128][512].
//   MX weights [G, N, K]: codes tiled as the FP8 weights
//     [G][ceil(N/256)][K/128][256][128], then the chunks
//     [G][ceil(N/256)][K/128][2][512] (the two 128-row halves of a 256-row tile).
//
// 4-bit form: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit), two in a
// byte, the even element in the low nibble; e the smallest integer with
// max |x_i| 2^-e <= 6 (bf16 magnitudes give e <= 126: every 2^-e is a normal
// fp32 number).  E2M1 has no NaN and no infinity, so a block that holds one gets
// the scale byte 255 (UE8M0's NaN) and its products are NaN.
//   MX matrix: codes [rows128][cols / 2 bytes], chunks as above.
//   MX weights: codes tiled [G][ceil(N/256)][ceil(K/256)][256][128 bytes] (256
//     elements of K a tile row; past K zero), chunks as above.
#pragma once

#include "fp8.cuh"

namespace fs {

constexpr int kMxBlock = 32;

__host__ __device__ inline long long mx_rows128(long long rows) { return (rows + 127) / 128 * 128; }
// Bytes of a row's codes.
__host__ __device__ inline int mx_row_bytes(bool f4, int cols) { return f4 ? cols / 2 : cols; }
__host__ __device__ inline size_t mx_sf_offset(bool f4, long long rows, int cols) {
    return (static_cast<size_t>(mx_rows128(rows)) * static_cast<size_t>(mx_row_bytes(f4, cols)) + 255) / 256 * 256;
}
__host__ __device__ inline size_t mx_rows_bytes(bool f4, long long rows, int cols) {
    return mx_sf_offset(f4, rows, cols) + static_cast<size_t>(mx_rows128(rows) / 128) * (cols / 128) * 512;
}
// Byte of row m's scale of block b (32 elements) in an MX matrix's chunks.
__host__ __device__ inline size_t mx_sf_byte(long long m, int b, int cols) {
    return (static_cast<size_t>(m >> 7) * (cols >> 7) + (b >> 2)) * 512 + (m & 31) * 16 + ((m & 127) >> 5) * 4 +
           (b & 3);
}
// Weights: tile nt of group g, row r of the 256-row tile, block b along K.
__host__ __device__ inline size_t mx_w_sf_byte(long long g, int NB, int nt, int r, int b, int K) {
    return ((static_cast<size_t>(g) * NB + nt) * (K >> 7) + (b >> 2)) * 1024 + (r >> 7) * 512 + (r & 31) * 16 +
           ((r & 127) >> 5) * 4 + (b & 3);
}
inline size_t mx_w_codes_bytes(bool f4, int G, int N, int K) {
    const size_t tiles = static_cast<size_t>(G) * ((static_cast<size_t>(N) + 255) / 256);
    return f4 ? tiles * 256 * 128 * ((static_cast<size_t>(K) + 255) / 256) : tiles * 256 * K;
}
inline size_t mx_w_bytes(bool f4, int G, int N, int K) {
    return mx_w_codes_bytes(f4, G, N, K) + static_cast<size_t>(G) * ((static_cast<size_t>(N) + 255) / 256) * (K / 128) * 1024;
}

// Quantisation of one block from its largest magnitude: the UE8M0 byte and the
// multiplier 2^-e (fp32 normal unless `wide`, then applied in double).
struct MxQuant {
    RowQuant q;
    uint8_t ue8m0;
};
__device__ __forceinline__ MxQuant mx_quant(float amax) {
    int e = fp8_row_exp(amax);
    e = e < -127 ? -127 : (e > 127 ? 127 : e);
    MxQuant m;
    m.q.e = e;
    m.q.wide = (e < -127 || e > 126);
    m.q.mult = m.q.wide ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    m.q.scale = 0.0f;   // not used: the scale travels as the UE8M0 byte
    m.ue8m0 = static_cast<uint8_t>(e + 127);
    return m;
}

// 4-bit block: the multiplier 2^-e and the scale byte from the fp32 bits of its
// largest magnitude (compared as integers, so that a NaN is the largest).
struct Mx4Quant {
    float mult;
    uint8_t ue8m0;
};
__device__ __forceinline__ Mx4Quant mx4_scale(uint32_t amax_bits) {
    Mx4Quant m;
    int e = static_cast<int>(amax_bits >> 23) - 127 - ((amax_bits & 0x7FFFFFu) <= 0x400000u ? 2 : 1);   // 6 = 1.5 * 2^2
    if (e < -127) e = -127;                    // subnormal and smallest normal magnitudes
    if (amax_bits == 0) e = 0;
    const bool finite = amax_bits < 0x7F800000u;
    m.mult = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
    m.ue8m0 = finite ? static_cast<uint8_t>(e + 127) : 255;
    return m;
}
// E2M1 codes of 8 values, element 0 in the lowest nibble (nearest, ties to even).
__device__ __forceinline__ uint32_t cvt_e2m1x8(float a0, float a1, float a2, float a3, float a4, float a5, float a6,
                                               float a7) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a0), "f"(a1), "f"(a2), "f"(a3), "f"(a4), "f"(a5), "f"(a6), "f"(a7));
    return r;
}
// Largest magnitude of the bf16 pairs, as fp32 bits.
template <int N>
__device__ __forceinline__ uint32_t absmax_bits(const uint32_t (&w)[N]) {
    uint32_t top = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < N; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    return max(top << 16, top & 0xFFFF0000u);
}
// Codes of 8 bf16 values.
__device__ __forceinline__ uint32_t mx4_codes8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float mult) {
    return cvt_e2m1x8(bf16lo(w0) * mult, bf16hi(w0) * mult, bf16lo(w1) * mult, bf16hi(w1) * mult, bf16lo(w2) * mult,
                      bf16hi(w2) * mult, bf16lo(w3) * mult, bf16hi(w3) * mult);
}

// Largest magnitude over the 4-lane group holding one 32-element block (lanes
// 4q .. 4q+3 of the warp, 8 elements each).
__device__ __forceinline__ float group4_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    return v;
}

__device__ __forceinline__ uint32_t group4_max(uint32_t v) {
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 2));
    return v;
}

// The codes of a lane's 8 elements and its block's scale byte; the 4 lanes of a
// block call it together.
template <bool F4>
struct MxLane;
template <>
struct MxLane<false> {
    using Codes = uint2;
    static __device__ __forceinline__ Codes zero() { return make_uint2(0, 0); }
    static __device__ __forceinline__ Codes quant(const uint4& a, uint8_t* byte) {
        const MxQuant m = mx_quant(group4_max(absmax_bf16x8(a)));
        *byte = m.ue8m0;
        return quant_bf16x8(a, m.q);
    }
};
template <>
struct MxLane<true> {
    using Codes = uint32_t;
    static __device__ __forceinline__ Codes zero() { return 0; }
    static __device__ __forceinline__ Codes quant(const uint4& a, uint8_t* byte) {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        const Mx4Quant m = mx4_scale(group4_max(absmax_bits(w)));
        *byte = m.ue8m0;
        return mx4_codes8(w[0], w[1], w[2], w[3], m.mult);
    }
};

}  // namespace fs
