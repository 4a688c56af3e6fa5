// latent_cache.cu -- writing token rows into the paged latent cache (bf16, or
// quantised to FP8 with one power-of-two scale per token; the rotary key rotated
// on the way) and reading records back as bf16 rows.
//
// Memory bound: 1,152 bytes of bf16 rows on one side, a record (1,152 or 656
// bytes) on the other.  A warp takes a token at a time: each lane holds 16
// consecutive latent elements, so the row maximum is one warp reduction, 16 codes
// leave as one 16-byte store, and nothing is read twice; the 32 lanes carry the 32
// rotated pairs, one sine and cosine each.  A lane's frequency stays in a register
// over the warp's tokens (a lane-dependent read of the parameter bank is 32 reads).
// Measured, 65,533 tokens, FP8: written in 27.2 us (4.4 TB/s; 40.5 with eight lanes
// rotating four pairs each), read in 21.4 us (5.5 TB/s).  A writing warp asks for its next
// two tokens only when these are stored, so its loads stand still meanwhile.
#include "kernels.h"
#include "latent.cuh"

namespace fs {

template <bool FP8>
__global__ void __launch_bounds__(256)
cache_write_kernel(const __grid_constant__ RopeTab tab, long long T, const __nv_bfloat16* __restrict__ c,
                   long long c_row, const __nv_bfloat16* __restrict__ kr, long long kr_row,
                   const int32_t* __restrict__ pos, const int64_t* __restrict__ slots, uint8_t* __restrict__ cache,
                   long long n_slots, int* err) {
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * 8;
    const uint64_t frac = pos ? tab.frac[lane] : 0;
    const bool half = pos && tab.half;               // lane's pair: elements lane, lane + 32, else 2 lane, 2 lane + 1
    for (long long t0 = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t0 < T; t0 += 2 * step) {
        // two tokens' loads in flight, which do not wait for their slots
        long long slot[2];
        uint4 v0[2], v1[2];
        uint32_t w[2];
        int p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long t = t0 + i * step < T ? t0 + i * step : t0;
            slot[i] = __ldg(slots + t);
            const uint4* src = reinterpret_cast<const uint4*>(c + t * c_row) + 2 * lane;
            v0[i] = __ldg(src);
            v1[i] = __ldg(src + 1);
            const uint16_t* k = reinterpret_cast<const uint16_t*>(kr + t * kr_row);
            w[i] = half ? __ldg(k + lane) | static_cast<uint32_t>(__ldg(k + lane + 32)) << 16
                        : __ldg(reinterpret_cast<const uint32_t*>(k) + lane);
            p[i] = pos ? __ldg(pos + t) : 0;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i && t0 + step >= T) break;
            if (slot[i] < 0) continue;               // a padding row: nothing is written
            if (slot[i] >= n_slots) {
                if (lane == 0) set_dev_error(err, DEV_ERR_PAGE);
                continue;
            }
            uint8_t* rec = cache + slot[i] * (FP8 ? kRecFp8 : kRecBf16);
            if (pos) {
                const float2 cs = rope_cs(frac, tab.mscale, tab.inverse, p[i]);
                const float a = bf16lo(w[i]), b = bf16hi(w[i]);
                w[i] = pack_bf16x2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
            }
            uint8_t* rope = rec + (FP8 ? kFp8RopeOff : 2 * kLatent);
            if (half) {
                reinterpret_cast<uint16_t*>(rope)[lane] = static_cast<uint16_t>(w[i]);
                reinterpret_cast<uint16_t*>(rope)[lane + 32] = static_cast<uint16_t>(w[i] >> 16);
            } else {
                reinterpret_cast<uint32_t*>(rope)[lane] = w[i];
            }
            if constexpr (FP8) {
                const RowQuant q = row_quant(warp_max(fmaxf(absmax_bf16x8(v0[i]), absmax_bf16x8(v1[i]))));
                const uint2 a = quant_bf16x8(v0[i], q), b = quant_bf16x8(v1[i], q);
                reinterpret_cast<uint4*>(rec)[lane] = make_uint4(a.x, a.y, b.x, b.y);
                if (lane == 8) *reinterpret_cast<uint4*>(rec + kFp8ScaleOff) = make_uint4(__float_as_uint(q.scale), 0, 0, 0);
            } else {
                reinterpret_cast<uint4*>(rec)[2 * lane] = v0[i];
                reinterpret_cast<uint4*>(rec)[2 * lane + 1] = v1[i];
            }
        }
    }
}

template <bool FP8>
__global__ void __launch_bounds__(256)
cache_read_kernel(long long T, const int64_t* __restrict__ slots, const uint8_t* __restrict__ cache,
                  long long n_slots, __nv_bfloat16* __restrict__ c, long long c_row, __nv_bfloat16* __restrict__ kr,
                  long long kr_row, int* err) {
    const int lane = threadIdx.x & 31;
    const long long t = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (t >= T) return;
    const long long slot = __ldg(slots + t);
    if (slot < 0) return;                        // a padding row: left as it was
    if (slot >= n_slots) {
        if (lane == 0) set_dev_error(err, DEV_ERR_PAGE);
        return;
    }
    const uint8_t* rec = cache + slot * (FP8 ? kRecFp8 : kRecBf16);
    uint4 o0, o1;
    if constexpr (FP8) {
        const uint4 w = *(reinterpret_cast<const uint4*>(rec) + lane);
        const float s = *reinterpret_cast<const float*>(rec + kFp8ScaleOff);
        o0 = make_uint4(e4m3x2_to_bf16x2(w.x & 0xffffu, s), e4m3x2_to_bf16x2(w.x >> 16, s),
                        e4m3x2_to_bf16x2(w.y & 0xffffu, s), e4m3x2_to_bf16x2(w.y >> 16, s));
        o1 = make_uint4(e4m3x2_to_bf16x2(w.z & 0xffffu, s), e4m3x2_to_bf16x2(w.z >> 16, s),
                        e4m3x2_to_bf16x2(w.w & 0xffffu, s), e4m3x2_to_bf16x2(w.w >> 16, s));
    } else {
        o0 = reinterpret_cast<const uint4*>(rec)[2 * lane];
        o1 = reinterpret_cast<const uint4*>(rec)[2 * lane + 1];
    }
    uint4* dst = reinterpret_cast<uint4*>(c + t * c_row) + 2 * lane;
    dst[0] = o0;
    dst[1] = o1;
    if (lane < 8)
        *reinterpret_cast<uint4*>(kr + t * kr_row + 8 * lane) =
            *reinterpret_cast<const uint4*>(rec + (FP8 ? kFp8RopeOff : 2 * kLatent) + 16 * lane);
}

// Blocks of the write, each warp taking every 4,864th pair of tokens: three or four an SM 51.4 us for the FP8 write and
// read of 65,533 tokens, six 55.2, eight 53.2 (one token in flight a warp, six blocks: 53.3).
constexpr long long kWriteBlocks = 152 * 4;

cudaError_t launch_cache_write(const RopeTab* tab, bool fp8, long long T, const void* c, long long c_row,
                               const void* kr, long long kr_row, const int32_t* pos, const int64_t* slots, void* cache,
                               long long n_slots, cudaStream_t st) {
    static const RopeTab none{};
    const RopeTab& rt = tab ? *tab : none;
    const int32_t* p = tab ? pos : nullptr;
    const unsigned blocks = static_cast<unsigned>(min((T + 7) / 8, kWriteBlocks));
    auto* cc = static_cast<const __nv_bfloat16*>(c);
    auto* kk = static_cast<const __nv_bfloat16*>(kr);
    auto* out = static_cast<uint8_t*>(cache);
    int* err = dev_error_ptr();
    if (fp8)
        cache_write_kernel<true><<<blocks, 256, 0, st>>>(rt, T, cc, c_row, kk, kr_row, p, slots, out, n_slots, err);
    else
        cache_write_kernel<false><<<blocks, 256, 0, st>>>(rt, T, cc, c_row, kk, kr_row, p, slots, out, n_slots, err);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_read(bool fp8, long long T, const int64_t* slots, const void* cache, long long n_slots,
                              void* c, long long c_row, void* kr, long long kr_row, cudaStream_t st) {
    const unsigned blocks = static_cast<unsigned>((T + 7) / 8);
    auto* in = static_cast<const uint8_t*>(cache);
    auto* cc = static_cast<__nv_bfloat16*>(c);
    auto* kk = static_cast<__nv_bfloat16*>(kr);
    int* err = dev_error_ptr();
    if (fp8)
        cache_read_kernel<true><<<blocks, 256, 0, st>>>(T, slots, in, n_slots, cc, c_row, kk, kr_row, err);
    else
        cache_read_kernel<false><<<blocks, 256, 0, st>>>(T, slots, in, n_slots, cc, c_row, kk, kr_row, err);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fs
