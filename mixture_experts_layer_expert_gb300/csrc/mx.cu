// mx.cu -- quantisation kernels of the block-scaled (MX) expert paths, E4M3 or (F4) E2M1:
// bf16 rows to an MX matrix (the shared experts' token rows), the quantising
// Dispatch copy (each token row quantised once, its codes and block scales
// written to all of its k permuted rows), and the one-time packing of bf16
// expert weights into MX codes and scale chunks (layouts in mx.cuh).
//
// In every kernel a warp walks a row 8 elements (one 16-byte vector) per lane
// and step, so the 4 lanes 4q .. 4q+3 of a step hold one 32-element block:
// its largest magnitude is a 4-lane shuffle maximum, and lane 4q writes the
// block's scale byte.  The steps are counted for the whole warp (a row of
// 16-byte vectors that is not a multiple of 32 leaves lanes idle in its last
// step, they still take part in the shuffles).
#include "kernels.h"
#include "mx.cuh"

namespace fs {

// One warp per row r < rows128 (grid-stride): x [rows, cols] bf16 -> q, an MX
// matrix; rows past `rows` get zero codes and unit scales.
__global__ void __launch_bounds__(256)
quant_rows_mx_kernel(const uint4* __restrict__ x, long long rows, int cols, uint8_t* __restrict__ q) {
    const int lane = threadIdx.x & 31;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    const int nv = cols / 8;
    uint8_t* sf = q + mx_sf_offset(false, rows, cols);
    const long long r128 = mx_rows128(rows);
    for (long long r = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < r128; r += nwarps) {
        uint2* dst = reinterpret_cast<uint2*>(q + r * cols);
        for (int v0 = 0; v0 < nv; v0 += 32) {
            const int v = v0 + lane;
            const bool act = v < nv;
            if (r < rows) {
                const uint4 a = act ? __ldg(x + r * nv + v) : make_uint4(0, 0, 0, 0);
                uint8_t byte;
                const uint2 c = MxLane<false>::quant(a, &byte);
                if (act) {
                    dst[v] = c;
                    if ((lane & 3) == 0) sf[mx_sf_byte(r, v / 4, cols)] = byte;
                }
            } else if (act) {
                dst[v] = make_uint2(0, 0);
                if ((lane & 3) == 0) sf[mx_sf_byte(r, v / 4, cols)] = 127;
            }
        }
    }
}

// One warp per token: u[t] quantised in 32-element blocks once; its codes and
// scale bytes go to every slot's row pos[t, s] of x_q (an MX matrix of
// rows_cap rows) and, when u_q is set, to row t of u_q (an MX matrix [T, d]).
__global__ void __launch_bounds__(256)
dispatch_copy_mx_kernel(const uint4* __restrict__ u, int T, int d, int k, const int32_t* __restrict__ pos,
                        uint8_t* __restrict__ x_q, long long rows_cap, uint8_t* __restrict__ u_q) {
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
    if (t >= T) return;
    const int nv = d / 8;
    const int my_p = lane < k ? pos[static_cast<long long>(t) * k + lane] : -1;
    uint8_t* xsf = x_q + mx_sf_offset(false, rows_cap, d);
    uint8_t* usf = u_q ? u_q + mx_sf_offset(false, T, d) : nullptr;
    const uint4* src = u + static_cast<long long>(t) * nv;
    for (int v0 = 0; v0 < nv; v0 += 32) {
        const int v = v0 + lane;
        const bool act = v < nv;
        const uint4 a = act ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
        uint8_t byte;
        const uint2 c = MxLane<false>::quant(a, &byte);
        const bool lead = (lane & 3) == 0;
        for (int s = 0; s < k; ++s) {
            const int p = __shfl_sync(0xffffffffu, my_p, s);
            if (p < 0 || !act) continue;
            reinterpret_cast<uint2*>(x_q + static_cast<long long>(p) * d)[v] = c;
            if (lead) xsf[mx_sf_byte(p, v / 4, d)] = byte;
        }
        if (u_q && act) {
            reinterpret_cast<uint2*>(u_q + static_cast<long long>(t) * d)[v] = c;
            if (lead) usf[mx_sf_byte(t, v / 4, d)] = byte;
        }
    }
}

// ---- 4-bit codes.  A lane holds 16 elements, half a block: 8 bytes of codes, so that a
// warp's store of 512 elements is 256 consecutive bytes, and the four scale bytes of a chunk's
// row (8 lanes) leave as one word.  Two such steps are in flight.  A row is shared by gridDim.y
// warps of `per` steps each where there are fewer rows than warps that fill the SMs.

// The codes of a lane's 16 elements; *word: in lanes 0, 8, 16, 24 the four scale bytes of the 8 lanes.
__device__ __forceinline__ uint2 mx4_lane16(const uint4& a, const uint4& b, uint32_t* word) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t top = absmax_bits(w);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const Mx4Quant m = mx4_scale(top);
    uint32_t s = m.ue8m0;
    s |= __shfl_down_sync(0xffffffffu, s, 2) << 8;
    s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
    *word = s;
    return make_uint2(mx4_codes8(w[0], w[1], w[2], w[3], m.mult), mx4_codes8(w[4], w[5], w[6], w[7], m.mult));
}

// x [rows, cols] -> q.  Zero rows behind them have zero codes and unit scales by themselves.  Bound by HBM: 16,381 x 7,168
// 45 us, 6.7 TB/s of rows in and codes out.
__global__ void __launch_bounds__(256)
quant_rows_mx4_kernel(const uint4* x, long long rows, int cols, int per, uint8_t* q) {
    const int lane = threadIdx.x & 31;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    const int n16 = cols / 16;
    const int first = blockIdx.y * per * 32, last = min(n16, first + per * 32);
    uint8_t* sf = q + mx_sf_offset(true, rows, cols);
    const long long r128 = mx_rows128(rows);
    cudaGridDependencySynchronize();
    for (long long r = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < r128; r += nwarps) {
        const uint4* src = x + r * 2 * n16;
        uint2* dst = reinterpret_cast<uint2*>(q + r * (cols / 2));
        for (int v0 = first; v0 < last; v0 += 64) {
            uint4 a[2], b[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int v = v0 + 32 * s + lane;
                const bool act = r < rows && v < last;
                a[s] = act ? src[2 * v] : make_uint4(0, 0, 0, 0);
                b[s] = act ? src[2 * v + 1] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int v = v0 + 32 * s + lane;
                if (v0 + 32 * s >= last) break;
                uint32_t word;
                const uint2 c = mx4_lane16(a[s], b[s], &word);
                if (v < last) {
                    dst[v] = c;
                    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(sf + mx_sf_byte(r, v / 2, cols)) = word;
                }
            }
        }
    }
}

// As dispatch_copy_mx_kernel.  8,192 x 7,168 to 8 rows each 74 us: HBM, 120 MB of rows in and 250 MB of codes out.
__global__ void __launch_bounds__(256)
dispatch_copy_mx4_kernel(const uint4* u, int T, int d, int k, const int32_t* pos, int per, uint8_t* x_q,
                         long long rows_cap, uint8_t* u_q) {
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
    if (t >= T) return;
    cudaGridDependencySynchronize();
    const int n16 = d / 16, rb = d / 2;
    const int first = blockIdx.y * per * 32, last = min(n16, first + per * 32);
    const int my_p = lane < k ? pos[static_cast<long long>(t) * k + lane] : -1;
    uint8_t* xsf = x_q + mx_sf_offset(true, rows_cap, d);
    uint8_t* usf = u_q ? u_q + mx_sf_offset(true, T, d) : nullptr;
    const uint4* src = u + static_cast<long long>(t) * 2 * n16;
    const bool lead = (lane & 7) == 0;
    for (int v0 = first; v0 < last; v0 += 64) {
        uint2 c[2];
        uint32_t word[2];
        uint4 a[2], b[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int v = v0 + 32 * s + lane;
            a[s] = v < last ? src[2 * v] : make_uint4(0, 0, 0, 0);
            b[s] = v < last ? src[2 * v + 1] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) c[s] = mx4_lane16(a[s], b[s], &word[s]);
        for (int slot = 0; slot <= k; ++slot) {              // the last one: u_q's row
            const bool own = slot == k;
            if (own && !u_q) break;
            const int p = own ? t : __shfl_sync(0xffffffffu, my_p, slot);
            if (p < 0) continue;
            uint2* dst = reinterpret_cast<uint2*>((own ? u_q : x_q) + static_cast<long long>(p) * rb);
            uint8_t* sf = own ? usf : xsf;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int v = v0 + 32 * s + lane;
                if (v < last) {
                    dst[v] = c[s];
                    if (lead) *reinterpret_cast<uint32_t*>(sf + mx_sf_byte(p, v / 2, d)) = word[s];
                }
            }
        }
    }
}

// One warp per packed row (grid-stride over G * NB * 256 rows): codes into the
// tiled layout, scale bytes into the tile's chunks; rows past N: zero codes,
// unit scales.  (E2M1 with K not a multiple of 256: the walk goes on to the end
// of the last tile and fills it with zero codes.)
template <bool F4>
__global__ void __launch_bounds__(256)
pack_mx_kernel(PackSrc src, int G, int NB, uint8_t* __restrict__ codes, uint8_t* __restrict__ sf) {
    const int lane = threadIdx.x & 31;
    using Codes = typename MxLane<F4>::Codes;
    constexpr int TILE_K = F4 ? 256 : 128;                 // elements of a tile's 128-byte rows
    const int K = src.K, N = src.N, KB = (K + TILE_K - 1) / TILE_K, nv = K / 8, nv_tiles = KB * (TILE_K / 8);
    const long long total = static_cast<long long>(G) * NB * 256;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    for (long long R = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; R < total; R += nwarps) {
        const long long g = R / (static_cast<long long>(NB) * 256);
        const int nr = static_cast<int>(R - g * NB * 256);
        const int nb = nr >> 8, rr = nr & 255;
        uint8_t* blk0 = codes + ((g * NB + nb) * KB) * 32768LL + rr * 128;
        for (int v0 = 0; v0 < nv_tiles; v0 += 32) {
            const int v = v0 + lane;
            const bool act = v < nv;
            const int kb = v * static_cast<int>(sizeof(Codes));        // byte along K
            Codes c = MxLane<F4>::zero();
            uint8_t byte = 127;
            if (nr < N) {
                const uint4 a = act ? __ldg(src.chunk(g, nr, v)) : make_uint4(0, 0, 0, 0);
                c = MxLane<F4>::quant(a, &byte);
            }
            if (v < nv_tiles) {
                *reinterpret_cast<Codes*>(blk0 + (kb >> 7) * 32768LL + (kb & 127)) = c;
                if (act && (lane & 3) == 0) sf[mx_w_sf_byte(g, NB, nb, rr, v / 4, K)] = byte;
            }
        }
    }
}

static int mx_grid(long long warps_needed) {
    long long blocks = (warps_needed + 7) / 8;
    const long long cap = 152LL * 16;
    if (blocks > cap) blocks = cap;
    return static_cast<int>(blocks < 1 ? 1 : blocks);
}

size_t packed_bytes_mx(bool f4, int G, int N, int K) { return mx_w_bytes(f4, G, N, K); }

const uint8_t* packed_sf_mx(bool f4, const void* packed, int G, int N, int K) {
    return static_cast<const uint8_t*>(packed) + mx_w_codes_bytes(f4, G, N, K);
}

static cudaError_t launch_pack_mx(bool f4, const PackSrc& src, int G, void* out, cudaStream_t st) {
    const int NB = (src.N + 255) / 256;
    uint8_t* codes = static_cast<uint8_t*>(out);
    uint8_t* sf = codes + mx_w_codes_bytes(f4, G, src.N, src.K);
    const int grid = mx_grid(static_cast<long long>(G) * NB * 256);
    if (f4) pack_mx_kernel<true><<<grid, 256, 0, st>>>(src, G, NB, codes, sf);
    else pack_mx_kernel<false><<<grid, 256, 0, st>>>(src, G, NB, codes, sf);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_pack_w13_mx(bool f4, int G, int c, int d, const void* w1, const void* w2, void* w13, cudaStream_t st) {
    PackSrc s{static_cast<const uint4*>(w1), static_cast<const uint4*>(w2), 0, 2 * c, d, c, 0};
    return launch_pack_mx(f4, s, G, w13, st);
}

cudaError_t launch_pack_w3_mx(bool f4, int G, int d, int c, const void* w3, void* w3p, cudaStream_t st) {
    PackSrc s{static_cast<const uint4*>(w3), nullptr, 1, d, c, 0, 0};
    return launch_pack_mx(f4, s, G, w3p, st);
}

cudaError_t launch_pack_w3_shared_mx(bool f4, int ns, int cs, int d, const void* w3s, void* w3cat, cudaStream_t st) {
    PackSrc s{static_cast<const uint4*>(w3s), nullptr, 2, d, ns * cs, 0, cs};
    return launch_pack_mx(f4, s, 1, w3cat, st);
}

// Steps of 512 elements that a warp takes of a row, so that `rows` rows give 152 x 16 warps where they can.
static int mx4_steps(long long rows, int cols) {
    const int steps = (cols + 511) / 512;
    long long split = 152LL * 16 / rows;
    split = split < 1 ? 1 : (split > steps ? steps : split);
    return static_cast<int>((steps + split - 1) / split);
}

cudaError_t launch_quant_rows_mx(bool f4, const void* x, long long rows, int cols, void* q, cudaStream_t st) {
    const long long r128 = mx_rows128(rows);
    const uint4* src = static_cast<const uint4*>(x);
    uint8_t* dst = static_cast<uint8_t*>(q);
    count_launch();
    if (f4) {
        const int per = mx4_steps(r128, cols);
        return launch_after(quant_rows_mx4_kernel, dim3(mx_grid(r128), ((cols + 511) / 512 + per - 1) / per), dim3(256), 0, st,
                            src, rows, cols, per, dst);
    }
    quant_rows_mx_kernel<<<mx_grid(r128), 256, 0, st>>>(src, rows, cols, dst);
    return cudaGetLastError();
}

cudaError_t launch_dispatch_copy_mx(bool f4, const void* u, int T, int d, int k, const int32_t* pos, void* x_q,
                                    long long rows_cap, void* u_q, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) + 7) / 8);
    const uint4* src = static_cast<const uint4*>(u);
    uint8_t *xq = static_cast<uint8_t*>(x_q), *uq = static_cast<uint8_t*>(u_q);
    count_launch();
    if (f4) {
        const int per = mx4_steps(T, d);
        return launch_after(dispatch_copy_mx4_kernel, dim3(grid, ((d + 511) / 512 + per - 1) / per), dim3(256), 0, st, src, T, d,
                            k, pos, per, xq, rows_cap, uq);
    }
    dispatch_copy_mx_kernel<<<grid, 256, 0, st>>>(src, T, d, k, pos, xq, rows_cap, uq);
    return cudaGetLastError();
}

}  // namespace fs
