// balance.cu -- the router's balance loss with per-expert token counts, and its
// gradient with respect to the router logits.
//
// Per sequence q of n counted tokens (its rows of the batch with mask != 0):
//   s_te  softmax(z_t + b) for the softmax gates, sigma(z_te + b_e) / sum_j sigma(z_tj + b_j)
//         for the sigmoid gates
//   c_e   tokens' slots that chose e,  f_e = E c_e / (k n),  P_e = mean_t s_te
//   loss  = coef / S sum_q sum_e f_e P_e
//   dz_te = g coef / (S n) s_te (f_e - sum_j f_j s_tj), times (1 - sigma_te) for the sigmoid gates (computed from f - 1)
// The counts carry no gradient.
//
// Both directions read every logit once and are bound by HBM; the work per logit is
// one exponential (two and a reciprocal for the sigmoids).  A warp owns a token: its
// row sits in registers (E <= 512: 16 a lane), the next two or four rows on their way, max and sums by
// shuffles.  Up to 1,024 rows of one sequence are one block's work, in one launch.  Otherwise,
// forward: the token axis is cut into equal ranges, one per block, whatever
// the sequences' lengths; what a block finds of a sequence goes to slot (block + sequence)
// of the workspace, which no other pair has because both only grow along the axis.  A second
// kernel adds a sequence's slots in order.  No float atomics: results repeat bit for bit.
// Measured: 65,536 x 256, sigmoids, forward 20 us + 7.5 (3.5 TB/s of logits and indices: a block an SM with 96 KB of rows in
// flight, and the ramps at both ends), backward 21 us (6.4 TB/s); 256 x 8 4 us each, latency.
#include "common.cuh"
#include "kernels.h"

namespace fs {
namespace bal {

// Warps of a block and tokens a warp has in flight, by elements a lane: one block fills an SM.
template <int EPL>
struct Cfg {
    static constexpr int WARPS = EPL == 16 ? 12 : 24;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int U = EPL == 4 ? 4 : 2;              // (more spill, and are slower)
};
constexpr int FIN_E = 32;                 // experts per block of the second kernel
constexpr int FIN_P = 32;                 // slots it reads at a time
constexpr int ONE_ROWS = 1024;            // at most this many rows of one sequence in one block

struct Args {
    const float* z;
    long long z_row;
    const float* bias;
    const int32_t* idx;
    const uint8_t* mask;
    const int32_t* cu;                    // null: one sequence of all rows
    int T, E, k, S, chunk, blocks;
    float coef;
    int* bad;                             // [blocks] a block's share of the borders is inconsistent
    float* part;                          // [slots][E] sums of scores
    int32_t* part_c;                      // [slots][E] counts
    int32_t* part_n;                      // [slots] counted tokens
    float* loss_part;                     // [S][expert blocks]
    unsigned* done;                       // blocks of the second kernel that have finished
    int32_t* counts;
    int32_t* tokens;
    float* probs;
    float* loss;
    int* err;
};

// Lane's element j of a row: vectors of 4 along the row, or one element per lane and step.
template <bool VEC>
__device__ __forceinline__ int elem(int j, int lane) {
    return VEC ? 128 * (j >> 2) + 4 * lane + (j & 3) : 32 * j + lane;
}

template <int EPL, bool VEC>
__device__ __forceinline__ void load_row(const float* p, int E, int lane, float pad, float (&v)[EPL]) {
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
            const int e = elem<VEC>(j, lane);
            float4 x = make_float4(pad, pad, pad, pad);
            if (e < E) x = *reinterpret_cast<const float4*>(p + e);
            v[j] = x.x; v[j + 1] = x.y; v[j + 2] = x.z; v[j + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = elem<VEC>(j, lane);
            v[j] = e < E ? p[e] : pad;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_top(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float recip(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Logits -> scores times *inv.  rest (sigmoids): 1 - sigma.  A row of -infinity scores zero.  Sigmoids
// of a row whose logits all lie below -60 are exponentials to fp32, and their ratios a softmax's.
template <int EPL, bool SIG>
__device__ __forceinline__ void scores(float (&v)[EPL], float (&rest)[EPL], float* inv) {
    float top = v[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, v[j]);
    float sum = 0.0f;
    if (SIG && __any_sync(0xffffffffu, top > -60.0f)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float u = __expf(-v[j]);
            v[j] = recip(1.0f + u);
            rest[j] = u == INFINITY ? 1.0f : u * v[j];
            sum += v[j];
        }
    } else {
        top = warp_top(top);
        const float m = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            v[j] = __expf(v[j] - m);
            rest[j] = 1.0f;
            sum += v[j];
        }
    }
    sum = warp_sum(sum);
    *inv = sum == 0.0f ? 0.0f : 1.0f / sum;
}

// First sequence that may hold row t or a later one: the last q with cu[q] <= t (0 if none).
__device__ __forceinline__ int first_seq(const int32_t* cu, int S, int t) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// A sequence's results from its sums: P, f P summed over the calling threads' experts (loss term not yet scaled).
__device__ __forceinline__ float finish(const Args& a, int q, int e, float sum, int c, int n) {
    const float p = n > 0 ? sum / static_cast<float>(n) : 0.0f;
    const long long at = static_cast<long long>(q) * a.E + e;
    a.probs[at] = p;
    a.counts[at] = c;
    return n > 0 ? static_cast<float>(a.E) * static_cast<float>(c) / (static_cast<float>(a.k) * static_cast<float>(n)) * p
                 : 0.0f;
}

// ONE: a single block over one sequence, which finishes it too.
template <int EPL, bool VEC, bool SIG, bool ONE>
__global__ void __launch_bounds__(Cfg<EPL>::THREADS, 1)
piece_kernel(const Args a) {
    constexpr int WARPS = Cfg<EPL>::WARPS, THREADS = Cfg<EPL>::THREADS, U = Cfg<EPL>::U;
    __shared__ float sums[WARPS][32 * EPL];
    __shared__ int cnt[32 * EPL];
    __shared__ int ntok;
    __shared__ float terms[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x * a.chunk, c1 = a.T - c0 < a.chunk ? a.T : c0 + a.chunk;     // no sum past an int
    cudaGridDependencySynchronize();
    if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    bool bad = false;
    if (!ONE && a.cu)
        for (int i = blockIdx.x * THREADS + threadIdx.x; i <= a.S; i += gridDim.x * THREADS) {
            const int at = a.cu[i];
            bad |= at < 0 || at > a.T || (i < a.S && a.cu[i + 1] < at);
        }
    float bias[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = elem<VEC>(j, lane);
        bias[j] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    for (int q = a.cu ? first_seq(a.cu, a.S, c0) : 0; q < a.S; ++q) {
        const int q0 = a.cu ? a.cu[q] : 0, q1 = a.cu ? a.cu[q + 1] : a.T;
        if (!ONE && q0 >= c1) break;
        int lo = max(q0, c0), hi = min(q1, c1);
        if (ONE && (q0 < 0 || q1 < q0 || q1 > a.T)) {
            if (threadIdx.x == 0) set_dev_error(a.err, DEV_ERR_OFFSETS);
            lo = hi = 0;
        }
        if (!ONE && lo >= hi) continue;
        for (int e = threadIdx.x; e < a.E; e += THREADS) cnt[e] = 0;
        if (threadIdx.x == 0) ntok = 0;
        __syncthreads();
        float acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
        int n = 0;
        float v[U][EPL];
        bool on[U];
        int pick[U];
        auto fetch = [&](int u, int t) {           // a token's row on its way while others are worked on
            on[u] = t < hi && !(a.mask && a.mask[t] == 0);
            if (!on[u]) return;
            pick[u] = lane < a.k ? a.idx[static_cast<long long>(t) * a.k + lane] : -1;
            load_row<EPL, VEC>(a.z + t * a.z_row, a.E, lane, -INFINITY, v[u]);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u, lo + warp + u * WARPS);
        for (int t0 = lo + warp; t0 < hi; t0 += U * WARPS) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool now = on[u];
                const int e = pick[u];
                float w[EPL], rest[EPL], inv;
#pragma unroll
                for (int j = 0; j < EPL; ++j) w[j] = v[u][j] + bias[j];
                fetch(u, t0 + (u + U) * WARPS);
                if (!now) continue;
                ++n;
                if (lane < a.k) {
                    if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
                    else set_dev_error(a.err, DEV_ERR_EXPERT_INDEX);
                }
                scores<EPL, SIG>(w, rest, &inv);
#pragma unroll
                for (int j = 0; j < EPL; ++j) acc[j] += w[j] * inv;
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) sums[warp][elem<VEC>(j, lane)] = acc[j];
        if (lane == 0) atomicAdd(&ntok, n);
        __syncthreads();
        if constexpr (ONE) {
            float term = 0.0f;
            for (int e = threadIdx.x; e < a.E; e += THREADS) {
                float s = sums[0][e];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) s += sums[w][e];
                term += finish(a, 0, e, s, cnt[e], ntok);
            }
            term = warp_sum(term);
            if (lane == 0) terms[warp] = term;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < WARPS; ++w) term += terms[w];
                a.tokens[0] = ntok;
                *a.loss = a.coef * term;
            }
            return;
        }
        const long long slot = static_cast<long long>(blockIdx.x) + q;
        for (int e = threadIdx.x; e < a.E; e += THREADS) {
            float s = sums[0][e];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) s += sums[w][e];
            a.part[slot * a.E + e] = s;
            a.part_c[slot * a.E + e] = cnt[e];
        }
        if (threadIdx.x == 0) a.part_n[slot] = ntok;
        __syncthreads();
    }
    if (!ONE && a.cu) {
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) a.bad[blockIdx.x] = bad;
    }
}

// Block (expert block, sequence): the sequence's slots added in order, its counts, mean scores
// and share of the loss; the block that finishes last adds the shares.  Where any border is inconsistent sequences may
// share rows, and slots that no block filled be read: then every sequence counts as empty.
__global__ void __launch_bounds__(FIN_E * FIN_P)
finish_kernel(const Args a) {
    __shared__ float s_sum[FIN_P][FIN_E + 1];
    __shared__ int s_cnt[FIN_P][FIN_E + 1];
    __shared__ int s_n[FIN_P];
    __shared__ bool last;
    const int x = threadIdx.x % FIN_E, y = threadIdx.x / FIN_E;
    const int e = blockIdx.x * FIN_E + x, q = blockIdx.y;
    cudaGridDependencySynchronize();
    bool bad = a.cu && threadIdx.x < a.blocks && a.bad[threadIdx.x];
    int q0 = a.cu ? a.cu[q] : 0, q1 = a.cu ? a.cu[q + 1] : a.T;
    if (q0 < 0 || q1 < q0 || q1 > a.T) q0 = q1 = 0;
    const int b0 = q0 / a.chunk, b1 = q1 > q0 ? (q1 - 1) / a.chunk + 1 : b0;
    float sum = 0.0f;
    int cnt = 0, n = 0;
#pragma unroll 4
    for (int b = b0 + y; b < b1; b += FIN_P) {
        const long long slot = static_cast<long long>(b) + q;
        if (e < a.E) {
            sum += a.part[slot * a.E + e];
            cnt += a.part_c[slot * a.E + e];
        }
        if (x == 0) n += a.part_n[slot];
    }
    s_sum[y][x] = sum;
    s_cnt[y][x] = cnt;
    if (x == 0) s_n[y] = n;
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) set_dev_error(a.err, DEV_ERR_OFFSETS);
    if (y == 0) {
        n = 0;
        sum = 0.0f;
        cnt = 0;
#pragma unroll
        for (int p = 0; p < FIN_P; ++p) {
            n += s_n[p];
            sum += s_sum[p][x];
            cnt += s_cnt[p][x];
        }
        if (bad) {
            n = cnt = 0;
            sum = 0.0f;
        }
        float term = e < a.E ? finish(a, q, e, sum, cnt, n) : 0.0f;
        term = warp_sum(term);
        if (x == 0) {
            if (blockIdx.x == 0) a.tokens[q] = n;
            a.loss_part[static_cast<long long>(q) * gridDim.x + blockIdx.x] = term;
            __threadfence();
            last = atomicAdd(a.done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    const long long parts = static_cast<long long>(gridDim.x) * gridDim.y;
    float s = 0.0f;
    for (long long i = threadIdx.x; i < parts; i += FIN_E * FIN_P) s += __ldcg(a.loss_part + i);
    s = warp_sum(s);
    if (x == 0) s_sum[0][y] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0f;
        for (int p = 0; p < FIN_P; ++p) s += s_sum[0][p];
        *a.loss = a.coef * s / static_cast<float>(a.S);
    }
}

struct BwdArgs {
    const float* z;
    long long z_row;
    const float* bias;
    const uint8_t* mask;
    const int32_t* cu;
    const int32_t* counts;
    const int32_t* tokens;
    const float* d_loss;
    float* dz;
    long long dz_row;
    int T, E, k, S, chunk;
    float coef;
    int* err;
};

template <int EPL, bool VEC>
__device__ __forceinline__ void store_row(float* p, int E, int lane, const float (&v)[EPL]) {
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
            const int e = elem<VEC>(j, lane);
            if (e < E) *reinterpret_cast<float4*>(p + e) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = elem<VEC>(j, lane);
            if (e < E) p[e] = v[j];
        }
    }
}

template <int EPL, bool VEC, bool SIG>
__global__ void __launch_bounds__(Cfg<EPL>::THREADS, 1)
backward_kernel(const BwdArgs a) {
    constexpr int WARPS = Cfg<EPL>::WARPS, U = Cfg<EPL>::U;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x * a.chunk, c1 = a.T - c0 < a.chunk ? a.T : c0 + a.chunk;     // no sum past an int
    cudaGridDependencySynchronize();
    const float g = (a.d_loss ? *a.d_loss : 1.0f) * a.coef / static_cast<float>(a.S);
    float bias[EPL], f[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = elem<VEC>(j, lane);
        bias[j] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    for (int q = a.cu ? first_seq(a.cu, a.S, c0) : 0; q < a.S; ++q) {
        const int q0 = a.cu ? a.cu[q] : 0, q1 = a.cu ? a.cu[q + 1] : a.T;
        if (q0 >= c1) break;
        const int lo = max(q0, c0), hi = min(q1, c1);
        if (lo + warp >= hi) continue;
        if (q0 < 0 || q1 > a.T) {              // (the forward reports all inconsistent borders, and counts no tokens then)
            set_dev_error(a.err, DEV_ERR_OFFSETS);
            continue;
        }
        const int n = a.tokens[q];
        const float per = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
        // f - 1 instead of f: the scores' sum is one, so the gradient is the same, and it is exactly zero where all f are equal
        const float unit = per / static_cast<float>(a.k), scale = g * per;
        const long long even = static_cast<long long>(a.k) * n;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = elem<VEC>(j, lane);
            f[j] = e < a.E ? unit * static_cast<float>(static_cast<long long>(a.counts[static_cast<long long>(q) * a.E + e]) * a.E - even)
                           : 0.0f;
        }
        float v[U][EPL];
        bool on[U];
        auto fetch = [&](int u, int t) {
            on[u] = t < hi && !(a.mask && a.mask[t] == 0);
            if (on[u]) load_row<EPL, VEC>(a.z + t * a.z_row, a.E, lane, -INFINITY, v[u]);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u, lo + warp + u * WARPS);
        for (int t0 = lo + warp; t0 < hi; t0 += U * WARPS) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * WARPS;
                const bool now = on[u];
                float w[EPL], rest[EPL];
#pragma unroll
                for (int j = 0; j < EPL; ++j) w[j] = v[u][j] + bias[j];
                fetch(u, t + U * WARPS);
                if (t >= hi) break;
                if (now) {
                    float inv, dot = 0.0f;
                    scores<EPL, SIG>(w, rest, &inv);
#pragma unroll
                    for (int j = 0; j < EPL; ++j) dot += f[j] * w[j];
                    dot = warp_sum(dot) * inv;
                    const float by = scale * inv;
#pragma unroll
                    for (int j = 0; j < EPL; ++j) {
                        w[j] *= by * (f[j] - dot);
                        if constexpr (SIG) w[j] *= rest[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < EPL; ++j) w[j] = 0.0f;
                }
                store_row<EPL, VEC>(a.dz + t * a.dz_row, a.E, lane, w);
            }
        }
    }
}

// Rows a block takes: one block on each SM.
int chunk_rows(int T) {
    const long long c = (static_cast<long long>(T) + 151) / 152;
    return static_cast<int>((c + 7) / 8 * 8);
}
int blocks(int T) { return (T - 1) / chunk_rows(T) + 1; }       // no sum past an int
int expert_blocks(int E) { return (E + FIN_E - 1) / FIN_E; }

struct Layout {
    size_t part, part_c, part_n, loss_part, done, bad, end;
};
Layout layout(int T, int E, int S) {
    const size_t slots = static_cast<size_t>(blocks(T)) + S;
    Layout l;
    size_t o = 0;
    auto take = [&](size_t n) { const size_t at = o; o = (o + n + 255) / 256 * 256; return at; };
    l.part = take(slots * E * 4);
    l.part_c = take(slots * E * 4);
    l.part_n = take(slots * 4);
    l.loss_part = take(static_cast<size_t>(S) * expert_blocks(E) * 4);
    l.done = take(4);
    l.bad = take(static_cast<size_t>(blocks(T)) * 4);
    l.end = o;
    return l;
}

bool vec_ok(const void* p, long long row, int E) {
    return E % 4 == 0 && row % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

}  // namespace bal

size_t balance_ws_bytes(int T, int E, int S) { return bal::layout(T, E, S).end; }

// KERNEL<elements a lane, TAIL...> for E experts, launched while what comes before it on the stream drains (each
// waits for that before it reads).
#define FS_BALANCE(KERNEL, E, GRID, ARGS, ...)                                                                          \
    (E) <= 128 ? launch_after(KERNEL<4, __VA_ARGS__>, dim3(GRID), dim3(bal::Cfg<4>::THREADS), 0, st, ARGS)               \
    : (E) <= 256 ? launch_after(KERNEL<8, __VA_ARGS__>, dim3(GRID), dim3(bal::Cfg<8>::THREADS), 0, st, ARGS)             \
                 : launch_after(KERNEL<16, __VA_ARGS__>, dim3(GRID), dim3(bal::Cfg<16>::THREADS), 0, st, ARGS)

template <bool SIG>
static cudaError_t balance_fwd(const bal::Args& a, cudaStream_t st) {
    const bool vec = bal::vec_ok(a.z, a.z_row, a.E);
    count_launch();
    if (a.S == 1 && a.T <= bal::ONE_ROWS)
        return vec ? (FS_BALANCE(bal::piece_kernel, a.E, 1, a, true, SIG, true))
                   : (FS_BALANCE(bal::piece_kernel, a.E, 1, a, false, SIG, true));
    const cudaError_t e = vec ? (FS_BALANCE(bal::piece_kernel, a.E, bal::blocks(a.T), a, true, SIG, false))
                              : (FS_BALANCE(bal::piece_kernel, a.E, bal::blocks(a.T), a, false, SIG, false));
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_after(bal::finish_kernel, dim3(bal::expert_blocks(a.E), a.S), dim3(bal::FIN_E * bal::FIN_P), 0, st, a);
}

template <bool SIG>
static cudaError_t balance_bwd(const bal::BwdArgs& a, cudaStream_t st) {
    const bool vec = bal::vec_ok(a.z, a.z_row, a.E) && bal::vec_ok(a.dz, a.dz_row, a.E);
    count_launch();
    return vec ? (FS_BALANCE(bal::backward_kernel, a.E, bal::blocks(a.T), a, true, SIG))
               : (FS_BALANCE(bal::backward_kernel, a.E, bal::blocks(a.T), a, false, SIG));
}

cudaError_t launch_balance(const BalanceArgs& b, void* ws, cudaStream_t st) {
    const bal::Layout l = bal::layout(b.T, b.E, b.S);
    uint8_t* w = static_cast<uint8_t*>(ws);
    bal::Args a;
    a.z = b.z; a.z_row = b.z_row; a.bias = b.bias; a.idx = b.idx; a.mask = b.mask; a.cu = b.cu;
    a.T = b.T; a.E = b.E; a.k = b.k; a.S = b.S;
    a.chunk = b.S == 1 && b.T <= bal::ONE_ROWS ? bal::ONE_ROWS : bal::chunk_rows(b.T);
    a.coef = b.coef;
    a.part = reinterpret_cast<float*>(w + l.part);
    a.part_c = reinterpret_cast<int32_t*>(w + l.part_c);
    a.part_n = reinterpret_cast<int32_t*>(w + l.part_n);
    a.loss_part = reinterpret_cast<float*>(w + l.loss_part);
    a.done = reinterpret_cast<unsigned*>(w + l.done);
    a.bad = reinterpret_cast<int*>(w + l.bad);
    a.blocks = bal::blocks(b.T);
    a.counts = b.counts; a.tokens = b.tokens; a.probs = b.probs; a.loss = b.loss;
    a.err = dev_error_ptr();
    return b.sigmoid ? balance_fwd<true>(a, st) : balance_fwd<false>(a, st);
}

cudaError_t launch_balance_backward(const BalanceArgs& b, const float* d_loss, float* dz, long long dz_row,
                                    cudaStream_t st) {
    bal::BwdArgs a;
    a.z = b.z; a.z_row = b.z_row; a.bias = b.bias; a.mask = b.mask; a.cu = b.cu;
    a.counts = b.counts; a.tokens = b.tokens; a.d_loss = d_loss; a.dz = dz; a.dz_row = dz_row;
    a.T = b.T; a.E = b.E; a.k = b.k; a.S = b.S; a.chunk = bal::chunk_rows(b.T); a.coef = b.coef;
    a.err = dev_error_ptr();
    return b.sigmoid ? balance_bwd<true>(a, st) : balance_bwd<false>(a, st);
}

}  // namespace fs
