// gemm_mx.cu -- persistent grouped GEMM on block-scaled operands (the MX expert
// paths): E4M3 codes with tcgen05.mma kind::mxf8f6f4.block_scale, or E2M1 codes
// (4 bits) with kind::mxf4.block_scale, in shared memory (TMA, 128-byte swizzle)
// and one UE8M0 scale per row per 32 elements of K for each operand, the scales
// copied into TMEM with tcgen05.cp (layouts in mx.cuh).  fp32 accumulate in TMEM.
//
// The grouped structure, warp roles, tile order and bounded waits are those of
// gemm_tc.cu (one CTA per SM, 10 warps: TMA producer, MMA issuer, 8 epilogue
// warps), with two differences forced by the scales:
//  * TMEM holds one 128 x 256 fp32 accumulator (256 columns) plus a ring of
//    scale-factor slots; two accumulators would fill all 512 columns.  So the
//    epilogue warps first copy their whole share of the accumulator into
//    registers (128 columns each), release TMEM, and only then compute and
//    store: the next tile's MMAs wait for that copy only.
//  * every group's rows start at a multiple of 128 (the MX Dispatch pads each
//    expert's segment), so an A tile's scales are one 512-byte chunk per stage.
// One stage = 128 bytes of K: A 128 x 128 B + B 256 x 128 B of codes.
//   E4M3: 128 elements, one chunk of scales (512 B of A, 1 KB of B); 4 MMAs of
//         128 x 256 x 32, MMA kk using byte kk of each scale word.
//   E2M1: 256 elements, two chunks; 4 MMAs of 128 x 256 x 64, MMA kk using bytes
//         2 (kk & 1) and + 1 of chunk kk / 2.  K is a multiple of 128, so a row's
//         last stage may be half full: it has one chunk and two MMAs (the codes
//         behind it are zeros of the weight tile or of the TMA load's fill).
//
// Measured, E2M1 and few rows (many run in gemm_mx_pair.cu): 61 tokens x 6 over 64 experts, d = 2,048, c = 1,408, gate/up
// 36 us and down 22, 4.7 TB/s of weights: HBM behind the latency of the first stages and the epilogue.
//
// Epilogues: EPI_SWIGLU writes the hidden h = SiLU(g) u rounded to bf16 and
// quantised in blocks of 32 straight into an MX matrix (codes and scales: the
// down projection's A operand); EPI_BF16 writes y (bf16); EPI_F32 writes fp32.
#include <cudaTypedefs.h>
#include <cstring>

#include "gemm_mx.cuh"

namespace fs {
namespace mx {

constexpr int BM = 128;
constexpr int BK = 128;                       // bytes of K per stage
constexpr int A_STAGE = BM * BK;              // 16 KB
constexpr int SFA_CHUNK = 512;                // scales of 128 rows x 4 blocks
constexpr int BAR_BYTES = 256;
constexpr int TMEM_COLS = 512;

// What differs between the two element formats and the tile widths.  BN = 64 (E2M1, one group) is for
// products with too few tiles of 256 columns for the SMs: four times the blocks stream the weights.
template <bool F4, int BN>
struct Fmt {
    static constexpr int STAGES = BN == 256 ? 4 : 8;
    static constexpr int B_STAGE = BN * BK;                   // 32 KB (8 KB)
    static constexpr int STAGE_BYTES = A_STAGE + B_STAGE;
    static constexpr int CHUNKS = F4 ? 2 : 1;                 // scale chunks (128 elements) per stage
    // groups of the plan (E2M1: its second chunk takes the room of half of them)
    static constexpr int MAX_GROUPS = BN < 256 ? 1 : (F4 ? kMaxExperts : kMaxGroups);
    static constexpr int SFB_CHUNK = BN == 256 ? 1024 : 512;  // of 256 rows x 4 blocks (128 rows: a tile of 64 is half of one)
    static constexpr int SFA_BYTES = CHUNKS * SFA_CHUNK;
    static constexpr int SF_STAGE = CHUNKS * (SFA_CHUNK + SFB_CHUNK);
    static constexpr int SFB_COLS = SFB_CHUNK / 128;          // TMEM columns of a chunk of B
    static constexpr int SF_COLS = CHUNKS * (4 + SFB_COLS);   // per slot: A's columns, then B's
    static constexpr int SF_SLOTS = 2 * STAGES;               // scale-factor slots in TMEM, a ring
    static constexpr int SF_COL0 = BN;                        // behind the accumulator
    static constexpr int SF_OFF = STAGES * STAGE_BYTES;       // shared memory: scale chunks after the code stages
    static constexpr int BAR_OFF = SF_OFF + STAGES * SF_STAGE;
    static constexpr int PLAN_OFF = BAR_OFF + BAR_BYTES;
    static constexpr int PIECE_OFF = (PLAN_OFF + 2 * (MAX_GROUPS + 1) * 4 + 1023) / 1024 * 1024;
    static constexpr size_t SMEM_BYTES = 1024 + PIECE_OFF + EPI_WARPS * PIECE_BYTES;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(SF_COL0 + SF_COLS * SF_SLOTS <= TMEM_COLS, "TMEM columns");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// TMEM <- shared memory scale chunk: 32 rows of 16 bytes, each row i copied to
// lane i of every lane quarter, 4 columns (tcgen05.cp 32x128b.warpx4).  The
// source descriptor: start >> 4, no swizzle, 8-row core groups 128 B apart.
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t saddr) {
    uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    desc |= static_cast<uint64_t>(128u >> 4) << 16;
    desc |= static_cast<uint64_t>(128u >> 4) << 32;
    desc |= 1ull << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D (fp32, TMEM) (+)= (A * sA) (B * sB)^T, E4M3 or E2M1 codes with UE8M0 block scales.
template <bool F4>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
    if constexpr (F4)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

template <int EPI, bool F4, int BN>
__global__ void __launch_bounds__(THREADS, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmO, const Args args) {
    using F = Fmt<F4, BN>;
    constexpr int STAGES = F::STAGES, STAGE_BYTES = F::STAGE_BYTES, SFB_CHUNK = F::SFB_CHUNK, SFB_COLS = F::SFB_COLS;
    constexpr int HALF = BN / 2;                // columns of an epilogue warp
    static_assert(BN == 256 || EPI != EPI_SWIGLU, "the hidden's blocks need gate and up in one warp's columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::BAR_OFF);
    uint64_t* full = bars;                 // [STAGES]
    uint64_t* empty = bars + STAGES;       // [STAGES]
    uint64_t* tfull = bars + 2 * STAGES;   // [1]
    uint64_t* tempty = tfull + 1;          // [1]
    uint64_t* fin = tempty + 1;            // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* mt_start = reinterpret_cast<int*>(smem + F::PLAN_OFF);
    int* row_start = mt_start + (args.G + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = args.G;

    if constexpr (F4) cudaGridDependencySynchronize();
    if constexpr (F4) {
        make_plan<BM>(args, mt_start, row_start);
    } else {
        for (int i = threadIdx.x; i < 2 * (G + 1); i += THREADS) mt_start[i] = args.plan[i];
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), EPI_WARPS);
        mbar_init(smem_u32(fin), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    int total_mtiles = mt_start[G];
    if (total_mtiles < 0 || total_mtiles > args.max_mtiles) {
        if (threadIdx.x == 0) set_dev_error(args.err, DEV_ERR_OFFSETS);
        total_mtiles = 0;
    }
    const int total = total_mtiles * args.n_tiles;
    const int chunks = args.K / 128;                              // scale chunks along K
    const int num_kb = (chunks + F::CHUNKS - 1) / F::CHUNKS;      // stages
    constexpr int SUB = 256 / BN;                                 // tiles per 256-row block of the packed weights
    const int tiles256 = (args.n_tiles + SUB - 1) / SUB;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile tl = decode<BM>(t, mt_start, row_start, G, args.n_tiles);
                const uint8_t* sfa = args.a_sf + static_cast<size_t>(tl.a_row / BM) * chunks * SFA_CHUNK;
                const uint8_t* sfb = args.b_sf + (static_cast<size_t>(tl.g) * tiles256 + tl.n / SUB) * chunks * 1024 +
                                     (BN == 256 ? 0 : (tl.n % SUB) / 2 * 512);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.err)) { ok = false; break; }
                    const uint32_t fb = smem_u32(&full[stage]);
                    const int nc = min(F::CHUNKS, chunks - kb * F::CHUNKS);
                    mbar_arrive_expect_tx(fb, STAGE_BYTES + nc * (SFA_CHUNK + SFB_CHUNK));
                    uint8_t* sa = smem + stage * STAGE_BYTES;
                    uint8_t* sf = smem + F::SF_OFF + stage * F::SF_STAGE;
                    tma_load_2d(smem_u32(sa), &tmA, fb, kb * BK, tl.a_row);
                    tma_load_3d(smem_u32(sa + A_STAGE), &tmB, fb, 0, tl.n % SUB * BN, (tl.g * tiles256 + tl.n / SUB) * num_kb + kb);
                    bulk_load(smem_u32(sf), sfa + static_cast<size_t>(kb) * F::SFA_BYTES, nc * SFA_CHUNK, fb);
                    if constexpr (BN == 256) {
                        bulk_load(smem_u32(sf + F::SFA_BYTES), sfb + static_cast<size_t>(kb) * F::CHUNKS * 1024, nc * 1024, fb);
                    } else {
                        for (int q = 0; q < nc; ++q)
                            bulk_load(smem_u32(sf + F::SFA_BYTES + q * 512), sfb + (static_cast<size_t>(kb) * F::CHUNKS + q) * 1024,
                                      512, fb);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            const int pending = issued < STAGES ? issued : STAGES;
            for (int j = 1; j <= pending; ++j) {
                int s = stage - j;
                uint32_t ph = phase;
                if (s < 0) { s += STAGES; ph ^= 1u; }
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(smem_u32(&full[s]), ph)) {
                    if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMA
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int it = 0;
            uint32_t slot = 0;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++it) {
                const Tile tl = decode<BM>(t, mt_start, row_start, G, args.n_tiles);
                // the epilogue has copied the previous tile out of TMEM
                if (!mbar_wait(smem_u32(tempty), (static_cast<uint32_t>(it) & 1u) ^ 1u, abort_flag, args.err)) break;
                tc_fence_after();
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, args.err)) { ok = false; break; }
                    tc_fence_after();
                    uint8_t* sa = smem + stage * STAGE_BYTES;
                    const uint32_t sf = smem_u32(smem + F::SF_OFF + stage * F::SF_STAGE);
                    // chunk q: A's columns at tsa + 4 q, B's behind them (rows 0..127, then 128..255)
                    const uint32_t tsa = tmem_base + F::SF_COL0 + static_cast<uint32_t>(F::SF_COLS) * slot;
                    const uint32_t tsb = tsa + 4u * F::CHUNKS;
                    const uint64_t adesc = smem_desc_sw128(smem_u32(sa));
                    const uint64_t bdesc = smem_desc_sw128(smem_u32(sa + A_STAGE));
#pragma unroll
                    for (int q = 0; q < F::CHUNKS; ++q) {
                        if (q > 0 && kb * F::CHUNKS + q >= chunks) break;
                        sf_copy(tsa + 4u * q, sf + q * SFA_CHUNK);
                        const uint32_t tb = tsb + static_cast<uint32_t>(SFB_COLS) * q;
                        sf_copy(tb, sf + F::SFA_BYTES + q * SFB_CHUNK);
                        if constexpr (BN == 256) sf_copy(tb + 4u, sf + F::SFA_BYTES + q * SFB_CHUNK + 512u);
                        constexpr int MMAS = 4 / F::CHUNKS;
#pragma unroll
                        for (int j = 0; j < MMAS; ++j) {
                            const int kk = q * MMAS + j;
                            mma_mx<F4>(tmem_base, adesc + 2ull * kk, bdesc + 2ull * kk, idesc_mx<F4>(BM, BN, j * F::CHUNKS),
                                       tsa + 4u * q, tb + (BN == 256 ? 0u : 2u * (tl.n & 1)), (kb > 0 || kk > 0) ? 1u : 0u);
                        }
                    }
                    tc_commit(smem_u32(&empty[stage]));
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    slot = (slot + 1u) % F::SF_SLOTS;
                }
                if (!ok) break;
                tc_commit(smem_u32(tfull));
            }
            tc_commit(smem_u32(fin));
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(fin), 0)) {
                if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;          // which 128 columns of the tile
        const int r = quarter * 32 + lane;
        uint8_t* piece = smem + F::PIECE_OFF + (warp - 2) * PIECE_BYTES;
        int it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
            const Tile tl = decode<BM>(t, mt_start, row_start, G, args.n_tiles);
            if (!mbar_wait(smem_u32(tfull), static_cast<uint32_t>(it) & 1u, abort_flag, args.err)) break;
            tc_fence_after();
            // this warp's 32 rows and half of the columns, copied out of TMEM at once
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * HALF);
            uint32_t v[HALF];
#pragma unroll
            for (int c = 0; c < HALF; c += 32) tmem_ld32_sync(tb + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(tempty));
            epilogue<EPI, F4, HALF>(v, args, &tmO, tl.n, half, tl.a_row, tl.rows_valid, r, piece);
        }
        if (args.tma_out && lane == 0) bulk_wait0();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace mx

// ------------------------------------------------------------------- host
cudaError_t encode_map(CUtensorMap* m, CUtensorMapDataType type, int rank, void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle,
                       CUtensorMapL2promotion promotion) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = fn(m, type, rank, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace mx {
// The output map of a launch whose epilogue stores pieces by TMA: 32 x 32 of bf16, 32 x 16 of fp32.
cudaError_t out_map(CUtensorMap* m, int epi, void* out, long long rows, int cols, long long ldo, int* tma_out) {
    *tma_out = 0;
    const int es = epi == EPI_F32 ? 4 : 2;
    if ((epi != EPI_BF16 && epi != EPI_F32) || ldo * es % 16 || (reinterpret_cast<uintptr_t>(out) & 15u)) return cudaSuccess;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldo) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / es), 32};
    *tma_out = 1;
    return encode_map(m, epi == EPI_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims,
                      strides, box, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}
}  // namespace mx

template <int EPI, bool F4, int BN = 256>
static cudaError_t launch_mx_impl(const void* A, long long a_rows, const uint8_t* a_sf, const void* B,
                                  const uint8_t* b_sf, int G, int N, int K, const int* plan, const int* offsets, int rows, int max_mtiles, void* out,
                                  long long ldo, int out_cols, uint8_t* h_sf, cudaStream_t st) {
    static bool set_mx[kMaxDevices];
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(mx::mx_gemm_kernel<EPI, F4, BN>), mx::Fmt<F4, BN>::SMEM_BYTES, set_mx);
    if (e != cudaSuccess) return e;
    if (K % 128 || N % (F4 ? 8 : 128) || a_rows % 128 || G < 1 || G > mx::Fmt<F4, BN>::MAX_GROUPS) return cudaErrorInvalidValue;
    const int row_bytes = F4 ? K / 2 : K;
    const int stages = (row_bytes + mx::BK - 1) / mx::BK;      // the last one of a 4-bit row may be half full
    CUtensorMap ta, tb, to;
    e = make_map(&ta, A, a_rows, row_bytes, 128, true);
    if (e != cudaSuccess) return e;
    const int n_tiles = (N + BN - 1) / BN;
    e = make_map_blocked(&tb, B, static_cast<long long>(G) * ((N + 255) / 256) * stages, BN, true);
    if (e != cudaSuccess) return e;
    mx::Args args;
    args.plan = plan;
    args.offsets = offsets;
    args.G = G;
    args.rows = rows;
    args.N = N;
    args.K = K;
    args.n_tiles = n_tiles;
    args.max_mtiles = max_mtiles;
    args.a_sf = a_sf;
    args.b_sf = b_sf;
    args.out = out;
    args.ldo = ldo;
    args.out_cols = out_cols;
    args.h_sf = h_sf;
    args.err = dev_error_ptr();
    args.tma_out = 0;
    to = ta;
    if (F4) {
        e = mx::out_map(&to, EPI, out, offsets ? a_rows : rows, out_cols, ldo, &args.tma_out);
        if (e != cudaSuccess) return e;
    } else if (EPI == EPI_BF16 && out_cols % 32 == 0 && ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
        e = make_out_map_bf16(&to, out, a_rows, out_cols, ldo);
        if (e != cudaSuccess) return e;
        args.tma_out = 1;
    }
    if (EPI == EPI_SWIGLU && (!h_sf || ldo < (F4 ? out_cols / 2 : out_cols))) return cudaErrorInvalidValue;
    int sms = 0;
    e = num_sms(&sms);
    if (e != cudaSuccess) return e;
    const long long max_tiles = static_cast<long long>(max_mtiles) * n_tiles;
    int grid = static_cast<int>(max_tiles < sms ? max_tiles : sms);
    if (grid < 1) grid = 1;
    count_launch();
    if (F4)         // set up while the kernel before it drains; it waits for that one's end before it reads
        return launch_after(mx::mx_gemm_kernel<EPI, F4, BN>, dim3(grid), dim3(mx::THREADS), mx::Fmt<F4, BN>::SMEM_BYTES, st,
                            ta, tb, to, args);
    mx::mx_gemm_kernel<EPI, F4, BN><<<grid, mx::THREADS, mx::Fmt<F4, BN>::SMEM_BYTES, st>>>(ta, tb, to, args);
    return cudaGetLastError();
}

template <bool F4>
static cudaError_t launch_mx_fmt(int epi, const void* A, long long a_rows, const uint8_t* a_sf, const void* B,
                                 const uint8_t* b_sf, int G, int N, int K, const int* plan, const int* offsets, int rows, int max_mtiles,
                                 void* out, long long ldo, int out_cols, uint8_t* h_sf, cudaStream_t st) {
    if constexpr (F4) {
        // one group whose tiles of 256 columns would leave half of the SMs idle
        int sms = 0;
        const cudaError_t e = num_sms(&sms);
        if (e != cudaSuccess) return e;
        if (!offsets && 2LL * max_mtiles * ((N + 255) / 256) <= sms) {
            if (epi == EPI_BF16)
                return launch_mx_impl<EPI_BF16, F4, 64>(A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo,
                                                        out_cols, h_sf, st);
            if (epi == EPI_F32)
                return launch_mx_impl<EPI_F32, F4, 64>(A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo,
                                                       out_cols, h_sf, st);
        }
    }
    switch (epi) {
        case EPI_SWIGLU:
            return launch_mx_impl<EPI_SWIGLU, F4>(A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo,
                                                  out_cols, h_sf, st);
        case EPI_BF16:
            return launch_mx_impl<EPI_BF16, F4>(A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo,
                                                out_cols, h_sf, st);
        case EPI_F32:
            return launch_mx_impl<EPI_F32, F4>(A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo,
                                               out_cols, h_sf, st);
        default:
            return cudaErrorInvalidValue;
    }
}

cudaError_t launch_mx_gemm(bool f4, int epi, const void* A, long long a_rows, const uint8_t* a_sf, const void* B,
                           const uint8_t* b_sf, int G, int N, int K, const int* plan, const int* offsets, int rows,
                           int max_mtiles, void* out, long long ldo, int out_cols, uint8_t* h_sf, cudaStream_t st) {
    return f4 ? launch_mx_fmt<true>(epi, A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo, out_cols,
                                    h_sf, st)
              : launch_mx_fmt<false>(epi, A, a_rows, a_sf, B, b_sf, G, N, K, plan, offsets, rows, max_mtiles, out, ldo, out_cols,
                                     h_sf, st);
}

}  // namespace fs
