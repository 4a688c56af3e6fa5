// gemm_mx_pair.cu -- the 4-bit grouped GEMM of gemm_mx.cu on CTA pairs: 256 x 256 tiles,
// tcgen05.mma cta_group::2 kind::mxf4 issued by the even CTA.
//
// The single-CTA kernel moves 51 KB of codes and scales into shared memory per 128 x 256 x 256
// stage, and at E2M1's rate that is what bounds it: a stage took 980 cycles where its MMAs take 512.
// A pair's CTA loads its own 128 rows of A and half of B's, 35 KB a stage, which leaves the
// MMAs and the output in front.  Each CTA's TMEM holds its 128 rows of the accumulator, the scales
// of its A rows and those of all 256 B rows: the scale copies are 2-CTA copies, each CTA's
// from its own shared memory.
//   full[s]  (even CTA)  both CTAs' loads complete on it;  empty[s] (each)  the pair's MMAs have read stage s
//   tfull    (each)      the tile is complete;             tempty (even)    16 warps have copied it out
// The scales come by tensor maps of 512-byte and 1 KB rows: those carry an mbarrier of the other CTA
// and fill with zeros past the end (an odd number of chunks, a pair's second half past the last row).
// Measured: 65,536 rows of 32 experts, gate/up (K = 7,168) 521 us, 7.4 PFLOP/s; down (K = 2,048) 370 us, 5.2;
// 16,381 x 2,048 of K = 7,168 76 us, 6.3.  What bounds it: L2 to shared memory, 18 TB/s in the gate/up product (a stage's
// 35 KB take 560 cycles at 64 bytes a cycle), and some 3,000 cycles between two tiles, in which the
// accumulator is copied out and handed back (there is no room in TMEM for a second one beside the scales).
#include "gemm_mx.cuh"

namespace fs {
namespace mx {
namespace pair {

constexpr int BM = 256;
constexpr int BN = 256;
constexpr int BK = 128;                        // bytes of K per stage: 256 elements
constexpr int STAGES = 5;
constexpr int A_STAGE = 128 * BK;              // this CTA's rows of A
constexpr int B_STAGE = 128 * BK;              // its half of B's
constexpr int SFA_BYTES = 2 * 512;             // two chunks of 128 elements
constexpr int SFB_BYTES = 2 * 1024;
constexpr int SF_STAGE = SFA_BYTES + SFB_BYTES;
constexpr int STAGE_BYTES = A_STAGE + B_STAGE;
constexpr int SF_OFF = STAGES * STAGE_BYTES;
constexpr int BAR_OFF = SF_OFF + STAGES * SF_STAGE;
constexpr int PLAN_OFF = BAR_OFF + 256;
constexpr int MAX_GROUPS = kMaxExperts;
constexpr int PIECE_OFF = (PLAN_OFF + 2 * (MAX_GROUPS + 1) * 4 + 1023) / 1024 * 1024;
constexpr size_t SMEM_BYTES = 1024 + PIECE_OFF + EPI_WARPS * PIECE_BYTES;
constexpr int TMEM_COLS = 512;
constexpr int SF_SLOTS = 10;                   // two per stage
constexpr int SF_COL0 = BN, SF_COLS = 24;      // slot: A's 2 x 4 columns, B's 2 x 8
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(SF_COL0 + SF_COLS * SF_SLOTS <= TMEM_COLS, "TMEM columns");

__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t saddr) {
    uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    desc |= static_cast<uint64_t>(128u >> 4) << 16;
    desc |= static_cast<uint64_t>(128u >> 4) << 32;
    desc |= 1ull << 46;
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
mx4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmO, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint64_t* full = bars;
    uint64_t* empty = bars + STAGES;
    uint64_t* tfull = bars + 2 * STAGES;
    uint64_t* tempty = tfull + 1;
    uint64_t* fin = tempty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* mt_start = reinterpret_cast<int*>(smem + PLAN_OFF);
    int* row_start = mt_start + (args.G + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = args.G;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), 2 * EPI_WARPS);
        mbar_init(smem_u32(fin), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    cudaGridDependencySynchronize();
    make_plan<BM>(args, mt_start, row_start);
    tc_fence_before();
    __syncthreads();
    cluster_sync();              // the even CTA's barriers exist before the odd CTA signals them
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    int total_mtiles = mt_start[G];
    if (total_mtiles < 0 || total_mtiles > args.max_mtiles) {
        if (threadIdx.x == 0) set_dev_error(args.err, DEV_ERR_OFFSETS);
        total_mtiles = 0;
    }
    const int total = total_mtiles * args.n_tiles;
    const int chunks = args.K / 128;
    const int num_kb = (chunks + 1) / 2;
    const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(nclusters_x());

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            tma_prefetch_desc(&tmSA);
            tma_prefetch_desc(&tmSB);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += ncl) {
                const Tile tl = decode<BM>(t, mt_start, row_start, G, args.n_tiles);
                const int a_row = tl.a_row + static_cast<int>(rank) * 128;
                const int bt = tl.g * args.n_tiles + tl.n;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.err)) { ok = false; break; }
                    const uint32_t fb_local = smem_u32(&full[stage]);
                    if (leader) mbar_arrive_expect_tx(fb_local, 2 * (STAGE_BYTES + SF_STAGE));
                    const uint32_t fb = map_to_cta(fb_local, 0);
                    const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                    const uint32_t sf = smem_u32(smem + SF_OFF + stage * SF_STAGE);
                    tma_load_2d_pair(sa, &tmA, fb, kb * BK, a_row);
                    tma_load_3d_pair(sa + A_STAGE, &tmB, fb, 0, static_cast<int>(rank) * 128, bt * num_kb + kb);
                    tma_load_2d_pair(sf, &tmSA, fb, 0, a_row / 128 * chunks + 2 * kb);
                    tma_load_2d_pair(sf + SFA_BYTES, &tmSB, fb, 0, bt * chunks + 2 * kb);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (leader) {        // the loads of both CTAs complete on this CTA's barriers
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
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMA
        if (leader) {
            int stage = 0, it = 0;
            uint32_t phase = 0, slot = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += ncl, ++it) {
                // both CTAs' epilogues have copied the previous tile out of TMEM
                if (!mbar_wait(smem_u32(tempty), (static_cast<uint32_t>(it) & 1u) ^ 1u, abort_flag, args.err)) break;
                tc_fence_after();
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, args.err)) { ok = false; break; }
                    tc_fence_after();
                    __syncwarp();
                    if (elect_one()) {
                        const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                        const uint32_t sf = smem_u32(smem + SF_OFF + stage * SF_STAGE);
                        const uint32_t tsa = tmem_base + SF_COL0 + SF_COLS * slot, tsb = tsa + 8u;
                        const uint64_t adesc = smem_desc_sw128(sa), bdesc = smem_desc_sw128(sa + A_STAGE);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (q == 1 && 2 * kb + 1 >= chunks) break;
                            sf_copy(tsa + 4u * q, sf + q * 512);
                            sf_copy(tsb + 8u * q, sf + SFA_BYTES + q * 1024);
                            sf_copy(tsb + 8u * q + 4u, sf + SFA_BYTES + q * 1024 + 512);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int kk = 2 * q + j;
                                mma(tmem_base, adesc + 2ull * kk, bdesc + 2ull * kk, idesc_mx<true>(BM, BN, 2 * j), tsa + 4u * q,
                                    tsb + 8u * q, (kb > 0 || kk > 0) ? 1u : 0u);
                            }
                        }
                        tc_commit_pair_multicast(smem_u32(&empty[stage]), 0x3);
                        if (kb == num_kb - 1) tc_commit_pair_multicast(smem_u32(tfull), 0x3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    slot = slot + 1 == SF_SLOTS ? 0 : slot + 1;
                }
            }
            __syncwarp();
            if (elect_one()) tc_commit_pair_multicast(smem_u32(fin), 0x3);
            __syncwarp();
        }
        // both CTAs: every MMA writing this CTA's TMEM has completed
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(fin), 0)) {
            if (globaltimer_ns() - t0 > kWaitLimitNs) { set_dev_error(args.err, DEV_ERR_TIMEOUT); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const int r = quarter * 32 + lane;
        uint8_t* piece = smem + PIECE_OFF + (warp - 2) * PIECE_BYTES;
        int it = 0;
        for (int t = cid; t < total; t += ncl, ++it) {
            const Tile tl = decode<BM>(t, mt_start, row_start, G, args.n_tiles);
            const int a_row = tl.a_row + static_cast<int>(rank) * 128;
            const int left = tl.rows_valid - static_cast<int>(rank) * 128;      // of this CTA's rows, may be none
            if (!mbar_wait(smem_u32(tfull), static_cast<uint32_t>(it) & 1u, abort_flag, args.err)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 128);
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) tmem_ld32_sync(tb + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_tmem(map_to_cta(smem_u32(tempty), 0));
            epilogue<EPI, true, 128>(v, args, &tmO, tl.n, half, a_row, left < 128 ? left : 128, r, piece);
        }
        if (args.tma_out && lane == 0) bulk_wait0();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();              // neither CTA releases TMEM or leaves while the pair still works
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// Tensor map of `rows` rows of `words` 32-bit words, boxes of two rows.
cudaError_t scale_map(CUtensorMap* map, const void* base, long long rows, int words) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(words), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(words) * 4};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(words), 2};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int EPI>
cudaError_t launch(const void* A, long long a_rows, const uint8_t* a_sf, const void* B, const uint8_t* b_sf, int G, int N, int K,
                   const int* offsets, int rows, int max_mtiles, void* out, long long ldo, int out_cols, uint8_t* h_sf,
                   cudaStream_t st) {
    static bool set[kMaxDevices];
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(mx4_pair_kernel<EPI>), SMEM_BYTES, set);
    if (e != cudaSuccess) return e;
    if (K % 128 || N % 8 || a_rows % 128 || G < 1 || G > MAX_GROUPS) return cudaErrorInvalidValue;
    const int n_tiles = (N + BN - 1) / BN, stages = (K / 2 + BK - 1) / BK;
    CUtensorMap ta, tb, sa, sb, to;
    e = make_map(&ta, A, a_rows, K / 2, 128, true);
    if (e == cudaSuccess) e = make_map_blocked(&tb, B, static_cast<long long>(G) * n_tiles * stages, 128, true);
    if (e == cudaSuccess) e = scale_map(&sa, a_sf, a_rows / 128 * (K / 128), 128);
    if (e == cudaSuccess) e = scale_map(&sb, b_sf, static_cast<long long>(G) * n_tiles * (K / 128), 256);
    if (e != cudaSuccess) return e;
    Args args{};
    args.offsets = offsets;
    args.G = G;
    args.rows = rows;
    args.N = N;
    args.K = K;
    args.n_tiles = n_tiles;
    args.max_mtiles = max_mtiles;
    args.out = out;
    args.ldo = ldo;
    args.out_cols = out_cols;
    args.h_sf = h_sf;
    args.err = dev_error_ptr();
    to = ta;
    e = out_map(&to, EPI, out, offsets ? a_rows : rows, out_cols, ldo, &args.tma_out);
    if (e != cudaSuccess) return e;
    if (EPI == EPI_SWIGLU && (!h_sf || ldo < out_cols / 2)) return cudaErrorInvalidValue;
    int sms = 0;
    e = num_sms(&sms);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>(max_mtiles) * n_tiles;
    const int clusters = static_cast<int>(tiles < sms / 2 ? (tiles < 1 ? 1 : tiles) : sms / 2);
    count_launch();
    return launch_after(mx4_pair_kernel<EPI>, dim3(2 * clusters), dim3(THREADS), SMEM_BYTES, st, ta, tb, sa, sb, to, args);
}

}  // namespace pair
}  // namespace mx

cudaError_t launch_mx4_pair_gemm(int epi, const void* A, long long a_rows, const uint8_t* a_sf, const void* B,
                                 const uint8_t* b_sf, int G, int N, int K, const int* offsets, int rows, int max_mtiles,
                                 void* out, long long ldo, int out_cols, uint8_t* h_sf, cudaStream_t st) {
    switch (epi) {
        case EPI_SWIGLU:
            return mx::pair::launch<EPI_SWIGLU>(A, a_rows, a_sf, B, b_sf, G, N, K, offsets, rows, max_mtiles, out, ldo, out_cols,
                                                h_sf, st);
        case EPI_BF16:
            return mx::pair::launch<EPI_BF16>(A, a_rows, a_sf, B, b_sf, G, N, K, offsets, rows, max_mtiles, out, ldo, out_cols,
                                              h_sf, st);
        case EPI_F32:
            return mx::pair::launch<EPI_F32>(A, a_rows, a_sf, B, b_sf, G, N, K, offsets, rows, max_mtiles, out, ldo, out_cols,
                                             h_sf, st);
        default:
            return cudaErrorInvalidValue;
    }
}

}  // namespace fs
