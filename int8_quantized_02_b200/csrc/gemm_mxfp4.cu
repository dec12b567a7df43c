// The MXFP4 product on the 5th-generation tensor cores of sm_100a:
//     Y[m, n] = sum_k X[m, k] W[n, k] + bias[n]
// X [M, K] and W [N, K] as e2m1 codes with one e8m0 scale to 32 columns, tcgen05.mma kind::mxf4
// (the tensor core applies both scales to each 32-column partial product), fp32 accumulators in
// TMEM, one rounding to the 16-bit output.
//
// A k-tile is 256 columns: 128 bytes of codes a row (the 128-byte swizzle's row, as in the int8
// product) and the 1024 bytes of a scale tile for each 128 rows, which is laid out in global
// memory as tcgen05.cp wants it: 32 lanes x 16 bytes for 128 columns, copied to four TMEM columns
// and broadcast to the four lane quadrants.  One k-tile is four MMAs of 64 columns; the scales of
// a pair of them are one copy, and the two pairs of a k-tile use two TMEM regions in turn.
// (Copies and MMAs of one thread execute in the order issued.)
//
// Two kernels:
//   pair  two CTAs of a cluster share 256 x 256 output tiles (cta_group::2; 128 rows of X and half
//         of the weight rows each), persistent, 6 stages.  Two 256-column accumulators and 24
//         columns of scales do not fit TMEM's 512, so the two accumulators overlap by 32 columns:
//         the epilogue takes those first, and the next tile's MMAs wait for them alone.
//   band  few rows of X: the weight is the MMA's 128-row operand and up to 64 rows of X its
//         columns, so each weight byte enters one SM once.  The k range of a band of 128 weight
//         rows is split over the S CTAs of a cluster, which add their partial sums through
//         distributed shared memory in rank order (the result does not depend on timing).
//         Up to 8 rows of X come unquantised: the epilogue's warps quantise each k-tile's rows
//         straight into its stage, in turns, while the weight streams in, and the layer is one
//         launch (us, one / two launches: 1 x 4096 x 4096 5.0 / 7.2, 8 x 16384 x 4096 10.3 / 11.8,
//         8 x 49152 x 12288 50.8 / 52.5; 16 rows do not fit the time that a k-tile of the weight
//         takes, 16 x 16384 x 4096 17.1 / 11.9).
// Every wait on an mbarrier is bounded (BoundedWait), as in the int8 product.
#include <mutex>

#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"

namespace llmint8 {

namespace {

constexpr int KB = 128;                  // bytes of codes of a k-tile's row
constexpr int ROWS = 128;                // rows of one CTA's X (pair) or weight (band) tile

// ------------------------------------------------------------------- tcgen05 forms ------
// Instruction descriptor of kind::mxf4: bits 4-5 the scales of B (which half of each 32-bit
// word: 0 or 2), 7-9 and 10-11 the operand types (1 = e2m1), 17-22 N / 8, 23 e8m0 scales,
// 27-28 M / 128, 29-30 the scales of A.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, int half) {
    return ((uint32_t)half << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           (1u << 23) | ((uint32_t)(m >> 7) << 27) | ((uint32_t)half << 29);
}

template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// 512 bytes of scales (128 rows x 128 columns) from shared memory to four TMEM columns.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle; 8 rows of 16 bytes to a core matrix, 128 bytes from one to the next
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) |
                          ((uint64_t)1u << 46);
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
}

// The MMAs of one k-tile.  `n_mma` (1 to 4) leaves out 64-column steps past K.
// TMEM at `sf`: for each pair of steps 4 columns of A's scales, then 4 for each 128 rows of B, of
// which B's rows begin at column `b0` (a column holds 32 rows; the address must be even, so tiles
// of B begin at multiples of 64 rows).
template <bool PAIR, int M, int N>
__device__ __forceinline__ void mma_ktile(uint32_t d, uint32_t sa, uint32_t sb, uint32_t ssfa,
                                          uint32_t ssfb, uint32_t sf, uint32_t b0, int n_mma,
                                          bool first) {
    constexpr int NB = (N + 127) / 128;
    constexpr uint32_t kCols = 4 + 4 * NB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (2 * h >= n_mma) break;
        const uint32_t t = sf + (uint32_t)h * kCols;
        copy_scales<PAIR>(t, ssfa + h * 512);
#pragma unroll
        for (int b = 0; b < NB; ++b) copy_scales<PAIR>(t + 4 + 4 * b, ssfb + b * kMxTile + h * 512);
#pragma unroll
        for (int k = 2 * h; k < 2 * h + 2; ++k)
            if (k < n_mma)
                mma_mxf4<PAIR>(d, sw128_desc(sa + 32 * k), sw128_desc(sb + 32 * k),
                               idesc_mxf4(M, N, 2 * (k & 1)), t, t + 4 + b0, !first || k != 0);
    }
}

// ------------------------------------------------------------------------- pair ---------
constexpr int BN = 256;                  // columns of an output tile
constexpr int EPI_WARPS = 8;             // two to a TMEM lane quadrant
constexpr int P_THREADS = 64 + 32 * EPI_WARPS;
constexpr int P_STAGES = 6;
constexpr int P_STAGE = 2 * ROWS * KB + 3 * kMxTile;   // X, half of W, scales of X and of W
constexpr int P_SHIFT = 224;             // first column of the second accumulator
constexpr int P_SF = 480;                // first column of the scales
// Staging of a warp's 32 x 32 outputs, 64 bytes a row in the order of TMA's 64-byte swizzle.
constexpr int P_STAGE_OUT = 32 * 64;
constexpr int P_STAGING = EPI_WARPS * P_STAGE_OUT;
static_assert(P_SHIFT + BN <= P_SF && P_SF + 2 * 12 <= 512, "TMEM columns");

struct PairTail {
    uint64_t full[P_STAGES];
    uint64_t empty[P_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t shared_empty;               // the columns both accumulators hold are read out
    uint64_t mma_done;
    uint64_t peer_loads;                 // leader: peer_issued holds the second CTA's count
    uint64_t loads_drained;              // second CTA: the leader is done, its loads drained
    uint64_t peer_exit;                  // leader: the second CTA made its last arrive
    uint32_t tmem_base;
    uint32_t peer_issued;
    int abort_flag;
};
constexpr int P_SMEM = P_STAGES * P_STAGE + P_STAGING + (int)sizeof(PairTail);
static_assert(P_SMEM <= 232448, "fits the opt-in shared memory of one CTA");

struct PArgs {
    const void *bias;
    void *Y;
    StatusRef status;
    int M, N;
    int tiles_k, last_mma;               // k-tiles; 64-column steps in the last one
    int tiles_m, tiles_n;
    uint64_t timeout_ns;
};

template <int DT>
__device__ __forceinline__ float load16(const void *p, int64_t i) {
    if constexpr (DT == kF16) return __half2float(static_cast<const __half *>(p)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store16(void *p, int64_t i, float v) {
    if constexpr (DT == kF16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

template <int DT>
__global__ void __launch_bounds__(P_THREADS, 1)
mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmXS, const __grid_constant__ CUtensorMap tmWS,
                  const __grid_constant__ CUtensorMap tmY, const PArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *staging = smem + P_STAGES * P_STAGE;
    PairTail *tail = reinterpret_cast<PairTail *>(smem + P_STAGES * P_STAGE + P_STAGING);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(smem_addr(&tail->full[s]), 1);
            mbar_init(smem_addr(&tail->empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&tail->acc_full[s]), 1);
            mbar_init(smem_addr(&tail->acc_empty[s]), 2 * EPI_WARPS);
        }
        mbar_init(smem_addr(&tail->shared_empty), EPI_WARPS);   // half of each CTA's warps
        mbar_init(smem_addr(&tail->mma_done), 1);
        mbar_init(smem_addr(&tail->peer_loads), 1);
        mbar_init(smem_addr(&tail->loads_drained), 1);
        mbar_init(smem_addr(&tail->peer_exit), 1);
        tail->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmXS);
        tma_prefetch_desc(&tmWS);
    }
    if (warp == 1) tmem_alloc_pair(smem_addr(&tail->tmem_base), 512);
    // a pair's barriers are initialized in both CTAs before either may use the other's
    cluster_barrier_all();
    // X's codes and scales are complete after this
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem_base;
    const BoundedWait wait{&tail->abort_flag, a.status, a.timeout_ns};
    LLMINT8_DCHECK((smem_addr(smem) & 1023u) == 0, a.status);
    const int total = a.tiles_m * a.tiles_n;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.status.set(LLMINT8_OK);

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer ----
        if (elect_one()) {
            const uint64_t keep = l2_policy_evict_last();
            int stage = 0;
            uint32_t phase = 0, issued = 0;      // k-tiles whose loads are on their way
            for (int tile = unit; tile < total; tile += units) {
                const int mt = (tile % a.tiles_m) * 2 + (int)rank;   // this CTA's 128 rows of X
                const int nt = (tile / a.tiles_m) * 2;               // the tile's 256 of W
                int kr = first_kblock(tile / a.tiles_m, a.tiles_k);
                for (int kb = 0; kb < a.tiles_k; ++kb) {
                    LLMINT8_DCHECK(kr >= 0 && kr < a.tiles_k && nt / 2 < a.tiles_n, a.status);
                    if (!wait(smem_addr(&tail->empty[stage]), phase ^ 1)) goto drain;
                    const uint32_t full = smem_addr(&tail->full[stage]);
                    const uint32_t sa = smem_addr(smem + stage * P_STAGE);
                    // the leader's barrier counts the bytes of both CTAs
                    if (leader) mbar_arrive_expect_tx(full, 2 * P_STAGE);
                    const uint32_t fbar = map_to_rank(full, 0);
                    tma_load_2d_pair_hint(sa, &tmX, kr * KB, mt * ROWS, fbar, keep);
                    tma_load_2d_pair(sa + ROWS * KB, &tmW, kr * KB, (nt + (int)rank) * ROWS, fbar);
                    // scale tiles past the last row of tiles read as zero
                    const uint32_t ss = sa + 2 * ROWS * KB;
                    tma_load_2d_pair_hint(ss, &tmXS, 0, mt * a.tiles_k + kr, fbar, keep);
                    tma_load_2d_pair(ss + kMxTile, &tmWS, 0, nt * a.tiles_k + kr, fbar);
                    tma_load_2d_pair(ss + 2 * kMxTile, &tmWS, 0, (nt + 1) * a.tiles_k + kr, fbar);
                    ++issued;
                    if (++kr == a.tiles_k) kr = 0;
                    if (++stage == P_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        drain:
            // the next kernel may set up while the last tiles are finished
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            // Every copy that signals the leader's barriers lands before either CTA exits.  After a
            // wait that gave up, one CTA may have issued k-tiles that the other did not: the
            // leader then takes the missing copies' bytes off, or expects those it did not.
            if (tail->abort_flag)
                st_cluster_u32(map_to_rank(smem_addr(&tail->abort_flag), rank ^ 1u), 1u);
            if (leader) {
                drain_wait(smem_addr(&tail->peer_loads), 0, a.status);
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                const uint32_t theirs = *reinterpret_cast<volatile uint32_t *>(&tail->peer_issued);
                for (uint32_t it = theirs; it < issued; ++it)
                    mbar_complete_tx(smem_addr(&tail->full[it % P_STAGES]), P_STAGE);
                for (uint32_t it = issued; it < theirs; ++it)
                    mbar_arrive_expect_tx(smem_addr(&tail->full[it % P_STAGES]), P_STAGE);
                const uint32_t all = max(issued, theirs);
                for (uint32_t it = all - min(all, (uint32_t)P_STAGES); it < all; ++it)
                    drain_wait(smem_addr(&tail->full[it % P_STAGES]), (it / P_STAGES) & 1u,
                               a.status);
            } else {
                st_cluster_u32(map_to_rank(smem_addr(&tail->peer_issued), 0), issued);
                mbar_arrive_cluster(map_to_rank(smem_addr(&tail->peer_loads), 0));
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMA issuer ----
        if (leader && elect_one()) {
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            int acc = 0, done = 0;
            for (int tile = unit; tile < total; tile += units, ++done) {
                if (!wait(smem_addr(&tail->acc_empty[acc]), acc_phase ^ 1)) break;
                if (done > 0 &&
                    !wait(smem_addr(&tail->shared_empty), (uint32_t)(done - 1) & 1u))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * P_SHIFT);
                bool ok = true;
                int kr = first_kblock(tile / a.tiles_m, a.tiles_k);
                for (int kb = 0; kb < a.tiles_k; ++kb) {
                    if (!wait(smem_addr(&tail->full[stage]), phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * P_STAGE);
                    mma_ktile<true, 2 * ROWS, BN>(
                        d, sa, sa + ROWS * KB, sa + 2 * ROWS * KB, sa + 2 * ROWS * KB + kMxTile,
                        tmem + P_SF, 0, kr == a.tiles_k - 1 ? a.last_mma : 4, kb == 0);
                    tc_commit_pair_multicast(smem_addr(&tail->empty[stage]));
                    if (++kr == a.tiles_k) kr = 0;
                    if (++stage == P_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair_multicast(smem_addr(&tail->acc_full[acc]));
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            // every MMA issued by this thread has completed once mma_done arrives
            tc_commit_pair_multicast(smem_addr(&tail->mma_done));
            drain_wait(smem_addr(&tail->mma_done), 0, a.status);
        }
    } else {
        // ----------------------------------------------------------------- epilogue ----
        const int q = warp & 3;                        // TMEM lane quadrant of this warp
        const int half = (warp - 2) / 4;               // its half of the tile's columns
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        uint8_t *stg = staging + (warp - 2) * P_STAGE_OUT;
        const bool vec = (a.N & 7) == 0;               // rows of Y start on 16 bytes
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = unit; tile < total; tile += units) {
            const int m0 = (tile % a.tiles_m) * 2 * ROWS + (int)rank * ROWS + q * 32;
            const int n0 = (tile / a.tiles_m) * BN;
            int ok = 0;
            if (lane == 0) ok = wait(smem_addr(&tail->acc_full[acc]), acc_phase) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                // of 8 chunks of 32 columns, the one that the other accumulator shares first:
                // the last of the first accumulator, the first of the second
                const int c = half ? 4 + ((i + 3) & 3) : i;
                const int nb = n0 + c * 32;
                uint32_t v[32];
                tmem_ld_32x32(tl + (uint32_t)(acc * P_SHIFT + c * 32), v);
                tmem_wait_ld();
                if (i == 0 && half == 1 - acc) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(smem_addr(&tail->shared_empty));
                        else mbar_arrive_cluster(map_to_rank(smem_addr(&tail->shared_empty), 0));
                    }
                }
                if (nb >= a.N) continue;
                if (a.bias) {
                    if (nb + 32 <= a.N) {
                        const uint4 *bp = reinterpret_cast<const uint4 *>(
                            static_cast<const uint8_t *>(a.bias) + (int64_t)nb * 2);
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint4 b4 = __ldg(bp + g);
                            Chunk<DT> bc;
                            bc.w[0] = b4.x;
                            bc.w[1] = b4.y;
                            bc.w[2] = b4.z;
                            bc.w[3] = b4.w;
                            float f[8];
                            unpack_chunk<DT>(bc, f);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                v[g * 8 + e] =
                                    __float_as_uint(__uint_as_float(v[g * 8 + e]) + f[e]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (nb + j < a.N)
                                v[j] = __float_as_uint(__uint_as_float(v[j]) +
                                                       load16<DT>(a.bias, nb + j));
                    }
                }
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    p[j] = pack_pair<DT>(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                // the warp's last stores have read the staging
                if (vec && lane == 0) bulk_wait_read();
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<uint4 *>(stg + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]);
                if (vec) {
                    fence_proxy_async_shared();
                    __syncwarp();
                    // what lies past M or N is left out by the tensor map
                    LLMINT8_DCHECK(m0 >= 0 && nb >= 0 && nb < a.N, a.status);
                    if (lane == 0 && m0 < a.M) tma_store_2d(&tmY, smem_addr(stg), nb, m0);
                    continue;
                }
                // rows of any alignment: neighbouring lanes write neighbouring values, in pairs
                // where rows start on 4 bytes
                __syncwarp();
                const int rows = min(32, a.M - m0);
                LLMINT8_DCHECK(rows <= 32 && (rows <= 0 || m0 + rows <= a.M), a.status);
                uint16_t *y = static_cast<uint16_t *>(a.Y) + (int64_t)m0 * a.N;
                const auto word_at = [&](int r, int w) {
                    return stg + r * 64 + (((w >> 2) ^ ((r >> 1) & 3)) << 4) + (w & 3) * 4;
                };
                if ((a.N & 1) == 0) {
                    const int n = nb + 2 * (lane & 15);
                    if (n < a.N) {
#pragma unroll 8
                        for (int r = lane >> 4; r < rows; r += 2)
                            *reinterpret_cast<uint32_t *>(y + (int64_t)r * a.N + n) =
                                *reinterpret_cast<const uint32_t *>(word_at(r, lane & 15));
                    }
                } else if (nb + lane < a.N) {
#pragma unroll 8
                    for (int r = 0; r < rows; ++r)
                        y[(int64_t)r * a.N + nb + lane] = reinterpret_cast<const uint16_t *>(
                            word_at(r, lane >> 1))[lane & 1];
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(smem_addr(&tail->acc_empty[acc]));
                else mbar_arrive_cluster(map_to_rank(smem_addr(&tail->acc_empty[acc]), 0));
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    // Winding down.  The waits from here on have a fixed limit, so they begin only now: a launch may take
    // longer than that, and the two CTAs reach this point at nearly the same time.
    if (threadIdx.x == 0) {
        // a CTA that gave up takes the other along (which is still there: the leader until peer_exit,
        // the second CTA until loads_drained)
        if (tail->abort_flag)
            st_cluster_u32(map_to_rank(smem_addr(&tail->abort_flag), rank ^ 1u), 1u);
        if (leader) {
            mbar_arrive_cluster(map_to_rank(smem_addr(&tail->loads_drained), 1));
            // the second CTA has made its last arrive on this CTA's barriers
            drain_wait(smem_addr(&tail->peer_exit), 0, a.status);
        } else {
            // the leader has seen every copy of this CTA land; then release the leader
            drain_wait(smem_addr(&tail->loads_drained), 0, a.status);
            mbar_arrive_cluster(map_to_rank(smem_addr(&tail->peer_exit), 0));
        }
    }
    if (warp == 1) {
        // the second CTA's TMEM and shared memory are the leader's MMA operands until its last MMA has
        // completed
        if (!leader && lane == 0) drain_wait(smem_addr(&tail->mma_done), 0, a.status);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------------------- band ---------
constexpr int B_THREADS = 192;           // producer, MMA issuer, four epilogue warps

template <int NT>
struct Band {
    static constexpr int NB = (NT + 127) / 128;        // scale tiles of X
    static constexpr int STAGE = ROWS * KB + NT * KB + (1 + NB) * kMxTile;
    // Stages of a CTA that has an SM, or half of one, to itself: about 100 KB, so that two fit; and
    // where the grid fills the machine more than twice, about 60 KB, so that a third CTA covers the
    // others' first loads and last stores (8 x 49152 x 12288: 53.7 us with 5 stages, 50.2 with 3).
    // The CTAs of one such grid that fit an SM's shared memory hold 512 columns of TMEM at most, so none of
    // them waits for another's.
    static constexpr int STAGES = 104 * 1024 / STAGE;
    static constexpr int FEW = NT == 64 ? 2 : 3;
    static constexpr uint32_t SF = NT;                 // TMEM: accumulator, then the scales
    static constexpr uint32_t COLS_USED = NT + 2 * (4 + 4 * NB);
    static constexpr uint32_t COLS = COLS_USED <= 32    ? 32
                                     : COLS_USED <= 64  ? 64
                                                        : 128;
    static_assert(COLS_USED <= COLS, "TMEM columns");
    static_assert(STAGE % 1024 == 0, "stages keep the swizzle's alignment");
    static_assert(FEW * STAGE >= NT * ROWS * 4, "the partial sums fit the stages");
};
constexpr int kBandMaxStages = 5;

struct BandTail {
    uint64_t full[kBandMaxStages];       // the copies into a stage have landed
    uint64_t quantised[kBandMaxStages];  // fused: X's rows are in it
    uint64_t empty[kBandMaxStages];
    uint64_t acc_full;
    uint32_t tmem_base;
    int abort_flag;
};
template <int NT>
constexpr int band_smem(int stages) {
    return stages * Band<NT>::STAGE + (int)sizeof(BandTail);
}

struct BArgs {
    const uint8_t *X;                    // fused: X itself, its row pitch in bytes, chunks of a row
    int64_t row_bytes;
    int64_t chunks;
    const void *bias;
    void *Y;
    StatusRef status;
    int M, N;
    int tiles_k, last_mma;
    int splits;                          // CTAs of a cluster
    int stages;
    uint64_t timeout_ns;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int DT, int NT, bool FUSED>
__global__ void __launch_bounds__(B_THREADS)
mxfp4_band_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmXS, const __grid_constant__ CUtensorMap tmWS,
                  const BArgs a) {
    using C = Band<NT>;
    static_assert(C::STAGES <= kBandMaxStages, "barriers");
    static_assert(!FUSED || (NT >= kMxfp4FusedRows && kMxfp4FusedRows <= 8), "rows of one swizzle atom");
    const int stages = a.stages;
    extern __shared__ __align__(1024) uint8_t smem[];
    BandTail *tail = reinterpret_cast<BandTail *>(smem + stages * C::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.splits;
    const int rank = (int)(blockIdx.x % (unsigned)S);
    const int band = (int)(blockIdx.x / (unsigned)S);
    const int m0 = (int)blockIdx.y * NT;               // more than one tile only with NT = 64
    // this CTA's k-tiles
    const int k_begin = (int)((int64_t)a.tiles_k * rank / S);
    const int k_count = (int)((int64_t)a.tiles_k * (rank + 1) / S) - k_begin;
    // ... from a place that depends on the band, so that the CTAs do not all read the same part of X, nor
    // the same columns of the weight, at one time (16 x 16384 x 4096: 11.4 us without, 10.7 with)
    const int k_first = first_kblock(band, k_count);
    const auto ktile = [&](int it) {
        const int k = k_first + it;
        return k_begin + (k >= k_count ? k - k_count : k);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_addr(&tail->full[s]), 1);
            mbar_init(smem_addr(&tail->quantised[s]), 1);
            mbar_init(smem_addr(&tail->empty[s]), 1);
        }
        mbar_init(smem_addr(&tail->acc_full), 1);
        tail->abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmWS);
        if (!FUSED) {
            tma_prefetch_desc(&tmX);
            tma_prefetch_desc(&tmXS);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&tail->tmem_base), C::COLS);
        // The next kernel may set up, and ask L2 for its weight, while this one runs.  Not before this
        // CTA has its columns of TMEM, so the warp that allocates them says so (one thread's word
        // counts for the CTA): a dependent that took them first would wait for this grid, and this
        // grid's allocation for the dependent.
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem_base;
    const BoundedWait wait{&tail->abort_flag, a.status, a.timeout_ns};
    LLMINT8_DCHECK((smem_addr(smem) & 1023u) == 0, a.status);

    const auto load = [&](int it, int stage) {
        const uint32_t full = smem_addr(&tail->full[stage]);
        const uint32_t sa = smem_addr(smem + stage * C::STAGE);
        const int kt = ktile(it);
        LLMINT8_DCHECK(kt >= k_begin && kt < k_begin + k_count && stage < stages, a.status);
        mbar_arrive_expect_tx(full, FUSED ? ROWS * KB + kMxTile : C::STAGE);
        tma_load_2d(sa, &tmW, kt * KB, band * ROWS, full);
        tma_load_2d(sa + (ROWS + NT) * KB, &tmWS, 0, band * a.tiles_k + kt, full);
        if (FUSED) return;
        tma_load_2d(sa + ROWS * KB, &tmX, kt * KB, m0, full);
        // scale tiles past the last row of tiles read as zero
#pragma unroll
        for (int b = 0; b < C::NB; ++b)
            tma_load_2d(sa + (ROWS + NT) * KB + (1 + b) * kMxTile, &tmXS, 0,
                        (m0 / kMxRows + b) * a.tiles_k + kt, full);
    };

    if (warp == 0) {
        if (elect_one()) {
            // The kernel that is still running may be writing the weight: L2, where every write lands,
            // is asked to fetch the first stages of it meanwhile.
            for (int it = 0; it < min(stages, k_count); ++it) {
                tma_prefetch_l2_2d(&tmW, ktile(it) * KB, band * ROWS);
                tma_prefetch_l2_2d(&tmWS, 0, band * a.tiles_k + ktile(it));
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int it = 0, stage = 0;
            uint32_t phase = 0;
            for (; it < k_count; ++it) {
                if (!wait(smem_addr(&tail->empty[stage]), phase ^ 1)) break;
                load(it, stage);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            // wait for every copy this thread issued to land before the CTA may exit
            for (int i = max(0, it - stages); i < it; ++i)
                drain_wait(smem_addr(&tail->full[i % stages]), (uint32_t)(i / stages) & 1u,
                           a.status);
        }
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (warp == 1 && elect_one()) {
            int stage = 0;
            uint32_t phase = 0;
            for (int it = 0; it < k_count; ++it) {
                if (!wait(smem_addr(&tail->full[stage]), phase)) break;
                if (FUSED && !wait(smem_addr(&tail->quantised[stage]), phase)) break;
                tc_fence_after();
                const uint32_t sa = smem_addr(smem + stage * C::STAGE);
                const uint32_t ss = sa + (ROWS + NT) * KB;
                mma_ktile<false, ROWS, NT>(tmem, sa, sa + ROWS * KB, ss, ss + kMxTile,
                                           tmem + C::SF, (uint32_t)(m0 & (kMxRows - 1)) >> 5,
                                           ktile(it) == a.tiles_k - 1 ? a.last_mma : 4,
                                           it == 0);
                tc_commit(smem_addr(&tail->empty[stage]));
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            // also after a wait that gave up: every MMA issued has completed once this arrives
            tc_commit(smem_addr(&tail->acc_full));
            drain_wait(smem_addr(&tail->acc_full), 0, a.status);
        }
        // Every `turns`-th k-tile is a warp's: X's rows to codes (a row of the swizzled operand, 16-byte
        // pieces XOR the row) and scales (a word a half tile), as the copies would have left them.
        // No more turns than stages: a warp that waits for stage k-tile `it` then knows that the
        // k-tile before the one there was consumed, so the barrier's parity tells the two apart.
        const int turns = min(4, stages);
        if (FUSED && warp >= 2 && warp - 2 < turns) {
            for (int it = warp - 2; it < k_count; it += turns) {
                const int stage = it % stages;
                const int64_t ch = (int64_t)ktile(it) * 32 + lane;
                LLMINT8_DCHECK(stage < stages && a.M <= kMxfp4FusedRows && ktile(it) < a.tiles_k, a.status);
                Chunk<DT> c[kMxfp4FusedRows];
#pragma unroll
                for (int m = 0; m < kMxfp4FusedRows; ++m)
                    c[m] = m < a.M && ch < a.chunks ? load_chunk<DT>(a.X + m * a.row_bytes, ch)
                                                    : zero_chunk<DT>();
                int ok = 0;
                if (lane == 0)
                    ok = wait(smem_addr(&tail->empty[stage]), (uint32_t)(it / stages + 1) & 1u);
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
                uint8_t *sx = smem + stage * C::STAGE + ROWS * KB;
                uint8_t *ss = sx + NT * KB + kMxTile;
#pragma unroll
                for (int m = 0; m < kMxfp4FusedRows; ++m) {
                    if (m >= a.M) break;
                    uint32_t word;
                    const uint32_t q = quantize_chunk<DT>(c[m], word, lane);
                    *reinterpret_cast<uint32_t *>(sx + m * KB + (((lane >> 2) ^ m) << 4) +
                                                  (lane & 3) * 4) = q;
                    if ((lane & 15) == 0)
                        *reinterpret_cast<uint32_t *>(ss + (lane >> 4) * 512 + m * 16) = word;
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&tail->quantised[stage]));
            }
        }
    }
    __syncwarp();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 32) a.status.set(LLMINT8_OK);
    tc_fence_before();

    // The partial sums of this CTA, [row of X][row of the band] fp32, in its stages: every copy
    // and MMA that used them has completed (the issuer drained acc_full, the producer the
    // copies, and both come before this barrier).
    __syncthreads();
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);
    const int rows = min(NT, a.M - m0);
    if (warp >= 2) {
        const int q = warp & 3;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < NT; c += 16) {
            if (c >= rows) break;
            uint32_t v[16];
            tmem_ld_32x16(tl + (uint32_t)c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                part[(c + j) * ROWS + q * 32 + lane] = __uint_as_float(v[j]);
        }
        tc_fence_before();
    }
    __syncwarp();
    if (S > 1) cluster_barrier_all();
    else __syncthreads();

    // Each CTA of the cluster finishes every S-th row of X; a lane four columns of Y.
    const int n = band * ROWS + lane * 4;
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) b[e] = load16<DT>(a.bias, n + e);
    }
    for (int m = rank + S * warp; m < rows; m += S * (B_THREADS / 32)) {
        const uint32_t at = smem_addr(part + m * ROWS + lane * 4);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (S == 1) {
            const float4 v = *reinterpret_cast<const float4 *>(part + m * ROWS + lane * 4);
            y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
        } else {
            for (int r = 0; r < S; ++r) {
                const float4 v = ld_cluster_f4(map_to_rank(at, (uint32_t)r));
                y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
            }
        }
        const int64_t o = (int64_t)(m0 + m) * a.N + n;
        LLMINT8_DCHECK(m < NT && m0 + m < a.M && ((a.N & 3) || n >= a.N || n + 4 <= a.N), a.status);
        if ((a.N & 3) == 0) {
            if (n < a.N)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.Y) + o) =
                    make_uint2(pack_pair<DT>(y[0] + b[0], y[1] + b[1]),
                               pack_pair<DT>(y[2] + b[2], y[3] + b[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) store16<DT>(a.Y, o + e, y[e] + b[e]);
        }
    }
    __syncwarp();
    // the other CTAs are done with this one's sums before it exits
    if (S > 1) cluster_barrier_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

// ------------------------------------------------------------------------ launch --------
struct Maps {
    CUtensorMap X, W, XS, WS;
};

bool make_maps(Maps *t, const Mxfp4Gemm &g, uint32_t x_rows, bool fused = false) {
    const int64_t tiles_k = ceil_div(g.K, kMxCols);
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    const auto flat = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (fused) memset(t, 0, sizeof(*t));
    return (fused ||
            (make_map(&t->X, g.Xc, u8, 1, g.K / 2, g.M, g.K / 2, KB, x_rows) &&
             make_map(&t->XS, g.Xs, u32, 4, kMxTile / 4, ceil_div(g.M, kMxRows) * tiles_k,
                      kMxTile / 4, kMxTile / 4, 1, flat))) &&
           make_map(&t->W, g.Wc, u8, 1, g.K / 2, g.N, g.K / 2, KB, ROWS) &&
           make_map(&t->WS, g.Ws, u32, 4, kMxTile / 4, ceil_div(g.N, kMxRows) * tiles_k,
                    kMxTile / 4, kMxTile / 4, 1, flat);
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int NT>
cudaError_t allow_band() {
    constexpr int smem = band_smem<NT>(Band<NT>::STAGES);
    cudaError_t e = allow_smem(mxfp4_band_kernel<kF16, NT, false>, smem);
    if (e == cudaSuccess) e = allow_smem(mxfp4_band_kernel<kBF16, NT, false>, smem);
    if constexpr (NT == 16) {
        if (e == cudaSuccess) e = allow_smem(mxfp4_band_kernel<kF16, NT, true>, smem);
        if (e == cudaSuccess) e = allow_smem(mxfp4_band_kernel<kBF16, NT, true>, smem);
    }
    return e;
}

// Shared-memory limits, once per device; the SM count.
cudaError_t device_setup(int *sms) {
    static std::mutex mu;
    static int known[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        int n = 0;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = allow_smem(mxfp4_pair_kernel<kF16>, P_SMEM)) != cudaSuccess ||
            (e = allow_smem(mxfp4_pair_kernel<kBF16>, P_SMEM)) != cudaSuccess ||
            (e = allow_band<16>()) != cudaSuccess || (e = allow_band<32>()) != cudaSuccess ||
            (e = allow_band<64>()) != cudaSuccess)
            return e;
        known[dev] = n;
    }
    *sms = known[dev];
    return cudaSuccess;
}

// Launch in clusters of `cluster` CTAs, as a programmatic dependent.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, int cluster,
                           cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// CTAs that share a band's k.  As many as still leave each an SM of its own and four k-tiles: past
// that the exchange costs more than the shorter k saves (1 x 4096 x 4096: 8.4 us in one part, 7.1 in
// four, 7.6 in eight; 1 x 1024 x 1024, four k-tiles: 3.8 in one, 4.5 in four).
int band_splits(int64_t tiles, int tiles_k, int sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({8, sms / tiles, (int64_t)tiles_k / 4}));
}

// The band kernel for tiles of NT rows of X.
template <int NT>
cudaError_t band(const Mxfp4Gemm &g, int tiles_k, int last_mma, int sms, cudaStream_t s) {
    const bool fused = g.X != nullptr;
    Maps t;
    if (!make_maps(&t, g, NT, fused)) return cudaErrorInvalidValue;
    const int64_t tiles = ceil_div(g.N, ROWS) * ceil_div(g.M, NT);
    BArgs a;
    a.X = static_cast<const uint8_t *>(g.X);
    a.row_bytes = g.ldx * 2;
    a.chunks = g.K / 8;
    a.bias = g.bias;
    a.Y = g.Y;
    a.status = g.status;
    a.M = (int)g.M;
    a.N = (int)g.N;
    a.tiles_k = tiles_k;
    a.last_mma = last_mma;
    a.timeout_ns = g.timeout_ns;
    a.splits = band_splits(tiles, tiles_k, sms);
    a.stages = tiles * a.splits > 2 * sms ? Band<NT>::FEW : Band<NT>::STAGES;
    const dim3 grid((unsigned)(ceil_div(g.N, ROWS) * a.splits), (unsigned)ceil_div(g.M, NT));
    auto k = g.dtype == kF16 ? mxfp4_band_kernel<kF16, NT, false>
                             : mxfp4_band_kernel<kBF16, NT, false>;
    if constexpr (NT == 16) {
        if (fused)
            k = g.dtype == kF16 ? mxfp4_band_kernel<kF16, NT, true>
                                : mxfp4_band_kernel<kBF16, NT, true>;
    }
    return launch_cluster(k, grid, B_THREADS, band_smem<NT>(a.stages), a.splits, s, t.X, t.W, t.XS,
                          t.WS, a);
}

// The band kernel takes up to 64 rows of X, and more in tiles of 64 while each tile has an SM of its
// own.  (us, band / pair: 64 x 49152 x 12288 56.1 / 63.4, 256 x 1024 x 8192 9.0 / 15.3,
// 128 x 5120 x 5120 11.1 / 11.5; past that rule, 128 x 16384 x 4096 13.0 / 12.1, 256 x 16384 x 4096
// 18.1 / 12.9, 300 x 4096 x 4096 10.1 / 11.2.)
bool use_band(int64_t M, int64_t N, int sms) {
    return M <= 64 || ceil_div(M, 64) * ceil_div(N, ROWS) <= sms;
}

cudaError_t gemm(const Mxfp4Gemm &g, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = device_setup(&sms);
    if (e != cudaSuccess) return e;
    const int tiles_k = (int)ceil_div(g.K, kMxCols);
    const int last_mma = (int)ceil_div(g.K - (int64_t)(tiles_k - 1) * kMxCols, 64);
    if (use_band(g.M, g.N, sms))
        return g.M <= 16   ? band<16>(g, tiles_k, last_mma, sms, s)
               : g.M <= 32 ? band<32>(g, tiles_k, last_mma, sms, s)
                           : band<64>(g, tiles_k, last_mma, sms, s);
    Maps t;
    if (!make_maps(&t, g, ROWS)) return cudaErrorInvalidValue;
    // rows of Y on 16 bytes are stored by TMA
    CUtensorMap tmY;
    memset(&tmY, 0, sizeof(tmY));
    if (g.N % 8 == 0 && !make_map(&tmY, g.Y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, g.N, g.M, g.N, 32,
                                  32, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    PArgs a;
    a.bias = g.bias;
    a.Y = g.Y;
    a.status = g.status;
    a.M = (int)g.M;
    a.N = (int)g.N;
    a.tiles_k = tiles_k;
    a.last_mma = last_mma;
    a.tiles_m = (int)ceil_div(g.M, 2 * ROWS);
    a.tiles_n = (int)ceil_div(g.N, BN);
    a.timeout_ns = g.timeout_ns;
    const int pairs = std::min(a.tiles_m * a.tiles_n, sms / 2);
    auto k = g.dtype == kF16 ? mxfp4_pair_kernel<kF16> : mxfp4_pair_kernel<kBF16>;
    return launch_cluster(k, dim3((unsigned)(2 * pairs)), P_THREADS, P_SMEM, 2, s, t.X, t.W, t.XS,
                          t.WS, tmY, a);
}

}  // namespace

cudaError_t launch_mxfp4_gemm(const Mxfp4Gemm &g, cudaStream_t s) {
    const cudaError_t e = gemm(g, s);
    note_launches(1);
    return e;
}

}  // namespace llmint8
