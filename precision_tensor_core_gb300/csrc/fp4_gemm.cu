// fp4_gemm.cu -- product of two microscaled 4-bit matrices on the block-scaled
// tensor cores (gemm_fp4 of include/ptc.h):
//
//   C[i][j] = out( G_A G_B  sum_b  sA[i][b] sB[j][b]  sum_{k in block b} a[i][k] b[j][k] )
//
// tcgen05.mma kind::mxf4 (a power of two per 32 elements) or kind::mxf4nvf4
// (E4M3 per 16 elements) multiplies the E2M1 codes and the block scales
// exactly and accumulates in FP32 in tensor memory; the matrix scales and the
// output rounding are the epilogue's.
//
// Operands arrive by TMA as rows of 128 bytes (256 codes) in the 128-byte
// swizzle, with the scale tiles (512 bytes: 128 rows x 4 blocks) that belong
// to them.  The issuing thread copies a stage's scale tiles from shared memory
// into tensor memory (tcgen05.cp, replicated to the four lane quarters) and
// then issues the stage's four MMAs of 64 codes; copies and MMAs of one
// thread execute in order.  The copies cost nothing (8192^3 in mxfp4: 169 us
// with and without them); writing the scales by four more warps with
// tcgen05.st took 253 us, for the barriers between them and the issuer.
//
// Tiles.  Large products run on CTA pairs (256 x 256 per pair, cta_group::2):
// each CTA holds 128 rows of A, 128 rows of B and the scales of its A rows and
// of all 256 B rows.  The FP32 accumulators take 256 of the 512 tensor-memory
// columns, so two of them and the scales do not fit; the two buffers overlap
// by 64 columns ([0, 256) and [192, 448), scales from 448).  The epilogue
// drains the shared columns first and then lets the next tile's MMAs start.
// Small products run on 128 x 128 or 128 x 64 tiles of one CTA, whole or in
// clusters of up to eight CTAs that share a tile's K range and add their
// partial sums through distributed shared memory in rank order.
//
// Rates: 8192^3 155 us in mxfp4 (7.1 PFLOP/s) and 160 in nvfp4, bound by the
// delivery of operands into the SMs (14.8 TB/s; the MMAs alone take 140);
// 2048^3 8.4 us, where the start of the call, eight stages and the output
// each take a third; 512^3 3.2 us.
//
// Every wait is bounded: on expiry the CTA raises its abort flag, records the
// error word that gemm_poll_device_error reads, and every role runs out; the CTA
// exits when its MMAs have ended and its copies in flight have landed.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "fp4.cuh"
#include "fp4.h"
#include "internal.h"
#include "ptc.h"
#include "ptx.cuh"

namespace ptc {
namespace {

__device__ uint32_t g_fp4_error = 0;

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kStageK = 256;  // codes of K per stage: rows of 128 bytes
constexpr int kMmaK = 64;
constexpr size_t kMaxSmem = 227 * 1024;

struct Fp4Args {
    void *C;
    int64_t ldc;
    int out_type;
    int M, N;
    int num_kb;    // stages of kStageK codes
    int k_steps;   // MMAs of kMmaK codes in all
    int tiles_m, tiles_n, num_tiles, group_m;
    int ks;        // CTAs per cluster sharing a tile's K range (one-CTA tiles)
    int stages;    // stages of the ring (fewer where C is staged)
    int vec;       // C's base and pitch are multiples of: 2: 32 bytes, 1: 16 bytes, 0: neither
    const float *ga, *gb;
    int stall_tile;
    uint64_t wait_limit;
};

template <int CTAS, int BN, bool NV>
struct Cfg4 {
    static constexpr int B_ROWS = BN / CTAS;
    static constexpr int NBLK = (BN + 127) / 128;
    static constexpr int KAT = NV ? 4 : 2;  // scale tiles per stage and 128 rows
    static constexpr int A_BYTES = 128 * 128, B_BYTES = B_ROWS * 128;
    static constexpr int SFA_BYTES = KAT * kScaleTile, SFB_BYTES = NBLK * KAT * kScaleTile;
    static constexpr int SF_BYTES = SFA_BYTES + SFB_BYTES;
    static constexpr int STAGE = A_BYTES + B_BYTES + SF_BYTES;
    static constexpr int STAGES = std::min(8, int((kMaxSmem - 2048) / STAGE));
    // Tensor-memory columns: two accumulators, then the scales.
    static constexpr int ACC1 = CTAS == 2 ? 192 : BN;
    static constexpr int SFA_COL = CTAS == 2 ? 448 : 2 * BN;
    static constexpr int SFB_COL = SFA_COL + 4 * KAT;
    static constexpr int COLS_USED = SFB_COL + 4 * KAT * NBLK;
    static constexpr int TMEM_COLS = COLS_USED <= 256 ? 256 : 512;
    static_assert(COLS_USED <= 512, "accumulators and scales fit tensor memory");
    static constexpr size_t SMEM = size_t(STAGES) * STAGE + 2048;
    static constexpr int TURN_STAGES = (kEpiWarps * 32 * 33 * 4 + STAGE - 1) / STAGE;  // of the ring, where C is staged
    static_assert(STAGES - TURN_STAGES >= 3, "a ring remains");
    static_assert(size_t(STAGES) * STAGE >= 128 * BN * 4 || CTAS == 2, "a K-split partial tile fits the ring");
};

template <int STAGES>
struct Tail4 {
    uint64_t full[STAGES], empty[STAGES], acc_full, acc_free, drain;
    uint32_t tmem_base;
    AbortState abort;
};

// Instruction descriptor of kind::mxf4 / mxf4nvf4 (dense, K = 64): bits 4-5
// the quarter of B's 32-bit scale words in use, 7-9 and 10-11 E2M1 operands,
// 17-22 N >> 3, 23 scale type (1 UE8M0, 0 UE4M3), 27-28 M >> 7, 29-30 A's quarter.
__host__ __device__ constexpr uint32_t instr_desc_fp4(bool nv, int m, int n, uint32_t quarter) {
    return (quarter << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (nv ? 0u : 1u << 23) |
           (uint32_t(m >> 7) << 27) | (quarter << 29);
}

template <int CTAS, bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
#define PTC_MMA4(GROUP, KIND)                                                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                            \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"( \
                     d),                                                                                       \
                 "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                               \
                 : "memory")
    if constexpr (CTAS == 1 && NV)
        PTC_MMA4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (CTAS == 1)
        PTC_MMA4("1", "mxf4.block_scale.scale_vec::2X");
    else if constexpr (NV)
        PTC_MMA4("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else
        PTC_MMA4("2", "mxf4.block_scale.scale_vec::2X");
#undef PTC_MMA4
}

// Shared-memory descriptors as two words: the high word is a constant, the low
// word the address (in 16 bytes) and the leading offset, so that an operand
// costs the issuing thread one addition.  K-major rows of 128 bytes in the
// 128-byte swizzle (eight rows 1024 bytes apart), and unswizzled rows of 16
// bytes (eight rows 128 bytes apart) for scale tiles.
constexpr uint32_t kDescLow = 1u << 16;
constexpr uint32_t kDescHighSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHighRows16 = (128u >> 4) | (1u << 14);

__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return (saddr >> 4) | kDescLow; }
__device__ __forceinline__ uint64_t desc_of(uint32_t low, uint32_t high) { return (uint64_t(high) << 32) | low; }

// One scale tile (32 rows of 16 bytes in shared memory) to four tensor-memory
// columns of every lane quarter; a pair copies in both CTAs.
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t low) {
    const uint64_t d = desc_of(low, kDescHighRows16);
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// 3-D tiled load of scale tiles (word, tile along K, tile of 128 rows).
template <int CTAS>
__device__ __forceinline__ void load_scales(uint32_t dst, const CUtensorMap *map, uint32_t bar, int kt, int rt) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(kt), "r"(rt), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(kt), "r"(rt), "r"(bar)
            : "memory");
}

// Arrives on a barrier of the cluster without ordering this thread's earlier
// global stores before it: what it announces is that tensor-memory loads are
// complete (their values are in registers), and a release would wait for the
// output stores of the tile before.
__device__ __forceinline__ void arrive_relaxed_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tile_of(int t, const Fp4Args &a, int &mb, int &nb) {
    const int per_group = a.group_m * a.tiles_n;
    const int g = t / per_group;
    const int first = g * a.group_m;
    const int rows = min(a.tiles_m - first, a.group_m);
    const int r = t - g * per_group;
    mb = first + r % rows;
    nb = r / rows;
}

__device__ __forceinline__ void st_global_v8(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_out(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return reinterpret_cast<const uint32_t &>(v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(v);
}

// CNT (4 or 32) consecutive results of one row, `valid` of them below N.
template <int CNT>
__device__ __forceinline__ void store_row(const Fp4Args &a, int64_t at, const float (&v)[CNT], int valid) {
    if (a.out_type == PTC_OUT_F32) {
        float *dst = static_cast<float *>(a.C) + at;
        if (valid >= CNT && a.vec >= 1) {
            if (CNT >= 8 && a.vec == 2) {
#pragma unroll
                for (int i = 0; i < CNT / 8; ++i) st_global_v8(dst + 8 * i, reinterpret_cast<const uint32_t *>(v) + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < CNT / 4; ++i)
                    reinterpret_cast<float4 *>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < CNT; ++j)
                if (j < valid) dst[j] = v[j];
        }
    } else {
        uint16_t *dst = static_cast<uint16_t *>(a.C) + at;
        uint32_t w[CNT / 2];
#pragma unroll
        for (int j = 0; j < CNT / 2; ++j) w[j] = pack_out(v[2 * j], v[2 * j + 1], a.out_type == PTC_OUT_BF16);
        if (valid >= CNT && a.vec >= 1) {
            if constexpr (CNT == 4) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            } else if (a.vec == 2) {
#pragma unroll
                for (int i = 0; i < CNT / 16; ++i) st_global_v8(dst + 16 * i, w + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < CNT / 8; ++i)
                    reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < CNT; ++j)
                if (j < valid) dst[j] = uint16_t((j & 1) ? w[j / 2] >> 16 : w[j / 2]);
        }
    }
}

__device__ __forceinline__ void store_one(const Fp4Args &a, int64_t at, float v) {
    if (a.out_type == PTC_OUT_F32)
        static_cast<float *>(a.C)[at] = v;
    else if (a.out_type == PTC_OUT_BF16)
        static_cast<__nv_bfloat16 *>(a.C)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(a.C)[at] = __float2half_rn(v);
}

template <int CTAS, int BN, bool NV>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const Fp4Args args) {
    using C_ = Cfg4<CTAS, BN, NV>;
    constexpr int STAGES = C_::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    const uint32_t ring = raw_addr + pad;  // stages: A, B, scales of A, scales of B
    Tail4<STAGES> *st = reinterpret_cast<Tail4<STAGES> *>(smem_raw + pad + STAGES * C_::STAGE);
    const int nst = args.stages;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint64_t limit = args.wait_limit;
    const int cl = CTAS == 2 ? 2 : args.ks;  // CTAs per cluster
    const uint32_t crank = cl == 1 ? 0u : cluster_ctarank();
    const uint32_t rank = CTAS == 2 ? crank : 0u;
    const int krank = CTAS == 2 ? 0 : int(crank);
    const int cluster = int(blockIdx.x) / cl, nclusters = int(gridDim.x) / cl;
    // This CTA's stages of K.
    const int kq = args.num_kb / (CTAS == 2 ? 1 : args.ks), kr = args.num_kb % (CTAS == 2 ? 1 : args.ks);
    const int kb0 = krank * kq + min(krank, kr), kb1 = kb0 + kq + (krank < kr ? 1 : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&st->full[s], 1);
            mbar_init(&st->empty[s], 1);
        }
        mbar_init(&st->acc_full, 1);
        mbar_init(&st->acc_free, kEpiWarps * CTAS);
        mbar_init(&st->drain, 1);
        st->abort.flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc<CTAS>(&st->tmem_base, C_::TMEM_COLS);
        tmem_relinquish<CTAS>();
    }
    tc_fence_before_sync();
    if constexpr (CTAS == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = st->tmem_base;
    griddep_wait();
    griddep_launch_dependents();

    uint32_t loaded = 0, loaded_phase = 0;  // producer: stages that hold or await a load, the phase of each
    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = cluster; t < args.num_tiles && ok; t += nclusters) {
                int mb, nb;
                tile_of(t, args, mb, nb);
                const int m0 = (mb * CTAS + int(rank)) * 128, n0 = nb * BN;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&st->empty[s], ph ^ 1u, &st->abort, &g_fp4_error, limit)) {
                        ok = false;
                        break;
                    }
                    if (!(t == args.stall_tile && kb == kb0 && rank == 0)) {
                        const uint32_t a = ring + s * C_::STAGE, b = a + C_::A_BYTES, sa = b + C_::B_BYTES;
                        uint8_t *ap = smem_raw + (a - raw_addr), *bp = smem_raw + (b - raw_addr);
                        if constexpr (CTAS == 1) {
                            mbar_arrive_expect_tx(&st->full[s], C_::STAGE);
                            tma_load_2d(ap, &tmA, &st->full[s], kb * 128, m0);
                            tma_load_2d(bp, &tmB, &st->full[s], kb * 128, n0);
                            load_scales<1>(sa, &tmSA, smem_u32(&st->full[s]), kb * C_::KAT, m0 / 128);
                            load_scales<1>(sa + C_::SFA_BYTES, &tmSB, smem_u32(&st->full[s]), kb * C_::KAT, n0 / 128);
                        } else {
                            if (rank == 0) mbar_arrive_expect_tx(&st->full[s], 2 * C_::STAGE);
                            const uint32_t bar = mapa_shared(smem_u32(&st->full[s]), 0);
                            tma_load_2d_pair(ap, &tmA, bar, kb * 128, m0);
                            tma_load_2d_pair(bp, &tmB, bar, kb * 128, n0 + int(rank) * C_::B_ROWS);
                            load_scales<2>(sa, &tmSA, bar, kb * C_::KAT, m0 / 128);
                            load_scales<2>(sa + C_::SFA_BYTES, &tmSB, bar, kb * C_::KAT, n0 / 128);
                        }
                        loaded |= 1u << s;
                        loaded_phase = (loaded_phase & ~(1u << s)) | (ph << s);
                    } else {
                        loaded &= ~(1u << s);
                    }
                    if (++s == nst) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        // The whole warp walks the stages and one elected lane issues, so that
        // addresses and descriptors stay uniform over the warp.  (Issued by
        // lane 0 in a branch of its own, every copy and MMA took about 45
        // clocks to issue: 8192^3 in mxfp4 took 237 us, in nvfp4 302 us.)
        if (rank == 0) {
            int s = 0, n = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = cluster; t < args.num_tiles && ok; t += nclusters, ++n) {
                int mb, nb;
                tile_of(t, args, mb, nb);
                if (n > 0)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st->acc_free, uint32_t(n - 1) & 1u, &st->abort, &g_fp4_error, limit));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem + ((n & 1) ? C_::ACC1 : 0);
                // A 64-column tile starts in the middle of a 128-row scale tile
                // when nb is odd: 64 rows are two 32-bit scale columns.
                const uint32_t sfa = tmem + C_::SFA_COL;
                const uint32_t sfb = tmem + C_::SFB_COL + (BN == 64 ? uint32_t(nb & 1) * 2u : 0u);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st->full[s], ph, &st->abort, &g_fp4_error, limit));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t a = desc_low(ring + s * C_::STAGE), b = a + C_::A_BYTES / 16;
                    const uint32_t sa = b + C_::B_BYTES / 16, sb = sa + C_::SFA_BYTES / 16;
                    const int steps = args.k_steps - kb * 4;  // of this stage: past K there is nothing
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < C_::KAT; ++j) {
                            copy_scales<CTAS>(tmem + C_::SFA_COL + 4 * j, sa + j * (kScaleTile / 16));
#pragma unroll
                            for (int q = 0; q < C_::NBLK; ++q)
                                copy_scales<CTAS>(tmem + C_::SFB_COL + 4 * (j * C_::NBLK + q),
                                                  sb + (q * C_::KAT + j) * (kScaleTile / 16));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k < steps) {
                                const int j = NV ? k : k / 2;  // scale tile of these 64 codes
                                const uint32_t idesc = instr_desc_fp4(NV, 128 * CTAS, BN, (!NV && (k & 1)) ? 2 : 0);
                                mma_fp4<CTAS, NV>(d, desc_of(a + 2 * k, kDescHighSw128), desc_of(b + 2 * k, kDescHighSw128),
                                                  idesc, sfa + 4 * j, sfb + 4 * (j * C_::NBLK), (kb > kb0 || k > 0) ? 1u : 0u);
                            }
                        }
                        if constexpr (CTAS == 1)
                            mma_commit<1>(&st->empty[s]);
                        else
                            mma_commit_pair(&st->empty[s], 3);
                        if (kb + 1 == kb1) {
                            if constexpr (CTAS == 1)
                                mma_commit<1>(&st->acc_full);
                            else
                                mma_commit_pair(&st->acc_full, 3);
                        }
                    }
                    __syncwarp();
                    if (++s == nst) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // The MMAs issued so far end before tensor memory is freed, also where it is
            // the epilogue that gave up.
            if (ok) {
                if (n > 0) mbar_wait(&st->acc_full, uint32_t(n - 1) & 1u, nullptr, nullptr, limit);
            } else {
                if (elect_one()) {
                    mma_commit<CTAS>(&st->drain);
                    mbar_wait(&st->drain, 0, nullptr, nullptr, limit);
                }
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------- epilogue
        const int ew = warp - 2, q = warp & 3, h = ew >> 2;
        // Rows that are not 16-byte aligned leave through the end of the ring.
        float *turn = reinterpret_cast<float *>(smem_raw + pad + nst * C_::STAGE) + ew * (32 * 33);
        constexpr int NCH = BN / 64;  // 32-column chunks per warp
        const float alpha = __fmul_rn(args.ga ? __ldg(args.ga) : 1.0f, args.gb ? __ldg(args.gb) : 1.0f);
        int n = 0;
        for (int t = cluster; t < args.num_tiles; t += nclusters, ++n) {
            int mb, nb;
            tile_of(t, args, mb, nb);
            const bool got = mbar_wait(&st->acc_full, uint32_t(n) & 1u, &st->abort, &g_fp4_error, limit);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + ((n & 1) ? C_::ACC1 : 0) + (uint32_t(32 * q) << 16);
            const int lrow = 32 * q + lane, row = (mb * CTAS + int(rank)) * 128 + lrow;
#pragma unroll 1
            for (int i = 0; i < NCH; ++i) {
                // The columns that the other buffer shares come first: this
                // tile's last 64 in the even buffer, its first 64 in the odd one.
                const int c = (CTAS == 2 && !(n & 1)) ? 2 * NCH - 1 - (2 * i + h) : 2 * i + h;
                uint32_t r[32];
                tmem_ld_32cols(acc + 32 * c, r);
                tmem_ld_wait();
                if (i == 0) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (CTAS == 1 || rank == 0)
                            mbar_arrive(&st->acc_free);
                        else
                            arrive_relaxed_cluster(mapa_shared(smem_u32(&st->acc_free), 0));
                    }
                }
                const int col = nb * BN + 32 * c;
                if (CTAS == 1 && args.ks > 1) {
                    // Partial sums to the idle ring: rows of BN floats, 16-byte
                    // pieces exchanged within groups of eight by the row.
                    if (row < args.M) {
                        const uint32_t base = ring + uint32_t(lrow) * (BN * 4);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared_v4(base + (uint32_t((8 * c + j) ^ (lrow & 7)) << 4), r[4 * j], r[4 * j + 1],
                                         r[4 * j + 2], r[4 * j + 3]);
                    }
                } else if (args.vec == 0) {
                    // A lane per row would write 32 scattered elements at a time;
                    // turned around, the warp writes 32 columns of one row.
#pragma unroll
                    for (int j = 0; j < 32; ++j) turn[lane * 33 + j] = __fmul_rn(__uint_as_float(r[j]), alpha);
                    __syncwarp();
                    const int first = row - lane, rows = min(32, args.M - first);
                    if (col + lane < args.N) {
                        int64_t at = int64_t(first) * args.ldc + col + lane;
#pragma unroll 4
                        for (int i2 = 0; i2 < rows; ++i2, at += args.ldc) store_one(args, at, turn[i2 * 33 + lane]);
                    }
                    __syncwarp();
                } else if (row < args.M && col < args.N) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(__uint_as_float(r[j]), alpha);
                    store_row<32>(args, int64_t(row) * args.ldc + col, v, args.N - col);
                }
            }
        }
        __syncwarp();
    }

    if (CTAS == 1 && args.ks > 1) {
        cluster_sync();
        // This CTA's share of the tile's pieces of four outputs: the partial
        // sums of all ranks, added in rank order.
        int mb, nb;
        tile_of(cluster, args, mb, nb);
        const float alpha = __fmul_rn(args.ga ? __ldg(args.ga) : 1.0f, args.gb ? __ldg(args.gb) : 1.0f);
        const int rows = min(128, args.M - mb * 128);
        for (int p = krank * kThreads + int(threadIdx.x); p < rows * (BN / 4); p += args.ks * kThreads) {
            const int lrow = p / (BN / 4), piece = p % (BN / 4);
            const uint32_t at = ring + uint32_t(lrow) * (BN * 4) + (uint32_t(piece ^ (lrow & 7)) << 4);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < args.ks; ++k) {
                const uint4 x = ld_shared_cluster_v4(mapa_shared(at, uint32_t(k)));
                v[0] = __fadd_rn(v[0], __uint_as_float(x.x));
                v[1] = __fadd_rn(v[1], __uint_as_float(x.y));
                v[2] = __fadd_rn(v[2], __uint_as_float(x.z));
                v[3] = __fadd_rn(v[3], __uint_as_float(x.w));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __fmul_rn(v[j], alpha);
            const int col = nb * BN + 4 * piece;
            if (col < args.N) store_row<4>(args, int64_t(mb * 128 + lrow) * args.ldc + col, v, args.N - col);
        }
        tc_fence_before_sync();
        cluster_sync();
        tc_fence_after_sync();
    } else {
        tc_fence_before_sync();
        if constexpr (CTAS == 2)
            cluster_sync();
        else
            __syncthreads();
        tc_fence_after_sync();
    }
    // Every role is done.  After an abort, of whichever role, copies in flight land
    // before the CTA exits: a pair's complete on the first CTA's barriers and get 200 us
    // (with one of its CTAs the other has given up too: its epilogue waits for the
    // same MMAs).
    if (warp == 0 && lane == 0 && st->abort.flag) {
        if constexpr (CTAS == 1) {
            for (int s = 0; s < STAGES; ++s)
                if (loaded >> s & 1u) mbar_wait(&st->full[s], loaded_phase >> s & 1u, nullptr, nullptr, limit);
        } else {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);
        }
    }
    if (warp == 1) tmem_dealloc<CTAS>(tmem, C_::TMEM_COLS);
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDim4 = int64_t(1) << 30;
constexpr int64_t kMaxLd4 = int64_t(1) << 36;
constexpr int kMaxDev = 64;

std::atomic<int> g_tile{0};    // "fp4_tile": 0 by size, 64, 128, 256 (CTA pairs)
std::atomic<int> g_split{0};   // "fp4_ksplit": 0 by size, 1, 2, 4, 8
std::atomic<int> g_raster{8};  // "fp4_group_m"

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape4 {
    int tile, ks;  // 256: CTA pairs
};

// The shape of least estimated time, in units of 0.01 us, fitted to every shape
// at 21 sizes (M 1 .. 2048, N 128 .. 16384, K 512 .. 8192): a call of 128 x 64
// tiles takes 2.6 us plus 0.25 us per stage and wave, of 128 x 128 tiles 3.4 and
// 0.27, of pairs 4.75 and 0.30; sharing K in a cluster costs 1.8 or 2.3 us and
// is taken where it saves a tenth.
Shape4 choose4(int64_t M, int64_t N, int num_kb, int sms) {
    const int tile = g_tile.load(), ks = g_split.load();
    const int64_t m128 = ceil_div(M, 128);
    Shape4 best{256, 1};
    int64_t best_cost = INT64_MAX;
    if (tile == 0 || tile == 256)
        best_cost = 475 + ceil_div(ceil_div(M, 256) * ceil_div(N, 256), sms / 2) * num_kb * 30;
    const ClusterCaps caps = cluster_caps(sms);
    for (int bn : {128, 64}) {
        if (tile != 0 && tile != bn) continue;
        const int64_t tiles = m128 * ceil_div(N, bn);
        for (int k : {1, 2, 4, 8}) {
            if ((ks != 0 && k != ks && k > 1) || num_kb < k) continue;
            if (ks == 0 && k > 1 && tiles > caps.of(k)) continue;  // one wave of clusters
            const int64_t waves = ceil_div(tiles * k, sms);
            int64_t cost = (bn == 64 ? 260 : 340) + waves * ceil_div(num_kb, k) * (bn == 64 ? 25 : 27);
            if (k > 1) cost = (cost + (bn == 64 ? 180 : 230)) * 11 / 10;
            if (k > 1 && k == ks) cost = tile == 0 ? cost : -1;  // asked for
            if (cost < best_cost) {
                best_cost = cost;
                best = {bn, k};
            }
        }
    }
    return best;
}

template <int CTAS, int BN, bool NV>
cudaError_t launch4(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &sa, const CUtensorMap &sb,
                    Fp4Args a, int sms, cudaStream_t stream) {
    using C_ = Cfg4<CTAS, BN, NV>;
    auto *fn = fp4_gemm_kernel<CTAS, BN, NV>;
    static std::atomic<int> clusters[kMaxDev];  // resident pairs + 1, once the kernel is set up
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C_::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    const int cl = CTAS == 2 ? 2 : a.ks;
    if (cl > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = unsigned(cl);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    int have = clusters[dev].load(std::memory_order_acquire);
    if (have == 0) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C_::SMEM));
        if (e != cudaSuccess) return e;
        have = sms;
        if constexpr (CTAS == 2) {
            cfg.gridDim = dim3(unsigned(sms / 2 * 2), 1, 1);
            e = cudaOccupancyMaxActiveClusters(&have, fn, &cfg);
            if (e != cudaSuccess) return e;
            if (have < 1) return cudaErrorInvalidConfiguration;
        }
        clusters[dev].store(have, std::memory_order_release);
    }
    if (pdl_enabled()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    a.stages = C_::STAGES - (a.vec == 0 && a.ks == 1 ? C_::TURN_STAGES : 0);
    // K-split clusters take one tile each; the others walk the tiles.
    const int units = a.ks > 1 ? a.num_tiles : std::min(a.num_tiles, have);
    cfg.gridDim = dim3(unsigned(units * cl), 1, 1);
    e = cudaLaunchKernelEx(&cfg, fn, ta, tb, sa, sb, a);
    if (e == cudaSuccess) {
        note_launches(1);
        note_fp4_launch(cfg.gridDim.x, cl, CTAS == 2 ? 1 : a.ks, BN);
    }
    return e;
}

}  // namespace

cudaError_t read_and_clear_fp4_error_word(uint32_t *out) {
    uint32_t v = 0;
    const uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_error, sizeof(v));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_fp4_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

bool set_fp4_tuning(const char *key, int64_t v) {
    if (std::strcmp(key, "fp4_tile") == 0 && (v == 0 || v == 64 || v == 128 || v == 256)) {
        g_tile.store(int(v));
        return true;
    }
    if (std::strcmp(key, "fp4_ksplit") == 0 && (v == 0 || v == 1 || v == 2 || v == 4 || v == 8)) {
        g_split.store(int(v));
        return true;
    }
    if (std::strcmp(key, "fp4_group_m") == 0 && v > 0 && v < (1 << 20)) {
        g_raster.store(int(v));
        return true;
    }
    return false;
}

}  // namespace ptc

using namespace ptc;

extern "C" int gemm_fp4(int64_t M, int64_t N, int64_t K, int format, const void *A, int64_t lda, const void *SA,
                        const float *GA, const void *B, int64_t ldb, const void *SB, const float *GB, void *C,
                        int64_t ldc, int out_type, void *stream) {
    set_message("");
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim4 || N > kMaxDim4 || K > kMaxDim4)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= M, N, K <= 2^30");
    if (ceil_div(M, 128) * ceil_div(N, 64) >= (int64_t(1) << 31))
        return fail_status(PTC_ERR_INVALID, "too many output tiles");
    if (format != PTC_FP4_MX && format != PTC_FP4_NV) return fail_status(PTC_ERR_INVALID, "unknown 4-bit format");
    if (out_type != PTC_OUT_F32 && out_type != PTC_OUT_BF16 && out_type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "unknown output type");
    if (M == 0 || N == 0) return PTC_OK;
    const bool nv = format == PTC_FP4_NV;
    const int es = out_type == PTC_OUT_F32 ? 4 : 2;
    if (!C || ldc < N || ldc > kMaxLd4) return fail_status(PTC_ERR_INVALID, "C is NULL, or ldc is not N .. 2^36");
    int rc;
    if (K > 0 && ((rc = check_fp4(A, lda, SA, GA, K, nv)) || (rc = check_fp4(B, ldb, SB, GB, K, nv)))) return rc;
    if (reinterpret_cast<uintptr_t>(C) % es) return fail_status(PTC_ERR_ALIGN, "C must be aligned to its element");
    const ByteRows c = elem_rows(C, M, N, ldc, es);
    if (K > 0 && (rows_overlap(c, fp4_code_rows(A, M, K, lda)) || rows_overlap(c, fp4_code_rows(B, N, K, ldb)) ||
                  rows_overlap(c, fp4_scale_rows(SA, M, K, nv)) || rows_overlap(c, fp4_scale_rows(SB, N, K, nv)) ||
                  rows_overlap(c, flat_bytes(GA, 4)) || rows_overlap(c, flat_bytes(GB, 4))))
        return fail_status(PTC_ERR_OVERLAP, "C overlaps an operand");
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const cudaError_t e = launch_zero_fill(C, ldc, int(M), int(N), es, sms * 4, s);
        if (e != cudaSuccess) return fail_launch(e, "zero-fill launch");
        note_launches(1);
        return PTC_OK;
    }
    Fp4Args a;
    std::memset(&a, 0, sizeof(a));
    a.C = C;
    a.ldc = ldc;
    a.out_type = out_type;
    a.M = int(M);
    a.N = int(N);
    const int64_t kp = ceil_div(K, 32) * 32;  // codes per row, zeros past K
    a.num_kb = int(ceil_div(kp, kStageK));
    a.k_steps = int(ceil_div(kp, kMmaK));
    const Shape4 sh = choose4(M, N, a.num_kb, sms);
    const int ctas = sh.tile == 256 ? 2 : 1, bn = sh.tile;
    a.tiles_m = int(ceil_div(M, 128 * ctas));
    a.tiles_n = int(ceil_div(N, bn));
    a.num_tiles = a.tiles_m * a.tiles_n;
    a.group_m = std::min(g_raster.load(), a.tiles_m);
    a.ks = sh.ks;
    const uintptr_t at = reinterpret_cast<uintptr_t>(C);
    a.vec = (at % 32 == 0 && ldc * es % 32 == 0) ? 2 : (at % 16 == 0 && ldc * es % 16 == 0) ? 1 : 0;
    a.ga = GA;
    a.gb = GB;
    a.stall_tile = take_stall_tile();
    a.wait_limit = wait_limit_ns();
    const int64_t blocks = ceil_div(K, nv ? 16 : 32), ktiles = ceil_div(blocks, 4);
    CUtensorMap ta, tb, sa, sb;
    if ((rc = encode_tmap_2d(&ta, true, A, uint64_t(kp / 2), uint64_t(M), uint64_t(lda), 128, 128)) ||
        (rc = encode_tmap_2d(&tb, true, B, uint64_t(kp / 2), uint64_t(N), uint64_t(ldb), 128, uint32_t(bn / ctas))) ||
        (rc = encode_tmap_scales(&sa, SA, uint64_t(ktiles), uint64_t(ceil_div(M, 128)), nv ? 4 : 2, 1)) ||
        (rc = encode_tmap_scales(&sb, SB, uint64_t(ktiles), uint64_t(ceil_div(N, 128)), nv ? 4 : 2, bn == 256 ? 2 : 1)))
        return rc;
    cudaError_t e;
    if (bn == 256)
        e = nv ? launch4<2, 256, true>(ta, tb, sa, sb, a, sms, s) : launch4<2, 256, false>(ta, tb, sa, sb, a, sms, s);
    else if (bn == 128)
        e = nv ? launch4<1, 128, true>(ta, tb, sa, sb, a, sms, s) : launch4<1, 128, false>(ta, tb, sa, sb, a, sms, s);
    else
        e = nv ? launch4<1, 64, true>(ta, tb, sa, sb, a, sms, s) : launch4<1, 64, false>(ta, tb, sa, sb, a, sms, s);
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "4-bit product launch");
}
