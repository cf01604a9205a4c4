// fp4_tokens.cu -- product of a few rows of 16-bit activations with a
// microscaled 4-bit matrix (gemm_a16_fp4 of include/ptc.h), the form a
// decoding step takes:
//
//   C[i][j] = out( G  sum_k x[i][k] (w[j][k] s[j][k / block]) )
//
// The weights are read once and bound the call: 0.53 or 0.56 bytes each, at
// the HBM rate some 12 T weights per second, so every instruction per weight
// counts.  The products run on mma.sync m16n8k16 with the weights as the
// 16-row operand and eight tokens as the columns; the sums stay in FP32.
//
// Layout.  The eight warps of a CTA are R row groups x S shares of K; a warp
// owns 16 rows of a 128-row scale tile.  A ninth warp brings the weights of
// each share to shared memory by TMA, 256 codes (128 bytes of each of the
// share's 16 R rows) and their scales per stage, kStages stages deep: whole
// 128-byte lines, many of them in flight, at no cost in registers.  The order
// of k within an MMA is free as long as both operands agree: of the 16 bytes of
// a row's block of 32 codes lane t of a quad takes word t (eight codes), and two
// MMAs multiply codes 0 .. 3 and 4 .. 7 of the four words with the same eight
// activations, 16 contiguous bytes of x, so that a pair of MMAs covers one
// block.  The activations of a chunk of stages lie in shared memory too (two
// buffers, filled by asynchronous copies).  Few tokens take R = 1, S = 8: many
// CTAs without a cluster, each reading all of x; many take R = 8, so that x is
// read once per 128 rows.
//
// Arithmetic.  A code becomes binary16 exactly, by one instruction per two.
// nvfp4 codes are multiplied by their E4M3 scale, still exactly (six
// significant bits within 2^-10 .. 2688).  mxfp4 scales exceed binary16, so
// each block's FP32 partial sum is multiplied by its row's scale instead.
// bfloat16 activations become binary16 relative to a power of two per token
// and block of 32, which brings the block's largest to [2^15, 2^16) and
// multiplies the block's partial sum: exact for elements down to 2^-32 of the
// largest, off by at most 2^-40 of the largest below that.  (bfloat16 MMAs
// need no such step, but take three more integer instructions per two weights:
// 16.8 us instead of 12.2 for one token and 8192 x 8192 mxfp4 weights.)  A block of
// codes times bfloat16's largest values lies beyond FP32 before its mxfp4 scale
// brings it back, so with those the sums are held 2^-8 times their size: the
// powers of two carry the factor, and the output's rounding takes it out.  At
// that size bfloat16's smallest number times the smallest code is still 2^-142,
// which FP32 holds.
//
// The partial sums of the S shares are added in order in shared memory; where
// that leaves SMs idle K is also shared by a cluster of up to eight CTAs, whose
// sums are added in rank order through distributed shared memory.
//
// Rates (weights from HBM): one token 6.1 us with 4096 x 4096 mxfp4 weights and
// 20 us with 16384 x 8192 (3.5 TB/s); 16 binary16 tokens 28 us with 16384 x 8192
// nvfp4 (2.7 TB/s, bound by the instructions per weight), 16 bfloat16 tokens 42.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "fp4.cuh"
#include "fp4.h"
#include "internal.h"
#include "ptc.h"
#include "ptx.cuh"

namespace ptc {
namespace {

constexpr int kWarps = 8, kTokThreads = 32 * (kWarps + 1);
constexpr int kGroup = 256;     // codes per stage
constexpr int kPieceBytes = 2 * kGroup;  // one token's activations of a stage
constexpr int kStages = 3;
constexpr int kCodeBytes = 128 * 128;    // codes of a stage, all shares

__device__ uint32_t g_tok_error = 0;

struct TokArgs {
    const void *x;
    int64_t ldx;
    const float *g;
    void *C;
    int64_t ldc;
    int M, N, K;
    int groups;          // stages of 256 codes in K
    int chunk;           // stages of each K share held in a buffer of activations
    int r_log2;          // log2 of the row groups per CTA
    int ks;              // CTAs per cluster
    int xvec;
    int stall;           // test hook: this CTA's weights never arrive (-1: none)
    uint64_t wait_limit;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two E4M3 bytes as binary16, each in both halves of a word.
__device__ __forceinline__ void scales_nv(uint32_t two, uint32_t &lo, uint32_t &hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
    lo = __byte_perm(h, 0, 0x1010);
    hi = __byte_perm(h, 0, 0x3232);
}

// Two power-of-two scale bytes as FP32 (0xFF: NaN).
__device__ __forceinline__ void scales_mx(uint32_t two, float &lo, float &hi) {
    uint32_t b;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"(uint16_t(two)));
    lo = __uint_as_float(b << 16);
    hi = __uint_as_float(b & 0xFFFF0000u);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 2-D box of 128-byte rows of codes, and of scale words (word, tile along K,
// tile of 128 rows).
__device__ __forceinline__ void load_scale_box(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int word, int kt, int rt) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(word), "r"(kt), "r"(rt), "r"(smem_u32(bar))
        : "memory");
}

// mxfp4 with bfloat16 tokens: the sums' size.  A block's sum of 32 codes of at most 6
// and activations below 2^16 is below 2^24, its power of two at most 2^112.
constexpr float kSumSize = 0x1p-8f;

struct TokTail {
    uint64_t full[kWarps][kStages], empty[kWarps][kStages];  // per share
    AbortState abort;
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// Row i (0 .. 15) of row group rg's MMAs: quarter q of the 128-row tile and row l
// of the CTA's 4 R rows there.  With R = 1 four rows of each quarter; otherwise
// eight rows of two quarters, so that the eight rows read together differ in
// the swizzle.
__device__ __forceinline__ void mma_row(int r_log2, int rg, int i, int &q, int &l) {
    if (r_log2 == 0) {
        q = i >> 2;
        l = i & 3;
    } else {
        q = 2 * (rg & 1) + (i >> 3);
        l = 8 * (rg >> 1) + (i & 7);
    }
}

template <bool NV, bool BF16, int NT>
__global__ void __launch_bounds__(kTokThreads, 2)
    tokens_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS, const TokArgs a) {
    constexpr int TOK = 8 * NT;
    constexpr int KAT = NV ? 4 : 2;                    // scale tiles per stage
    constexpr int STAGE = kCodeBytes + 512 * KAT;      // of all shares
    using X = typename ElemOf<BF16 ? Elem::BF16 : Elem::F16>::type;
    extern __shared__ uint8_t smem_raw[];
    // [stage]: codes [share][row], scales [share]; then activations
    // [buffer][share][token][stage] and, for bfloat16, their powers of two
    // [share][stage][block][token]; partial sums take the activations' place.
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *xs_base = smem + kStages * STAGE;
    __shared__ TokTail st;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int krank = a.ks == 1 ? 0 : int(cluster_ctarank());
    const int R = 1 << a.r_log2, S = kWarps >> a.r_log2;
    const int unit = int(blockIdx.x) / a.ks;                            // S units per 128 rows
    const int row0 = unit / S * 128, rg0 = unit % S * R;                // tile, first row group
    const int tok0 = int(blockIdx.y) * TOK;
    const int ntok = min(TOK, a.M - tok0);
    // This CTA's stages of K, then a share's: even shares, the first ones a stage longer.
    auto range = [](int first, int n, int parts, int i, int &lo, int &hi) {
        const int q = n / parts, r = n % parts;
        lo = first + i * q + min(i, r);
        hi = lo + q + (i < r ? 1 : 0);
    };
    int c0, c1;
    range(0, a.groups, a.ks, krank, c0, c1);
    const int longest = (c1 - c0 + S - 1) / S;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s)
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&st.full[s][i], 1);
                mbar_init(&st.empty[s][i], uint32_t(R));
            }
        st.abort.flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmS);
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

    int loaded = 0;  // stages that this lane of the ninth warp has asked for
    if (warp == kWarps) {
        // ---------------------------------------------------------- weights
        // Lane 4 s + q brings the 4 R rows 32 q + 4 rg0 .. of share s, lane
        // 4 s its scales too.
        const int sh = lane >> 2, q = lane & 3;
        int lo = 0, hi = 0;
        if (sh < S) range(c0, c1 - c0, S, sh, lo, hi);
        const uint32_t code_at = uint32_t(sh) * (16 * R * 128) + uint32_t(q) * (4 * R * 128);
        const uint32_t scale_at = kCodeBytes + uint32_t(sh) * (64 * R * KAT);
        bool ok = true;
        for (int i = 0; i < longest; ++i) {
            const int slot = i % kStages;
            if (ok && lo + i < hi) {
                ok = mbar_wait(&st.empty[sh][slot], uint32_t(i / kStages + 1) & 1u, &st.abort, &g_tok_error, a.wait_limit);
                if (ok && int(blockIdx.x) != a.stall) {
                    uint64_t *bar = &st.full[sh][slot];
                    uint8_t *stage = smem + slot * STAGE;
                    if (q == 0) {
                        mbar_arrive_expect_tx(bar, uint32_t(16 * R * 128 + 64 * R * KAT));
                        load_scale_box(smem_u32(stage) + scale_at, &tmS, bar, 16 * rg0, (lo + i) * KAT, row0 / 128);
                    }
                    tma_load_2d(stage + code_at, &tmW, bar, (lo + i) * 128, row0 + 32 * q + 4 * rg0);
                    loaded = i + 1;
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- products
        const int gr = lane >> 2, t = lane & 3;
        const int rg = warp & (R - 1), share = warp >> a.r_log2;
        int g0, g1;
        range(c0, c1 - c0, S, share, g0, g1);
        const uint32_t tok_bytes = uint32_t(a.chunk) * kPieceBytes, share_bytes = tok_bytes * uint32_t(ntok);
        const uint32_t pow_share = uint32_t(a.chunk) * (8 * TOK * 4);  // bytes of a share's powers of two
        const uint32_t pow_at = share_bytes * uint32_t(S), buf_bytes = pow_at + (BF16 ? pow_share * uint32_t(S) : 0u);
        // MMA rows gr and gr + 8 of this warp in the boxes of its share (see
        // mma_row): their codes, word t of each 16-byte piece in the 128-byte
        // swizzle, and their scale words.
        int q0, l0, q1, l1;
        mma_row(a.r_log2, rg, gr, q0, l0);
        mma_row(a.r_log2, rg, gr + 8, q1, l1);
        const uint32_t row_a = uint32_t(share) * (16 * R * 128) + uint32_t(q0 * 4 * R + l0) * 128u;
        const uint32_t row_b = uint32_t(share) * (16 * R * 128) + uint32_t(q1 * 4 * R + l1) * 128u;
        const uint32_t code_a = row_a + (((row_a >> 7) & 7u) << 4) + 4u * t;
        const uint32_t code_b = row_b + (((row_b >> 7) & 7u) << 4) + 4u * t;
        const uint32_t share_scale = kCodeBytes + uint32_t(share) * (64 * R * KAT);
        const uint32_t scale_a = share_scale + uint32_t(l0) * 16u + uint32_t(q0) * 4u;
        const uint32_t scale_b = share_scale + uint32_t(l1) * 16u + uint32_t(q1) * 4u;
        const uint32_t nv_pick = t < 2 ? 0x4420u : 0x4431u;  // this lane's half of a 32-code block: bytes 0, 2 or 1, 3
        // 16-byte piece 4 b + t (block b) of a token's stage lies at 4 (b ^ (token & 1)) + t.
        // (Tokens past the last read it again; their sums are dropped.)
        // Even blocks from x_at[n][0], odd ones from x_at[n][1], 128 bytes apart.
        uint32_t x_at[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int tok = min(8 * n + gr, ntok - 1);
            x_at[n][0] = uint32_t(share) * share_bytes + uint32_t(tok) * tok_bytes + (uint32_t(tok & 1) << 6) + uint32_t(t) * 16u;
            x_at[n][1] = x_at[n][0] ^ 64u;
        }
        // The activations of chunk `c` of every share: f(shared-memory offset of the
        // piece in buffer c & 1, offset of its block's power of two, source, valid
        // elements).  A warp takes a token's row of one share at a time, a lane a
        // piece, four consecutive lanes a block; every thread sees the same pieces
        // in each call.
        auto each_piece = [&](int c, auto f) {
            for (int line = warp; line < S * ntok; line += kWarps) {
                const int sh = line / ntok, tok = line - sh * ntok;
                int lo, hi;
                range(c0, c1 - c0, S, sh, lo, hi);
                lo += c * a.chunk;
                const int pieces = (min(hi, lo + a.chunk) - lo) * (kGroup / 8);  // a multiple of 32
                const X *row = static_cast<const X *>(a.x) + int64_t(tok0 + tok) * a.ldx + int64_t(lo) * kGroup;
                const uint32_t buf = uint32_t(c & 1) * buf_bytes;
                const uint32_t to = buf + uint32_t(sh) * share_bytes + uint32_t(tok) * tok_bytes;
                const uint32_t pw = buf + pow_at + uint32_t(sh) * pow_share + uint32_t(tok) * 4u;
                const int valid = int(min(int64_t(pieces) * 8, int64_t(a.K) - int64_t(lo) * kGroup));  // elements
                for (int p = lane; p < pieces; p += 32)
                    f(to + (uint32_t(p ^ ((tok & 1) << 2)) << 4), pw + uint32_t(p >> 2) * (TOK * 4), row + 8 * p,
                      min(8, valid - 8 * p));
            }
        };
        // Copies of chunk c into its buffer; zeros past K.
        auto stage_x = [&](int c) {
            each_piece(c, [&](uint32_t dst, uint32_t, const X *src, int n) {
                if (a.xvec != 0 && n >= 8) {
                    cp_async16(smem_u32(xs_base) + dst, src);
                } else {
                    const Pack8<X> v = load8(n > 0 ? src : static_cast<const X *>(a.x), n, false);
                    *reinterpret_cast<uint4 *>(xs_base + dst) = v.v[0];
                }
            });
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // bfloat16 pieces that this thread copied to binary16, in place.
        auto convert_x = [&](int c) {
            each_piece(c, [&](uint32_t dst, uint32_t pw, const X *, int) {
                Pack8<__nv_bfloat16> v;
                v.v[0] = *reinterpret_cast<const uint4 *>(xs_base + dst);
                uint32_t m = 0;  // largest finite magnitude, as FP32 bits
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = __float_as_uint(to_float(v.get(j))) & 0x7FFFFFFFu;
                    m = max(m, u < kInfBits ? u : 0u);
                }
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const int e = max(int(m >> 23) - 127 - 15, -126);  // (the largest: 65280 of binary16's 65504)
                const float down = __uint_as_float(uint32_t(127 - e) << 23);
                Pack8<__half> h;
#pragma unroll
                for (int j = 0; j < 8; ++j) h.set(j, __float2half_rn(__fmul_rn(to_float(v.get(j)), down)));
                *reinterpret_cast<uint4 *>(xs_base + dst) = h.v[0];
                if (t == 0)
                    *reinterpret_cast<float *>(xs_base + pw) =
                        __fmul_rn(__uint_as_float(uint32_t(127 + e) << 23), NV ? 1.0f : kSumSize);
            });
        };

        stage_x(0);
        int slot = 0;
        uint32_t ph = 0;
        for (int c = 0; c * a.chunk < longest; ++c) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if constexpr (BF16) convert_x(c);
            consumers_sync();  // chunk c is there, and everyone is done with the buffer of chunk c + 1
            if ((c + 1) * a.chunk < longest) stage_x(c + 1);
            const uint8_t *xs = xs_base + uint32_t(c & 1) * buf_bytes;
            const uint8_t *pw = xs + pow_at + uint32_t(share) * pow_share + uint32_t(t) * 8u;
            const int end = min(g1, g0 + (c + 1) * a.chunk);
            for (int g = g0 + c * a.chunk; g < end; ++g, xs += kPieceBytes, pw += 8 * TOK * 4) {
                // (After an abort the waits return at once and the sums are not used.)
                mbar_wait(&st.full[share][slot], ph, &st.abort, &g_tok_error, a.wait_limit);
                __syncwarp();
                const uint8_t *stage = smem + slot * STAGE;
#pragma unroll
                for (int i = 0; i < KAT; ++i) {  // a scale tile: two blocks of 32 (nvfp4) or four (mxfp4)
                    const uint32_t qa = *reinterpret_cast<const uint32_t *>(stage + scale_a + uint32_t(i) * (64 * R));
                    const uint32_t qb = *reinterpret_cast<const uint32_t *>(stage + scale_b + uint32_t(i) * (64 * R));
                    constexpr int BPT = NV ? 2 : 4;
                    uint32_t na[2], nb[2];
                    float fa[4], fb[4];
                    if constexpr (NV) {
                        scales_nv(__byte_perm(qa, 0, nv_pick), na[0], na[1]);
                        scales_nv(__byte_perm(qb, 0, nv_pick), nb[0], nb[1]);
                    } else {
                        scales_mx(qa, fa[0], fa[1]);
                        scales_mx(qa >> 16, fa[2], fa[3]);
                        scales_mx(qb, fb[0], fb[1]);
                        scales_mx(qb >> 16, fb[2], fb[3]);
                    }
#pragma unroll
                    for (int j = 0; j < BPT; ++j) {
                        const int b = i * BPT + j;
                        uint32_t va[4], vb[4];
                        codes_to_f16(*reinterpret_cast<const uint32_t *>(stage + (code_a ^ (uint32_t(b) << 4))), va);
                        codes_to_f16(*reinterpret_cast<const uint32_t *>(stage + (code_b ^ (uint32_t(b) << 4))), vb);
                        if constexpr (NV) {
#pragma unroll
                            for (int i2 = 0; i2 < 4; ++i2) {
                                va[i2] = mul_f16x2(va[i2], na[j]);
                                vb[i2] = mul_f16x2(vb[i2], nb[j]);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(xs + x_at[n][b & 1] + (b >> 1) * 128);
                            if constexpr (NV && !BF16) {
                                mma16816(acc[n], va[0], vb[0], va[1], vb[1], x.x, x.y, acc[n]);
                                mma16816(acc[n], va[2], vb[2], va[3], vb[3], x.z, x.w, acc[n]);
                            } else {
                                const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                float s[4];
                                mma16816(s, va[0], vb[0], va[1], vb[1], x.x, x.y, zero);
                                mma16816(s, va[2], vb[2], va[3], vb[3], x.z, x.w, s);
                                if constexpr (BF16) {  // the two tokens' powers of two
                                    const float2 p = *reinterpret_cast<const float2 *>(pw + (b * TOK + 8 * n) * 4);
                                    if constexpr (NV) {
                                        acc[n][0] = __fmaf_rn(s[0], p.x, acc[n][0]);
                                        acc[n][1] = __fmaf_rn(s[1], p.y, acc[n][1]);
                                        acc[n][2] = __fmaf_rn(s[2], p.x, acc[n][2]);
                                        acc[n][3] = __fmaf_rn(s[3], p.y, acc[n][3]);
                                    } else {
                                        s[0] = __fmul_rn(s[0], p.x);
                                        s[1] = __fmul_rn(s[1], p.y);
                                        s[2] = __fmul_rn(s[2], p.x);
                                        s[3] = __fmul_rn(s[3], p.y);
                                    }
                                }
                                if constexpr (!NV) {
                                    acc[n][0] = __fmaf_rn(s[0], fa[j], acc[n][0]);
                                    acc[n][1] = __fmaf_rn(s[1], fa[j], acc[n][1]);
                                    acc[n][2] = __fmaf_rn(s[2], fb[j], acc[n][2]);
                                    acc[n][3] = __fmaf_rn(s[3], fb[j], acc[n][3]);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.empty[share][slot]);
                if (++slot == kStages) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
        }
        consumers_sync();
    }

    // Sums: [warp][row][token] in shared memory, added over the shares and then
    // over the cluster's ranks, both in order.
    if (warp < kWarps) {
        float *part = reinterpret_cast<float *>(xs_base) + warp * (16 * TOK);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int gr = lane >> 2, tk = 8 * n + 2 * (lane & 3);
            *reinterpret_cast<float2 *>(part + gr * TOK + tk) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2 *>(part + (gr + 8) * TOK + tk) = make_float2(acc[n][2], acc[n][3]);
        }
    }
    if (a.ks > 1)
        cluster_sync();
    else
        __syncthreads();
    // After an abort, of whichever role, copies in flight land before the CTA exits.
    if (warp == kWarps && st.abort.flag)
        for (int i = max(0, loaded - kStages); i < loaded; ++i)
            mbar_wait(&st.full[lane >> 2][i % kStages], uint32_t(i / kStages) & 1u, nullptr, nullptr, a.wait_limit);
    const float g = NV ? (a.g ? __ldg(a.g) : 1.0f) : BF16 ? 1.0f / kSumSize : 1.0f;
    const uint32_t base = smem_u32(xs_base);
    for (int i = krank * kTokThreads + int(threadIdx.x); i < R * 16 * TOK; i += a.ks * kTokThreads) {
        // Consecutive threads take consecutive rows of a row group.
        const int tk = i / (R * 16), r = i - tk * (R * 16), w = r >> 4, mrow = r & 15;
        float v = 0.0f;
        for (int k = 0; k < a.ks; ++k) {
            for (int sh = 0; sh < S; ++sh) {
                const uint32_t at = base + uint32_t(((sh << a.r_log2) + w) * (16 * TOK) + mrow * TOK + tk) * 4u;
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(a.ks == 1 ? at : mapa_shared(at, uint32_t(k))) : "memory");
                v = __fadd_rn(v, f);
            }
        }
        int q, l;
        mma_row(a.r_log2, w, mrow, q, l);
        const int row = row0 + 32 * q + 4 * rg0 + l;
        if (tk < ntok && row < a.N)
            static_cast<X *>(a.C)[int64_t(tok0 + tk) * a.ldc + row] = from_float<X>(__fmul_rn(v, g));
    }
    if (a.ks > 1) cluster_sync();
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDimT = int64_t(1) << 30;
constexpr int64_t kMaxLdT = int64_t(1) << 36;
constexpr int kMaxDevT = 64;
std::atomic<int> g_rows{0};   // "fp4_tokens_rows": 0 by size, 1, 2, 4, 8
std::atomic<int> g_split{0};  // "fp4_tokens_split": 0 by size, 1, 2, 4, 8
constexpr int kBufBytes = 28 * 1024;  // one buffer of activations (two per CTA, two CTAs per SM)
static_assert(16 * (kPieceBytes + 32) <= kBufBytes, "sixteen tokens fit with R = 8");

// Row groups per CTA (log2) and CTAs per cluster of least estimated time, in
// units of 0.01 us.  A wave of two CTAs per SM starts in 2.2 us, 3.2 with clusters
// of two, 3.6 and 0.02 per cluster of four, 5.5 and 0.11 per cluster of eight (few
// of those fit a GPC).  A stage takes 0.54 us for eight tokens (bfloat16 0.6) and
// 0.92 for sixteen, 1.8 times that where two CTAs share an SM, and 0.8 us more
// where it is a whole chunk of the activations.  Their reading takes 0.02 us per KB
// (bfloat16, which is converted, 0.1), 3.5 times that where rows are not aligned.
// (Fitted to the times of every shape at 25 sizes between 128 x 8000 and 16384 x
// 8192 weights with 1 to 16 tokens.  Its choice takes 1.02 times the fastest
// shape's time there and at 15 other sizes, 1.13 at most.)
// The keys take a part of the shapes, all of them where that leaves none.
void choose_tokens(int64_t N, int64_t K, int groups, int toks, int token_bytes, bool bf16, bool xvec, int64_t chunks,
                   int sms, int *r_log2, int *ks) {
    const int64_t per_stage = toks > 8 ? 92 : bf16 ? 60 : 54;
    const int rows = g_rows.load(), split = g_split.load();
    int64_t best = INT64_MAX;
    for (bool any : {false, true}) {
        for (int r = 3; r >= 0; --r) {
            const int S = 8 >> r, most = kBufBytes / (S * token_bytes);  // stages of a chunk
            if (most < 1) continue;                                      // (never with R = 8)
            for (int k = 1; k <= 8; k *= 2) {
                if (groups < S * k && (r < 3 || k > 1)) continue;
                if (!any && ((rows != 0 && rows != 1 << r) || (split != 0 && split != k))) continue;
                const int64_t ctas = (N + 127) / 128 * S * k * chunks;
                const int64_t waves = (ctas + 2 * sms - 1) / (2 * sms), clusters = ctas / k / waves;
                const int64_t stages = (groups + S * k - 1) / (S * k);
                const int64_t start = k == 1 ? 220 : k == 2 ? 320 : k == 4 ? 360 + 2 * clusters : 550 + 11 * clusters;
                const int64_t read = toks * K / k * 2 * (bf16 ? 10 : 2) * (xvec ? 2 : 7) / 2048;
                const int64_t cost = waves * (start + stages * per_stage * (ctas > sms ? 18 : 10) / 10 +
                                              (most == 1 ? stages * 80 : 0) + read);
                if (cost < best) {
                    best = cost;
                    *r_log2 = r;
                    *ks = k;
                }
            }
        }
        if (best != INT64_MAX) return;
    }
}

template <bool NV, bool BF16, int NT>
int launch_tokens(TokArgs a, const void *codes, int64_t pitch, const void *scales, int sms, cudaStream_t stream) {
    constexpr int TOK = 8 * NT, KAT = NV ? 4 : 2;
    constexpr int RING = kStages * (kCodeBytes + 512 * KAT) + 1024;
    auto *fn = tokens_kernel<NV, BF16, NT>;
    static std::atomic<int> ready[kMaxDevT];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_launch(e, "cudaGetDevice");
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, RING + 2 * kBufBytes);
        if (e != cudaSuccess) return fail_launch(e, "4-bit weight product set-up");
        ready[dev].store(1, std::memory_order_release);
    }
    const int64_t tiles = (a.N + 127) / 128, chunks = (a.M + TOK - 1) / TOK;
    const int toks = std::min(a.M, TOK);
    // Bytes of a stage's activations and powers of two.
    const int token_bytes = toks * kPieceBytes + (BF16 ? 8 * TOK * 4 : 0);
    choose_tokens(a.N, a.K, a.groups, toks, token_bytes, BF16, a.xvec != 0, chunks, sms, &a.r_log2, &a.ks);
    const int ks = a.ks, S = kWarps >> a.r_log2;
    const int per = ((a.groups + ks - 1) / ks + S - 1) / S;         // stages of the longest share
    const int most = kBufBytes / (S * token_bytes);                // of a buffer
    a.chunk = std::min(per, most);
    const int bufs = per > a.chunk ? 2 : 1;
    const size_t smem =
        RING + std::max(size_t(bufs) * S * a.chunk * token_bytes, size_t(kWarps) * 16 * TOK * 4);
    const int R = 1 << a.r_log2;
    const int64_t kp = (int64_t(a.K) + 31) / 32 * 32, block = NV ? 16 : 32;
    CUtensorMap tw, ts;
    int rc = encode_tmap_2d(&tw, true, codes, uint64_t(kp / 2), uint64_t(a.N), uint64_t(pitch), 128, uint32_t(4 * R));
    if (!rc)
        rc = encode_tmap_scales(&ts, scales, uint64_t(((a.K + block - 1) / block + 3) / 4), uint64_t(tiles), KAT, 1,
                                uint32_t(16 * R));
    if (rc) return rc;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = dim3(unsigned(tiles * S * ks), unsigned(chunks), 1);
    cfg.blockDim = dim3(kTokThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (ks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = unsigned(ks);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (pdl_enabled()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    e = cudaLaunchKernelEx(&cfg, fn, tw, ts, a);
    if (e != cudaSuccess) return fail_launch(e, "4-bit weight product launch");
    note_launches(1);
    note_fp4_launch(int64_t(cfg.gridDim.x) * cfg.gridDim.y, ks, ks, 16 * R);
    return PTC_OK;
}

template <bool NV, bool BF16>
int launch_width(const TokArgs &a, const void *codes, int64_t pitch, const void *scales, int sms, cudaStream_t s) {
    return a.M <= 8 ? launch_tokens<NV, BF16, 1>(a, codes, pitch, scales, sms, s)
                    : launch_tokens<NV, BF16, 2>(a, codes, pitch, scales, sms, s);
}

}  // namespace

bool set_tokens_tuning(const char *key, int64_t v) {
    if (v != 0 && v != 1 && v != 2 && v != 4 && v != 8) return false;
    if (std::strcmp(key, "fp4_tokens_rows") == 0)
        g_rows.store(int(v));
    else if (std::strcmp(key, "fp4_tokens_split") == 0)
        g_split.store(int(v));
    else
        return false;
    return true;
}

cudaError_t read_and_clear_tokens_error_word(uint32_t *out) {
    uint32_t v = 0;
    const uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tok_error, sizeof(v));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tok_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace ptc

using namespace ptc;

extern "C" int gemm_a16_fp4(int64_t M, int64_t N, int64_t K, int type, const void *X, int64_t ldx, int format,
                            const void *W, int64_t ldw, const void *SW, const float *GW, void *C, int64_t ldc,
                            void *stream) {
    set_message("");
    if (M < 0 || N < 0 || K < 0 || M > kMaxDimT || N > kMaxDimT || K > kMaxDimT)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= M, N, K <= 2^30");
    if (M > 65535 * 16) return fail_status(PTC_ERR_INVALID, "at most 1048560 rows of activations");
    if (type != PTC_OUT_BF16 && type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "activations are PTC_OUT_BF16 or PTC_OUT_F16");
    if (format != PTC_FP4_MX && format != PTC_FP4_NV) return fail_status(PTC_ERR_INVALID, "unknown 4-bit format");
    if (M == 0 || N == 0) return PTC_OK;
    const bool nv = format == PTC_FP4_NV;
    if (!C || ldc < N || ldc > kMaxLdT) return fail_status(PTC_ERR_INVALID, "C is NULL, or ldc is not N .. 2^36");
    if (K > 0 && (!X || ldx < K || ldx > kMaxLdT))
        return fail_status(PTC_ERR_INVALID, "X is NULL, or ldx is not K .. 2^36");
    int rc;
    if (K > 0 && (rc = check_fp4(W, ldw, SW, GW, K, nv))) return rc;
    if (reinterpret_cast<uintptr_t>(C) % 2 || (K > 0 && reinterpret_cast<uintptr_t>(X) % 2))
        return fail_status(PTC_ERR_ALIGN, "X and C must be aligned to their elements");
    const ByteRows c = elem_rows(C, M, N, ldc, 2);
    if (K > 0 && (rows_overlap(c, elem_rows(X, M, K, ldx, 2)) || rows_overlap(c, fp4_code_rows(W, N, K, ldw)) ||
                  rows_overlap(c, fp4_scale_rows(SW, N, K, nv)) || rows_overlap(c, flat_bytes(GW, 4))))
        return fail_status(PTC_ERR_OVERLAP, "C overlaps an operand");
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const cudaError_t e = launch_zero_fill(C, ldc, int(M), int(N), 2, sms * 4, s);
        if (e != cudaSuccess) return fail_launch(e, "zero-fill launch");
        note_launches(1);
        return PTC_OK;
    }
    TokArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = X;
    a.ldx = ldx;
    a.g = GW;
    a.C = C;
    a.ldc = ldc;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.groups = int((K + kGroup - 1) / kGroup);
    a.xvec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
    a.stall = take_stall_tile();
    a.wait_limit = wait_limit_ns();
    if (type == PTC_OUT_BF16)
        return nv ? launch_width<true, true>(a, W, ldw, SW, sms, s) : launch_width<false, true>(a, W, ldw, SW, sms, s);
    return nv ? launch_width<true, false>(a, W, ldw, SW, sms, s) : launch_width<false, false>(a, W, ldw, SW, sms, s);
}
