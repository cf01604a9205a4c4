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
// Layout.  A warp owns 16 rows of a 128-row scale tile, rows 4 w + {0..3} +
// {0, 32, 64, 96}, so that its scale words are 64 contiguous bytes.  In each
// step of 128 codes a lane loads the 16 bytes (32 codes) of its two rows that
// lie in block lane % 4: the order of k within an MMA is free as long as both
// operands agree, so MMA i of the step multiplies codes 4 i .. 4 i + 3 of each
// of the four lanes' pieces with the same four activations, eight contiguous
// bytes of x.  The x rows of the CTA's K range lie in shared memory, their
// 16-byte pieces exchanged so that the loads do not conflict.
//
// Weights are expanded exactly: nvfp4 with binary16 activations to binary16
// (code x E4M3 scale has 6 significant bits and lies in 2^-10 .. 2688);
// otherwise to bfloat16 (code x scale has at most 6 bits).  A code is
// first converted to binary16 by one instruction per two codes; moved down by
// three bits it is the same value times 2^-112 in bfloat16, and one
// multiplication by 2^112 x scale finishes it (two where 2^112 x scale is too
// large).  Binary16 activations with mxfp4 weights are split into two
// bfloat16 terms (8 + 3 bits), exactly.
//
// K is shared by a cluster of up to eight CTAs; the partial sums are added in
// rank order through distributed shared memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "fp4.cuh"
#include "internal.h"
#include "ptc.h"
#include "ptx.cuh"

namespace ptc {
namespace {

constexpr int kWarps = 8, kTokThreads = 32 * kWarps;
constexpr int kRows = 128;      // weight rows per CTA
constexpr int kGroup = 128;     // codes per step
constexpr int kPieceBytes = 2 * kGroup;  // one token's activations of a step

struct TokArgs {
    const void *x;
    int64_t ldx;
    const uint8_t *codes;
    int64_t pitch;
    const uint8_t *scales;
    const float *g;
    void *C;
    int64_t ldc;
    int M, N, K;
    int64_t ktiles;      // scale tiles per 128 rows
    int groups;          // steps of 128 codes in K
    int slice;           // steps held in shared memory at a time
    int ks;              // CTAs per cluster
    int xvec;
};

// How the operands of the MMAs are made.
enum class Form { F16 = 0, BF16 = 1, SPLIT = 2 };

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The multiplier(s) of one block's codes, both halves of a word alike.
struct Mult {
    uint32_t m, post;  // post: the second factor, used when `wide` is set
    bool wide;
};

template <bool NV, Form F>
__device__ __forceinline__ Mult multiplier(uint32_t byte) {
    Mult r{0u, 0u, false};
    if constexpr (NV && F == Form::F16) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(byte | (byte << 8))));
        r.m = h;
    } else if constexpr (NV) {
        // 2^112 x scale: at most 448 x 2^112, four significant bits.
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(byte)));
        const float s = __half2float(__ushort_as_half(uint16_t(h))) * 5192296858534827628530496329220096.0f;  // 2^112
        r.m = uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(s))) * 0x10001u;
    } else {
        // 2^(byte - 127 + 112) while that is at most 2^127; above, 2^112 and 2^(byte - 127).
        const bool wide = byte > 142u;
        r.m = (wide ? (112u + 127u) << 7 : (byte + 112u) << 7) * 0x10001u;
        const uint32_t own = byte == 255u ? 0x7FC0u : byte << 7;
        r.post = own * 0x10001u;
        r.wide = wide;
    }
    return r;
}

// Eight codes times their block's scale as four words of two values.
template <bool NV, Form F>
__device__ __forceinline__ void expand8(uint32_t w, const Mult &s, bool any_wide, uint32_t (&v)[4]) {
    codes_to_f16(w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F == Form::F16) {
            v[i] = mul_f16x2(v[i], s.m);
        } else {
            const uint32_t b = ((v[i] >> 3) & 0x0FFF0FFFu) | (v[i] & 0x80008000u);
            v[i] = mul_bf16x2(b, s.m);
            if constexpr (!NV)
                if (any_wide && s.wide) v[i] = mul_bf16x2(v[i], s.post);
        }
    }
}

// Offset of 16-byte piece p (0 .. 15) of a token's step in shared memory.
__device__ __forceinline__ uint32_t piece_at(int token, int p) {
    const int t = p >> 2, j = p & 3;
    return uint32_t(4 * t + (j ^ t ^ (token & 1))) << 4;
}

template <bool NV, Form F, int NT>
__global__ void __launch_bounds__(kTokThreads, 2) tokens_kernel(const TokArgs a) {
    constexpr int PARTS = F == Form::SPLIT ? 2 : 1;
    constexpr int TOK = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];  // [part][token][slice] pieces, then partial sums
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gr = lane >> 2, t = lane & 3;
    const int krank = a.ks == 1 ? 0 : int(cluster_ctarank());
    const int row0 = int(blockIdx.x) / a.ks * kRows;
    const int tok0 = int(blockIdx.y) * TOK;
    const int ntok = min(TOK, a.M - tok0);
    const int kq = a.groups / a.ks, kr = a.groups % a.ks;
    const int g0 = krank * kq + min(krank, kr), g1 = g0 + kq + (krank < kr ? 1 : 0);
    const uint32_t row_bytes = uint32_t(a.slice) * kPieceBytes;
    // MMA row i of this warp: row 4 warp + i % 4 + 32 (i / 4) of the tile.
    const int lr0 = 4 * warp + (gr & 3) + 32 * (gr >> 2), lr1 = lr0 + 64;
    const bool in0 = row0 + lr0 < a.N, in1 = row0 + lr1 < a.N;
    const uint8_t *p0 = a.codes + int64_t(in0 ? row0 + lr0 : 0) * a.pitch, *p1 = a.codes + int64_t(in1 ? row0 + lr1 : 0) * a.pitch;
    const uint8_t *s0 = a.scales + scale_word(row0 + lr0, 0, a.ktiles), *s1 = a.scales + scale_word(row0 + lr1, 0, a.ktiles);
    const int blocks32 = (a.K + 31) / 32;

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

    struct Step {
        uint4 w0, w1;
        uint32_t c0, c1;  // scale bytes of the lane's block (nvfp4: of its two blocks)
    };
    auto fetch = [&](int g) {
        Step s;
        s.w0 = s.w1 = make_uint4(0, 0, 0, 0);
        s.c0 = s.c1 = 0u;
        const int b = 4 * g + t;  // block of 32 codes
        if (b < blocks32) {
            if (in0) s.w0 = __ldcs(reinterpret_cast<const uint4 *>(p0 + int64_t(b) * 16));
            if (in1) s.w1 = __ldcs(reinterpret_cast<const uint4 *>(p1 + int64_t(b) * 16));
            if constexpr (NV) {
                const int64_t o = int64_t(2 * g + (t >> 1)) * kScaleTile + 2 * (t & 1);
                if (in0) s.c0 = *reinterpret_cast<const uint16_t *>(s0 + o);
                if (in1) s.c1 = *reinterpret_cast<const uint16_t *>(s1 + o);
            } else {
                const int64_t o = int64_t(g) * kScaleTile + t;
                if (in0) s.c0 = s0[o];
                if (in1) s.c1 = s1[o];
            }
        }
        return s;
    };

    griddep_wait();
    griddep_launch_dependents();
    constexpr int AHEAD = 3;
    Step next[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (g0 + i < g1) next[i] = fetch(g0 + i);

    for (int base = g0; base < g1; base += a.slice) {
        const int end = min(g1, base + a.slice);
        if (base > g0) __syncthreads();
        // Activations of this slice; zeros past K and past the last token.
        for (int i = int(threadIdx.x); i < TOK * (end - base) * 16; i += kTokThreads) {
            const int per = (end - base) * 16, tok = i / per, p = i - tok * per;
            const int64_t k = int64_t(base) * kGroup + p * 8;
            const int n = tok < ntok ? int(max(int64_t(0), min(int64_t(8), int64_t(a.K) - k))) : 0;
            const uint32_t dst = uint32_t(tok) * row_bytes + uint32_t(p >> 4) * kPieceBytes + piece_at(tok, p & 15);
            using X = typename ElemOf<F == Form::BF16 ? Elem::BF16 : Elem::F16>::type;
            const X *src = static_cast<const X *>(a.x) + (n > 0 ? int64_t(tok0 + tok) * a.ldx + k : 0);
            const Pack8<X> v = load8(src, n, a.xvec != 0);
            if constexpr (F == Form::SPLIT) {
                Pack8<__nv_bfloat16> hi, lo;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = to_float(v.get(j));
                    hi.set(j, __float2bfloat16_rn(f));
                    // (an infinity or NaN is in the first term alone)
                    const float rest = f - __bfloat162float(hi.get(j));
                    lo.set(j, __float2bfloat16_rn(fabsf(f) <= 65504.0f ? rest : 0.0f));
                }
                *reinterpret_cast<uint4 *>(smem + dst) = hi.v[0];
                *reinterpret_cast<uint4 *>(smem + TOK * row_bytes + dst) = lo.v[0];
            } else {
                *reinterpret_cast<uint4 *>(smem + dst) = v.v[0];
            }
        }
        __syncthreads();
        for (int gb = base; gb < end; gb += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int g = gb + u;
                if (g >= end) break;
                const Step s = next[u];
                if (g + AHEAD < g1) next[u] = fetch(g + AHEAD);
                Mult m0[NV ? 2 : 1], m1[NV ? 2 : 1];
                m0[0] = multiplier<NV, F>(s.c0 & 0xFFu);
                m1[0] = multiplier<NV, F>(s.c1 & 0xFFu);
                if constexpr (NV) {
                    m0[1] = multiplier<NV, F>(s.c0 >> 8);
                    m1[1] = multiplier<NV, F>(s.c1 >> 8);
                }
                bool wide = false;
                if constexpr (!NV) wide = __any_sync(0xFFFFFFFFu, m0[0].wide || m1[0].wide);
                const uint32_t xs = smem_u32(smem) + uint32_t(g - base) * kPieceBytes;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w0 = j == 0 ? s.w0.x : j == 1 ? s.w0.y : j == 2 ? s.w0.z : s.w0.w;
                    const uint32_t w1 = j == 0 ? s.w1.x : j == 1 ? s.w1.y : j == 2 ? s.w1.z : s.w1.w;
                    uint32_t v0[4], v1[4];
                    expand8<NV, F>(w0, m0[NV ? j / 2 : 0], wide, v0);
                    expand8<NV, F>(w1, m1[NV ? j / 2 : 0], wide, v1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int tok = 8 * n + gr;
                        const uint32_t at = xs + uint32_t(tok) * row_bytes + piece_at(tok, 4 * t + j);
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            const uint4 x = ld_shared_v4(at + uint32_t(part) * (TOK * row_bytes));
                            mma16816<F == Form::F16>(acc[n], v0[0], v1[0], v0[1], v1[1], x.x, x.y);
                            mma16816<F == Form::F16>(acc[n], v0[2], v1[2], v0[3], v1[3], x.z, x.w);
                        }
                    }
                }
            }
        }
    }

    // Sums: [row][token] in shared memory, added over the cluster's ranks.
    __syncthreads();
    float *part = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int tk = 8 * n + 2 * t;
        *reinterpret_cast<float2 *>(part + lr0 * TOK + tk) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2 *>(part + lr1 * TOK + tk) = make_float2(acc[n][2], acc[n][3]);
    }
    if (a.ks > 1)
        cluster_sync();
    else
        __syncthreads();
    const float g = a.g ? __ldg(a.g) : 1.0f;
    const uint32_t base = smem_u32(smem);
    for (int i = krank * kTokThreads + int(threadIdx.x); i < kRows * TOK; i += a.ks * kTokThreads) {
        const int r = i % kRows, tk = i / kRows;
        float v = 0.0f;
        for (int k = 0; k < a.ks; ++k) {
            const uint32_t at = base + uint32_t(r * TOK + tk) * 4u;
            float f;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(a.ks == 1 ? at : mapa_shared(at, uint32_t(k))) : "memory");
            v = __fadd_rn(v, f);
        }
        if (tk < ntok && row0 + r < a.N) {
            using X = typename ElemOf<F == Form::BF16 ? Elem::BF16 : Elem::F16>::type;
            static_cast<X *>(a.C)[int64_t(tok0 + tk) * a.ldc + row0 + r] = from_float<X>(__fmul_rn(v, g));
        }
    }
    if (a.ks > 1) cluster_sync();
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDimT = int64_t(1) << 30;
constexpr int64_t kMaxLdT = int64_t(1) << 36;
constexpr int kMaxDevT = 64;
constexpr int kSliceBytes = 96 * 1024;  // activations in shared memory: two CTAs per SM

template <bool NV, Form F, int NT>
cudaError_t launch_tokens(TokArgs a, int sms, cudaStream_t stream) {
    constexpr int PARTS = F == Form::SPLIT ? 2 : 1, TOK = 8 * NT;
    auto *fn = tokens_kernel<NV, F, NT>;
    static std::atomic<int> ready[kMaxDevT];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceBytes);
        if (e != cudaSuccess) return e;
        ready[dev].store(1, std::memory_order_release);
    }
    const int64_t tiles = (a.N + kRows - 1) / kRows, chunks = (a.M + TOK - 1) / TOK;
    // As many K shares as fill two CTAs per SM in one wave, at least two steps each.
    int ks = 8;
    while (ks > 1 && (tiles * chunks * ks > 2 * sms || a.groups < 2 * ks)) ks /= 2;
    a.ks = ks;
    const int per = (a.groups + ks - 1) / ks, most = kSliceBytes / (PARTS * TOK * kPieceBytes);
    a.slice = std::min(per, most);
    const size_t smem = std::max(size_t(PARTS) * TOK * a.slice * kPieceBytes, size_t(kRows) * TOK * 4);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = dim3(unsigned(tiles * ks), unsigned(chunks), 1);
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
    e = cudaLaunchKernelEx(&cfg, fn, a);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

template <bool NV, Form F>
cudaError_t launch_width(const TokArgs &a, int sms, cudaStream_t s) {
    return a.M <= 8 ? launch_tokens<NV, F, 1>(a, sms, s) : launch_tokens<NV, F, 2>(a, sms, s);
}

}  // namespace
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
    if (K > 0 && (rc = check_fp4(W, ldw, SW, GW, N, K, nv))) return rc;
    if (reinterpret_cast<uintptr_t>(C) % 2 || (K > 0 && reinterpret_cast<uintptr_t>(X) % 2))
        return fail_status(PTC_ERR_ALIGN, "X and C must be aligned to their elements");
    const uint64_t cb = span_of(M, N, ldc, 2);
    if (K > 0 && (ranges_overlap(C, cb, X, span_of(M, K, ldx, 2)) || ranges_overlap(C, cb, W, fp4_code_span(N, K, ldw)) ||
                  ranges_overlap(C, cb, SW, fp4_scale_bytes(N, K, nv)) || (GW && ranges_overlap(C, cb, GW, 4))))
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
    a.codes = static_cast<const uint8_t *>(W);
    a.pitch = ldw;
    a.scales = static_cast<const uint8_t *>(SW);
    a.g = GW;
    a.C = C;
    a.ldc = ldc;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    const int64_t block = nv ? 16 : 32;
    a.ktiles = ((K + block - 1) / block + 3) / 4;
    a.groups = int((K + kGroup - 1) / kGroup);
    a.xvec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
    cudaError_t e;
    if (type == PTC_OUT_BF16)
        e = nv ? launch_width<true, Form::BF16>(a, sms, s) : launch_width<false, Form::BF16>(a, sms, s);
    else
        e = nv ? launch_width<true, Form::F16>(a, sms, s) : launch_width<false, Form::SPLIT>(a, sms, s);
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "4-bit weight product launch");
}
