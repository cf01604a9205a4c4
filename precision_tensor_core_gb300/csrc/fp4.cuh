// fp4.cuh -- device primitives of the microscaled 4-bit formats and of the
// counter-based generator: E2M1 codes, block scales, the tiled scale layout,
// and 16 random bits per element.
//
// Formats (include/ptc.h, "Microscaled 4-bit matrices"): a block of
// consecutive elements of a row shares one scale byte,
//   mxfp4  32 elements, scale 2^(byte - 127), 0xFF: NaN
//   nvfp4  16 elements, E4M3 scale, 0x7F: NaN, and one FP32 scale per matrix
// and each element is an E2M1 code (sign, 0 / 0.5 / 1 / 1.5 / 2 / 3 / 4 / 6).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

namespace ptc {

// ------------------------------------------------------------ generator
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit products.  One
// call gives the 16 bits of eight consecutive elements of a row.  The ten
// rounds' keys are made on the host, so that a round is two products and two
// three-way exclusive ors with a kernel parameter.
struct RngArgs {
    uint32_t key[20];         // of round i: key[2 i], key[2 i + 1]
    uint32_t off_lo, off_hi;  // offset (63 bits)
};

inline RngArgs make_rng(uint64_t seed, uint64_t offset) {
    RngArgs r;
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
    for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
        r.key[2 * i] = k0;
        r.key[2 * i + 1] = k1;
    }
    r.off_lo = uint32_t(offset);
    r.off_hi = uint32_t(offset >> 32);
    return r;
}

// What a stream of random bits is for: its own counters for each.
constexpr uint32_t kRngDropout = 0, kRngRounding = 1;

// The 16-bit numbers of elements (row, 8 group .. 8 group + 7): element j has
// bits 16 (j & 1) .. of word j >> 1.
__device__ __forceinline__ uint4 random_bits8(const RngArgs &g, uint32_t purpose, uint32_t row, uint32_t group) {
    uint32_t c0 = group, c1 = row, c2 = g.off_lo, c3 = g.off_hi | (purpose << 31);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = uint64_t(0xD2511F53u) * c0, p1 = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(p1 >> 32) ^ c1 ^ g.key[2 * i];
        c1 = uint32_t(p1);
        c2 = uint32_t(p0 >> 32) ^ c3 ^ g.key[2 * i + 1];
        c3 = uint32_t(p0);
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint32_t bits16(const uint4 &w, int j) {
    const uint32_t x = (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w;
    return (j & 1) ? x >> 16 : x & 0xFFFFu;
}

// ------------------------------------------------------------ element types
enum class Elem : int { F32 = 0, BF16 = 1, F16 = 2 };  // the values of PTC_OUT_*

template <Elem E>
struct ElemOf;
template <>
struct ElemOf<Elem::F32> {
    using type = float;
};
template <>
struct ElemOf<Elem::BF16> {
    using type = __nv_bfloat16;
};
template <>
struct ElemOf<Elem::F16> {
    using type = __half;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
    return __float2half_rn(v);
}

// Eight consecutive elements as they lie in memory (16 or 32 bytes).
template <typename T>
struct Pack8 {
    static constexpr int W = sizeof(T) * 8 / 16;
    uint4 v[W];
    __device__ __forceinline__ T get(int j) const { return reinterpret_cast<const T *>(v)[j]; }
    __device__ __forceinline__ void set(int j, T x) { reinterpret_cast<T *>(v)[j] = x; }
};

// Eight FP32 values rounded to the element type, two per conversion.
template <typename T>
__device__ __forceinline__ Pack8<T> round8(const float (&v)[8]) {
    Pack8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.set(j, v[j]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = reinterpret_cast<const uint32_t &>(h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = reinterpret_cast<const uint32_t &>(h);
            }
        }
        r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}

// `n` (1 .. 8) elements at p; the others +0.  `vec`: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ Pack8<T> load8(const T *p, int n, bool vec) {
    Pack8<T> r;
    if (vec && n >= 8) {
#pragma unroll
        for (int w = 0; w < Pack8<T>::W; ++w) r.v[w] = reinterpret_cast<const uint4 *>(p)[w];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.set(j, j < n ? p[j] : from_float<T>(0.0f));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const Pack8<T> &r, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
        for (int w = 0; w < Pack8<T>::W; ++w) reinterpret_cast<uint4 *>(p)[w] = r.v[w];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = r.get(j);
    }
}

// ------------------------------------------------------------ scales
constexpr int kScaleTile = 512;  // bytes of a tile of 128 rows x 4 blocks

// Offset of row r's four scale bytes of blocks 4 kt .. 4 kt + 3.
__host__ __device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t ktiles) {
    return ((r >> 7) * ktiles + kt) * kScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// A scale byte as FP32.
template <bool NV>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    if constexpr (NV) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(byte)));
        return __half2float(__ushort_as_half(uint16_t(h)));
    } else {
        return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
    }
}

constexpr uint32_t kInfBits = 0x7F800000u;

// a / b rounded to FP32, `inverse` being 1 / b rounded: the product with it is
// corrected by its remainder (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990), without which exact midpoints of the
// codes could fall to either side.  A quotient beyond FP32 is NaN.
__device__ __forceinline__ float quotient(float a, float b, float inverse) {
    const float q = __fmul_rn(a, inverse);
    return __fmaf_rn(__fmaf_rn(-q, b, a), inverse, q);
}

// The matrix scale G (0 .. 2^100) of an nvfp4 matrix, and 6 G by which blocks' largest
// magnitudes are divided.  (One division per call of 6 G's reciprocal in place of
// one per block: 8192 x 8192 bfloat16 both ways 64.0 -> 62.6 us.)
// Small: G is below 2^-20, and then 6 G, blocks' largest magnitudes, their scales and
// elements are taken times 2^64 (LIFT below), which keeps remainders above FP32's
// smallest number and reciprocals of the smallest scales below its largest.  An
// element that this takes beyond FP32 is far above its block's largest code.  With
// G = 0 scales and codes are 0.  (Kernels hold the two forms apart: a test per eight
// elements costs a stochastic call 5%.)
template <bool NV>
struct MatrixScale {
    float g = 1.0f, six = 6.0f, inverse = 0.0f;
    bool small = false;
    __device__ __forceinline__ explicit MatrixScale(const float *p) {
        if constexpr (NV) {
            if (p != nullptr) g = __ldg(p);
            small = g < 0x1p-20f;
            six = __fmul_rn(g, 6.0f);
            inverse = g > 0.0f ? __frcp_rn(small ? __fmul_rn(six, 0x1p64f) : six) : 0.0f;
        }
    }
    // a / (6 G), or 0 where G is; at least 2^14 where the quotient is beyond FP32.
    template <bool LIFT>
    __device__ __forceinline__ float sixths(float a) const {
        if constexpr (LIFT)
            return six > 0.0f ? fminf(quotient(__fmul_rn(a, 0x1p64f), __fmul_rn(six, 0x1p64f), inverse), 0x1p14f) : 0.0f;
        return fminf(quotient(a, six, inverse), 0x1p14f);
    }
};

// A block's scale: the reciprocal it is applied by, and for nvfp4 the scale, both
// for lifted elements where G is small.
template <bool NV>
struct BlockScale {
    float inverse, d;
    // Eight elements as the other functions take them.
    template <bool LIFT>
    __device__ __forceinline__ void lift8(float (&v)[8]) const {
        if constexpr (LIFT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = d > 0.0f ? __fmul_rn(v[j], 0x1p64f) : 0.0f;
        }
    }
    // x / scale rounded to FP32.  mxfp4 scales are powers of two, so the
    // product is exact.
    __device__ __forceinline__ float apply(float x) const {
        const float q = __fmul_rn(x, inverse);
        if constexpr (!NV) return q;
        // (Far above the largest code, where the remainder could overflow, q saturates as it is.)
        return fabsf(q) < 16.0f ? quotient(x, d, inverse) : q;
    }
    // The smaller of |x| / scale and 6 for stochastic rounding.  mxfp4's scale
    // is then at least a sixth of the block's largest magnitude.  (nvfp4: a quotient
    // so large that its remainder is NaN is 6 too.)
    __device__ __forceinline__ float magnitude(float x) const {
        if constexpr (!NV) return __fmul_rn(fabsf(x), inverse);
        return fminf(fabsf(quotient(x, d, inverse)), 6.0f);
    }
};

// Scale byte and scale of a block whose largest magnitude has the
// FP32 bits `amax` (at least kInfBits: some element is not finite).
//   mxfp4, nearest:    2^(floor(log2 amax) - 2): elements in (6, 8) x scale
//                      saturate, the rule of the OCP microscaling format
//   mxfp4, stochastic: the least power of two with amax <= 6 x scale, so that
//                      no element saturates and the rounding has no bias
//   nvfp4:             amax / (6 G) rounded to E4M3 (stochastic: up to the next
//                      one where amax would saturate), G the matrix scale
// LIFT: the scale is that of lifted elements.
template <bool NV, bool SR, bool LIFT>
__device__ __forceinline__ BlockScale<NV> block_scale(uint32_t amax, const MatrixScale<NV> &g, uint32_t &byte) {
    BlockScale<NV> s{0.0f, 0.0f};
    const bool finite = amax < kInfBits;
    if constexpr (!NV) {
        int e = int(amax >> 23) - 2;
        if constexpr (SR) e += (amax & 0x7FFFFFu) > 0x400000u ? 1 : 0;
        e = e < 0 ? 0 : e;
        byte = finite ? uint32_t(e) : 255u;
        s.inverse = __uint_as_float(uint32_t(254 - (finite ? e : 0)) << 23);
    } else {
        const float a = __uint_as_float(amax);
        uint16_t q;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(0.0f), "f"(g.template sixths<LIFT>(a)));
        uint32_t b = q & 0x7Fu;
        if constexpr (SR)
            if (__fmul_rn(g.six, scale_value<true>(b)) < a && b < 0x7Eu && !(LIFT && g.six == 0.0f)) ++b;
        s.d = __fmul_rn(scale_value<true>(b), g.g);
        if constexpr (LIFT) s.d = __fmul_rn(s.d, 0x1p64f);
        byte = finite ? b : 0x7Fu;
        s.inverse = s.d > 0.0f ? __frcp_rn(s.d) : 0.0f;
    }
    return s;
}

// ------------------------------------------------------------ codes
// Eight FP32 values to eight codes, nearest with ties to even, at most 6 in
// magnitude; value j in bits 4 j .. 4 j + 3.
__device__ __forceinline__ uint32_t codes_nearest(const float (&v)[8]) {
    uint32_t q;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(q)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return q;
}

// The magnitude u (at most 6) of a scaled value rounded down or up to the
// neighbouring codes, up when its remainder (in 1/65536 of the gap) plus r
// reaches 65536; the code in the top byte of the result.  From 1 up the codes are floats of one mantissa
// bit, so bits 22 .. 24 of u are the code rounded down (plus a constant) and the 22
// bits below are the remainder: adding r << 6 carries exactly where the code goes
// up.  Below 1 the grid is uniform with the gap of [1, 2): (u + 1) / 2 lies one
// binade lower, which makes its first code 0.  It is made as u + (1 - u) / 2, whose
// second term saturates at 0 from 1 up, and rounded down keeps all 16 bits of the
// remainder that count: the second term is rounded by at most 2^-26, and to the
// nearest, so that the sum passes a multiple of 2^-18 only where the exact one
// does.  `r8` is (r + 4 * 65536) * 256; the 4 makes up for the exponent's bias
// (2 * 126 = -4 modulo 8) and the product by 4 takes the constant out at the top.
// The signs join the packed codes, four at a time (joined to each code: 8192 x 8192
// bfloat16 to mxfp4 both ways 90 us instead of 81).
__device__ __forceinline__ uint32_t code_stochastic(float u, uint32_t r8) {
    float half_gap;  // (1 - u) / 2, or 0
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(half_gap) : "f"(u), "f"(-0.5f), "f"(0.5f));
    const float w = __fadd_rd(u, half_gap);
    return 4u * __float_as_uint(w) + r8;
}

// Bytes picked from two words; a selector's bit 3 spreads the byte's top bit.
template <uint32_t SELECT>
__device__ __forceinline__ uint32_t pick_bytes(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(SELECT));
    return r;
}

// Of eight values: byte j is 0xFF where value 2 j (`even`) or 2 j + 1 is negative.
struct Signs8 {
    uint32_t even, odd;
};

__device__ __forceinline__ Signs8 signs8(const float (&v)[8]) {
    uint32_t p[4];  // values 0 and 2, 1 and 3, 4 and 6, 5 and 7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = (i >> 1) * 4 + (i & 1);
        p[i] = pick_bytes<0x00FB>(__float_as_uint(v[j]), __float_as_uint(v[j + 2]));
    }
    return {pick_bytes<0x5410>(p[0], p[2]), pick_bytes<0x5410>(p[1], p[3])};
}

// Of four words of two 16-bit values: byte j is 0xFF where word j's low (`low`) or
// high value is negative.
__device__ __forceinline__ void half_signs(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t &low,
                                           uint32_t &high) {
    const uint32_t p = pick_bytes<0x7351>(w0, w1), q = pick_bytes<0x7351>(w2, w3);
    low = pick_bytes<0xDC98>(p, q);
    high = pick_bytes<0xFEBA>(p, q);
}

// The signs of eight elements as they came.
template <typename T>
__device__ __forceinline__ Signs8 signs8(const Pack8<T> &p) {
    Signs8 s;
    if constexpr (sizeof(T) == 2) {
        const uint4 &w = p.v[0];
        half_signs(w.x, w.y, w.z, w.w, s.even, s.odd);
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_float(p.get(j));
        s = signs8(v);
    }
    return s;
}

// Eight codes of code_stochastic with their signs, value j in bits 4 j .. 4 j + 3.
__device__ __forceinline__ uint32_t pack_stochastic(const uint32_t (&c)[8], const Signs8 &s) {
    const uint32_t e = pick_bytes<0x5410>(pick_bytes<0x0073>(c[0], c[2]), pick_bytes<0x0073>(c[4], c[6]));
    const uint32_t o = pick_bytes<0x5410>(pick_bytes<0x0073>(c[1], c[3]), pick_bytes<0x0073>(c[5], c[7]));
    const uint32_t sign = (s.even & 0x0F0F0F0Fu) | (s.odd & 0xF0F0F0F0u);
    return (e + 16u * o) | (sign & 0x88888888u);
}

// (r + 4 * 65536) * 256 of element j of eight (bits as random_bits8 gives them),
// and of the low and high half of a word.
__device__ __forceinline__ uint32_t low_r8(uint32_t w) { return __byte_perm(w, 4u, 0x4105); }
__device__ __forceinline__ uint32_t high_r8(uint32_t w) { return __byte_perm(w, 4u, 0x4325); }
__device__ __forceinline__ uint32_t bits_r8(const uint4 &w, int j) {
    const uint32_t x = (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w;
    return (j & 1) ? high_r8(x) : low_r8(x);
}

// Eight codes (a 32-bit word) as eight binary16 values, exactly: word i of the
// result holds values 2 i (low half) and 2 i + 1.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

}  // namespace ptc
