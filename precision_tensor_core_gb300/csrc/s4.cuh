// s4.cuh -- device primitives of the products with grouped 4-bit integer weights
// (s4_tokens.cu, s4_experts.cu): 16-bit activations relative to a power of two,
// weight codes as binary16 operands, and one stage of 128 codes on the tensor cores.
//
// Weights.  A weight is (c - z) s: code c in -8 .. 7, scale s and zero z per row and
// group of 32, 64 or a multiple of 128 codes.  With n = c + 8 (the code with its top
// bit turned over, 0 .. 15) the nibbles lie where a binary16 subnormal has its mantissa:
// the word's bits 0 .. 3 of each half are the number n 2^-24, and bits 4 .. 7 are 16 n
// 2^-24.  So one three-input logic operation makes two operands of the tensor cores,
// exact as they are (converting them takes two), and a group's sum is
//   s 2^24 (sum of n 2^-24 x  -  (8 + z) 2^-24 sum of x).
// A word of eight codes gives four operands: codes (0, 4) and (2, 6), and with 16 n (1, 5)
// and (3, 7), whose activations are held divided by 16.  The order of k within an MMA is
// free as long as both operands agree.
//
// Activations.  Each block of 32, 64 or 128 (the smaller of that and the group) is held
// as binary16 relative to a power of two that brings its largest into [2^14, 2^15).  Those
// divided by 16 lose what lies below 2^-20 before: bfloat16's eight bits are exact from 2^-13
// on, 2^-27 of the largest, binary16's eleven from 2^-10 on, 2^-24 of it (the others four
// binary digits further); off by at most half of 2^-20, 2^-35 of the largest,
// below that, for either 16-bit type.  The block's power of two, times 2^12, and its sum
// of x 2^-24 stand beside it; the other 2^12 is the output's factor, so that neither
// bfloat16's largest nor its smallest numbers leave FP32.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "fp4.cuh"
#include "ptx.cuh"

namespace ptc {

constexpr int kS4Half = 128;         // codes of a row that one call of s4_half multiplies
constexpr int kS4Stage = 256;        // codes of a row per stage of a ring
constexpr int kS4RowBytes = 128;     // their bytes
constexpr int kS4TileBytes = 2048;   // of 16 rows
constexpr int kS4XBytes = 256;       // a token's activations of half a stage
constexpr float kS4Out = 0x1p12f;    // the output's factor

// Codes per block of activations, in units of 32, for a group size; groups per stage.
__host__ __device__ constexpr int s4_unit(int64_t group) { return group == 32 ? 1 : group == 64 ? 2 : 4; }

// ------------------------------------------------------------ activations
// The power of two of a block whose largest magnitude has the FP32 bits m (at least
// kInfBits: the token is NaN anyway), as the factor that brings it to [2^14, 2^15) and
// the block's factor.
__device__ __forceinline__ void s4_powers(uint32_t m, float &down, float &factor) {
    const int e = min(max(int(m >> 23) - 127 - 14, -126), 113);
    down = __uint_as_float(uint32_t(127 - e) << 23);
    factor = __uint_as_float(uint32_t(127 + 12 + e) << 23);
}

__device__ __forceinline__ uint32_t s4_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return reinterpret_cast<const uint32_t &>(h);
}

// Eight consecutive 16-bit activations of a block that 4 UNIT consecutive lanes hold, as
// operands (16 bytes, see above), and the block's factor and sum (in every lane).  The
// sum is that of the elements before they are held, which differ by 2^-35 of the largest
// at most.
template <int UNIT, typename X>
__device__ __forceinline__ uint4 s4_operands(const uint4 &raw, float2 &factor_sum) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
    for (int o = 1; o < 4 * UNIT; o *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float v[8];
    if constexpr (std::is_same_v<X, __half>) {
        m = __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(reinterpret_cast<const __half2 &>(w[j]));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    } else {
        m <<= 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
    float down, factor;
    s4_powers(m, down, factor);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = __fmul_rn(v[j], down);
        sum = __fadd_rn(sum, v[j]);
    }
#pragma unroll
    for (int o = 1; o < 4 * UNIT; o *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    factor_sum = make_float2(factor, __fmul_rn(sum, 0x1p-24f));
#pragma unroll
    for (int j = 1; j < 8; j += 2) v[j] = __fmul_rn(v[j], 0x1p-4f);
    return make_uint4(s4_pair(v[0], v[4]), s4_pair(v[2], v[6]), s4_pair(v[1], v[5]), s4_pair(v[3], v[7]));
}

// One FP32 activation of a block that a warp's 32 lanes hold, as one operand of 11 bits (hi,
// rounded to binary16) or, with PARTS 2, two whose sum has 22 (lo: what that left), and the
// block's factor and sum: that of the numbers held, as n = c + 8 multiplies those and (8 + z)
// takes their sum off again.  (A sum of the numbers before they are held would leave 8 + z times
// what the rounding took, about four times the codes' own size.)
template <int PARTS>
__device__ __forceinline__ void s4_operand32(float v, int lane, __half &hi, __half &lo, float2 &factor_sum) {
    float down, factor;
    s4_powers(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu), down, factor);
    const float part = __fmul_rn(__fmul_rn(v, down), (lane & 1) ? 0x1p-4f : 1.0f);
    hi = __float2half_rn(part);
    float held = __half2float(hi);
    lo = __float2half_rn(__fsub_rn(part, held));
    if constexpr (PARTS == 2) held = __fadd_rn(held, __half2float(lo));
    float sum = __fmul_rn(held, (lane & 1) ? 0x1p4f : 1.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    factor_sum = make_float2(factor, __fmul_rn(sum, 0x1p-24f));
}
// Where element e (0 .. 7) of a word lies among its operands' halves: 0, 4, 2, 6, 1, 5, 3, 7.
__device__ __forceinline__ int s4_half(int e) { return ((e & 1) << 2) | (e & 2) | (e >> 2); }

// ------------------------------------------------------------ copies
// `bytes` (a multiple of 16) from 16-byte aligned global to shared memory, signalled on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Box of a 3-D tensor: bytes of a row, rows, experts.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// A stage's rows of 128 bytes lie in the 128-byte swizzle: 16-byte piece c of row r at
// c ^ (r & 7), on 1024 bytes.  In half a stage (four pieces) the lanes of a quad take the
// words in one of two ways.  With UNIT 4, where all of it is one block, lane t takes piece
// t by one load, and the i-th pair of MMAs multiplies its word i: codes 32 t + 8 i .. + 7.
// Otherwise lane t takes word t of each piece, and the i-th pair multiplies block i.
//
// MMA rows gr and gr + 8 are the tile's rows 2 f and 2 f + 1, whose scales one load takes;
// f is such that rows whose pieces are read together differ in the swizzle's top bit.
__device__ __forceinline__ int s4_pair_of(int gr) { return ((gr & 1) << 1) | ((gr >> 1) & 1) | (gr & 4); }

// This lane's piece (UNIT 4) or word (of piece 0) of row 2 f in the first half of a stage's
// codes; the second half is 64 further by exclusive or, row 2 f + 1 at s4_next_row.
template <int UNIT>
__device__ __forceinline__ uint32_t s4_code_at(int lane) {
    const int r = 2 * s4_pair_of(lane >> 2), t = lane & 3;
    return uint32_t(r) * kS4RowBytes + (UNIT == 4 ? uint32_t(t ^ (r & 7)) << 4 : uint32_t(r & 7) << 4 | uint32_t(t) << 2);
}
__device__ __forceinline__ uint32_t s4_next_row(uint32_t at) { return (at ^ 16u) + kS4RowBytes; }

// Where the operands of activations 8 c .. 8 c + 7 of half a stage lie: 64 bytes for each
// pair of MMAs, 16 for each lane of a quad.
template <int UNIT>
__device__ __forceinline__ uint32_t s4_x_piece(int c) {
    return uint32_t(UNIT == 4 ? (c & 3) * 4 + (c >> 2) : c) << 4;
}

// ------------------------------------------------------------ products
__device__ __forceinline__ void s4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// (a & b) ^ c in one instruction (written out as C++ it became two: 23.1 us instead of 19.6 for
// one token with 16384 x 8192 weights).
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Eight codes as four operands (see the top).
__device__ __forceinline__ void s4_codes(uint32_t w, uint32_t (&a)[4]) {
    const uint32_t w8 = w >> 8;
    a[0] = and_xor(w, 0x000F000Fu, 0x00080008u);
    a[1] = and_xor(w8, 0x000F000Fu, 0x00080008u);
    a[2] = and_xor(w, 0x00F000F0u, 0x00800080u);
    a[3] = and_xor(w8, 0x00F000F0u, 0x00800080u);
}

// The scales (zeros) of two rows that lie side by side at p, or (ODD) at p and `second` on.
template <bool ODD>
__device__ __forceinline__ float2 s4_row_scales(const uint8_t *p, uint32_t second, bool bf16) {
    uint32_t u;
    if constexpr (ODD)
        u = uint32_t(*reinterpret_cast<const uint16_t *>(p)) | uint32_t(*reinterpret_cast<const uint16_t *>(p + second)) << 16;
    else
        u = *reinterpret_cast<const uint32_t *>(p);
    return bf16 ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u))
                : __half22float2(reinterpret_cast<const __half2 &>(u));
}

// Half a stage: MT tiles of 16 rows of codes with NT sets of eight tokens.  Offsets in
// shared memory (`smem`): codes, this lane's s4_code_at of the half; scales[m], those of this
// lane's row 2 f in the half's first group (ODD: that of row 2 f + 1 is second[m] on), `step` bytes
// from group to group, the zeros `zeros` bytes behind (0: none).  x(i, n, p): the operands
// of this lane's token of set n for the i-th pair of MMAs, p 1 those of the low parts (PARTS
// 2); ps(g, n): factor and sum of block g of this lane's two tokens of set n.  The half has
// 4 / UNIT blocks, of which `blocks` are there, in SG groups.
// tot += s factor (sum of n x - (8 + z) sum of x).
template <int MT, int NT, int UNIT, int SG, int PARTS, bool ODD, typename OPERANDS, typename SUMS>
__device__ __forceinline__ void s4_half_stage(float (&tot)[MT][NT][4], const uint8_t *smem, uint32_t codes,
                                              const uint32_t (&scales)[MT], const uint32_t (&second)[MT], uint32_t step,
                                              uint32_t zeros, bool bf16, OPERANDS x, SUMS ps, int blocks) {
    constexpr int BLOCKS = 4 / UNIT;
    uint4 wide[MT][2];
    if constexpr (UNIT == 4) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wide[m][h] = *reinterpret_cast<const uint4 *>(smem + (h ? s4_next_row(codes) : codes) + m * kS4TileBytes);
    }
#pragma unroll
    for (int g = 0; g < BLOCKS; ++g) {
        if (BLOCKS > 1 && g >= blocks) break;
        float d[MT][NT][4];
#pragma unroll
        for (int u = 0; u < UNIT; ++u) {
            const int i = g * UNIT + u;
            uint4 xv[NT][PARTS];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    xv[n][p] = x(i, n, p);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t w[2], a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (UNIT == 4)
                        w[h] = i == 0 ? wide[m][h].x : i == 1 ? wide[m][h].y : i == 2 ? wide[m][h].z : wide[m][h].w;
                    else
                        w[h] = *reinterpret_cast<const uint32_t *>(smem + ((h ? s4_next_row(codes) : codes) ^ (uint32_t(i) << 4)) +
                                                                   m * kS4TileBytes);
                    s4_codes(w[h], a[h]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        if (u == 0 && p == 0)
                            s4_mma(d[m][n], a[0][0], a[1][0], a[0][1], a[1][1], xv[n][p].x, xv[n][p].y, zero);
                        else
                            s4_mma(d[m][n], a[0][0], a[1][0], a[0][1], a[1][1], xv[n][p].x, xv[n][p].y, d[m][n]);
                        s4_mma(d[m][n], a[0][2], a[1][2], a[0][3], a[1][3], xv[n][p].z, xv[n][p].w, d[m][n]);
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t *at = smem + scales[m] + uint32_t(g * SG / BLOCKS) * step;
            const float2 s = s4_row_scales<ODD>(at, second[m], bf16);
            float2 z = make_float2(8.0f, 8.0f);
            if (zeros != 0) {
                const float2 more = s4_row_scales<ODD>(at + zeros, second[m], bf16);
                z = make_float2(__fadd_rn(z.x, more.x), __fadd_rn(z.y, more.y));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 q = ps(g, n);
                float(&o)[4] = tot[m][n];
                const float(&v)[4] = d[m][n];
                o[0] = __fmaf_rn(s.x, __fmul_rn(q.x, __fmaf_rn(-z.x, q.y, v[0])), o[0]);
                o[1] = __fmaf_rn(s.x, __fmul_rn(q.z, __fmaf_rn(-z.x, q.w, v[1])), o[1]);
                o[2] = __fmaf_rn(s.y, __fmul_rn(q.x, __fmaf_rn(-z.y, q.y, v[2])), o[2]);
                o[3] = __fmaf_rn(s.y, __fmul_rn(q.z, __fmaf_rn(-z.y, q.w, v[3])), o[3]);
            }
        }
    }
}

// ------------------------------------------------------------ host side
// Weights of one matrix (or of the experts') as the C entry points take them.
struct S4Weights {
    const void *codes;
    int64_t pitch;    // bytes between rows
    int64_t expert;   // bytes between experts' matrices (0: one)
    const void *scales, *zeros;
    int64_t rows, cols, group, experts;
    int64_t groups() const { return (cols + group - 1) / group; }
    int64_t tiles() const { return (rows + 15) / 16; }
    uint64_t scale_bytes() const { return uint64_t(experts) * uint64_t(tiles()) * uint64_t(groups()) * 32u; }
};

}  // namespace ptc
