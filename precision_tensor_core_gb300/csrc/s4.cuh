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
// as binary16 relative to a power of two that brings its largest into [2^14, 2^15): exact
// for elements down to 2^-28 of the largest, off by at most 2^-35 of the largest
// below that, for either 16-bit type.  The block's power of two, times 2^12, and its sum
// of x 2^-24 stand beside it; the other 2^12 is the output's factor, so that neither
// bfloat16's largest nor its smallest numbers leave FP32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "ptx.cuh"

namespace ptc {

constexpr int kS4Stage = 128;        // codes of a row per stage
constexpr int kS4RowBytes = 64;      // their bytes
constexpr int kS4TileBytes = 1024;   // of 16 rows
constexpr int kS4XBytes = 256;       // a token's activations of a stage
constexpr float kS4Out = 0x1p12f;    // the output's factor

// Codes per block of activations, in units of 32, for a group size; groups per stage.
__host__ __device__ constexpr int s4_unit(int64_t group) { return group == 32 ? 1 : group == 64 ? 2 : 4; }

// ------------------------------------------------------------ activations
// Eight consecutive activations of a block that 4 UNIT consecutive lanes hold, as
// operands (a word of 16 bytes, see above), and the block's factor and sum (in every
// lane).  LO also gives the operands of what the rounding to binary16 left, for FP32
// values: 22 bits in all.
template <int UNIT, bool LO>
__device__ __forceinline__ void s4_operands(const float (&v)[8], uint4 &hi, uint4 &lo, float2 &factor_sum) {
    uint32_t m = 0;  // largest finite magnitude, as FP32 bits
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t u = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        m = max(m, u < kInfBits ? u : 0u);
    }
#pragma unroll
    for (int o = 1; o < 4 * UNIT; o *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const int e = max(int(m >> 23) - 127 - 14, -126);
    const float down = __uint_as_float(uint32_t(127 - e) << 23);
    __half h[8], l[8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float part = (j & 1) ? 0x1p-4f : 1.0f;
        const float x = __fmul_rn(__fmul_rn(v[j], down), part);
        h[j] = __float2half_rn(x);
        float held = __half2float(h[j]);
        if constexpr (LO) {
            l[j] = __float2half_rn(__fsub_rn(x, held));
            held = __fadd_rn(held, __half2float(l[j]));
        }
        sum = __fmaf_rn(held, (j & 1) ? 0x1p4f : 1.0f, sum);
    }
#pragma unroll
    for (int o = 1; o < 4 * UNIT; o *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    factor_sum = make_float2(__uint_as_float(uint32_t(127 + 12 + e) << 23), __fmul_rn(sum, 0x1p-24f));
    auto pair = [](__half a, __half b) { return uint32_t(__half_as_ushort(a)) | uint32_t(__half_as_ushort(b)) << 16; };
    hi = make_uint4(pair(h[0], h[4]), pair(h[2], h[6]), pair(h[1], h[5]), pair(h[3], h[7]));
    if constexpr (LO) lo = make_uint4(pair(l[0], l[4]), pair(l[2], l[6]), pair(l[1], l[5]), pair(l[3], l[7]));
}

// ------------------------------------------------------------ copies
// 16 (8) bytes to shared memory, `n` of them from global memory and zeros after them.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Where 16-byte piece c (0 .. 3) of row r of a tile of 16 rows lies: rows that are read
// together differ in their banks.
__device__ __forceinline__ uint32_t s4_piece(int r, int c) { return uint32_t(r) * kS4RowBytes + (uint32_t(c ^ ((r >> 1) & 3)) << 4); }

// Where 16-byte piece c (block c / 4, lane c % 4) of token j's stage lies, from the token's start.
__device__ __forceinline__ uint32_t s4_x_piece(int j, int c) { return uint32_t(c ^ ((j & 1) << 2)) << 4; }

// A scale or zero of either 16-bit type.
__device__ __forceinline__ float s4_scale(const uint8_t *p, bool bf16) {
    const uint16_t u = *reinterpret_cast<const uint16_t *>(p);
    return bf16 ? __uint_as_float(uint32_t(u) << 16) : __half2float(__ushort_as_half(u));
}

// ------------------------------------------------------------ products
__device__ __forceinline__ void s4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Eight codes as four operands (see the top).
__device__ __forceinline__ void s4_codes(uint32_t w, uint32_t (&a)[4]) {
    const uint32_t w8 = w >> 8;
    a[0] = (w & 0x000F000Fu) ^ 0x00080008u;
    a[1] = (w8 & 0x000F000Fu) ^ 0x00080008u;
    a[2] = (w & 0x00F000F0u) ^ 0x00800080u;
    a[3] = (w8 & 0x00F000F0u) ^ 0x00800080u;
}

// One stage: MT tiles of 16 rows of codes (`codes`: of this lane's word of row 0, see
// code_at) with NT sets of eight tokens.  `scales` (and `zeros`, or NULL): [tile][group][16]
// of this stage; x[n]: this lane's operands of token set n (of block 0), x_lo: those of
// the low parts, PARTS 2; ps: factors and sums, [block of activations][8 NT tokens].
// tot += s factor (sum of n x - (8 + z) sum of x).
template <int MT, int NT, int UNIT, int PARTS>
__device__ __forceinline__ void s4_stage(float (&tot)[MT][NT][4], const uint8_t *codes, const uint8_t *scales,
                                         const uint8_t *zeros, bool bf16, const uint8_t *const (&x)[NT], uint32_t x_lo,
                                         const uint8_t *ps, int lane) {
    constexpr int GROUPS = 4 / UNIT;
    const int gr = lane >> 2, t = lane & 3;
    const uint32_t turn = uint32_t((gr >> 1) & 3);   // the same for rows gr and gr + 8
    const uint32_t x_turn = uint32_t(gr & 1);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        float d[MT][NT][4];
#pragma unroll
        for (int u = 0; u < UNIT; ++u) {
            const int b = g * UNIT + u;
            uint4 xv[NT][PARTS];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    xv[n][p] = *reinterpret_cast<const uint4 *>(x[n] + ((uint32_t(b) ^ x_turn) << 6) + uint32_t(p) * x_lo);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint8_t *row = codes + m * kS4TileBytes + ((uint32_t(b) ^ turn) << 4);
                uint32_t a[4], c[4];
                s4_codes(*reinterpret_cast<const uint32_t *>(row), a);
                s4_codes(*reinterpret_cast<const uint32_t *>(row + 8 * kS4RowBytes), c);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        if (u == 0 && p == 0)
                            s4_mma(d[m][n], a[0], c[0], a[1], c[1], xv[n][p].x, xv[n][p].y, zero);
                        else
                            s4_mma(d[m][n], a[0], c[0], a[1], c[1], xv[n][p].x, xv[n][p].y, d[m][n]);
                        s4_mma(d[m][n], a[2], c[2], a[3], c[3], xv[n][p].z, xv[n][p].w, d[m][n]);
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t at = uint32_t((m * GROUPS + g) * 16 + gr) * 2u;
            const float s0 = s4_scale(scales + at, bf16), s1 = s4_scale(scales + at + 16, bf16);
            float z0 = 8.0f, z1 = 8.0f;
            if (zeros != nullptr) {
                z0 = __fadd_rn(z0, s4_scale(zeros + at, bf16));
                z1 = __fadd_rn(z1, s4_scale(zeros + at + 16, bf16));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 q = *reinterpret_cast<const float4 *>(ps + (g * 8 * NT + 8 * n + 2 * t) * 8);
                float(&o)[4] = tot[m][n];
                const float(&v)[4] = d[m][n];
                o[0] = __fmaf_rn(s0, __fmul_rn(q.x, __fmaf_rn(-z0, q.y, v[0])), o[0]);
                o[1] = __fmaf_rn(s0, __fmul_rn(q.z, __fmaf_rn(-z0, q.w, v[1])), o[1]);
                o[2] = __fmaf_rn(s1, __fmul_rn(q.x, __fmaf_rn(-z1, q.y, v[2])), o[2]);
                o[3] = __fmaf_rn(s1, __fmul_rn(q.z, __fmaf_rn(-z1, q.w, v[3])), o[3]);
            }
        }
    }
}

// This lane's word of row lane / 4 in a stage's codes.
__device__ __forceinline__ uint32_t s4_code_at(int lane) { return uint32_t(lane >> 2) * kS4RowBytes + uint32_t(lane & 3) * 4u; }

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
