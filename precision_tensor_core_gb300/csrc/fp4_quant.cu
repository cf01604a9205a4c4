// fp4_quant.cu -- dropout, quantisation to the microscaled 4-bit formats and
// the way back (ptc_dropout, ptc_quantize_fp4, ptc_dequantize_fp4 of
// include/ptc.h).  All of them read and write each byte once and are bound by
// memory traffic; the random numbers are made where they are used, so no mask
// is ever stored.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
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

// Position of a thread in a rows x groups walk with a fixed stride: one
// division at the start, additions after it.
struct Walk {
    int64_t row, drow;
    uint32_t group, dgroup, groups;
    __device__ __forceinline__ Walk(int64_t index, int64_t stride, uint32_t groups_) : groups(groups_) {
        row = index / groups;
        group = uint32_t(index - row * groups);
        drow = stride / groups;
        dgroup = uint32_t(stride - drow * groups);
    }
    __device__ __forceinline__ void next() {
        row += drow;
        group += dgroup;
        if (group >= groups) {
            group -= groups;
            ++row;
        }
    }
};

using yes = std::integral_constant<bool, true>;
using no = std::integral_constant<bool, false>;

struct DropArgs {
    uint32_t kept;  // of 65536; 65536: nothing is dropped
    float scale;    // 65536 / kept
    RngArgs rng;
};

// ------------------------------------------------------------ dropout
// y = [r < kept] x * (65536 / kept) (+ residual), eight elements of a row per
// step: 2 to 3 times 16 bytes of traffic and one generator call, whose twenty
// wide products (a quarter of the integer rate each) come close to the traffic's
// time.  8192 x 8192 bfloat16: 60.6 us with a residual (6.6 TB/s, the copy
// rate), 50.4 us without (5.3 TB/s, bound by the random numbers); 4096 x 2048 float32
// to bfloat16 8.1 us.
//
// O is the type of y: T, or a 16-bit type for FP32 x (no residual then), so that
// an FP32 product is dropped out and rounded once.
template <typename T, typename O, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, int64_t ldx, const O *res, int64_t ldr, O *y,
                                                      int64_t ldy, int64_t rows, int64_t cols, DropArgs d) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t groups = uint32_t((cols + 7) / 8);
    Walk w(int64_t(blockIdx.x) * blockDim.x + threadIdx.x, int64_t(gridDim.x) * blockDim.x, groups);
    for (; w.row < rows; w.next()) {
        const int64_t c = int64_t(w.group) * 8;
        const int n = int(min(int64_t(8), cols - c));
        const Pack8<T> a = load8(x + w.row * ldx + c, n, true);
        Pack8<O> r;
        float o[8];
        if constexpr (RES) r = load8(res + w.row * ldr + c, n, true);
        const uint4 bits = random_bits8(d.rng, kRngDropout, uint32_t(w.row), w.group);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // Selected, not multiplied by zero: a dropped infinity or NaN leaves +0.
            float v = bits16(bits, j) < d.kept ? __fmul_rn(to_float(a.get(j)), d.scale) : 0.0f;
            if constexpr (RES) v = __fadd_rn(v, to_float(r.get(j)));
            o[j] = v;
        }
        store8(y + w.row * ldy + c, round8<O>(o), n, true);
    }
}

// The same for rows that are not 16-byte aligned: a warp takes 256 columns of a
// row, each lane makes the eight keep bits of its group, and loads and stores
// take 32 consecutive elements at a time, whose bits come from the lane that
// made them.  (Eight elements per lane, one store each, touched every sector
// eight times: 2047 x 1003 binary16 took 7.5 us, and takes 3.9; 8191 x 8191
// float32 84 us, 6.4 TB/s.)
template <typename T, typename O, bool RES>
__global__ void __launch_bounds__(256) dropout_ragged_kernel(const T *x, int64_t ldx, const O *res, int64_t ldr, O *y,
                                                             int64_t ldy, int64_t rows, int64_t cols, DropArgs d) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    Walk w((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32, int64_t(gridDim.x) * blockDim.x / 32,
           uint32_t((cols + 255) / 256));
    for (; w.row < rows; w.next()) {
        const int64_t c0 = int64_t(w.group) * 256;
        const int n = int(min(int64_t(256), cols - c0));
        const T *xr = x + w.row * ldx + c0;
        const O *rr = RES ? res + w.row * ldr + c0 : nullptr;
        O *yr = y + w.row * ldy + c0;
        T a[8];
        O r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 32 * i + lane;
            a[i] = c < n ? xr[c] : from_float<T>(0.0f);
            if constexpr (RES) r[i] = c < n ? rr[c] : from_float<O>(0.0f);
        }
        const uint4 bits = random_bits8(d.rng, kRngDropout, uint32_t(w.row), uint32_t(c0 / 8) + lane);
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) keep |= (bits16(bits, j) < d.kept ? 1u : 0u) << j;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 32 * i + lane;
            const uint32_t k = __shfl_sync(0xFFFFFFFFu, keep, 4 * i + (lane >> 3)) >> (lane & 7);
            float v = (k & 1u) ? __fmul_rn(to_float(a[i]), d.scale) : 0.0f;
            if constexpr (RES) v = __fadd_rn(v, to_float(r[i]));
            if (c < n) yr[c] = from_float<O>(v);
        }
    }
}

// ------------------------------------------------------------ quantisation
struct QuantArgs {
    int64_t rows, cols, ldx;
    uint8_t *codes;   // rows of the matrix: codes, pitch, tiled scales
    int64_t pitch;
    uint8_t *scales;
    uint8_t *codes_t;  // its columns
    int64_t pitch_t;
    uint8_t *scales_t;
    const float *g;  // matrix scale (NULL: 1)
    DropArgs drop;
    int vec;
};

// FP32 values of eight loaded elements after dropout.
template <typename T, bool DROP>
__device__ __forceinline__ void dropped8(const Pack8<T> &a, const DropArgs &d, int64_t row, uint32_t group,
                                         float (&v)[8]) {
    if constexpr (DROP) {
        const uint4 bits = random_bits8(d.rng, kRngDropout, uint32_t(row), group);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = bits16(bits, j) < d.kept ? __fmul_rn(to_float(a.get(j)), d.scale) : 0.0f;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_float(a.get(j));
    }
}

// The FP32 bits of the largest magnitude of eight elements as they came; of
// 16-bit elements in pairs (their bits order like the magnitudes).
template <typename T>
__device__ __forceinline__ uint32_t max_abs8(const Pack8<T> &p) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(to_float(p.get(j))) & 0x7FFFFFFFu);
        return m;
    } else {
        const uint4 &w = p.v[0];
        constexpr uint32_t K = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(w.x & K, w.y & K), __vmaxu2(w.z & K, w.w & K));
        const uint16_t top = uint16_t(max(m & 0xFFFFu, m >> 16));
        return __float_as_uint(to_float(reinterpret_cast<const T &>(top)));
    }
}

__device__ __forceinline__ uint32_t max_abs8(const float (&v)[8]) {
    uint32_t m = 0;  // of the bits, so that infinities and NaN come out on top
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
}

// The bits of a magnitude after dropout's scaling (monotonic, so the largest
// stays the largest; a NaN stays one, whatever its sign).
__device__ __forceinline__ uint32_t scaled_bits(uint32_t m, float scale) {
    return __float_as_uint(__fmul_rn(__uint_as_float(m), scale)) & 0x7FFFFFFFu;
}

// Eight codes of values v, whose signs are those of `from`, with the block's scale.
// (v is lifted in place.)
template <bool NV, bool SR, bool LIFT, typename S>
__device__ __forceinline__ uint32_t codes8(float (&v)[8], const S &from, uint32_t amax, const BlockScale<NV> &scale,
                                           const uint4 &bits) {
    uint32_t q = 0;
    scale.template lift8<LIFT>(v);
    if constexpr (SR) {
        uint32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = code_stochastic(scale.magnitude(v[j]), bits_r8(bits, j));
        q = pack_stochastic(c, signs8(from));
    } else {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = scale.apply(v[j]);
        q = codes_nearest(s);
    }
    return amax < kInfBits ? q : 0u;
}

// Rows only.  A warp takes U x 256 columns of a row, a lane U times eight of
// them, all loads before the first use: the block's maximum by one or two
// shuffles, codes as 4 bytes per lane (128 contiguous bytes per warp), scales
// gathered to one 4-byte store per tile.  Rows past the last one to the end of
// the scale tile get zero scales.  8192 x 8192 bfloat16: 28.4 us to mxfp4 (6.0
// TB/s, 90% of the copy rate) and 39.0 to nvfp4 to nearest, where the elements'
// quotients show; 56 and 67 us stochastically, bound by the issue of
// instructions (random numbers and rounding).  8191 x 8191, whose rows are not
// aligned: 53 us to mxfp4.
template <typename T, bool NV, bool SR, bool DROP, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T *x, const QuantArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LPB = NV ? 2 : 4;          // lanes per block
    constexpr int LPT = 4 * LPB;             // lanes per scale word
    const int lane = threadIdx.x & 31;
    const MatrixScale<NV> g(a.g);
    const int64_t ktiles = (a.cols + 8 * LPT - 1) / (8 * LPT);
    const int64_t rows_p = (a.rows + 127) / 128 * 128;
    const int cols = int(a.cols);
    Walk w((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32, int64_t(gridDim.x) * blockDim.x / 32,
           uint32_t((cols + 256 * U - 1) / (256 * U)));
    for (; w.row < rows_p; w.next()) {
        const int c0 = int(w.group) * (256 * U);
        uint8_t *const scale_row = a.scales + scale_word(w.row, 0, ktiles);
        if (w.row >= a.rows) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t kt = (c0 + 256 * u + lane * 8) / (8 * LPT);
                if (lane % LPT == 0 && kt < ktiles) *reinterpret_cast<uint32_t *>(scale_row + kt * kScaleTile) = 0u;
            }
            continue;
        }
        const T *const row = x + w.row * a.ldx;
        uint8_t *const code_row = a.codes + w.row * a.pitch;
        // Whole: 256 U aligned columns that all exist.  Lifted:
        // the matrix scale is small (MatrixScale).
        auto chunk = [&](auto whole, auto lifted) {
            constexpr bool WHOLE = decltype(whole)::value, LIFT = decltype(lifted)::value;
            Pack8<T> p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + 256 * u + lane * 8;
                const int n = WHOLE ? 8 : max(0, min(8, cols - c));
                p[u] = load8(row + (n > 0 ? c : 0), n, WHOLE || a.vec != 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + 256 * u + lane * 8;
                if (!WHOLE && c0 + 256 * u >= cols) break;  // (uniform)
                float v[8];
                uint32_t m;
                if constexpr (DROP) {
                    dropped8<T, DROP>(p[u], a.drop, w.row, uint32_t(c / 8), v);
                    if (!WHOLE && c + 8 > cols) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j >= cols) v[j] = 0.0f;
                    }
                    m = max_abs8(v);
                } else {
                    dropped8<T, DROP>(p[u], a.drop, w.row, uint32_t(c / 8), v);
                    m = max_abs8(p[u]);
                }
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                if constexpr (!NV) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                uint32_t byte;
                const BlockScale<NV> scale = block_scale<NV, SR, LIFT>(m, g, byte);
                uint4 bits = make_uint4(0, 0, 0, 0);
                if constexpr (SR) bits = random_bits8(a.drop.rng, kRngRounding, uint32_t(w.row), uint32_t(c / 8));
                uint32_t q;
                if constexpr (DROP)
                    q = codes8<NV, SR, LIFT>(v, v, m, scale, bits);
                else
                    q = codes8<NV, SR, LIFT>(v, p[u], m, scale, bits);
                if (WHOLE || c < (cols + 31) / 32 * 32) *reinterpret_cast<uint32_t *>(code_row + c / 2) = q;
                // Four blocks' bytes to one word (held by the first lane of the four).
                uint32_t word = byte;
                word |= __shfl_down_sync(0xFFFFFFFFu, word, LPB) << 8;
                word |= __shfl_down_sync(0xFFFFFFFFu, word, 2 * LPB) << 16;
                const int64_t kt = c / (8 * LPT);
                if (lane % LPT == 0 && (WHOLE || kt < ktiles))
                    *reinterpret_cast<uint32_t *>(scale_row + kt * kScaleTile) = word;
            }
        };
        if (NV && __builtin_expect(g.small, 0))
            chunk(no(), std::integral_constant<bool, NV>());
        else if (a.vec != 0 && c0 + 256 * U <= cols)
            chunk(yes(), no());
        else
            chunk(no(), no());
    }
}

// Columns (and rows).  A CTA takes 128 rows x 64 columns: read once (four
// loads per thread in flight), dropped out, kept in shared memory as they came
// (dropped ones +0) beside their rounding bits; rows are quantised on the way
// in, eight lanes per row.  For the columns a lane takes two adjacent columns
// and a warp 16 rows: a block of nvfp4, half of one of mxfp4, whose maximum two
// warps share.  Codes and scale bytes go through shared memory so that a
// column's 64 bytes are written together.  8192 x 8192 bfloat16 to mxfp4 both
// ways: 44 us to nearest (30.6 us of traffic), 81 us stochastically, with an
// instruction issued in 79% of the cycles (19 per code: 7.6 integer, 7.6 multiply).
// Positions are 32-bit steps from the tile's corner and tiles that exist whole
// test nothing: 64-bit ones and their tests took 53 and 105 us.  (128 x 128 tiles
// of one column per thread took 33 us for 2047 x 1003 both ways, these take 6.7:
// four times the CTAs.  Five or six CTAs per SM instead of four made no
// difference.)
constexpr int kTileR = 128, kTileC = 64;
constexpr int kCodePitch = 80;  // of a column's 64 code bytes in shared memory

template <typename T, bool SR>
constexpr size_t tile_smem() {
    return size_t(kTileR) * kTileC * (sizeof(T) + (SR ? 2 : 0));
}

template <typename T, bool NV, bool SR, bool DROP, bool ROWS>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const T *x, const QuantArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    T *xs = reinterpret_cast<T *>(smem);
    uint16_t *rs = reinterpret_cast<uint16_t *>(smem + size_t(kTileR) * kTileC * sizeof(T));
    __shared__ __align__(16) uint8_t ct[kTileC * kCodePitch];
    __shared__ __align__(8) uint8_t sct[kTileC * 8];
    __shared__ uint32_t top[NV ? 1 : 8 * kTileC];
    griddep_wait();
    griddep_launch_dependents();
    constexpr int KW = NV ? 64 : 128;  // columns (rows) per scale word
    const MatrixScale<NV> g(a.g);
    const int64_t tiles_c = (a.cols + kTileC - 1) / kTileC;
    const int64_t kt_rows = (a.cols + KW - 1) / KW, kt_cols = (a.rows + KW - 1) / KW;
    const int64_t r0 = blockIdx.x / tiles_c * kTileR, c0 = (blockIdx.x % tiles_c) * kTileC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Whole: all rows and columns of the tile exist, and rows are aligned.  Lifted: as above.
    auto rows_in = [&](auto whole, auto lifted) {
        constexpr bool WHOLE = decltype(whole)::value, LIFT = decltype(lifted)::value;
        const int grp = threadIdx.x & 7, lr0 = threadIdx.x >> 3;
        const int rows_left = WHOLE ? kTileR : int(min(int64_t(kTileR), a.rows - r0));
        const int n_cols = WHOLE ? 8 : int(max(int64_t(0), min(int64_t(8), a.cols - c0 - grp * 8)));
        const T *px = x + (r0 + lr0) * a.ldx + c0 + grp * 8;
        const int64_t x_step = 32 * a.ldx, code_step = 32 * a.pitch;
        uint8_t *code = nullptr, *scale_at = nullptr;
        bool code_exists = true;
        if constexpr (ROWS) {
            code = a.codes + (r0 + lr0) * a.pitch + (c0 + grp * 8) / 2;
            code_exists = WHOLE || c0 + grp * 8 < (a.cols + 31) / 32 * 32;
            scale_at = a.scales + scale_word(r0 + lr0, c0 / KW, kt_rows);  // 32 rows further: 4 bytes
        }
        const uint32_t row = uint32_t(r0) + lr0, group = uint32_t(c0 / 8) + grp;
        Pack8<T> p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = WHOLE || lr0 + 32 * i < rows_left ? n_cols : 0;
            p[i] = load8(n > 0 ? px + i * x_step : x, n, WHOLE || a.vec != 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int lr = lr0 + 32 * i;
            const bool exists = WHOLE || lr < rows_left;
            if constexpr (DROP) {
                const uint4 bits = random_bits8(a.drop.rng, kRngDropout, row + 32 * i, group);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (bits16(bits, j) >= a.drop.kept) p[i].set(j, from_float<T>(0.0f));
            }
            uint4 bits = make_uint4(0, 0, 0, 0);
            if constexpr (SR) {
                bits = random_bits8(a.drop.rng, kRngRounding, row + 32 * i, group);
                *reinterpret_cast<uint4 *>(rs + lr * kTileC + grp * 8) = bits;
            }
#pragma unroll
            for (int w = 0; w < Pack8<T>::W; ++w) reinterpret_cast<uint4 *>(xs + lr * kTileC + grp * 8)[w] = p[i].v[w];
            if constexpr (ROWS) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = DROP ? __fmul_rn(to_float(p[i].get(j)), a.drop.scale) : to_float(p[i].get(j));
                uint32_t m = max_abs8(p[i]);
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                if constexpr (!NV) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                if constexpr (DROP) m = scaled_bits(m, a.drop.scale);
                uint32_t byte;
                const BlockScale<NV> scale = block_scale<NV, SR, LIFT>(m, g, byte);
                const uint32_t q = codes8<NV, SR, LIFT>(v, p[i], m, scale, bits);
                if (exists && code_exists) *reinterpret_cast<uint32_t *>(code + i * code_step) = q;
                // The row's scale bytes of these 64 columns: a word (nvfp4), or half
                // of one; a last first half also clears the other.
                uint32_t word = exists ? byte : 0u;
                uint8_t *dst = scale_at + 4 * i;
                if constexpr (NV) {
                    word |= __shfl_down_sync(0xFFFFFFFFu, word, 2) << 8;
                    word |= __shfl_down_sync(0xFFFFFFFFu, word, 4) << 16;
                    if (grp == 0) *reinterpret_cast<uint32_t *>(dst) = word;
                } else {
                    word |= __shfl_down_sync(0xFFFFFFFFu, word, 4) << 8;
                    if (grp == 0) {
                        const int half = int(c0 / kTileC) & 1;
                        if (half == 0 && c0 + kTileC >= a.cols)
                            *reinterpret_cast<uint32_t *>(dst) = word & 0xFFFFu;
                        else
                            *reinterpret_cast<uint16_t *>(dst + 2 * half) = uint16_t(word);
                    }
                }
            }
        }
    };
    if (NV && __builtin_expect(g.small, 0))
        rows_in(no(), std::integral_constant<bool, NV>());
    else if (a.vec != 0 && r0 + kTileR <= a.rows && c0 + kTileC <= a.cols)
        rows_in(yes(), no());
    else
        rows_in(no(), no());
    __syncthreads();

    struct alignas(2 * sizeof(T)) Two {
        T a, b;
    };
    Two t[16];  // columns 2 lane and 2 lane + 1, rows 16 warp ..
    uint32_t ma = 0, mb = 0;
    uint32_t both = 0;  // largest magnitudes of 16-bit elements, in pairs
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        t[i] = *reinterpret_cast<const Two *>(xs + (16 * warp + i) * kTileC + 2 * lane);
        if constexpr (sizeof(T) == 2) {
            both = __vmaxu2(both, reinterpret_cast<const uint32_t &>(t[i]) & 0x7FFF7FFFu);
        } else {
            ma = max(ma, __float_as_uint(t[i].a) & 0x7FFFFFFFu);
            mb = max(mb, __float_as_uint(t[i].b) & 0x7FFFFFFFu);
        }
    }
    if constexpr (sizeof(T) == 2) {
        const Two top2 = reinterpret_cast<const Two &>(both);
        ma = __float_as_uint(to_float(top2.a));
        mb = __float_as_uint(to_float(top2.b));
    }
    if constexpr (DROP) {
        ma = scaled_bits(ma, a.drop.scale);
        mb = scaled_bits(mb, a.drop.scale);
    }
    if constexpr (!NV) {
        top[warp * kTileC + 2 * lane] = ma;
        top[warp * kTileC + 2 * lane + 1] = mb;
        __syncthreads();
        ma = max(ma, top[(warp ^ 1) * kTileC + 2 * lane]);
        mb = max(mb, top[(warp ^ 1) * kTileC + 2 * lane + 1]);
    }
    uint32_t ba, bb;
    uint32_t qa[2] = {0u, 0u}, qb[2] = {0u, 0u};
    auto columns = [&](auto lifted) {
        constexpr bool LIFT = decltype(lifted)::value;
        const BlockScale<NV> sa = block_scale<NV, SR, LIFT>(ma, g, ba), sb = block_scale<NV, SR, LIFT>(mb, g, bb);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float va[8], vb[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                va[j] = to_float(t[8 * w + j].a);
                vb[j] = to_float(t[8 * w + j].b);
                if constexpr (DROP) {
                    va[j] = __fmul_rn(va[j], a.drop.scale);
                    vb[j] = __fmul_rn(vb[j], a.drop.scale);
                }
            }
            sa.template lift8<LIFT>(va);
            sb.template lift8<LIFT>(vb);
            if constexpr (SR) {
                uint32_t ca[8], cb[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t r = *reinterpret_cast<const uint32_t *>(rs + (16 * warp + 8 * w + j) * kTileC + 2 * lane);
                    ca[j] = code_stochastic(sa.magnitude(va[j]), low_r8(r));
                    cb[j] = code_stochastic(sb.magnitude(vb[j]), high_r8(r));
                }
                Signs8 na, nb;
                if constexpr (sizeof(T) == 2) {
                    auto word = [&](int j) { return reinterpret_cast<const uint32_t &>(t[8 * w + j]); };
                    half_signs(word(0), word(2), word(4), word(6), na.even, nb.even);
                    half_signs(word(1), word(3), word(5), word(7), na.odd, nb.odd);
                } else {
                    na = signs8(va);
                    nb = signs8(vb);
                }
                qa[w] = pack_stochastic(ca, na);
                qb[w] = pack_stochastic(cb, nb);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    va[j] = sa.apply(va[j]);
                    vb[j] = sb.apply(vb[j]);
                }
                qa[w] = codes_nearest(va);
                qb[w] = codes_nearest(vb);
            }
            qa[w] = ma < kInfBits ? qa[w] : 0u;
            qb[w] = mb < kInfBits ? qb[w] : 0u;
        }
    };
    if (NV && __builtin_expect(g.small, 0))
        columns(std::integral_constant<bool, NV>());
    else
        columns(no());
    *reinterpret_cast<uint2 *>(ct + (2 * lane) * kCodePitch + 8 * warp) = make_uint2(qa[0], qa[1]);
    *reinterpret_cast<uint2 *>(ct + (2 * lane + 1) * kCodePitch + 8 * warp) = make_uint2(qb[0], qb[1]);
    if (NV || (warp & 1) == 0) {
        const int at = NV ? warp : warp >> 1;
        sct[(2 * lane) * 8 + at] = uint8_t(ba);
        sct[(2 * lane + 1) * 8 + at] = uint8_t(bb);
    }
    __syncthreads();
    {
        const int lc = threadIdx.x >> 2, piece = threadIdx.x & 3;
        const int64_t col = c0 + lc;
        if (col < a.cols && r0 + 32 * piece < a.rows)
            *reinterpret_cast<uint4 *>(a.codes_t + col * a.pitch_t + r0 / 2 + 16 * piece) =
                *reinterpret_cast<const uint4 *>(ct + lc * kCodePitch + 16 * piece);
        // Scale words: one (mxfp4) or two (nvfp4) per column; columns past the last
        // to the end of the 128-row scale tile get zeros.
        constexpr int W = NV ? 2 : 1;
        if (piece < W) {
            const int64_t kt = r0 / KW + piece;
            if (kt < kt_cols) {
                const uint32_t word = *reinterpret_cast<const uint32_t *>(sct + lc * 8 + 4 * piece);
                *reinterpret_cast<uint32_t *>(a.scales_t + scale_word(col, kt, kt_cols)) = col < a.cols ? word : 0u;
                if (c0 + kTileC >= a.cols && c0 % 128 == 0)
                    *reinterpret_cast<uint32_t *>(a.scales_t + scale_word(col + kTileC, kt, kt_cols)) = 0u;
            }
        }
    }
}

// ------------------------------------------------------------ back to values
// value = code x scale (x matrix scale), each product in FP32, rounded once
// more to the output type.  A warp takes U x 256 columns of a row, a lane U
// times eight of them, all loads before the first use.  8192 x 8192 mxfp4 to
// bfloat16: 31.0 us, 5.5 TB/s, bound by the writes.
template <typename T, bool NV, int U>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *codes, int64_t pitch, const uint8_t *scales,
                                                         const float *gp, int64_t rows, int64_t cols, T *y,
                                                         int64_t ldy, int vec) {
    griddep_wait();
    griddep_launch_dependents();
    const bool has_g = gp != nullptr;
    const float g = has_g ? __ldg(gp) : 1.0f;
    constexpr int EPB = NV ? 16 : 32;
    const int64_t ktiles = (cols + 4 * EPB - 1) / (4 * EPB);
    const int lane = threadIdx.x & 31;
    Walk w((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32, int64_t(gridDim.x) * blockDim.x / 32,
           uint32_t((cols + 256 * U - 1) / (256 * U)));
    __shared__ __align__(16) T turn[8][256];  // a warp's 256 values where rows are not aligned
    for (; w.row < rows; w.next()) {
        const int64_t c0 = int64_t(w.group) * (256 * U) + lane * 8;
        uint32_t q[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + 256 * u;
            q[u] = b[u] = 0u;
            if (c < cols) {
                q[u] = __ldcs(reinterpret_cast<const uint32_t *>(codes + w.row * pitch + c / 2));
                const int64_t blk = c / EPB;
                b[u] = scales[scale_word(w.row, blk >> 2, ktiles) + (blk & 3)];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + 256 * u;
            if (c - lane * 8 >= cols) break;  // (uniform)
            const float s = scale_value<NV>(b[u]);
            uint32_t h[4];
            codes_to_f16(q[u], h);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(reinterpret_cast<const __half2 &>(h[i]));
                v[2 * i] = __fmul_rn(f.x, s);
                v[2 * i + 1] = __fmul_rn(f.y, s);
                if (has_g) {
                    v[2 * i] = __fmul_rn(v[2 * i], g);
                    v[2 * i + 1] = __fmul_rn(v[2 * i + 1], g);
                }
            }
            const Pack8<T> o = round8<T>(v);
            if (vec != 0) {
                if (c < cols) store8(y + w.row * ldy + c, o, int(min(int64_t(8), cols - c)), true);
            } else {
                // Turned around, so that a store writes 32 consecutive elements.
                T *t = turn[threadIdx.x >> 5];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < Pack8<T>::W; ++i) reinterpret_cast<uint4 *>(t + lane * 8)[i] = o.v[i];
                __syncwarp();
                T *dst = y + w.row * ldy + (c - lane * 8);
                const int n = int(min(int64_t(256), cols - (c - lane * 8)));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (32 * i + lane < n) dst[32 * i + lane] = t[32 * i + lane];
            }
        }
    }
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxLd = int64_t(1) << 36;

int elem_bytes(int type) { return type == PTC_OUT_F32 ? 4 : 2; }
bool known_type(int type) { return type == PTC_OUT_F32 || type == PTC_OUT_BF16 || type == PTC_OUT_F16; }
bool multiple_of(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// 16-byte accesses: base and row pitch are multiples of 16 bytes.
bool wide_rows(const void *p, int64_t ld, int esize) { return multiple_of(p, 16) && (ld * esize) % 16 == 0; }

template <typename... P, typename... A>
cudaError_t launch(void (*fn)(P...), int64_t blocks, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (pdl_enabled()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

int64_t grid_for(int64_t threads, int sms) {
    const int64_t blocks = (threads + 255) / 256, most = int64_t(sms) * 16;
    return blocks < most ? blocks : most;
}

// Dropout probability to the kept count of 65536, the generator's key and counter.
DropArgs drop_args(double p, uint64_t seed, uint64_t offset) {
    DropArgs d;
    d.kept = uint32_t((1.0 - p) * 65536.0 + 0.5);
    d.scale = float(65536.0 / (d.kept > 0 ? d.kept : 1u));
    d.rng = make_rng(seed, offset);
    return d;
}

int check_random(double p, uint64_t offset) {
    if (!(p >= 0.0 && p <= 1.0)) return fail_status(PTC_ERR_INVALID, "p must be in [0, 1]");
    if (offset >> 63) return fail_status(PTC_ERR_INVALID, "offset must be below 2^63");
    return PTC_OK;
}

template <typename T, typename O>
int run_dropout(int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *res, int64_t ldr, void *y,
                int64_t ldy, const DropArgs &d, int sms, cudaStream_t s) {
    const int vec = wide_rows(x, ldx, sizeof(T)) && wide_rows(y, ldy, sizeof(O)) &&
                    (res == nullptr || wide_rows(res, ldr, sizeof(O)));
    const T *xp = static_cast<const T *>(x);
    const O *rp = static_cast<const O *>(res);
    O *yp = static_cast<O *>(y);
    auto go = [&](auto wide, auto ragged) {
        const int64_t threads = rows * (vec ? (cols + 7) / 8 : (cols + 255) / 256 * 32);
        return launch(vec ? wide : ragged, grid_for(threads, sms), 256, 0, s, xp, ldx, rp, ldr, yp, ldy, rows, cols, d);
    };
    cudaError_t e;
    if constexpr (std::is_same_v<T, O>)
        e = res ? go(dropout_kernel<T, O, true>, dropout_ragged_kernel<T, O, true>)
                : go(dropout_kernel<T, O, false>, dropout_ragged_kernel<T, O, false>);
    else
        e = go(dropout_kernel<T, O, false>, dropout_ragged_kernel<T, O, false>);
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "dropout launch");
}

template <typename T, bool NV, bool SR, bool DROP>
cudaError_t launch_quantize(const T *x, const QuantArgs &a, int sms, cudaStream_t s) {
    if (a.codes_t == nullptr) {
        // Four loads in flight per lane where rows are long enough and there is more than a wave of them.
        const int64_t rows_p = (a.rows + 127) / 128 * 128;
        const int64_t warps = rows_p * ((a.cols + 1023) / 1024);
        if (a.cols > 512 && warps >= int64_t(sms) * 64)
            return launch(quantize_rows_kernel<T, NV, SR, DROP, 4>, grid_for(warps * 32, sms), 256, 0, s, x, a);
        return launch(quantize_rows_kernel<T, NV, SR, DROP, 1>, grid_for(rows_p * ((a.cols + 255) / 256) * 32, sms), 256, 0, s,
                      x, a);
    }
    const int64_t tiles = ((a.rows + kTileR - 1) / kTileR) * ((a.cols + kTileC - 1) / kTileC);
    if (tiles >= int64_t(1) << 31) return cudaErrorInvalidConfiguration;  // (more elements than a GPU holds)
    constexpr size_t smem = tile_smem<T, SR>();
    auto *fn = a.codes ? quantize_tile_kernel<T, NV, SR, DROP, true> : quantize_tile_kernel<T, NV, SR, DROP, false>;
    if (smem + 8192 > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    return launch(fn, tiles, 256, smem, s, x, a);
}

template <typename T>
cudaError_t run_quantize(const void *x, const QuantArgs &a, bool nv, bool sr, int sms, cudaStream_t s) {
    const T *p = static_cast<const T *>(x);
    const bool drop = a.drop.kept < 65536u;
    auto go = [&](auto n, auto r) {
        return drop ? launch_quantize<T, decltype(n)::value, decltype(r)::value, true>(p, a, sms, s)
                    : launch_quantize<T, decltype(n)::value, decltype(r)::value, false>(p, a, sms, s);
    };
    if (nv) return sr ? go(yes(), yes()) : go(yes(), no());
    return sr ? go(no(), yes()) : go(no(), no());
}

}  // namespace

ByteRows fp4_scale_rows(const void *scales, int64_t rows, int64_t cols, bool nv) {
    const int64_t block = nv ? 16 : 32, blocks = (cols + block - 1) / block;
    return flat_bytes(scales, uint64_t((rows + 127) / 128) * uint64_t((blocks + 3) / 4) * kScaleTile);
}

ByteRows fp4_code_rows(const void *codes, int64_t rows, int64_t cols, int64_t pitch) {
    return elem_rows(codes, rows, (cols + 31) / 32 * 16, pitch, 1);
}

// Checks of a 4-bit matrix with rows of `cols` values.
int check_fp4(const void *codes, int64_t pitch, const void *scales, const void *g, int64_t cols, bool nv) {
    if (!codes || !scales) return fail_status(PTC_ERR_INVALID, "codes or scales is NULL");
    if (pitch < (cols + 31) / 32 * 16 || pitch > kMaxLd)
        return fail_status(PTC_ERR_INVALID, "the code pitch must hold whole 32-element blocks (16 bytes each)");
    if (g && !nv) return fail_status(PTC_ERR_INVALID, "mxfp4 has no matrix scale");
    if (!multiple_of(codes, 16) || !multiple_of(scales, 16) || pitch % 16)
        return fail_status(PTC_ERR_ALIGN, "codes, scales must be 16-byte aligned with a code pitch that is a multiple of 16");
    if (g && !multiple_of(g, 4)) return fail_status(PTC_ERR_ALIGN, "matrix scales must be 4-byte aligned");
    return PTC_OK;
}

}  // namespace ptc

using namespace ptc;

extern "C" {

int ptc_dropout_to(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, const void *residual, int64_t ldr,
                   void *y, int64_t ldy, int out_type, double p, uint64_t seed, uint64_t offset, void *stream) {
    set_message("");
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= rows, cols <= 2^30");
    if (!known_type(type) || !known_type(out_type)) return fail_status(PTC_ERR_INVALID, "unknown element type");
    if (out_type != type && (type != PTC_OUT_F32 || residual))
        return fail_status(PTC_ERR_INVALID, "y has x's type, or a 16-bit type for float32 x without a residual");
    int rc = check_random(p, offset);
    if (rc) return rc;
    if (rows == 0 || cols == 0) return PTC_OK;
    if (!x || !y) return fail_status(PTC_ERR_INVALID, "x or y is NULL");
    if (ldx < cols || ldy < cols || (residual && ldr < cols) || ldx > kMaxLd || ldy > kMaxLd || (residual && ldr > kMaxLd))
        return fail_status(PTC_ERR_INVALID, "leading dimensions must be cols .. 2^36");
    const int es = elem_bytes(type), os = elem_bytes(out_type);
    if (!multiple_of(x, es) || !multiple_of(y, os) || (residual && !multiple_of(residual, os)))
        return fail_status(PTC_ERR_ALIGN, "pointers must be aligned to the element");
    const ByteRows yr = elem_rows(y, rows, cols, ldy, os);
    if ((y != x || ldy != ldx || out_type != type) && rows_overlap(yr, elem_rows(x, rows, cols, ldx, es)))
        return fail_status(PTC_ERR_OVERLAP, "y overlaps x without being x");
    if (residual && (y != residual || ldy != ldr) && rows_overlap(yr, elem_rows(residual, rows, cols, ldr, os)))
        return fail_status(PTC_ERR_OVERLAP, "y overlaps the residual without being it");
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    const DropArgs d = drop_args(p, seed, offset);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto run) { return run(rows, cols, x, ldx, residual, ldr, y, ldy, d, sms, s); };
    if (type == PTC_OUT_BF16) return go(run_dropout<__nv_bfloat16, __nv_bfloat16>);
    if (type == PTC_OUT_F16) return go(run_dropout<__half, __half>);
    return out_type == PTC_OUT_F32    ? go(run_dropout<float, float>)
           : out_type == PTC_OUT_BF16 ? go(run_dropout<float, __nv_bfloat16>)
                                      : go(run_dropout<float, __half>);
}

int ptc_dropout(int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *residual, int64_t ldr, void *y,
                int64_t ldy, int type, double p, uint64_t seed, uint64_t offset, void *stream) {
    return ptc_dropout_to(rows, cols, x, ldx, type, residual, ldr, y, ldy, type, p, seed, offset, stream);
}

int ptc_quantize_fp4(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, int format, int rounding,
                     const float *matrix_scale, void *codes, int64_t pitch, void *scales, void *codes_t,
                     int64_t pitch_t, void *scales_t, double p, uint64_t seed, uint64_t offset, void *stream) {
    set_message("");
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= rows, cols <= 2^30");
    if (!known_type(type)) return fail_status(PTC_ERR_INVALID, "unknown element type");
    if (format != PTC_FP4_MX && format != PTC_FP4_NV) return fail_status(PTC_ERR_INVALID, "unknown 4-bit format");
    if (rounding != PTC_ROUND_NEAREST && rounding != PTC_ROUND_STOCHASTIC)
        return fail_status(PTC_ERR_INVALID, "unknown rounding");
    int rc = check_random(p, offset);
    if (rc) return rc;
    if (rows == 0 || cols == 0) return PTC_OK;
    if (!x) return fail_status(PTC_ERR_INVALID, "x is NULL");
    if (!codes && !codes_t) return fail_status(PTC_ERR_INVALID, "neither rows nor columns are asked for");
    if (ldx < cols || ldx > kMaxLd) return fail_status(PTC_ERR_INVALID, "ldx must be cols .. 2^36");
    const bool nv = format == PTC_FP4_NV;
    const int es = elem_bytes(type);
    if (codes && (rc = check_fp4(codes, pitch, scales, matrix_scale, cols, nv))) return rc;
    if (codes_t && (rc = check_fp4(codes_t, pitch_t, scales_t, matrix_scale, rows, nv))) return rc;
    if (!multiple_of(x, es)) return fail_status(PTC_ERR_ALIGN, "x must be aligned to its element");
    const ByteRows r[6] = {elem_rows(x, rows, cols, ldx, es),
                           flat_bytes(matrix_scale, 4),
                           fp4_code_rows(codes, rows, cols, pitch),
                           fp4_scale_rows(codes ? scales : nullptr, rows, cols, nv),
                           fp4_code_rows(codes_t, cols, rows, pitch_t),
                           fp4_scale_rows(codes_t ? scales_t : nullptr, cols, rows, nv)};
    for (int i = 0; i < 6; ++i)
        for (int j = std::max(i + 1, 2); j < 6; ++j)  // (the outputs)
            if (rows_overlap(r[i], r[j])) return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    QuantArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.codes = static_cast<uint8_t *>(codes);
    a.pitch = pitch;
    a.scales = static_cast<uint8_t *>(scales);
    a.codes_t = static_cast<uint8_t *>(codes_t);
    a.pitch_t = pitch_t;
    a.scales_t = static_cast<uint8_t *>(scales_t);
    a.g = matrix_scale;
    a.drop = drop_args(p, seed, offset);
    a.vec = wide_rows(x, ldx, es);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool sr = rounding == PTC_ROUND_STOCHASTIC;
    const cudaError_t e = type == PTC_OUT_F32    ? run_quantize<float>(x, a, nv, sr, sms, s)
                          : type == PTC_OUT_BF16 ? run_quantize<__nv_bfloat16>(x, a, nv, sr, sms, s)
                                                 : run_quantize<__half>(x, a, nv, sr, sms, s);
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "quantisation launch");
}

int ptc_dequantize_fp4(int64_t rows, int64_t cols, const void *codes, int64_t pitch, const void *scales, int format,
                       const float *matrix_scale, void *y, int64_t ldy, int type, void *stream) {
    set_message("");
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= rows, cols <= 2^30");
    if (!known_type(type)) return fail_status(PTC_ERR_INVALID, "unknown element type");
    if (format != PTC_FP4_MX && format != PTC_FP4_NV) return fail_status(PTC_ERR_INVALID, "unknown 4-bit format");
    if (rows == 0 || cols == 0) return PTC_OK;
    const bool nv = format == PTC_FP4_NV;
    if (!y) return fail_status(PTC_ERR_INVALID, "y is NULL");
    if (ldy < cols || ldy > kMaxLd) return fail_status(PTC_ERR_INVALID, "ldy must be cols .. 2^36");
    int rc = check_fp4(codes, pitch, scales, matrix_scale, cols, nv);
    if (rc) return rc;
    const int es = elem_bytes(type);
    if (!multiple_of(y, es)) return fail_status(PTC_ERR_ALIGN, "y must be aligned to its element");
    const ByteRows yr = elem_rows(y, rows, cols, ldy, es);
    if (rows_overlap(yr, fp4_code_rows(codes, rows, cols, pitch)) || rows_overlap(yr, fp4_scale_rows(scales, rows, cols, nv)) ||
        rows_overlap(yr, flat_bytes(matrix_scale, 4)))
        return fail_status(PTC_ERR_OVERLAP, "y overlaps an input");
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int vec = wide_rows(y, ldy, es);
    const uint8_t *cp = static_cast<const uint8_t *>(codes), *sp = static_cast<const uint8_t *>(scales);
    const bool many = cols > 512 && rows * ((cols + 1023) / 1024) >= int64_t(sms) * 64;
    const int64_t grid = grid_for(rows * (many ? (cols + 1023) / 1024 : (cols + 255) / 256) * 32, sms);
    auto go = [&](auto one, auto four, auto *out) {
        return launch(many ? four : one, grid, 256, 0, s, cp, pitch, sp, matrix_scale, rows, cols, out, ldy, vec);
    };
    cudaError_t e;
    if (type == PTC_OUT_F32)
        e = nv ? go(dequantize_kernel<float, true, 1>, dequantize_kernel<float, true, 4>, static_cast<float *>(y))
               : go(dequantize_kernel<float, false, 1>, dequantize_kernel<float, false, 4>, static_cast<float *>(y));
    else if (type == PTC_OUT_BF16)
        e = nv ? go(dequantize_kernel<__nv_bfloat16, true, 1>, dequantize_kernel<__nv_bfloat16, true, 4>,
                    static_cast<__nv_bfloat16 *>(y))
               : go(dequantize_kernel<__nv_bfloat16, false, 1>, dequantize_kernel<__nv_bfloat16, false, 4>,
                    static_cast<__nv_bfloat16 *>(y));
    else
        e = nv ? go(dequantize_kernel<__half, true, 1>, dequantize_kernel<__half, true, 4>, static_cast<__half *>(y))
               : go(dequantize_kernel<__half, false, 1>, dequantize_kernel<__half, false, 4>, static_cast<__half *>(y));
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "dequantisation launch");
}

}  // extern "C"
