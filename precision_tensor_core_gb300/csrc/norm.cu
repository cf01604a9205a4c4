// norm.cu -- root-mean-square norm of rows, with the residual's addition and an
// output in the element type or in 8 bits with a scale per row, and its gradient
// (ptc_rms_norm, ptc_rms_norm_s8, ptc_rms_norm_backward of include/ptc.h).
//
// Every byte is read and written once: rows of up to 16384 elements stay in
// registers between the sum of squares and the output.  The 16-bit norm is bound
// by memory traffic (8192 x 8192 bfloat16 with a residual 85 us, 92% of the copy rate), the norm
// to 8 bits by its instructions (the same without one 56 us), the gradient by both (99 us with
// dsum, 80% of the copy rate; 88 without, 67%); a row of one token by the start of a kernel and one reduction (2.2 us).
//
// In 8 bits the row's 1 / rms cancels out of the codes: with t = s w and a the
// row's largest |t|, y / (max |y| / 127) = 127 t / a.  So the sum of squares and the
// largest magnitude are reduced together, and a code depends on no sum's order.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "fp4.cuh"
#include "fp4.h"
#include "internal.h"
#include "ptc.h"
#include "ptx.cuh"

namespace ptc {
namespace {

struct NormArgs {
    const void *x;
    int64_t ldx;
    const void *res;  // NULL: none
    int64_t ldr;
    void *sum;  // with a residual
    int64_t lds;
    const void *w;  // NULL: ones
    int w_f32;      // w is float32 (else of x's type)
    void *y;        // or the 8-bit codes
    int64_t ldy;
    float *scale;  // 8 bits: a scale per row
    int64_t rows, cols;
    float eps, inv_cols;
};

struct GradArgs {
    const void *dy, *s, *ds;  // ds NULL: none
    int64_t lddy, lds, ldds;
    const void *w;
    int w_f32;
    void *dx;
    int64_t lddx;
    float *part;     // [gridDim.x][cols]: sums of dy s r
    float2 *stat;    // long rows: r and r mean(g s) of every row
    int64_t rows, cols;
    float eps, inv_cols;
};

// How a thread meets its chunk i of eight elements of a row: eight consecutive ones, of
// rows that are 16-byte aligned, or (kShifted, loads only) of any; eight of a 16-byte word (32
// bytes of float32) of rows that all lie alike within one (kAlike, the weights shifted); or one of
// each run of the row's threads (kSpread).  A warp's accesses are consecutive in all of them.
constexpr int kSpread = 0, kWide = 1, kShifted = 2, kAlike = 3;

// Elements of a row's first word that lie before the row.
template <typename T>
__device__ __forceinline__ int row_shift(const T *p) { return int((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)); }

template <int HOW>
__device__ __forceinline__ int64_t column(int i, int e, int tid, int threads) {
    return HOW != kSpread ? (int64_t(i) * threads + tid) * 8 + e : (int64_t(i) * 8 + e) * threads + tid;
}

// Eight elements at p, which is aligned to them alone, from the aligned words around them;
// `before`, `after`: elements of the row before p, and from p on.  (A word that reaches past
// the row is not read: those at the row's ends come one by one.)
template <typename T>
__device__ __forceinline__ Pack8<T> load_shifted(const T *p, int64_t before, int64_t after) {
    constexpr int W = Pack8<T>::W, PER = 16 / int(sizeof(T));
    const int m = int((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    if (m > before || after < 8 + (m ? PER - m : 0)) return load8(p, int(min(int64_t(8), after)), false);
    const uint4 *from = reinterpret_cast<const uint4 *>(p - m);
    uint4 words[W + 1];
#pragma unroll
    for (int i = 0; i < W; ++i) words[i] = from[i];
    words[W] = m ? from[W] : make_uint4(0, 0, 0, 0);
    uint32_t r[4 * W + 4];
#pragma unroll
    for (int i = 0; i <= W; ++i) r[4 * i] = words[i].x, r[4 * i + 1] = words[i].y, r[4 * i + 2] = words[i].z, r[4 * i + 3] = words[i].w;
    const int bytes = m * int(sizeof(T));
#pragma unroll
    for (int i = 0; i < 4 * W + 2; ++i) r[i] = bytes & 8 ? r[i + 2] : r[i];
#pragma unroll
    for (int i = 0; i < 4 * W + 1; ++i) r[i] = bytes & 4 ? r[i + 1] : r[i];
    if constexpr (sizeof(T) == 2)
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], bytes & 2 ? 16 : 0);
    Pack8<T> o;
#pragma unroll
    for (int i = 0; i < W; ++i) o.v[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    return o;
}

// (Elements past the row are +0.)
template <int HOW, typename T>
__device__ __forceinline__ Pack8<T> load_chunk(const T *p, int i, int tid, int threads, int64_t cols) {
    const int64_t c = column<HOW>(i, 0, tid, threads);
    if constexpr (HOW == kWide) {
        if (c + 8 <= cols) return load8(p + c, 8, true);
        return load8(c < cols ? p + c : p, c < cols ? int(cols - c) : 0, false);
    } else if constexpr (HOW == kShifted) {
        return c < cols ? load_shifted(p + c, c, cols - c) : load8(p, 0, false);
    } else if constexpr (HOW == kAlike) {
        const int64_t at = c - row_shift(p);
        if (at >= 0 && at + 8 <= cols) return load8(p + at, 8, true);
        Pack8<T> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.set(e, at + e >= 0 && at + e < cols ? p[at + e] : from_float<T>(0.0f));
        return r;
    } else {
        Pack8<T> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = column<kSpread>(i, e, tid, threads);
            r.set(e, at < cols ? p[at] : from_float<T>(0.0f));
        }
        return r;
    }
}

template <int HOW, typename T>
__device__ __forceinline__ void store_chunk(T *p, const Pack8<T> &v, int i, int tid, int threads, int64_t cols) {
    if constexpr (HOW == kAlike) {
        const int64_t at = column<HOW>(i, 0, tid, threads) - row_shift(p);
        if (at >= 0 && at + 8 <= cols) {
            store8(p + at, v, 8, true);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e >= 0 && at + e < cols) p[at + e] = v.get(e);
        }
    } else if constexpr (HOW != kSpread) {
        const int64_t c = column<HOW>(i, 0, tid, threads);
        if (c < cols) store8(p + c, v, int(min(int64_t(8), cols - c)), HOW == kWide);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = column<kSpread>(i, e, tid, threads);
            if (c < cols) p[c] = v.get(e);
        }
    }
}

// Weights of a chunk; `shift`: the row's (kAlike).
template <int HOW, typename W>
__device__ __forceinline__ Pack8<W> weight_chunk(const W *w, int i, int tid, int threads, int64_t cols, int shift) {
    if constexpr (HOW == kAlike) {
        const int64_t at = column<HOW>(i, 0, tid, threads) - shift;
        if (at >= 0) return at < cols ? load_shifted(w + at, at, cols - at) : load8(w, 0, false);
        Pack8<W> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.set(e, at + e >= 0 && at + e < cols ? w[at + e] : from_float<W>(0.0f));
        return r;
    } else {
        return load_chunk<HOW>(w, i, tid, threads, cols);
    }
}

// Eight weights as FP32; 1 where there are none, +0 or 1 past the row.
template <int HOW, typename T>
__device__ __forceinline__ void load_weight(float (&o)[8], const void *w, int w_f32, int i, int tid, int threads, int64_t cols,
                                            int shift = 0) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 1.0f;
    } else if (w_f32) {
        const Pack8<float> v = weight_chunk<HOW>(static_cast<const float *>(w), i, tid, threads, cols, shift);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v.get(e);
    } else {
        const Pack8<T> v = weight_chunk<HOW>(static_cast<const T *>(w), i, tid, threads, cols, shift);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = to_float(v.get(e));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The larger of `m` and |t| as bits; a NaN is the largest.
__device__ __forceinline__ uint32_t larger(uint32_t m, float t) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(__uint_as_float(m)), "f"(fabsf(t)));
    return __float_as_uint(o);
}

// The sum of `a` and the largest `m` over the row's threads (a warp, or the CTA).
// `buf`: 2 x 32 words that no thread still reads.
template <bool WARP, bool MAX>
__device__ __forceinline__ void reduce_row(float &a, uint32_t &m, uint32_t *buf) {
    a = warp_sum(a);
    if constexpr (MAX) m = __reduce_max_sync(0xFFFFFFFFu, m);
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        if (lane == 0) {
            buf[warp] = __float_as_uint(a);
            if constexpr (MAX) buf[32 + warp] = m;
        }
        __syncthreads();
        a = warp_sum(lane < warps ? __uint_as_float(buf[lane]) : 0.0f);
        if constexpr (MAX) m = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? buf[32 + lane] : 0u);
    }
}

__device__ __forceinline__ float inverse_rms(float squares, float inv_cols, float eps) {
    return __frcp_rn(__fsqrt_rn(__fmaf_rn(squares, inv_cols, eps)));
}

// Row s of a chunk: x, or x + residual rounded to the type, which is also stored.
template <int HOW, typename T>
__device__ __forceinline__ Pack8<T> sum_chunk(const NormArgs &a, int64_t row, int i, int tid, int threads) {
    Pack8<T> v = load_chunk<HOW>(static_cast<const T *>(a.x) + row * a.ldx, i, tid, threads, a.cols);
    if (a.res != nullptr) {
        const Pack8<T> r = load_chunk<HOW>(static_cast<const T *>(a.res) + row * a.ldr, i, tid, threads, a.cols);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fadd_rn(to_float(v.get(e)), to_float(r.get(e)));
        v = round8<T>(f);
    }
    return v;
}

constexpr float kNear = 0.49999f;

// 127 t / a rounded to nearest, ties to even, for a quotient next to a border: decided in 64
// bits, where both products are exact.
__device__ __noinline__ int border_code(float t, float a, float inverse) {
    const float low = floorf(__fmul_rn(t, inverse));
    const double d = 127.0 * double(t) - (double(low) + 0.5) * double(a);
    return int(d > 0.0 ? low + 1.0f : d < 0.0 ? low : 2.0f * rintf(0.5f * low + 0.25f));
}

// One chunk's output in the element type; `r`: 1 / rms.
template <int HOW, typename T>
__device__ __forceinline__ void put_chunk(const NormArgs &a, int64_t row, const Pack8<T> &s, float r, int i, int tid, int threads) {
    T *const y = static_cast<T *>(a.y) + row * a.ldy;
    float w[8], o[8];
    load_weight<HOW, T>(w, a.w, a.w_f32, i, tid, threads, a.cols, HOW == kAlike ? row_shift(y) : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __fmul_rn(__fmul_rn(to_float(s.get(e)), r), w[e]);
    store_chunk<HOW>(y, round8<T>(o), i, tid, threads, a.cols);
}

// One chunk's t = s w.
template <int HOW, typename T>
__device__ __forceinline__ void products(float (&t)[8], const NormArgs &a, const Pack8<T> &s, int i, int tid, int threads) {
    load_weight<HOW, T>(t, a.w, a.w_f32, i, tid, threads, a.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = __fmul_rn(to_float(s.get(e)), t[e]);
}

// Of a row in 8 bits: its largest |t|, 127 of which one is a code's step.  The smallest rows
// are lifted, exactly, so that 127 / |t| is a number.
struct CodeScale {
    float largest, lift, inverse;  // (lifted)
    bool blank;  // an infinity or NaN in the row, or nothing but zeros
    __device__ __forceinline__ explicit CodeScale(uint32_t bits) {
        const float a = __uint_as_float(bits);
        lift = a < 0x1p-100f ? 0x1p100f : 1.0f;
        largest = __fmul_rn(a, lift);
        inverse = __fdiv_rn(127.0f, largest);
        blank = bits >= kInfBits || bits == 0;
    }
};

// One chunk's codes of t (lifted).  With 3 2^22 added the sum's low byte is the code of the
// FP32 quotient, which is within 127 2^-24 of the quotient: its own code but for 2 in 10^5,
// next to a border.
template <int HOW>
__device__ __forceinline__ void put_codes(const NormArgs &a, int64_t row, const float (&t)[8], const CodeScale &c, int i, int tid, int threads) {
    uint32_t q[8];
    float near = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float u = __fmaf_rn(t[e], c.inverse, 0x1.8p23f);
        near = fmaxf(near, fabsf(__fmaf_rn(t[e], c.inverse, -__fsub_rn(u, 0x1.8p23f))));
        q[e] = __float_as_uint(u);
    }
    if (c.blank) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = 0;
    } else if (near > kNear) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (fabsf(__fmaf_rn(t[e], c.inverse, -rintf(__fmul_rn(t[e], c.inverse)))) > kNear)
                q[e] = uint32_t(border_code(t[e], c.largest, c.inverse));
    }
    int8_t *p = static_cast<int8_t *>(a.y) + row * a.ldy;
    if constexpr (HOW != kSpread) {
        const int64_t at = column<HOW>(i, 0, tid, threads);
        if (at + 8 <= a.cols) {
            uint32_t two[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) two[e] = __byte_perm(q[2 * e], q[2 * e + 1], 0x0040);
            *reinterpret_cast<uint2 *>(p + at) = make_uint2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[2], two[3], 0x5410));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e < a.cols) p[at + e] = int8_t(q[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = column<HOW>(i, e, tid, threads);
            if (at < a.cols) p[at] = int8_t(q[e]);
        }
    }
}

__device__ __forceinline__ float scale_of(uint32_t largest, float r) {
    return largest < kInfBits ? __fdiv_rn(__fmul_rn(__uint_as_float(largest), r), 127.0f) : __uint_as_float(0x7FC00000u);
}

// A row per CTA, or (WARP) per warp; CH chunks of eight elements per thread.
template <typename T, bool S8, int HOW, int CH, bool WARP>
__global__ void __launch_bounds__(CH == 1 ? 1024 : 512) norm_kernel(const NormArgs a) {
    __shared__ uint32_t buf[64];
    griddep_wait();
    griddep_launch_dependents();
    const int threads = WARP ? 32 : int(blockDim.x), tid = WARP ? int(threadIdx.x) % 32 : int(threadIdx.x);
    const int64_t row = WARP ? int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : int64_t(blockIdx.x);
    if (row >= a.rows) return;  // (whole warps, and never with a CTA per row)
    Pack8<T> s[CH];
    float t[CH][8];  // 8 bits: what is coded
#pragma unroll
    for (int i = 0; i < CH; ++i) s[i] = sum_chunk<HOW, T>(a, row, i, tid, threads);
    float squares = 0.0f;
    uint32_t largest = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) squares = __fmaf_rn(to_float(s[i].get(e)), to_float(s[i].get(e)), squares);
        if constexpr (S8) {
            products<HOW, T>(t[i], a, s[i], i, tid, threads);
#pragma unroll
            for (int e = 0; e < 8; ++e) largest = larger(largest, t[i][e]);
        }
        if (a.res != nullptr)
            store_chunk<HOW>(static_cast<T *>(a.sum) + row * a.lds, s[i], i, tid, threads, a.cols);
    }
    reduce_row<WARP, S8>(squares, largest, buf);
    const float r = inverse_rms(squares, a.inv_cols, a.eps);
    if constexpr (S8) {
        const CodeScale c(largest);
        if (c.lift != 1.0f)
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = __fmul_rn(t[i][e], c.lift);
#pragma unroll
        for (int i = 0; i < CH; ++i) put_codes<HOW>(a, row, t[i], c, i, tid, threads);
        if (tid == 0) a.scale[row] = scale_of(largest, r);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) put_chunk<HOW>(a, row, s[i], r, i, tid, threads);
    }
}

// Rows beyond the registers: s is read again after the sums (by the thread that
// stored it).
template <typename T, bool S8, int HOW>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    __shared__ uint32_t buf[64];
    griddep_wait();
    griddep_launch_dependents();
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    const int chunks = int((a.cols + (HOW == kAlike ? 7 : 0) + int64_t(8) * threads - 1) / (int64_t(8) * threads));
    float squares = 0.0f;
    uint32_t largest = 0;
    for (int i = 0; i < chunks; ++i) {
        const Pack8<T> s = sum_chunk<HOW, T>(a, row, i, tid, threads);
        float part = 0.0f;  // (chunk by chunk: long sums stay exact to a few ulps)
#pragma unroll
        for (int e = 0; e < 8; ++e) part = __fmaf_rn(to_float(s.get(e)), to_float(s.get(e)), part);
        squares += part;
        if constexpr (S8) {
            float t[8];
            products<HOW, T>(t, a, s, i, tid, threads);
#pragma unroll
            for (int e = 0; e < 8; ++e) largest = larger(largest, t[e]);
        }
        if (a.res != nullptr) store_chunk<HOW>(static_cast<T *>(a.sum) + row * a.lds, s, i, tid, threads, a.cols);
    }
    reduce_row<false, S8>(squares, largest, buf);
    const float r = inverse_rms(squares, a.inv_cols, a.eps);
    const CodeScale c(largest);
    const T *again = a.res != nullptr ? static_cast<const T *>(a.sum) + row * a.lds : static_cast<const T *>(a.x) + row * a.ldx;
    for (int i = 0; i < chunks; ++i) {
        const Pack8<T> s = load_chunk<HOW>(again, i, tid, threads, a.cols);
        if constexpr (S8) {
            float t[8];
            products<HOW, T>(t, a, s, i, tid, threads);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = __fmul_rn(t[e], c.lift);
            put_codes<HOW>(a, row, t, c, i, tid, threads);
        } else {
            put_chunk<HOW>(a, row, s, r, i, tid, threads);
        }
    }
    if (S8 && tid == 0) a.scale[row] = scale_of(largest, r);
}

// ------------------------------------------------------------ gradient
// With g = dy w, n columns and u = s r: dx = r (g - u m) (+ ds), m = r sum(g s) / n, dw =
// sum over rows of dy u.  Both row sums are reduced together.
__device__ __forceinline__ void reduce_two(float &p, float &q, float2 *buf) {
    p = warp_sum(p);
    q = warp_sum(q);
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) buf[warp] = make_float2(p, q);
    __syncthreads();
    const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
    p = warp_sum(v.x);
    q = warp_sum(v.y);
}

template <typename T, int HOW>
__device__ __forceinline__ void grad_chunk(const GradArgs &a, int64_t row, const Pack8<T> &s, const Pack8<T> &dy, float r,
                                           float m, float (&acc)[8], int i, int tid, int threads) {
    float w[8], o[8];
    load_weight<HOW, T>(w, a.w, a.w_f32, i, tid, threads, a.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float sv = to_float(s.get(e)), dv = to_float(dy.get(e));
        const float u = __fmul_rn(sv, r);
        o[e] = __fmul_rn(r, __fmaf_rn(-u, m, __fmul_rn(dv, w[e])));
        acc[e] = __fmaf_rn(dv, u, acc[e]);
    }
    if (a.ds != nullptr) {
        const Pack8<T> d = load_chunk<HOW>(static_cast<const T *>(a.ds) + row * a.ldds, i, tid, threads, a.cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __fadd_rn(o[e], to_float(d.get(e)));
    }
    store_chunk<HOW>(static_cast<T *>(a.dx) + row * a.lddx, round8<T>(o), i, tid, threads, a.cols);
}

// 16 bytes to shared memory, `n` of them from global memory and zeros after them.
__device__ __forceinline__ void copy16_or_zero(void *dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// Rows that are not aligned: a CTA takes rows blockIdx.x, + gridDim.x, ... and holds its columns' sums of the
// weight's gradient in registers; they leave as one row of partial sums per CTA,
// which column_sums_kernel adds in order.
template <typename T, int CH>
__global__ void __launch_bounds__(512) grad_kernel(const GradArgs a) {
    __shared__ float2 buf[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    float acc[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    int b = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, b ^= 1) {
        Pack8<T> s[CH], dy[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            s[i] = load_chunk<kSpread>(static_cast<const T *>(a.s) + row * a.lds, i, tid, threads, a.cols);
            dy[i] = load_chunk<kSpread>(static_cast<const T *>(a.dy) + row * a.lddy, i, tid, threads, a.cols);
        }
        float squares = 0.0f, gs = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float w[8];
            load_weight<kSpread, T>(w, a.w, a.w_f32, i, tid, threads, a.cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float sv = to_float(s[i].get(e));
                squares = __fmaf_rn(sv, sv, squares);
                gs = __fmaf_rn(__fmul_rn(to_float(dy[i].get(e)), w[e]), sv, gs);
            }
        }
        reduce_two(squares, gs, buf[b]);
        const float r = inverse_rms(squares, a.inv_cols, a.eps);
        const float m = __fmul_rn(r, __fmul_rn(gs, a.inv_cols));
#pragma unroll
        for (int i = 0; i < CH; ++i) grad_chunk<T, kSpread>(a, row, s[i], dy[i], r, m, acc[i], i, tid, threads);
    }
    float *part = a.part + int64_t(blockIdx.x) * a.cols;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = column<kSpread>(i, e, tid, threads);
            if (c < a.cols) part[c] = acc[i][e];
        }
}

// The same for aligned rows, which come through shared memory: every thread copies its own
// elements of the next rows there, `slots` rows deep, and waits for nobody else's.  (Loads
// at the row's beginning left the memory idle during the reduction and the stores: 8192 x
// 8192 bfloat16 with ds 259 us instead of 99.)  With rows that lie alike (kAlike) the grid is a
// multiple of eight wherever a CTA has several, so that all of a CTA's begin at the same
// element of a word and its columns stay where they are.
template <typename T, int CH, int HOW>
__global__ void __launch_bounds__(1024) grad_ring_kernel(const GradArgs a, int slots) {
    constexpr int W = Pack8<T>::W;
    extern __shared__ uint4 ring[];  // [slot][s, dy, ds][chunk][16 bytes][thread], then the weights [chunk][2][thread]
    __shared__ float2 buf[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    const int arrays = a.ds != nullptr ? 3 : 2, slot_size = arrays * CH * W * threads;
    const int shift = HOW == kAlike ? row_shift(static_cast<const T *>(a.s) + int64_t(blockIdx.x) * a.lds) : 0;
    uint4 *const weights = ring + slots * slot_size + tid;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        float w[8];
        load_weight<HOW, T>(w, a.w, a.w_f32, i, tid, threads, a.cols, shift);
        weights[(2 * i) * threads] = *reinterpret_cast<const uint4 *>(&w[0]);
        weights[(2 * i + 1) * threads] = *reinterpret_cast<const uint4 *>(&w[4]);
    }
    auto issue = [&](int64_t row, int slot) {
        if (row < a.rows) {
            const T *from[3] = {static_cast<const T *>(a.s) + row * a.lds, static_cast<const T *>(a.dy) + row * a.lddy,
                                static_cast<const T *>(a.ds) + row * a.ldds};
            uint4 *to = ring + slot * slot_size + tid;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < arrays)
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int64_t c = column<HOW>(i, 0, tid, threads) - shift;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            constexpr int PER = 16 / int(sizeof(T));
                            if (HOW == kAlike && w == 0 && c < 0) {
                                // The word that the row begins in: whole, with the end of the row
                                // before it (which `taken` clears), or where none is its elements.
                                uint4 *const at = to + ((k * CH + i) * W) * threads;
                                if (row > 0 && a.cols >= 8) {
                                    copy16_or_zero(at, from[k] + c, 16);
                                } else {
                                    Pack8<T> v;
#pragma unroll
                                    for (int e = 0; e < 8; ++e) v.set(e, c + e >= 0 && c + e < a.cols ? from[k][c + e] : from_float<T>(0.0f));
                                    *at = v.v[0];
                                }
                                continue;
                            }
                            const int have = c < a.cols ? int(max(int64_t(0), min(int64_t(PER), a.cols - c - w * PER))) : 0;
                            if (HOW == kAlike && have == 0) {  // (the row's first element is no address for 16 bytes, even of none)
                                to[((k * CH + i) * W + w) * threads] = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            copy16_or_zero(to + ((k * CH + i) * W + w) * threads, from[k] + (have > 0 ? c + w * PER : 0), have * int(sizeof(T)));
                        }
                    }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto taken = [&](int slot, int array, int i) {
        Pack8<T> v;
#pragma unroll
        for (int w = 0; w < W; ++w) v.v[w] = ring[slot * slot_size + ((array * CH + i) * W + w) * threads + tid];
        if (HOW == kAlike && i == 0 && tid == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < shift) v.set(e, from_float<T>(0.0f));
        return v;
    };
    auto weight = [&](int i, int e) { return reinterpret_cast<const float *>(weights + (2 * i + (e >> 2)) * threads)[e & 3]; };
    float acc[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    for (int k = 0; k < slots; ++k) issue(int64_t(blockIdx.x) + int64_t(k) * gridDim.x, k);
    int slot = 0, b = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, b ^= 1) {
        switch (slots) {  // (all but the copies of the last slots - 1 rows)
            case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
            case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
            case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
        Pack8<T> s[CH], dy[CH];
        float squares = 0.0f, gs = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            s[i] = taken(slot, 0, i);
            dy[i] = taken(slot, 1, i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float sv = to_float(s[i].get(e));
                squares = __fmaf_rn(sv, sv, squares);
                gs = __fmaf_rn(__fmul_rn(to_float(dy[i].get(e)), weight(i, e)), sv, gs);
            }
        }
        reduce_two(squares, gs, buf[b]);
        const float r = inverse_rms(squares, a.inv_cols, a.eps);
        const float m = __fmul_rn(r, __fmul_rn(gs, a.inv_cols));
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dv = to_float(dy[i].get(e)), u = __fmul_rn(to_float(s[i].get(e)), r);
                o[e] = __fmul_rn(r, __fmaf_rn(-u, m, __fmul_rn(dv, weight(i, e))));
                acc[i][e] = __fmaf_rn(dv, u, acc[i][e]);
            }
            if (a.ds != nullptr) {
                const Pack8<T> d = taken(slot, 2, i);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __fadd_rn(o[e], to_float(d.get(e)));
            }
            store_chunk<HOW>(static_cast<T *>(a.dx) + row * a.lddx, round8<T>(o), i, tid, threads, a.cols);
        }
        issue(row + int64_t(slots) * gridDim.x, slot);
        if (++slot == slots) slot = 0;
    }
    float *part = a.part + int64_t(blockIdx.x) * a.cols;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = column<HOW>(i, e, tid, threads) - shift;
            if (c >= 0 && c < a.cols) part[c] = acc[i][e];
        }
}

// Longer rows: the sums of every row first, then columns in pieces of 8 per thread
// (blockIdx.x) for the rows of each blockIdx.y.
template <typename T, int HOW>
__global__ void __launch_bounds__(1024) grad_stats_kernel(const GradArgs a) {
    __shared__ float2 buf[32];
    griddep_wait();
    griddep_launch_dependents();
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    const int chunks = int((a.cols + int64_t(8) * threads - 1) / (int64_t(8) * threads));
    float squares = 0.0f, gs = 0.0f;
    for (int i = 0; i < chunks; ++i) {
        const Pack8<T> s = load_chunk<HOW>(static_cast<const T *>(a.s) + row * a.lds, i, tid, threads, a.cols);
        const Pack8<T> dy = load_chunk<HOW>(static_cast<const T *>(a.dy) + row * a.lddy, i, tid, threads, a.cols);
        float w[8], p = 0.0f, q = 0.0f;
        load_weight<HOW, T>(w, a.w, a.w_f32, i, tid, threads, a.cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float sv = to_float(s.get(e));
            p = __fmaf_rn(sv, sv, p);
            q = __fmaf_rn(__fmul_rn(to_float(dy.get(e)), w[e]), sv, q);
        }
        squares += p;
        gs += q;
    }
    reduce_two(squares, gs, buf);
    const float r = inverse_rms(squares, a.inv_cols, a.eps);
    if (tid == 0) a.stat[row] = make_float2(r, __fmul_rn(r, __fmul_rn(gs, a.inv_cols)));
}

template <typename T, int HOW>
__global__ void __launch_bounds__(256) grad_columns_kernel(const GradArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int threads = int(blockDim.x), tid = int(threadIdx.x), i = int(blockIdx.x);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const Pack8<T> s = load_chunk<HOW>(static_cast<const T *>(a.s) + row * a.lds, i, tid, threads, a.cols);
        const Pack8<T> dy = load_chunk<HOW>(static_cast<const T *>(a.dy) + row * a.lddy, i, tid, threads, a.cols);
        const float2 st = a.stat[row];
        grad_chunk<T, HOW>(a, row, s, dy, st.x, st.y, acc, i, tid, threads);
    }
    float *part = a.part + int64_t(blockIdx.y) * a.cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t c = column<HOW>(i, e, tid, threads);
        if (c < a.cols) part[c] = acc[e];
    }
}

// dw[c] = sum over p of part[p][c]: 32 columns per CTA, eight warps a share of p each, in
// four sums per lane that are joined in pairs, as the warps' are: of 512 parts one passes
// through 20 additions at most (one after the other 71, and 333 x 777 f32 1.4e-7 from the
// exact sums instead of 1.0e-7, in the same time).
__global__ void __launch_bounds__(256) column_sums_kernel(const float *part, int parts, int64_t cols, float *dw) {
    __shared__ float sums[8][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < cols) {
#pragma unroll 8
        for (int p = warp; p < parts; p += 8) {  // (the four in turn)
            const float t = __fadd_rn(v[0], part[int64_t(p) * cols + c]);
            v[0] = v[1];
            v[1] = v[2];
            v[2] = v[3];
            v[3] = t;
        }
    }
    sums[warp][lane] = __fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3]));
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = sums[k][lane];
#pragma unroll
        for (int n = 4; n > 0; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) t[k] = __fadd_rn(t[k], t[k + n]);
        dw[c] = t[0];
    }
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDimN = int64_t(1) << 30;
constexpr int64_t kMaxLdN = int64_t(1) << 36;

int bytes_of(int type) { return type == PTC_OUT_F32 ? 4 : 2; }
bool type_known(int type) { return type == PTC_OUT_F32 || type == PTC_OUT_BF16 || type == PTC_OUT_F16; }
bool aligned_to(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool wide(const void *p, int64_t ld, int esize) { return aligned_to(p, 16) && (ld * esize) % 16 == 0; }

template <typename... P, typename... A>
cudaError_t launch_norm_smem(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = grid;
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

template <typename... P, typename... A>
cudaError_t launch_norm(void (*fn)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    return launch_norm_smem(fn, grid, threads, 0, stream, args...);
}

int round32(int64_t n) { return int((n + 31) / 32 * 32); }

// A few rows take a thread per eight elements, so that a row is one round of loads; many
// take four rounds per thread, whose loads are in flight together; rows of up to 1024
// elements a warp each.
template <typename T, bool S8, int HOW>
cudaError_t run_norm(const NormArgs &a, int sms, cudaStream_t s) {
    const int64_t chunks = (a.cols + 7) / 8 + (HOW == kAlike ? 1 : 0);
    if (chunks > 4 * 512)
        return launch_norm(norm_long_kernel<T, S8, HOW>, dim3(unsigned(a.rows)), 1024, s, a);
    if (a.rows > 2 * sms && chunks <= 128) {
        const dim3 grid(unsigned((a.rows + 7) / 8));
        return chunks <= 32 ? launch_norm(norm_kernel<T, S8, HOW, 1, true>, grid, 256, s, a)
                            : launch_norm(norm_kernel<T, S8, HOW, 4, true>, grid, 256, s, a);
    }
    const dim3 grid = dim3(unsigned(a.rows));
    if ((a.rows <= sms && chunks <= 1024) || chunks <= 32)
        return launch_norm(norm_kernel<T, S8, HOW, 1, false>, grid, round32(chunks), s, a);
    return launch_norm(norm_kernel<T, S8, HOW, 4, false>, grid, round32((chunks + 3) / 4), s, a);
}

template <bool S8>
int start_norm(NormArgs a, int type, int out_esize, cudaStream_t s) {
    int sms;
    const int rc = usable_device(&sms);
    if (rc) return rc;
    const int es = bytes_of(type);
    if (a.rows == 1) a.ldx = a.ldr = a.lds = a.ldy = 0;  // (one row has no pitch)
    const bool out = S8 ? aligned_to(a.y, 8) && a.ldy % 8 == 0 : wide(a.y, a.ldy, out_esize);
    const bool vec = out && wide(a.x, a.ldx, es) && (!a.res || (wide(a.res, a.ldr, es) && wide(a.sum, a.lds, es))) && aligned_to(a.w, 16);
    // Rows that lie as x's do within 16 bytes.
    auto alike = [&](const void *p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(a.x)) % 16 == 0 && (ld - a.ldx) * es % 16 == 0;
    };
    auto go = [&](auto t) {
        using T = decltype(t);
        if (vec) return run_norm<T, S8, kWide>(a, sms, s);
        if constexpr (S8)  // codes are stored eight at a time, and nothing else is
            if (out && !a.res) return run_norm<T, S8, kShifted>(a, sms, s);
        if constexpr (!S8)  // (2047 x 5003 f16 11.1 us instead of 15.8)
            if (alike(a.y, a.ldy) && (!a.res || (alike(a.res, a.ldr) && alike(a.sum, a.lds)))) return run_norm<T, S8, kAlike>(a, sms, s);
        return run_norm<T, S8, kSpread>(a, sms, s);
    };
    const cudaError_t e = type == PTC_OUT_F32 ? go(float()) : type == PTC_OUT_BF16 ? go(__nv_bfloat16()) : go(__half());
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "norm launch");
}

int check_sizes_n(int64_t rows, int64_t cols, int type, int w_type, float eps) {
    if (rows < 0 || cols < 0 || rows > kMaxDimN || cols > kMaxDimN)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= rows, cols <= 2^30");
    if (!type_known(type) || (w_type != type && w_type != PTC_OUT_F32))
        return fail_status(PTC_ERR_INVALID, "unknown element type, or a weight that is neither float32 nor of x's type");
    if (!(eps >= 0.0f) || eps > 3.0e38f) return fail_status(PTC_ERR_INVALID, "eps must be finite and not negative");
    return PTC_OK;
}

int check_rows(const void *p, int64_t cols, int64_t ld, int esize) {
    if (!p || ld < cols || ld > kMaxLdN)
        return fail_status(PTC_ERR_INVALID, "a matrix is NULL, or its leading dimension is not cols .. 2^36");
    if (!aligned_to(p, uintptr_t(esize))) return fail_status(PTC_ERR_ALIGN, "matrices must be aligned to their elements");
    return PTC_OK;
}

// `same`: an output may be exactly this input (a thread reads what it writes first).
bool clashes(const ByteRows &out, const ByteRows &in, bool same) {
    return rows_overlap(out, in) && !(same && out.p == in.p && (out.pitch == in.pitch || out.rows == 1));
}

// The checks that both forms share; `y` the output's bytes.
int check_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, const void *res, int64_t ldr, void *sum,
               int64_t lds, const void *w, int w_type, const ByteRows &y, bool same) {
    const int es = bytes_of(type);
    int rc = check_rows(x, cols, ldx, es);
    if (!rc && res) rc = check_rows(res, cols, ldr, es);
    if (!rc && res) rc = check_rows(sum, cols, lds, es);
    if (rc) return rc;
    if (!res && sum) return fail_status(PTC_ERR_INVALID, "a sum is written only with a residual");
    if (w && !aligned_to(w, uintptr_t(bytes_of(w_type)))) return fail_status(PTC_ERR_ALIGN, "weight must be aligned to its elements");
    const ByteRows bx = elem_rows(x, rows, cols, ldx, es), br = elem_rows(res, rows, cols, ldr, es),
                   bs = elem_rows(sum, rows, cols, lds, es), bw = flat_bytes(w, uint64_t(cols) * uint64_t(bytes_of(w_type)));
    if (clashes(y, bx, same) || clashes(y, br, same) || rows_overlap(y, bs) || rows_overlap(y, bw) || clashes(bs, bx, true) ||
        clashes(bs, br, true) || rows_overlap(bs, bw))
        return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
    return PTC_OK;
}

NormArgs norm_args(int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *res, int64_t ldr, void *sum,
                   int64_t lds, const void *w, int w_type, float eps, void *y, int64_t ldy, float *scale) {
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.ldx = ldx;
    a.res = res;
    a.ldr = ldr;
    a.sum = sum;
    a.lds = lds;
    a.w = w;
    a.w_f32 = w_type == PTC_OUT_F32;
    a.y = y;
    a.ldy = ldy;
    a.scale = scale;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.inv_cols = float(1.0 / double(cols));
    return a;
}

// Partial sums of the weight's gradient: rows of them, and of the row pieces of long rows.
constexpr int kMaxParts = 512;
bool grad_long(int64_t cols) { return cols > 16384; }
int64_t grad_pieces(int64_t cols) { return (cols + 2047) / 2048; }  // of 256 threads with eight columns each
// (Long rows: their pieces' CTAs, eight per SM in all, of 152.)
int64_t grad_parts(int64_t rows, int64_t cols) {
    return std::min<int64_t>(rows, grad_long(cols) ? std::max<int64_t>(1, 8 * 152 / grad_pieces(cols)) : kMaxParts);
}

// Of grad_ring_kernel: threads and their chunks, bytes of a row in flight and of the weights.
struct RingShape {
    int ch, threads;
    size_t row, weights;
};
constexpr size_t kRingMost = 225 * 1024;  // of an SM, and of a CTA

RingShape ring_shape(int64_t chunks, int arrays, size_t esize) {
    RingShape g;
    g.ch = chunks <= 1024 ? 1 : 2;
    g.threads = round32((chunks + g.ch - 1) / g.ch);
    g.row = size_t(arrays) * size_t(g.ch) * esize * 8 * size_t(g.threads);
    g.weights = size_t(g.ch) * 32 * size_t(g.threads);
    return g;
}

template <typename T, int HOW>
cudaError_t run_grad(GradArgs a, int sms, float *dw, cudaStream_t s) {
    const int64_t chunks = (a.cols + 7) / 8;
    int parts;
    cudaError_t e;
    constexpr int WIDE = HOW == kWide ? kWide : kSpread;
    if (grad_long(a.cols)) {
        const int64_t pieces = grad_pieces(a.cols);
        parts = int(grad_parts(a.rows, a.cols));
        e = launch_norm(grad_stats_kernel<T, WIDE>, dim3(unsigned(a.rows)), 1024, s, a);
        if (e == cudaSuccess) e = launch_norm(grad_columns_kernel<T, WIDE>, dim3(unsigned(pieces), unsigned(parts)), 256, s, a);
    } else if (const RingShape g = ring_shape(chunks + (HOW == kAlike ? 1 : 0), a.ds ? 3 : 2, sizeof(T));
               HOW != kSpread && g.weights + g.row <= kRingMost) {
        // Four rows in flight per CTA, fewer where they do not fit; up to three CTAs per SM.
        const int slots = int(std::min<size_t>(4, (kRingMost - g.weights) / g.row));
        const size_t smem = slots * g.row + g.weights;
        const int per_sm = int(std::max<size_t>(1, std::min<size_t>({3, size_t(2048 / g.threads), kRingMost / (smem + 2048)})));
        constexpr int RING = HOW == kAlike ? kAlike : kWide;
        auto *fn = g.ch == 1 ? grad_ring_kernel<T, 1, RING> : grad_ring_kernel<T, 2, RING>;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kRingMost));
        if (e != cudaSuccess) return e;
        parts = int(std::min<int64_t>(grad_parts(a.rows, a.cols), int64_t(sms) * per_sm));
        if (HOW == kAlike && parts < a.rows) parts = std::max(8, parts / 8 * 8);
        e = launch_norm_smem(fn, dim3(unsigned(parts)), g.threads, smem, s, a, slots);
    } else {
        // (also aligned FP32 rows of over 14336 elements with ds, of which the ring holds not one)
        const int ch = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
        const int threads = round32((chunks + ch - 1) / ch);
        const int per_sm = std::max(1, (sizeof(T) == 2 && ch <= 2 ? 1024 : 512) / threads);
        parts = int(std::min<int64_t>(grad_parts(a.rows, a.cols), int64_t(sms) * std::min(per_sm, 3)));
        const dim3 grid = dim3(unsigned(parts));
        e = ch == 1   ? launch_norm(grad_kernel<T, 1>, grid, threads, s, a)
            : ch == 2 ? launch_norm(grad_kernel<T, 2>, grid, threads, s, a)
                      : launch_norm(grad_kernel<T, 4>, grid, threads, s, a);
    }
    if (e == cudaSuccess)
        e = launch_norm(column_sums_kernel, dim3(unsigned((a.cols + 31) / 32)), 256, s, static_cast<const float *>(a.part), parts,
                        a.cols, dw);
    return e;
}

// `n` zeros: the sums of no rows.
int start_zeros(float *p, int64_t n, cudaStream_t s, const char *what) {
    int sms;
    const int rc = usable_device(&sms);
    if (rc) return rc;
    const cudaError_t e = launch_norm(column_sums_kernel, dim3(unsigned((n + 31) / 32)), 256, s,
                                      static_cast<const float *>(nullptr), 0, n, p);
    return e == cudaSuccess ? PTC_OK : fail_launch(e, what);
}

}  // namespace
}  // namespace ptc

using namespace ptc;

extern "C" {

int ptc_rms_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, const void *residual, int64_t ldr,
                 void *sum, int64_t lds, const void *weight, int weight_type, float eps, void *y, int64_t ldy, void *stream) {
    set_message("");
    int rc = check_sizes_n(rows, cols, type, weight_type, eps);
    if (rc || rows == 0 || cols == 0) return rc;
    rc = check_rows(y, cols, ldy, bytes_of(type));
    if (!rc)
        rc = check_norm(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type,
                        elem_rows(y, rows, cols, ldy, bytes_of(type)), true);
    if (rc) return rc;
    return start_norm<false>(norm_args(rows, cols, x, ldx, residual, ldr, sum, lds, weight, weight_type, eps, y, ldy, nullptr),
                             type, bytes_of(type), static_cast<cudaStream_t>(stream));
}

int ptc_rms_norm_s8(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, const void *residual, int64_t ldr,
                    void *sum, int64_t lds, const void *weight, int weight_type, float eps, int8_t *codes, int64_t ldc,
                    float *scale, void *stream) {
    set_message("");
    int rc = check_sizes_n(rows, cols, type, weight_type, eps);
    if (rc || rows == 0) return rc;
    if (cols > 0 && (rc = check_rows(codes, cols, ldc, 1))) return rc;
    if (!scale) return fail_status(PTC_ERR_INVALID, "scale is NULL");
    if (!aligned_to(scale, 4)) return fail_status(PTC_ERR_ALIGN, "scale must be 4-byte aligned");
    if (cols == 0) return start_zeros(scale, rows, static_cast<cudaStream_t>(stream), "norm launch");
    const ByteRows c = elem_rows(codes, rows, cols, ldc, 1), sc = flat_bytes(scale, uint64_t(rows) * 4);
    const int es = bytes_of(type);
    rc = check_norm(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type, c, false);
    if (rc) return rc;
    if (rows_overlap(sc, c) || rows_overlap(sc, elem_rows(x, rows, cols, ldx, es)) ||
        rows_overlap(sc, elem_rows(residual, rows, cols, ldr, es)) || rows_overlap(sc, elem_rows(sum, rows, cols, lds, es)) ||
        rows_overlap(sc, flat_bytes(weight, uint64_t(cols) * uint64_t(bytes_of(weight_type)))))
        return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
    return start_norm<true>(norm_args(rows, cols, x, ldx, residual, ldr, sum, lds, weight, weight_type, eps, codes, ldc, scale),
                            type, 1, static_cast<cudaStream_t>(stream));
}

int64_t ptc_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxDimN || cols > kMaxDimN) return 0;
    return grad_parts(rows, cols) * cols * 4 + (grad_long(cols) ? rows * 8 + 16 : 0);
}

int ptc_rms_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *s, int64_t lds, int type,
                          const void *ds, int64_t ldds, const void *weight, int weight_type, float eps, void *dx, int64_t lddx,
                          float *dweight, void *workspace, int64_t workspace_bytes, void *stream) {
    set_message("");
    int rc = check_sizes_n(rows, cols, type, weight_type, eps);
    if (rc || cols == 0) return rc;
    if (!dweight) return fail_status(PTC_ERR_INVALID, "dweight is NULL");
    if (!aligned_to(dweight, 4)) return fail_status(PTC_ERR_ALIGN, "dweight must be 4-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int sms;
    if (rows == 0) return start_zeros(dweight, cols, st, "norm gradient launch");
    const int es = bytes_of(type);
    rc = check_rows(dy, cols, lddy, es);
    if (!rc) rc = check_rows(s, cols, lds, es);
    if (!rc && ds) rc = check_rows(ds, cols, ldds, es);
    if (!rc) rc = check_rows(dx, cols, lddx, es);
    if (rc) return rc;
    if (weight && !aligned_to(weight, uintptr_t(bytes_of(weight_type))))
        return fail_status(PTC_ERR_ALIGN, "weight must be aligned to its elements");
    const int64_t need = ptc_rms_norm_backward_workspace(rows, cols);
    if (!workspace || workspace_bytes < need) return fail_status(PTC_ERR_INVALID, "the workspace is too small");
    if (!aligned_to(workspace, 16)) return fail_status(PTC_ERR_ALIGN, "the workspace must be 16-byte aligned");
    const ByteRows in[4] = {elem_rows(dy, rows, cols, lddy, es), elem_rows(s, rows, cols, lds, es),
                            elem_rows(ds, rows, cols, ldds, es), flat_bytes(weight, uint64_t(cols) * uint64_t(bytes_of(weight_type)))};
    const ByteRows bx = elem_rows(dx, rows, cols, lddx, es), bw = flat_bytes(dweight, uint64_t(cols) * 4),
                   bk = flat_bytes(workspace, uint64_t(need));
    bool bad = rows_overlap(bx, bw) || rows_overlap(bx, bk) || rows_overlap(bw, bk);
    for (int i = 0; i < 4; ++i)  // (with long rows dy and s are read by other threads than those that write dx)
        bad = bad || clashes(bx, in[i], i < 3) || rows_overlap(bw, in[i]) || rows_overlap(bk, in[i]);
    if (bad) return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
    if ((rc = usable_device(&sms))) return rc;
    GradArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dy = dy;
    a.lddy = lddy;
    a.s = s;
    a.lds = lds;
    a.ds = ds;
    a.ldds = ldds;
    a.w = weight;
    a.w_f32 = weight_type == PTC_OUT_F32;
    a.dx = dx;
    a.lddx = lddx;
    a.part = static_cast<float *>(workspace);
    a.stat = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + (grad_parts(rows, cols) * cols * 4 + 15) / 16 * 16);
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.inv_cols = float(1.0 / double(cols));
    if (rows == 1) a.lddy = a.lds = a.ldds = a.lddx = 0;  // (one row has no pitch)
    const bool vec = wide(dy, a.lddy, es) && wide(s, a.lds, es) && wide(dx, a.lddx, es) && (!ds || wide(ds, a.ldds, es)) &&
                     aligned_to(weight, 16);
    // Rows that lie as those of s do within 16 bytes.
    auto alike = [&](const void *p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(s)) % 16 == 0 && (ld - a.lds) * es % 16 == 0;
    };
    auto go = [&](auto t) {
        using T = decltype(t);
        if (vec) return run_grad<T, kWide>(a, sms, dweight, st);
        // (Without ds 2047 x 5003 f16 31.5 us instead of 50, 8192 x 8191 bf16 125 instead of 212; but with
        // few rows per SM there is nothing to copy ahead: 333 x 777 f32 7.4 instead of 6.1)
        if (rows > 4 * int64_t(sms) && alike(dy, a.lddy) && alike(dx, a.lddx) && (!ds || alike(ds, a.ldds))) return run_grad<T, kAlike>(a, sms, dweight, st);
        return run_grad<T, kSpread>(a, sms, dweight, st);
    };
    const cudaError_t e = type == PTC_OUT_F32 ? go(float()) : type == PTC_OUT_BF16 ? go(__nv_bfloat16()) : go(__half());
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "norm gradient launch");
}

}  // extern "C"
