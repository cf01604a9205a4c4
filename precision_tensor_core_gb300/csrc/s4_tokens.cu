// s4_tokens.cu -- product of a few rows of 16-bit activations with 4-bit integer
// weights that have group scales (gemm_a16_s4 of include/ptc.h).
//
// The weights, 0.5 bytes each and their scales, are read once per 16 tokens and are all that a
// call cannot do without.  The products run on mma.sync m16n8k16 with 16 rows of the weights as one operand and eight
// tokens as the other (s4.cuh); sums stay in FP32.
//
// Layout.  The sixteen warps of a CTA are R row groups x S shares of K; a warp owns 16 MT
// rows and every S-th stage of 256 codes.  One of its lanes brings them to the warp's own
// ring in shared memory: the rows by TMA, whole 128-byte lines, and their scales by bulk
// copies, so that no warp waits for another and the others spend no instruction on it.
// A few activations are made operands by every CTA; more by s4_operands_kernel once, and
// every CTA copies them, in chunks of K that fit, two of them in
// shared memory.  The shares' sums are added in order there, and where that leaves
// SMs idle K is also shared by a cluster of up to eight CTAs, whose sums are added in rank
// order through distributed shared memory.
//
// Rates (weights from HBM): one token 5.1 us with 4096 x 4096 weights in groups of 128 and 17.4
// with 16384 x 8192 (3.9 TB/s); sixteen 8.3 and 29 (2.4 TB/s).  No one unit bounds those: 409
// instructions per 16 rows x 256 codes and sixteen tokens take half of the issue slots, and 16 warps
// per SM (registers, shared memory) do not fill the other half while they wait for each other's results.
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
#include "s4.cuh"
#include "s4.h"

namespace ptc {
namespace {

constexpr int kWarps4 = 16, kThreads4 = 32 * kWarps4, kShares4Log2 = 4;
constexpr int kRing4 = 2;  // stages of a warp's ring

__device__ uint32_t g_s4_error = 0;

struct S4Args {
    const void *x;
    int64_t ldx;
    const uint8_t *scales, *zeros;  // tiles
    void *C;
    int64_t ldc;
    int M, N, K;
    int groups;          // per row
    int per_group;       // halves of a stage per group (1 for groups of up to 128)
    int halves;          // of stages, in K
    int stages;          // of K
    int chunk;           // stages of the CTA's K range whose activations are held at once
    int buffers;         // of activations
    int r_log2, ks;
    int xvec, bf16_scales;
    int ring_bytes;      // of all warps
    int sums_at;
    // Operands made by s4_operands_kernel: [token][stage][512 bytes], and factors and sums
    // [tile of tokens][block][token]; NULL: every CTA makes its own.
    uint8_t *xs;
    float2 *xps;
    int stall;           // test hook: this CTA's weights never arrive (-1: none)
    uint64_t wait_limit;
};

struct S4Tail {
    uint64_t full[kWarps4][kRing4], operands[2];
    AbortState abort;
};

// The tokens' operands, once for all CTAs (whole stages, zeros past K): 4 UNIT lanes a block.
// With more than a few tokens making them in every CTA costs as much as the products.
template <typename X, int UNIT>
__global__ void __launch_bounds__(256) s4_operands_kernel(const S4Args a, int tok_tile) {
    constexpr int LANES = 4 * UNIT, PER = 32 / LANES, BLOCKS = 4 / UNIT;
    griddep_wait();
    griddep_launch_dependents();  // (after the wait: what runs before this kernel is done when the product starts)
    const int lane = threadIdx.x % 32, part = lane % LANES;
    const int blocks = a.stages * 2 * BLOCKS, rounds = (blocks + PER - 1) / PER;
    for (int64_t u = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32; u < int64_t(rounds) * a.M; u += int64_t(gridDim.x) * 8) {
        const int tok = int(u / rounds), blk = int(u - int64_t(tok) * rounds) * PER + lane / LANES;
        const int k = blk * (32 * UNIT) + part * 8, have = max(0, min(8, a.K - k));
        const X *p = static_cast<const X *>(a.x) + (have > 0 ? int64_t(tok) * a.ldx + k : 0);
        float2 ps;
        const uint4 op = s4_operands<UNIT, X>(load8(p, have, a.xvec != 0).v[0], ps);
        if (blk >= blocks) continue;
        const int hf = blk / BLOCKS, g = blk % BLOCKS;
        *reinterpret_cast<uint4 *>(a.xs + (int64_t(tok) * a.stages * 2 + hf) * kS4XBytes + s4_x_piece<UNIT>(g * LANES + part)) = op;
        if (part == 0) a.xps[(int64_t(tok / tok_tile) * blocks + blk) * tok_tile + tok % tok_tile] = ps;
    }
}

template <typename X, int MT, int NT, int UNIT>
__global__ void __launch_bounds__(kThreads4, 1) s4_kernel(const __grid_constant__ CUtensorMap tm, const S4Args a) {
    constexpr int TOK = 8 * NT, BLOCKS = 4 / UNIT, D = kRing4, CODES = MT * kS4TileBytes;
    constexpr int SCALES = 2 * BLOCKS * 32;  // bytes of a tile's scales in a stage: two halves' groups
    extern __shared__ uint8_t smem4_raw[];
    uint8_t *const smem4 = smem4_raw + ((1024u - (smem_u32(smem4_raw) & 1023u)) & 1023u);
    __shared__ S4Tail st4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gr = lane >> 2, t = lane & 3;
    const int krank = a.ks == 1 ? 0 : int(cluster_ctarank());
    const int R = 1 << a.r_log2, S = kWarps4 >> a.r_log2;
    const int rg = warp & (R - 1), share = warp >> a.r_log2;
    // Row tiles of R 16 MT rows: this cluster's first, and from one to its next.
    const int tile0 = int(blockIdx.x) / a.ks, tile_step = int(gridDim.x) / a.ks;
    const int tile_rows = 16 * MT * R, tiles = (a.N + tile_rows - 1) / tile_rows;
    const int tok0 = int(blockIdx.y) * TOK, ntok = min(TOK, a.M - tok0);
    // This CTA's stages of K.
    const int q = a.stages / a.ks, rest = a.stages % a.ks;
    const int c0 = krank * q + min(krank, rest), c1 = c0 + q + (krank < rest ? 1 : 0);
    // Shared memory: every warp's codes (on 1024 bytes), every warp's scales and zeros, activations.
    const uint32_t scale_bytes = MT * SCALES * (a.zeros ? 2u : 1u);
    const uint32_t ring = uint32_t(warp * D * CODES), scale_ring = uint32_t(kWarps4 * D * CODES) + uint32_t(warp * D) * scale_bytes;
    const uint32_t xs_base = uint32_t(a.ring_bytes);
    // (Tokens lie an odd number of 64 bytes apart, so that two of them are read at once.)
    const uint32_t tok_bytes = uint32_t(a.chunk) * (2 * kS4XBytes) + 64u, ps_at = tok_bytes * uint32_t(ntok);
    const uint32_t buf_bytes = ps_at + uint32_t(a.chunk) * (2 * BLOCKS * TOK * 8);

    if (lane == 0)
        for (int i = 0; i < D; ++i) mbar_init(&st4.full[warp][i], 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&st4.operands[i], 1);
        st4.abort.flag = 0;
        tma_prefetch_desc(&tm);
    }
    fence_barrier_init();
    // (After s4_operands_kernel the weights may be read before it is done: see there.)
    if (a.xs == nullptr) griddep_wait();

    // Lane 0 brings this warp's stages c0 + share, + S, ... of tile after tile: the codes of
    // its rows (zeros past the matrix) and its tiles' scales and zeros.
    int asked = 0, taken = 0;
    int next = c0 + share, next_tile = next < c1 ? tile0 : tiles, into = 0;
    auto issue = [&]() {
        if (next_tile >= tiles) return;
        if (lane == 0 && int(blockIdx.x) != a.stall) {
            const int row0 = next_tile * tile_rows + rg * (16 * MT);
            uint64_t *bar = &st4.full[warp][into];
            const int g0 = a.per_group == 1 ? 2 * next * BLOCKS : 2 * next / a.per_group;
            const uint32_t bytes = uint32_t(min(2 * BLOCKS, a.groups - g0)) * 32u;
            mbar_arrive_expect_tx(bar, uint32_t(CODES) + MT * bytes * (a.zeros ? 2u : 1u));
            tma_load_2d(smem4 + ring + into * CODES, &tm, bar, next * kS4RowBytes, row0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // (rows past the last tile read it again; what they give is dropped)
                const int64_t at = (int64_t(min(row0 / 16 + m, (a.N + 15) / 16 - 1)) * a.groups + g0) * 32;
                const uint32_t dst = smem_u32(smem4) + scale_ring + uint32_t(into) * scale_bytes + m * SCALES;
                bulk_copy(dst, a.scales + at, bytes, bar);
                if (a.zeros) bulk_copy(dst + MT * SCALES, a.zeros + at, bytes, bar);
            }
        }
        next += S;
        if (next >= c1) {
            next = c0 + share;
            next_tile += tile_step;
        }
        ++asked;
        if (++into == D) into = 0;
    };
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D; ++i) issue();
    if (a.xs != nullptr) griddep_wait();
    griddep_launch_dependents();

    // Activations of chunk c to the buffer of the place-th chunk: 4 UNIT lanes a block, a warp 32 / (4 UNIT),
    // four loads in flight per lane.
    int chunks_done = 0;
    bool over = false;  // the CTA gave up: known to all of its threads
    int brought = 0;    // chunks of operands asked for, alternately on the two barriers
    auto load_x = [&](int c, int place) {
        ++brought;
        constexpr int LANES = 4 * UNIT, PER = 32 / LANES;
        const uint32_t buf = xs_base + (a.buffers == 2 && (place & 1) ? buf_bytes : 0u);
        const int first = c0 + c * a.chunk;
        if (a.xs != nullptr) {  // a copy per token, and one of the factors and sums
            if (threadIdx.x == 0) {
                const int n = min(a.chunk, c1 - first);
                uint64_t *bar = &st4.operands[place & 1];
                const uint32_t bytes = uint32_t(n) * (2 * kS4XBytes), sums = uint32_t(n) * (2 * BLOCKS * TOK * 8), to = smem_u32(smem4) + buf;
                fence_proxy_async_all();  // (what was read there before)
                mbar_arrive_expect_tx(bar, bytes * uint32_t(ntok) + sums);
                for (int j = 0; j < ntok; ++j)
                    bulk_copy(to + uint32_t(j) * tok_bytes, a.xs + (int64_t(tok0 + j) * a.stages + first) * (2 * kS4XBytes), bytes, bar);
                bulk_copy(to + ps_at, a.xps + (int64_t(blockIdx.y) * a.stages + first) * (2 * BLOCKS * TOK), sums, bar);
            }
            return;
        }
        const int blocks = min(2 * min(a.chunk, c1 - first), a.halves - 2 * first) * BLOCKS;
        const int part = lane % LANES, k0 = first * kS4Stage + part * 8;
        const int rounds = (blocks + PER - 1) / PER, all = rounds * ntok;
        for (int u0 = warp; u0 < all; u0 += 4 * kWarps4) {
            uint4 raw[4];
            int at[4], tk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = u0 + j * kWarps4;
                tk[j] = u / rounds;
                at[j] = (u - tk[j] * rounds) * PER + lane / LANES;  // block
                const int k = k0 + at[j] * (32 * UNIT);
                const int have = u < all && at[j] < blocks ? max(0, min(8, a.K - k)) : 0;
                const X *p = static_cast<const X *>(a.x) + (have > 0 ? int64_t(tok0 + tk[j]) * a.ldx + k : 0);
                raw[j] = load8(p, have, a.xvec != 0).v[0];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (u0 + j * kWarps4 >= all) break;
                float2 ps;
                const uint4 op = s4_operands<UNIT, X>(raw[j], ps);
                if (at[j] < blocks) {
                    const int hf = at[j] / BLOCKS, g = at[j] % BLOCKS;
                    *reinterpret_cast<uint4 *>(smem4 + buf + uint32_t(tk[j]) * tok_bytes + uint32_t(hf) * kS4XBytes +
                                               s4_x_piece<UNIT>(g * LANES + part)) = op;
                    if (part == 0) *reinterpret_cast<float2 *>(smem4 + buf + ps_at + uint32_t(at[j] * TOK + tk[j]) * 8u) = ps;
                }
            }
        }
    };
    load_x(0, 0);

    const uint32_t code_at = ring + s4_code_at<UNIT>(lane);
    const uint32_t zeros = a.zeros ? MT * SCALES : 0, scale_at = scale_ring + uint32_t(s4_pair_of(gr)) * 4u;
    uint32_t tok_at[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {  // (tokens past the last read it again; their sums are dropped)
        const int tok = min(8 * n + gr, ntok - 1);
        tok_at[n] = uint32_t(tok) * tok_bytes + uint32_t(t) * 16u;
    }
    int from = 0;  // place in the ring
    uint32_t parity = 0;
    bool ok = true;
    // Sums [warp][row][token].
    float *sums = reinterpret_cast<float *>(smem4 + a.sums_at);
    for (int tile = tile0; tile < tiles; tile += tile_step) {
        float tot[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[m][n][i] = 0.0f;
        for (int c = 0, st = c0 + share; c * a.chunk < c1 - c0; ++c) {
            // Chunk c is there, and everyone is done with the other buffer.  After an abort nothing more is brought: a
            // wait may have ended before its copies did, and their buffer and barrier are still theirs.
            if (a.buffers == 2 || tile == tile0) over = __syncthreads_or(int(st4.abort.flag)) != 0;
            ok = ok && !over;
            if (a.buffers == 2 && !over) {  // (the next tile begins with the first chunk again)
                const bool last = (c + 1) * a.chunk >= c1 - c0;
                if (!last || tile + tile_step < tiles) load_x(last ? 0 : c + 1, chunks_done + 1);
            }
            const uint32_t buf = xs_base + (a.buffers == 2 && (chunks_done & 1) ? buf_bytes : 0u);
            if (a.xs != nullptr && ok && (a.buffers == 2 || tile == tile0))
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st4.operands[chunks_done & 1], uint32_t(chunks_done >> 1) & 1u, &st4.abort,
                                                       &g_s4_error, a.wait_limit));
            ++chunks_done;
            const int first = c0 + c * a.chunk, end = min(c1, first + a.chunk);
            for (; ok && st < end; st += S) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st4.full[warp][from], parity, &st4.abort, &g_s4_error, a.wait_limit));
                if (!ok) break;  // (the sums are not used)
                const uint32_t local = uint32_t(st - first) * 2;
                // (groups of more than 128: the second half's may be the first's)
                const uint32_t second = a.per_group == 1 ? BLOCKS * 32u : uint32_t((2 * st + 1) / a.per_group - 2 * st / a.per_group) * 32u;
#pragma unroll 1
                for (uint32_t h = 0; h < 2; ++h) {
                    if (2 * st + int(h) >= a.halves) break;
                    uint32_t scales[MT];
                    const uint32_t second_row[MT] = {};
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        scales[m] = scale_at + uint32_t(from) * scale_bytes + uint32_t(m) * SCALES + h * second;
                    const uint8_t *xp = smem4 + buf + (local + h) * kS4XBytes;
                    const uint8_t *pp = smem4 + buf + ps_at + (local + h) * (BLOCKS * TOK * 8) + uint32_t(t) * 16u;
                    s4_half_stage<MT, NT, UNIT, BLOCKS, 1, false>(
                        tot, smem4, (code_at + uint32_t(from) * CODES) ^ (h << 6), scales, second_row, 32u, zeros, a.bf16_scales != 0,
                        [&](int i, int n, int) { return *reinterpret_cast<const uint4 *>(xp + tok_at[n] + i * 64); },
                        [&](int g, int n) { return *reinterpret_cast<const float4 *>(pp + (g * TOK + 8 * n) * 8); },
                        (a.K - (2 * st + int(h)) * kS4Half + 32 * UNIT - 1) / (32 * UNIT));
                }
                __syncwarp();  // (every lane has read the stage)
                ++taken;
                issue();
                if (++from == D) {
                    from = 0;
                    parity ^= 1u;
                }
            }
        }
        // Added over the shares and then over the cluster's ranks, both in order.
        float *part = sums + warp * (16 * MT * TOK);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = 16 * m + 2 * s4_pair_of(gr), tk = 8 * n + 2 * t;
                *reinterpret_cast<float2 *>(part + r * TOK + tk) = make_float2(tot[m][n][0], tot[m][n][1]);
                *reinterpret_cast<float2 *>(part + (r + 1) * TOK + tk) = make_float2(tot[m][n][2], tot[m][n][3]);
            }
        if (a.ks > 1)
            cluster_sync();
        else
            __syncthreads();
        // (Rows of a tile and of a row group are powers of two.)
        constexpr int GROUP_LOG2 = MT == 1 ? 4 : 5;
        const int rows_log2 = a.r_log2 + GROUP_LOG2, outs = ntok << rows_log2;
        const int from_share = (16 * MT * TOK) << a.r_log2;  // from a share's sums to the next one's
        const uint32_t base = smem_u32(sums);
        for (int o = krank * kThreads4 + int(threadIdx.x); o < outs; o += a.ks * kThreads4) {
            const int tk = o >> rows_log2, r = o & ((1 << rows_log2) - 1), row = tile * tile_rows + r;
            const int at = (r >> GROUP_LOG2) * (16 * MT * TOK) + (r & (16 * MT - 1)) * TOK + tk;
            float v = 0.0f;
            if (a.ks == 1) {
#pragma unroll 4
                for (int sh = 0; sh < S; ++sh) v = __fadd_rn(v, sums[at + sh * from_share]);
            } else {
                for (int k = 0; k < a.ks; ++k) {
                    const uint32_t peer = mapa_shared(base + uint32_t(at) * 4u, uint32_t(k));
#pragma unroll 4
                    for (int sh = 0; sh < S; ++sh) {
                        float f;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(peer + uint32_t(sh * from_share) * 4u) : "memory");
                        v = __fadd_rn(v, f);
                    }
                }
            }
            if (row < a.N) static_cast<X *>(a.C)[int64_t(tok0 + tk) * a.ldc + row] = from_float<X>(__fmul_rn(v, kS4Out));
        }
        if (tile + tile_step < tiles || a.ks > 1) {  // (the sums are read)
            if (a.ks > 1)
                cluster_sync();
            else
                __syncthreads();
        }
    }
    // After an abort copies in flight land before the CTA exits.
    // (Operands: the last chunk on each barrier.)
    if (st4.abort.flag && a.xs != nullptr)
        for (int c = max(0, brought - 2); c < brought; ++c)
            mbar_wait(&st4.operands[c & 1], uint32_t(c >> 1) & 1u, nullptr, nullptr, a.wait_limit);
    if (int(blockIdx.x) != a.stall)
        for (; taken < asked; ++taken)
            mbar_wait(&st4.full[warp][taken % D], uint32_t(taken / D) & 1u, nullptr, nullptr, a.wait_limit);
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxDim4 = int64_t(1) << 30;
constexpr int64_t kMaxLd4 = int64_t(1) << 36;
constexpr int kMaxDev4 = 64;
// Up to so many tokens, or stages of all tokens, every CTA makes the operands itself.  (A kernel
// for them takes 0.5 us, and 0.7 of the caller's time: 1024 codes of 8 tokens 4.6 us instead of
// 5.1, 4096 of 4 5.9 either way, 4096 of 5 6.9 instead of 5.9, 8192 of 16 51 instead of 12.)
constexpr int64_t kAlone4 = 2, kAloneStages4 = 64;
std::atomic<int> g_s4_rows{0};   // "s4_tokens_rows": 0 by size, 1, 2, 4, 8, 16
std::atomic<int> g_s4_split{0};  // "s4_tokens_split": 0 by size, 1, 2, 4, 8
std::atomic<int> g_s4_tiles{0};  // "s4_tokens_tiles": 0 by size, 1, 2

constexpr int kSmem4 = 227 * 1024;

// Rows and K shares of a launch, and how the activations are held.
struct S4Shape {
    int mt, r_log2, ks;
    int chunk, buffers;
    int sums_at;  // offset of the sums
    size_t smem;
};

// Bytes of all warps' rings: codes, scales, zeros.
int ring_bytes4(int mt, int blocks, const void *zeros) {
    return kWarps4 * kRing4 * mt * (kS4TileBytes + 2 * blocks * 32 * (zeros ? 2 : 1));
}

// Shared memory of a shape; false where a buffer does not hold a stage.
bool fit_s4(S4Shape &sh, const S4Args &a, int blocks, int toks, int tok) {
    const int S = kWarps4 >> sh.r_log2, ring = ring_bytes4(sh.mt, blocks, a.zeros), sums = kWarps4 * 16 * sh.mt * tok * 4;
    const int per_stage = 2 * (toks * kS4XBytes + blocks * tok * 8), more = toks * 64;
    const int range = (a.stages + sh.ks - 1) / sh.ks;  // the longest of a CTA
    const int most = (kSmem4 - 2048) / 256 * 256 - ring - sums;  // (alignment, barriers)
    sh.buffers = int64_t(range) * per_stage + more <= most ? 1 : 2;
    sh.chunk = sh.buffers == 1 ? range : (most / 2 - more) / per_stage;
    if (sh.buffers == 2 && sh.chunk > S) sh.chunk = sh.chunk / S * S;  // (whole rounds of the shares)
    sh.sums_at = ring + sh.buffers * (sh.chunk * per_stage + more);
    sh.smem = size_t(sh.sums_at + sums);
    return sh.chunk > 0;
}

// The shape of least estimated time, in units of 0.01 us.  A warp takes 1.1 us for a stage
// of 16 rows and up to eight tokens, 1.4 for sixteen, 1.9 and 3.0 for 32 rows; an eighth
// more with groups of 32, a tenth with 64.  A tile of rows takes 0.8 to 1.1 us more,
// 2.0 for 16 rows and sixteen tokens, its sums over a cluster 1.6, clusters of four 0.8 to
// start, of eight 2.0.  Operands that a CTA makes itself cost 0.03 us per stage and token, ones
// that do not fit 1.1 per chunk and tile.  (Fitted to the times of every shape at 44 sizes
// between 64 x 64 and 16384 x 8192 weights with 1 to 16 tokens; its choice takes 1.005
// times the fastest shape's time there, 1.07 at most.)
// The keys take a part of the shapes, all of them where that leaves none.
S4Shape choose_s4(const S4Args &a, int unit, int sms) {
    const int64_t chunks = (a.M + 15) / 16;
    const int stages = a.stages, toks = std::min(a.M, 16), nt = a.M > 8 ? 2 : 1;
    S4Shape best{1, 0, 1, 0, 0, 0, 0};
    const int rows = g_s4_rows.load(), split = g_s4_split.load(), tiles = g_s4_tiles.load();
    constexpr int kStage[2][2] = {{111, 139}, {188, 297}}, kTile4[2][2] = {{96, 203}, {84, 108}};
    int64_t cost_best = INT64_MAX;
    for (bool any : {false, true}) {
        for (int mt = 1; mt <= 2; ++mt)
            for (int r = 0; r <= kShares4Log2; ++r)
                for (int k = 1; k <= 8; k *= 2) {
                    const int S = kWarps4 >> r;
                    if (stages < S * k && (r < kShares4Log2 || k > 1)) continue;
                    if (!any && ((rows && rows != 1 << r) || (split && split != k) || (tiles && tiles != mt))) continue;
                    S4Shape sh{mt, r, k, 0, 0, 0, 0};
                    if (!fit_s4(sh, a, 4 / unit, toks, 8 * nt)) continue;
                    const int64_t per = int64_t(16) * mt << r, count = (a.N + per - 1) / per;
                    const int64_t clusters = std::min<int64_t>(count, std::max(1, sms / k));
                    const int64_t walk = (count + clusters - 1) / clusters * chunks;  // tiles of a CTA
                    const int range = (stages + k - 1) / k;
                    const int64_t stage = kStage[mt - 1][nt - 1] * (unit == 1 ? 113 : unit == 2 ? 109 : 100) / 100;
                    int64_t tile = kTile4[mt - 1][nt - 1] + (range + S - 1) / S * stage + (k > 1 ? 156 : 0);
                    if (sh.buffers == 2) tile += 111 * int64_t((range + sh.chunk - 1) / sh.chunk);
                    const int64_t start = (k == 4 ? 84 : k == 8 ? 203 : 0) + (a.xs ? 0 : 3 * int64_t(toks) * range) + ((nt * mt) << r) * 8 / 5;
                    const int64_t cost = start + walk * tile;
                    if (cost < cost_best) {
                        cost_best = cost;
                        best = sh;
                    }
                }
        if (cost_best != INT64_MAX) return best;
    }
    return best;
}

template <typename X, int MT, int NT, int UNIT>
int launch_s4(S4Args a, const void *codes, int64_t pitch, const S4Shape &sh, int sms, cudaStream_t stream) {
    constexpr int TOK = 8 * NT, BLOCKS = 4 / UNIT;
    auto *fn = s4_kernel<X, MT, NT, UNIT>;
    static std::atomic<int> ready[kMaxDev4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_launch(e, "cudaGetDevice");
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem4 - 1024);
        // (An SM changes its split between shared memory and cache only when it is idle.)
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(s4_operands_kernel<X, UNIT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return fail_launch(e, "grouped 4-bit product set-up");
        ready[dev].store(1, std::memory_order_release);
    }
    a.r_log2 = sh.r_log2;
    a.ks = sh.ks;
    a.ring_bytes = ring_bytes4(MT, BLOCKS, a.zeros);
    a.buffers = sh.buffers;
    a.chunk = sh.chunk;
    a.sums_at = sh.sums_at;
    const size_t smem = sh.smem + 1024;
    const int R = 1 << sh.r_log2;
    const int64_t per = int64_t(16) * MT * R, chunks = (a.M + TOK - 1) / TOK;
    const int64_t blocks = std::min((a.N + per - 1) / per, int64_t(std::max(1, sms / sh.ks))) * sh.ks;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = dim3(unsigned(blocks), unsigned(chunks), 1);
    cfg.blockDim = dim3(kThreads4, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (sh.ks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = unsigned(sh.ks);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (pdl_enabled()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    CUtensorMap tm;
    const int rc = encode_tmap_2d(&tm, true, codes, uint64_t(a.K + 1) / 2, uint64_t(a.N), uint64_t(pitch), kS4RowBytes, 16 * MT);
    if (rc) return rc;
    if (a.xs) {
        cudaLaunchConfig_t first = cfg;  // (no cluster)
        cudaLaunchAttribute alone[1];
        std::memset(alone, 0, sizeof(alone));
        const int64_t warps = (int64_t(a.stages) * 2 * BLOCKS * a.M + 8 / UNIT - 1) / (8 / UNIT);
        first.gridDim = dim3(unsigned(std::min<int64_t>((warps + 7) / 8, 4 * int64_t(sms))), 1, 1);
        first.blockDim = dim3(256, 1, 1);
        first.dynamicSmemBytes = 0;
        first.attrs = alone;
        first.numAttrs = 0;
        if (pdl_enabled()) {
            alone[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            alone[0].val.programmaticStreamSerializationAllowed = 1;
            first.numAttrs = 1;
        }
        e = cudaLaunchKernelEx(&first, s4_operands_kernel<X, UNIT>, a, TOK);
        if (e != cudaSuccess) return fail_launch(e, "grouped 4-bit product launch");
        note_launches(1);
    }
    e = cudaLaunchKernelEx(&cfg, fn, tm, a);
    if (e != cudaSuccess) return fail_launch(e, "grouped 4-bit product launch");
    note_launches(1);
    note_fp4_launch(int64_t(cfg.gridDim.x) * cfg.gridDim.y, sh.ks, sh.ks, 16 * MT * R);
    return PTC_OK;
}

template <typename X>
int run_s4(const S4Args &a, const void *codes, int64_t pitch, int64_t group, int sms, cudaStream_t s) {
    const bool wide = a.M > 8;
    const S4Shape sh = choose_s4(a, s4_unit(group), sms);
    auto unit = [&](auto u) {
        constexpr int U = decltype(u)::value;
        if (sh.mt == 1) return wide ? launch_s4<X, 1, 2, U>(a, codes, pitch, sh, sms, s) : launch_s4<X, 1, 1, U>(a, codes, pitch, sh, sms, s);
        return wide ? launch_s4<X, 2, 2, U>(a, codes, pitch, sh, sms, s) : launch_s4<X, 2, 1, U>(a, codes, pitch, sh, sms, s);
    };
    switch (s4_unit(group)) {
        case 1: return unit(std::integral_constant<int, 1>());
        case 2: return unit(std::integral_constant<int, 2>());
        default: return unit(std::integral_constant<int, 4>());
    }
}

bool at_multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

cudaError_t read_and_clear_s4_error_word(uint32_t *out) {
    uint32_t v = 0;
    const uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_s4_error, sizeof(v));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_s4_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

bool set_s4_tuning(const char *key, int64_t v) {
    const bool power = v == 0 || v == 1 || v == 2 || v == 4 || v == 8;
    if (std::strcmp(key, "s4_tokens_rows") == 0 && (power || v == 16))
        g_s4_rows.store(int(v));
    else if (std::strcmp(key, "s4_tokens_split") == 0 && power)
        g_s4_split.store(int(v));
    else if (std::strcmp(key, "s4_tokens_tiles") == 0 && v >= 0 && v <= 2)
        g_s4_tiles.store(int(v));
    else
        return false;
    return true;
}

int check_s4(const S4Weights &w) {
    if (!w.codes || !w.scales) return fail_status(PTC_ERR_INVALID, "codes or scales is NULL");
    if (w.group != 32 && w.group != 64 && (w.group <= 0 || w.group % 128 || w.group > kMaxDim4))
        return fail_status(PTC_ERR_INVALID, "groups are of 32, 64 or a multiple of 128 codes");
    if (w.pitch < (w.cols + 1) / 2 || w.pitch > kMaxLd4)
        return fail_status(PTC_ERR_INVALID, "the code pitch must hold a row's codes, two per byte");
    if (!at_multiple(w.codes, 16) || !at_multiple(w.scales, 16) || !at_multiple(w.zeros, 16) || w.pitch % 16 || w.expert % 16)
        return fail_status(PTC_ERR_ALIGN, "codes, scales and zeros must be 16-byte aligned, with pitches that are multiples of 16");
    return PTC_OK;
}

}  // namespace ptc

using namespace ptc;

// Operands of every token, and factors and sums of whole tiles of tokens, eight per stage at most.
extern "C" int64_t gemm_a16_s4_workspace(int64_t M, int64_t K) {
    if (M <= kAlone4 || K <= 0 || M > 65535 * 16 || K > kMaxDim4) return 0;
    const int64_t stages = (K + kS4Stage - 1) / kS4Stage, tile = M > 8 ? 16 : 8;
    return M * stages * (2 * kS4XBytes) + (M + tile - 1) / tile * tile * stages * 8 * 8;
}

extern "C" int gemm_a16_s4(int64_t M, int64_t N, int64_t K, int type, const void *X, int64_t ldx, const void *W, int64_t ldw,
                           int64_t group, int scale_type, const void *scales, const void *zeros, void *C, int64_t ldc,
                           void *workspace, int64_t workspace_bytes, void *stream) {
    set_message("");
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim4 || N > kMaxDim4 || K > kMaxDim4)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= M, N, K <= 2^30");
    if (M > 65535 * 16) return fail_status(PTC_ERR_INVALID, "at most 1048560 rows of activations");
    if (type != PTC_OUT_BF16 && type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "activations are PTC_OUT_BF16 or PTC_OUT_F16");
    if (scale_type != PTC_OUT_BF16 && scale_type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "scales are PTC_OUT_BF16 or PTC_OUT_F16");
    if (M == 0 || N == 0) return PTC_OK;
    if (!C || ldc < N || ldc > kMaxLd4) return fail_status(PTC_ERR_INVALID, "C is NULL, or ldc is not N .. 2^36");
    if (K > 0 && (!X || ldx < K || ldx > kMaxLd4)) return fail_status(PTC_ERR_INVALID, "X is NULL, or ldx is not K .. 2^36");
    const S4Weights w{W, ldw, 0, scales, zeros, N, K, group, 1};
    int rc;
    if (K > 0 && (rc = check_s4(w))) return rc;
    if (!at_multiple(C, 2) || (K > 0 && !at_multiple(X, 2)))
        return fail_status(PTC_ERR_ALIGN, "X and C must be aligned to their elements");
    const ByteRows c = elem_rows(C, M, N, ldc, 2);
    if (K > 0 && (rows_overlap(c, elem_rows(X, M, K, ldx, 2)) || rows_overlap(c, elem_rows(W, N, (K + 1) / 2, ldw, 1)) ||
                  rows_overlap(c, flat_bytes(scales, w.scale_bytes())) || rows_overlap(c, flat_bytes(zeros, w.scale_bytes()))))
        return fail_status(PTC_ERR_OVERLAP, "C overlaps an operand");
    const int64_t need = gemm_a16_s4_workspace(M, K);
    if (workspace && need > 0) {
        if (workspace_bytes < need) return fail_status(PTC_ERR_INVALID, "the workspace is too small");
        if (!at_multiple(workspace, 16)) return fail_status(PTC_ERR_ALIGN, "the workspace must be 16-byte aligned");
        const ByteRows b = flat_bytes(workspace, uint64_t(need));
        if (rows_overlap(b, c) || rows_overlap(b, elem_rows(X, M, K, ldx, 2)) || rows_overlap(b, elem_rows(W, N, (K + 1) / 2, ldw, 1)) ||
            rows_overlap(b, flat_bytes(scales, w.scale_bytes())) || rows_overlap(b, flat_bytes(zeros, w.scale_bytes())))
            return fail_status(PTC_ERR_OVERLAP, "the workspace overlaps another argument");
    }
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const cudaError_t e = launch_zero_fill(C, ldc, int(M), int(N), 2, sms * 4, s);
        if (e != cudaSuccess) return fail_launch(e, "zero-fill launch");
        note_launches(1);
        return PTC_OK;
    }
    S4Args a;
    std::memset(&a, 0, sizeof(a));
    a.x = X;
    a.ldx = ldx;
    a.scales = static_cast<const uint8_t *>(scales);
    a.zeros = static_cast<const uint8_t *>(zeros);
    a.C = C;
    a.ldc = ldc;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.groups = int(w.groups());
    a.per_group = int(group >= 128 ? group / 128 : 1);
    a.halves = int((K + kS4Half - 1) / kS4Half);
    a.stages = int((K + kS4Stage - 1) / kS4Stage);
    a.stall = take_stall_tile();
    a.wait_limit = wait_limit_ns();
    a.xvec = at_multiple(X, 16) && (M == 1 || ldx % 8 == 0);
    a.bf16_scales = scale_type == PTC_OUT_BF16;
    if (workspace && need > 0 && M * a.stages > kAloneStages4) {
        a.xs = static_cast<uint8_t *>(workspace);
        a.xps = reinterpret_cast<float2 *>(a.xs + M * a.stages * (2 * kS4XBytes));
    }
    return type == PTC_OUT_BF16 ? run_s4<__nv_bfloat16>(a, W, ldw, group, sms, s) : run_s4<__half>(a, W, ldw, group, sms, s);
}
