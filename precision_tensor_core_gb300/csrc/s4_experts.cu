// s4_experts.cu -- a whole mixture-of-experts layer for a few tokens, the experts' weights
// 4-bit integers with group scales (ptc_moe_a16_s4 of include/ptc.h), in two kernels.
//
//   logits = x R^T, the top_k largest of each token, p their softmax
//   h = silu(gate_e x) * (up_e x),  y = sum over the token's experts of p down_e h
//
// The active experts' weights are read once per eight of an expert's tokens and bound the
// call.  router_kernel makes the logits and the tokens' operands (s4.cuh).  Every CTA of
// experts_kernel finds the experts and their tokens from the logits, which is less than
// handing them over.  It then takes items: first, by tickets, 32 rows of h of an expert (32
// rows of gate and 32 of up, the eight warps two row halves by four shares of K), and when
// those are gone 32 rows of y of all experts, or of a share of their codes, which the warps share
// evenly.  The second kind waits until every item of the first kind is done.  A ticket is
// taken by a CTA that runs, and a CTA that waits holds no item of the first kind, so the wait
// ends whatever else holds the GPU.  h passes through memory as one or two binary16 numbers
// relative to a power of two per 32.  No sum's order depends on which CTA or warp takes what, nor
// on the other tokens: a token's products with an expert are summed in chunks of the expert's codes,
// whose sums pass through memory (L2) and are added by slot and chunk.
//
// Each warp brings its rows itself, by TMA, to a ring of its own in shared memory, and the
// next item's while it ends one.  The activations come from L2 into registers, half a stage
// ahead: an expert has few of them.
//
// Times: 16 tokens through 4 each of 32 experts of 4096 x 2048 in bfloat16 142 us (367 MB, 2.6 TB/s),
// in binary16 184; one token through 8 of 64 experts of 2048 x 1024 22 us, a chain of waits: router
// 3.3, routing 2.6, rows of h 8, all of them 3, rows of y 4, their sums 2.  No one unit bounds the
// first: about 410 instructions per 16 rows x 256 codes take 42% of the issue slots, and the 16 warps
// that the registers leave an SM wait for each other's results and for the activations from L2.  With 16
// rows of y per item instead of 32 it took a tenth more.  A fixed order of the sums, whichever warps
// take the chunks, costs it 3%: a sum in shared memory by each warp for what it held took 138.
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

constexpr int kMoeWarps = 8, kMoeThreads = 32 * kMoeWarps;
constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopK = 32, kMaxPairs = 512;
constexpr int kTile = 8;  // tokens of an expert per item
constexpr int kLogits = 4;  // tokens per CTA of the router
constexpr int kMaxRing = 6;  // places of a warp's ring, each a stage of 16 rows; taken in pairs
constexpr int kMaxParts4 = 1024;  // shares of all tiles of 32 rows of y, where they are shared
constexpr int kPlaces = 512;  // sets of chunks' sums: of a tile of 32 rows each, or (more tiles) of a CTA each
// Chunks of all pairs' codes, at least, where their codes have as many stages: enough for an even
// share of warps, few enough for their sums (16 tokens of 4 experts of 2048: 4 of two stages; twice
// as many chunks take the same time within 2%).
constexpr int kChunks = 256;

__device__ uint32_t g_moe_error = 0;

struct Experts {  // scales of one of the two weight matrices
    const uint8_t *scales, *zeros;
    int groups, tiles;
};

struct MoeArgs {
    const void *x, *router;
    int64_t ldx, ldr;
    int router_f32, xvec, rvec;
    void *y;
    int64_t ldy;
    int *ids;        // NULL, or [tokens][top_k]
    float *weights;  // NULL, or the same
    int tokens, hidden, inner, experts, top_k, renormalize;
    int bf16_scales, per_group;  // halves of a stage per group (1 for groups of up to 128)
    Experts gate_up, down;
    int halves, stages;              // of hidden
    int h_halves, h_stages, h_blocks;  // of inner; blocks of 32
    int chunk, chunks;               // stages per chunk of inner, and chunks
    int places, ring_bytes, scale_bytes;  // of a warp's ring (even); of all warps' codes; of a place's scales and zeros
    // Workspace.
    uint32_t *counters;   // tickets, items of the first kind that are done; shares of 32 rows of y that are
    float *parts;         // chunks' sums of rows of y: [place][token][slot][chunk][32]
    float *logits;        // [tokens][experts]
    uint8_t *xs;          // [token][stage] operands
    float2 *xps;          // [token][block] factors and sums
    uint8_t *hs;          // [pair][stage] operands, high parts and low parts
    float2 *hps;          // [pair][block of 32, eight per stage]
    int stall;            // test hook: this item is never done (-1: none)
    uint64_t wait_limit;
};

// ------------------------------------------------------------ router
// A CTA per expert and four tokens: their logits, every thread eight columns of each 2048;
// after them CTAs that make the tokens' operands.
template <typename X, int UNIT>
__global__ void __launch_bounds__(kMoeThreads) router_kernel(const MoeArgs a) {
    __shared__ float part[kMoeWarps][kLogits];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int logits = (a.tokens + kLogits - 1) / kLogits * a.experts;  // CTAs
    if (int(blockIdx.x) >= logits) {
        const int first = int(blockIdx.x) - logits, ctas = int(gridDim.x) - logits;
        if (first == 0)
            for (int i = threadIdx.x; i < 2 + kMaxParts4 / 2; i += kMoeThreads) a.counters[i] = 0;
        constexpr int LANES = 4 * UNIT, PER = 32 / LANES, GROUPS = 4 / UNIT;
        const int blocks = a.stages * 2 * GROUPS, rounds = (blocks + PER - 1) / PER, lane8 = lane % LANES;
        for (int u = first * kMoeWarps + warp; u < rounds * a.tokens; u += ctas * kMoeWarps) {
            const int tok = u / rounds, blk = (u - tok * rounds) * PER + lane / LANES;
            const int k = blk * (32 * UNIT) + lane8 * 8, have = max(0, min(8, a.hidden - k));
            const X *p = static_cast<const X *>(a.x) + (have > 0 ? int64_t(tok) * a.ldx + k : 0);
            float2 ps;
            const uint4 op = s4_operands<UNIT, X>(load8(p, have, a.xvec != 0).v[0], ps);
            if (blk >= blocks) continue;
            const int half = blk / GROUPS, g = blk % GROUPS;
            *reinterpret_cast<uint4 *>(a.xs + (int64_t(tok) * a.stages * 2 + half) * kS4XBytes + s4_x_piece<UNIT>(g * LANES + lane8)) = op;
            if (lane8 == 0) a.xps[int64_t(tok) * blocks + blk] = ps;
        }
        return;
    }
    const int e = int(blockIdx.x) % a.experts, t0 = int(blockIdx.x) / a.experts * kLogits;
    const X *x[kLogits];
    float acc[kLogits];
#pragma unroll
    for (int j = 0; j < kLogits; ++j) {  // (tokens past the last are the last again)
        x[j] = static_cast<const X *>(a.x) + int64_t(min(t0 + j, a.tokens - 1)) * a.ldx;
        acc[j] = 0.0f;
    }
#pragma unroll 2
    for (int k = int(threadIdx.x) * 8; k < a.hidden; k += kMoeThreads * 8) {
        const int have = min(8, a.hidden - k);
        float w[8];
        Pack8<X> v[kLogits];
#pragma unroll
        for (int j = 0; j < kLogits; ++j) v[j] = load8(x[j] + k, have, a.xvec != 0);
        if (a.router_f32) {
            const Pack8<float> r = load8(static_cast<const float *>(a.router) + int64_t(e) * a.ldr + k, have, a.rvec != 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = r.get(i);
        } else {
            const Pack8<X> r = load8(static_cast<const X *>(a.router) + int64_t(e) * a.ldr + k, have, a.rvec != 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = to_float(r.get(i));
        }
#pragma unroll
        for (int j = 0; j < kLogits; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j] = __fmaf_rn(to_float(v[j].get(i)), w[i], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < kLogits; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (int(threadIdx.x) < min(kLogits, a.tokens - t0)) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kMoeWarps; ++w) v += part[w][threadIdx.x];
        a.logits[int64_t(t0 + threadIdx.x) * a.experts + e] = v;
    }
}

// ------------------------------------------------------------ routing
// What every CTA finds from the logits.  A pair is a token and one of its experts; pairs
// lie by expert, then by token, and each expert's in tiles of up to eight.
struct Routing {
    uint8_t pair_token[kMaxPairs];
    uint16_t pair_slot[kMaxPairs];  // [token][slot]
    float pair_weight[kMaxPairs];
    uint16_t tile_expert[kMaxPairs], tile_first[kMaxPairs];
    uint8_t tile_count[kMaxPairs];
    int tiles;
    uint32_t ticket[4];
    bool last;  // of the shares of 32 rows of y
};
struct RoutingWork {  // in the ring's place, before it is used
    uint32_t mask[kMaxExperts][2];   // tokens of an expert
    uint16_t first[kMaxExperts];     // its first pair
    uint16_t id[kMaxPairs];          // [token][slot]
    float slot_weight[kMaxPairs];
};

struct MoeTail {
    uint64_t full[kMoeWarps][kMaxRing];
    AbortState abort;
};

// Order of logits as integers: NaN below every number, 0 for what is taken already.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) > kInfBits) return 1u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int PER>
__device__ __forceinline__ void choose_experts(const MoeArgs &a, RoutingWork &w) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int tok = warp; tok < a.tokens; tok += kMoeWarps) {
        const float *l = a.logits + int64_t(tok) * a.experts;
        float v[PER];
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < a.experts ? __ldcg(l + e) : 0.0f;
            key[i] = e < a.experts ? logit_key(v[i]) : 0u;
        }
        float largest = 0.0f, mine = 0.0f;  // of the logits; this lane's slot's
        int my_id = 0;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t k = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) k = max(k, key[i]);
            const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, k);
            int at = kMaxExperts;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == best) at = lane + 32 * i;
            const int e = __reduce_min_sync(0xFFFFFFFFu, at);
            float value = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i == e) {
                    key[i] = 0u;
                    value = v[i];
                }
            value = __shfl_sync(0xFFFFFFFFu, value, e & 31);
            if (j == 0) largest = value;
            if (lane == j) {
                mine = value;
                my_id = e;
            }
        }
        float sum = 0.0f;
        const float p = lane < a.top_k ? expf(mine - largest) : 0.0f;
        if (a.renormalize) {
            sum = p;
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < a.experts) sum += expf(v[i] - largest);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane < a.top_k) {
            const int s = tok * a.top_k + lane;
            const float share = __fdiv_rn(p, sum);
            w.id[s] = uint16_t(my_id);
            w.slot_weight[s] = share;
            atomicOr(&w.mask[my_id][tok >> 5], 1u << (tok & 31));
            if (blockIdx.x == 0) {
                if (a.ids) a.ids[s] = my_id;
                if (a.weights) a.weights[s] = share;
            }
        }
    }
}

__device__ __forceinline__ void route(const MoeArgs &a, Routing &r, RoutingWork &w) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int i = threadIdx.x; i < a.experts; i += kMoeThreads) w.mask[i][0] = w.mask[i][1] = 0;
    __syncthreads();
    if (a.experts <= 64)
        choose_experts<2>(a, w);
    else if (a.experts <= 128)
        choose_experts<4>(a, w);
    else
        choose_experts<kMaxExperts / 32>(a, w);
    __syncthreads();
    if (warp == 0) {  // pairs and tiles of the experts, in order
        int pairs = 0, tiles = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < a.experts ? __popc(w.mask[e][0]) + __popc(w.mask[e][1]) : 0, t = (c + kTile - 1) / kTile;
            int sum = c | t << 16;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += up;
            }
            const int p0 = pairs + (sum & 0xFFFF) - c, t0 = tiles + (sum >> 16) - t;
            if (e < a.experts) w.first[e] = uint16_t(p0);
            for (int i = 0; i < t; ++i) {
                r.tile_expert[t0 + i] = uint16_t(e);
                r.tile_first[t0 + i] = uint16_t(p0 + kTile * i);
                r.tile_count[t0 + i] = uint8_t(min(kTile, c - kTile * i));
            }
            const int total = __shfl_sync(0xFFFFFFFFu, sum, 31);
            pairs += total & 0xFFFF;
            tiles += total >> 16;
        }
        if (lane == 0) r.tiles = tiles;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < a.tokens * a.top_k; s += kMoeThreads) {
        const int tok = s / a.top_k, e = w.id[s];
        const uint32_t lo = w.mask[e][0], hi = w.mask[e][1];
        const int rank = tok < 32 ? __popc(lo & ((1u << tok) - 1u)) : __popc(lo) + __popc(hi & ((1u << (tok - 32)) - 1u));
        r.pair_token[w.first[e] + rank] = uint8_t(tok);
        r.pair_slot[w.first[e] + rank] = uint16_t(s);
        r.pair_weight[w.first[e] + rank] = w.slot_weight[s];
    }
    fence_proxy_async_all();  // (bulk copies write where this was held)
    __syncthreads();
}

// Waits until `count` items of the first kind are done; false after the limit.
__device__ __forceinline__ bool wait_done(const MoeArgs &a, uint32_t count) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.counters + 1) : "memory");
        if (v >= count) return true;
        if ((n & 15u) == 0 && globaltimer_ns() - t0 > a.wait_limit) {
            atomicCAS(&g_moe_error, 0u, kErrTimeout);
            return false;
        }
        __nanosleep(32);
    }
}

// ------------------------------------------------------------ experts
// What a warp brings next: stages of one item, in the order in which it takes them.
struct Bring {
    int left;         // stages of the item
    int second_kind;  // rows of y
    int tile, st;     // the next stage's tile of pairs and stage
    int row;          // the warp's first row of h, or the item's of y
    int expert;       // the tile's
    const uint8_t *scales, *more_scales;  // of the tiles of the first and second 16 rows, from group 0
};

template <typename X, int UNIT, bool ODD>
__global__ void __launch_bounds__(kMoeThreads, 2)
    experts_kernel(const __grid_constant__ CUtensorMap tm_up, const __grid_constant__ CUtensorMap tm_down, const MoeArgs a) {
    constexpr int SG = 4 / UNIT;            // scale groups (and, of x, blocks) per half stage
    constexpr int SCALES = 2 * SG * 32;     // bytes of a tile's scales in a stage
    constexpr int ZEROS = SCALES * (ODD ? 2 : 1);  // zeros from scales
    constexpr int CODES = kS4TileBytes;
    // Rows of y: with groups of 128 and more half a stage is one block, whose four blocks of
    // 32 of h are brought to one power of two as they are loaded.
    constexpr int UNIT_H = UNIT == 4 ? 4 : 1;
    // h as one binary16 number where y is bfloat16, two where it is binary16.  One is off by
    // 2^-11 of an element at most, an eighth of what y's own rounding is: as those errors are
    // weighted as h itself is, sqrt(1 + 1 / 64) = 1.008 times y's error without them.
    constexpr int PARTS = std::is_same_v<X, __half> ? 2 : 1;
    extern __shared__ uint8_t moe_raw[];
    uint8_t *const smem = moe_raw + ((1024u - (smem_u32(moe_raw) & 1023u)) & 1023u);
    __shared__ Routing r;
    __shared__ MoeTail st;
    __shared__ __align__(16) float2 factors[kMoeWarps][2][32];  // of half a stage, [block][token]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float2 *const mine = &factors[warp][0][0];
    const int f = s4_pair_of(lane >> 2), gr = lane >> 2, t = lane & 3;
    const int half = warp & 1, share = warp >> 1;  // of rows of h
    const uint32_t ring = uint32_t(warp * a.places * CODES), scale_ring = uint32_t(a.ring_bytes + warp * a.places * a.scale_bytes);
    float *const sums = reinterpret_cast<float *>(smem + a.ring_bytes + kMoeWarps * a.places * a.scale_bytes);
    if (lane == 0)
        for (int i = 0; i < a.places; ++i) mbar_init(&st.full[warp][i], 1);
    if (threadIdx.x == 0) {
        st.abort.flag = 0;
        tma_prefetch_desc(&tm_up);
        tma_prefetch_desc(&tm_down);
    }
    fence_barrier_init();
    griddep_wait();
    griddep_launch_dependents();
    // (Tickets are asked for where they are due and looked at later.)
    uint32_t asked_ticket = 0;
    if (threadIdx.x == 0) asked_ticket = atomicAdd(a.counters, 1u);
    route(a, r, *reinterpret_cast<RoutingWork *>(smem));
    if (threadIdx.x == 0) r.ticket[0] = asked_ticket;

    const int units = r.tiles * a.chunks;  // chunks of 32 rows of y, of all tiles of pairs
    const int row_tiles = (a.hidden + 31) / 32;
    // Shares of these chunks that are items of their own: what takes the least stages of a warp
    // in all rounds, two more per item.
    const int grid = int(gridDim.x);
    int shares = 1;
    {
        const int n = (lane & 7) + 1, items = row_tiles * n, warps = n * kMoeWarps;
        const uint32_t cost = uint32_t((items + grid - 1) / grid) * uint32_t((units + warps - 1) / warps * a.chunk + 2);
        const bool may = n == 1 || (items <= kMaxParts4 && cost < 1u << 28);
        shares = int(__reduce_min_sync(0xFFFFFFFFu, may ? min(cost, (1u << 28) - 1) * 8u + uint32_t(n - 1) : ~0u) & 7u) + 1;
    }
    // Items of the first kind are taken by tickets, which end the wait for them: whoever waits has
    // none that is not done.  Those of the second kind are every grid-th from this CTA's own number.
    const int first_items = r.tiles * a.h_blocks, second_items = row_tiles * shares;
    // With many items per CTA tickets are taken two items ahead, so that the next item's weights
    // are asked for before this one's end; with few that would leave CTAs without, and they are
    // taken when the item before begins.
    const bool early = first_items >= 4 * int(gridDim.x);
    if (early && threadIdx.x == 0) r.ticket[1] = atomicAdd(a.counters, 1u);
    __syncthreads();
    // This warp's chunks of a share, as stages of all tiles.
    auto units_of = [&](int part, int &u0, int &u1) {
        const int first = int(int64_t(units) * part / shares), n = int(int64_t(units) * (part + 1) / shares) - first;
        auto stage = [&](int u) { return u / a.chunks * a.h_stages + u % a.chunks * a.chunk; };
        u0 = stage(first + n * warp / kMoeWarps);
        u1 = stage(first + n * (warp + 1) / kMoeWarps);
    };
    // The item of a round: one of the first kind by its ticket, then those of the second kind; -1
    // after the last.  (Tickets rise, so that the rounds of the first kind come first;
    // `second_round` is the round of the first ticket past them, where it is known.)
    int second_round = 1 << 30;
    auto item_of = [&](int round) {
        if (round < second_round) {
            const uint32_t t = r.ticket[round & 3];
            if (t < uint32_t(first_items)) return int(t);
            second_round = round;
        }
        const int64_t second = int(blockIdx.x) + int64_t(round - second_round) * grid;
        return second < second_items ? first_items + int(second) : -1;
    };
    // From scales to zeros, of either matrix (0: it has none).
    const int64_t up_zeros = a.gate_up.zeros ? a.gate_up.zeros - a.gate_up.scales : 0;
    const int64_t down_zeros = a.down.zeros ? a.down.zeros - a.down.scales : 0;
    auto tile_scales = [](const Experts &w, int e, int tile) {  // (rows past the last tile read it again)
        return w.scales + (int64_t(e) * w.tiles + min(tile, w.tiles - 1)) * w.groups * 32;
    };
    // The stages of the item of a round; none past the last item.
    auto begin = [&](int round) {
        const int item = item_of(round);
        Bring b{0, 0, 0, 0, 0, 0, nullptr, nullptr};
        if (item < 0) return b;
        if (item < first_items) {
            b.tile = item / a.h_blocks;
            b.row = (item - b.tile * a.h_blocks) * 32 + half * 16;
            b.st = share;
            b.left = (a.stages - share + 3) / 4;  // share, share + 4, ...
            b.expert = r.tile_expert[b.tile];
            b.scales = tile_scales(a.gate_up, b.expert, b.row / 16);
            b.more_scales = tile_scales(a.gate_up, b.expert, (a.inner + b.row) / 16);
        } else {
            int u0, u1;
            units_of((item - first_items) / row_tiles, u0, u1);
            b.second_kind = 1;
            b.row = (item - first_items) % row_tiles * 32;
            b.tile = u0 / a.h_stages;
            b.st = u0 - b.tile * a.h_stages;
            b.left = u1 - u0;
            b.expert = r.tile_expert[min(b.tile, r.tiles - 1)];
            b.scales = tile_scales(a.down, b.expert, b.row / 16);
            b.more_scales = tile_scales(a.down, b.expert, b.row / 16 + 1);
        }
        return b;
    };
    // Lane 0 brings one stage: its codes (zeros past the matrix) and its tiles' scales and
    // zeros.  When the item's are all asked for, the next item's follow: the weights do
    // not depend on h.
    Bring b = begin(0);
    int bring_round = 0, into = 0, asked = 0, taken = 0;  // (in places)
    auto issue = [&](int round, bool ahead) {
        if (b.left == 0 && bring_round == round && ahead) b = begin(++bring_round);
        if (b.left == 0 || asked - taken + 2 > a.places) return false;
        if (lane == 0) {
            const CUtensorMap *const tm = b.second_kind ? &tm_down : &tm_up;
            const int groups = b.second_kind ? a.down.groups : a.gate_up.groups;
            const int64_t zeros = b.second_kind ? down_zeros : up_zeros;
            const int g0 = a.per_group == 1 ? 2 * b.st * SG : 2 * b.st / a.per_group;
            const uint32_t bytes = uint32_t(min(2 * SG, groups - g0)) * 32u, both = zeros ? 2u * bytes : bytes;
            const uint32_t codes = smem_u32(smem) + ring + into * CODES, scales = smem_u32(smem) + scale_ring + into * a.scale_bytes;
            uint64_t *const bar = &st.full[warp][into];
            const uint8_t *const from = b.scales + g0 * 32;
            mbar_arrive_expect_tx(bar, kS4TileBytes + both);
            tma_load_rows(codes, tm, bar, b.st * kS4RowBytes, b.row, b.expert);
            bulk_copy(scales, from, bytes, bar);
            if (zeros) bulk_copy(scales + ZEROS, from + zeros, bytes, bar);
            // (up's rows may begin in the middle of a tile and end in the next one)
            const uint32_t second = scales + a.scale_bytes;
            const uint8_t *const more = b.more_scales + g0 * 32;
            const int row = b.second_kind ? b.row + 16 : a.inner + b.row;
            const bool next = ODD && !b.second_kind && row / 16 + 1 < a.gate_up.tiles;
            mbar_arrive_expect_tx(bar + 1, kS4TileBytes + (next ? 2 * both : both));
            tma_load_rows(codes + CODES, tm, bar + 1, b.st * kS4RowBytes, row, b.expert);
            bulk_copy(second, more, bytes, bar + 1);
            if (zeros) bulk_copy(second + ZEROS, more + zeros, bytes, bar + 1);
            if (next) {
                bulk_copy(second + SCALES, more + groups * 32, bytes, bar + 1);
                if (zeros) bulk_copy(second + ZEROS + SCALES, more + groups * 32 + zeros, bytes, bar + 1);
            }
        }
        --b.left;
        if (b.second_kind) {
            if (++b.st == a.h_stages) {
                b.st = 0;
                ++b.tile;
                if (b.left > 0) {
                    const int e = r.tile_expert[b.tile];
                    const int64_t to = int64_t(e - b.expert) * a.down.tiles * a.down.groups * 32;
                    b.scales += to;
                    b.more_scales += to;
                    b.expert = e;
                }
            }
        } else {
            b.st += 4;
        }
        asked += 2;
        into += 2;
        if (into == a.places) into = 0;
        return true;
    };
    // Waits for the next stage to take; its place in the ring.
    bool ok = true;
    int from = 0;          // the place
    uint32_t parity = 0;
    auto arrived = [&](int places) {
        for (int i = 0; i < places; ++i)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st.full[warp][from + i], parity, &st.abort, &g_moe_error, a.wait_limit)) && ok;
        return ok;
    };
    // A stage has been read by every lane: its places are free.
    auto release = [&](int places) {
        __syncwarp();
        taken += places;
        from += places;
        if (from == a.places) {
            from = 0;
            parity ^= 1u;
        }
    };
    // Offset in a stage's scales of this lane's two rows, for the gate (and y) and up; from
    // the first to the second row.
    uint32_t row_at[2], row_more[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        auto at = [&](int i) { return uint32_t(i >> 4) * SCALES + uint32_t(i & 15) * 2u; };
        const int i = 2 * f + (ODD && m ? a.inner % 16 : 0);
        row_at[m] = at(i) + (m ? uint32_t(a.scale_bytes) : 0u);  // (up's are in the next place)
        row_more[m] = at(i + 1) - at(i);
    }
    // From the first to the second half of a stage: that of its scales.
    auto second_half = [&](int s) {
        return a.per_group == 1 ? SG * 32u : uint32_t((2 * s + 1) / a.per_group - 2 * s / a.per_group) * 32u;
    };

    __syncwarp();
    while (issue(0, early)) {}
    bool ready = false;  // every item of the first kind is done
    for (int round = 0;; ++round) {
        const int item = item_of(round);
        if (item < 0) break;
        const int later = (round + (early ? 2 : 1)) & 3;
        if (threadIdx.x == 0 && item < first_items) asked_ticket = atomicAdd(a.counters, 1u);
        if (item < first_items) {
            // ------------------------------------------------ rows of h
            const int tile = item / a.h_blocks, ib = item - tile * a.h_blocks;
            const int pair0 = r.tile_first[tile], n = r.tile_count[tile];
            float tot[2][1][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[m][0][i] = 0.0f;
            // Operands and factors of half a stage ahead: 16 bytes per pair of MMAs of this lane's
            // token, and an entry of the warp's [block][token].
            const uint8_t *const xs = a.xs + int64_t(r.pair_token[pair0 + min(gr, n - 1)]) * a.stages * (2 * kS4XBytes) + t * 16;
            const float2 *const ps = a.xps + int64_t(r.pair_token[pair0 + min(lane & 7, n - 1)]) * a.stages * (2 * SG) + min(lane >> 3, SG - 1);
            uint4 x[2][4];
            float2 p[2];
            auto load = [&](int hf, int at) {  // (the workspace holds whole stages)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[at][i] = *reinterpret_cast<const uint4 *>(xs + hf * kS4XBytes + i * 64);
                p[at] = ps[hf * SG];
            };
            if (share < a.stages) load(2 * share, 0);
            for (int s = share; s < a.stages && ok; s += 4) {
                if (!arrived(2)) break;
                const uint32_t more = second_half(s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 0)
                        load(2 * s + 1, 1);
                    else if (s + 4 < a.stages)
                        load(2 * (s + 4), 0);
                    if (2 * s + h < a.halves) {
                        if (lane < 8 * SG) mine[h * 32 + lane] = p[h];
                        __syncwarp();
                        const uint32_t at = scale_ring + uint32_t(from * a.scale_bytes) + uint32_t(h) * more;
                        const uint32_t scales[2] = {at + row_at[0], at + row_at[1]};
                        s4_half_stage<2, 1, UNIT, SG, 1, ODD>(
                            tot, smem, (ring + uint32_t(from) * CODES + s4_code_at<UNIT>(lane)) ^ (uint32_t(h) << 6), scales, row_more,
                            32u, a.gate_up.zeros ? ZEROS : 0u, a.bf16_scales != 0, [&](int i, int, int) { return x[h][i]; },
                            [&](int g, int) { return *reinterpret_cast<const float4 *>(mine + h * 32 + g * 8 + 2 * t); },
                            (a.hidden - (2 * s + h) * kS4Half + 32 * UNIT - 1) / (32 * UNIT));
                    }
                }
                release(2);
                issue(round, early);
            }
            // Sums of the shares: [share][half][gate, up][row][token].
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float *p = sums + ((warp * 2 + m) * 16 + 2 * f) * kTile + 2 * t;
                *reinterpret_cast<float2 *>(p) = make_float2(tot[m][0][0], tot[m][0][1]);
                *reinterpret_cast<float2 *>(p + kTile) = make_float2(tot[m][0][2], tot[m][0][3]);
            }
            __syncthreads();
            if (st.abort.flag) break;
            if (warp < n) {  // token `warp`, a lane a row
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float *p = sums + ((s * 2 + (lane >> 4)) * 2 * 16 + (lane & 15)) * kTile + warp;
                    gate = __fadd_rn(gate, p[0]);
                    up = __fadd_rn(up, p[16 * kTile]);
                }
                gate = __fmul_rn(gate, kS4Out);
                up = __fmul_rn(up, kS4Out);
                const float h = ib * 32 + lane < a.inner ? __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up) : 0.0f;
                __half hi, lo;
                float2 ps;
                s4_operand32<PARTS>(h, lane, hi, lo, ps);
                const int64_t pair = pair0 + warp;
                // [pair][stage][high parts of 256, low parts]
                uint8_t *p = a.hs + (pair * a.h_stages + ib / 8) * (4 * kS4XBytes) + ((ib >> 2) & 1) * kS4XBytes +
                             s4_x_piece<UNIT_H>((ib & 3) * 4 + (lane >> 3)) + s4_half(lane & 7) * 2;
                *reinterpret_cast<__half *>(p) = hi;
                if (PARTS == 2) *reinterpret_cast<__half *>(p + 2 * kS4XBytes) = lo;
                if (lane == 0) a.hps[pair * a.h_stages * 8 + ib] = ps;
            }
            __syncthreads();
            if (threadIdx.x == 0 && item != a.stall)  // (released for the whole CTA)
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counters + 1) : "memory");
        } else {
            // ------------------------------------------------ rows of y
            if (!ready) {
                if (threadIdx.x == 0 && !wait_done(a, uint32_t(first_items))) st.abort.flag = 1;
                __syncthreads();
                if (st.abort.flag) break;
                ready = true;
            }
            const int part = (item - first_items) / row_tiles, row_tile = (item - first_items) % row_tiles, row0 = row_tile * 32;
            int u0, u1;
            units_of(part, u0, u1);
            // (32 bits: 512 places of at most 767 sums)
            const int place = (row_tiles <= kPlaces ? row_tile : int(blockIdx.x)) * (a.tokens * a.top_k * a.chunks);
            float tot[2][1][4] = {{{0.0f, 0.0f, 0.0f, 0.0f}}, {{0.0f, 0.0f, 0.0f, 0.0f}}};
            int tile = u0 / a.h_stages, s = u0 - tile * a.h_stages, chunk = s / a.chunk;
            // Half a stage ahead where the registers hold it (not with two parts), of the pairs of
            // a tile (h comes from other SMs): operands, and the factor and sum of one block of one
            // token: UNIT_H 4 those of this lane's operands.
            constexpr int AHEAD = PARTS == 1 ? 1 : 0;
            uint4 x[1 + AHEAD][4][PARTS];
            float2 p[1 + AHEAD];
            const uint8_t *xs = nullptr;
            const float2 *ps = nullptr;
            auto point = [&](int tl) {  // to a tile's pairs
                const int pair0 = r.tile_first[tl], n = r.tile_count[tl];
                const int token = UNIT_H == 4 ? gr : lane & 7, block = UNIT_H == 4 ? t : lane >> 3;
                xs = a.hs + int64_t(pair0 + min(gr, n - 1)) * a.h_stages * (4 * kS4XBytes) + t * 16;
                ps = a.hps + int64_t(pair0 + min(token, n - 1)) * a.h_stages * 8 + block;
            };
            auto load = [&](int hf, int at) {
                const uint8_t *const from = xs + (hf >> 1) * (4 * kS4XBytes) + (hf & 1) * kS4XBytes;
                const bool there = UNIT_H == 1 || hf * 4 + t < a.h_blocks;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        x[at][i][part] = there ? __ldcg(reinterpret_cast<const uint4 *>(from + i * 64 + part * 2 * kS4XBytes)) : make_uint4(0, 0, 0, 0);
                p[at] = there ? __ldcg(ps + hf * 4) : make_float2(0x1p-114f, 0.0f);
            };
            if (u0 < u1) {
                point(tile);
                load(2 * s, 0);
            }
            for (int u = u0; u < u1 && ok; ++u) {
                if (!arrived(2)) break;
                const uint32_t more = second_half(s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int now = h * AHEAD;
                    if (!AHEAD) {
                        if (h == 1) load(2 * s + 1, 0);
                    } else if (h == 0) {
                        load(2 * s + 1, 1);
                    } else if (u + 1 < u1) {
                        const bool over = s + 1 == a.h_stages;
                        if (over) point(tile + 1);
                        load(over ? 0 : 2 * (s + 1), 0);
                    }
                    if (2 * s + h < a.h_halves) {
                        if constexpr (UNIT_H == 4) {
                            float most = fmaxf(p[now].x, __shfl_xor_sync(0xFFFFFFFFu, p[now].x, 1));
                            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                            // (powers of two: the inverse and the quotient are exact)
                            const float rel = __fmul_rn(p[now].x, __uint_as_float((254u << 23) - __float_as_uint(most)));
                            // (binary16 as what it multiplies: 0 below 2^-24)
                            const __half2 by = __float2half2_rn(rel);
                            float sum = __fmul_rn(p[now].y, __low2float(by));
                            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                            if (t == 0) mine[h * 32 + gr] = make_float2(most, sum);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int part = 0; part < PARTS; ++part) {
                                    __half2 *v = reinterpret_cast<__half2 *>(&x[now][i][part]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) v[k] = __hmul2(v[k], by);
                                }
                        } else {
                            mine[h * 32 + lane] = p[now];
                        }
                        __syncwarp();
                        const uint32_t at = scale_ring + uint32_t(from * a.scale_bytes) + uint32_t(h) * more + row_at[0];
                        const uint32_t scales[2] = {at, at + uint32_t(a.scale_bytes)}, next_row[2] = {2u, 2u};
                        s4_half_stage<2, 1, UNIT_H, SG, PARTS, false>(
                            tot, smem, (ring + uint32_t(from) * CODES + s4_code_at<UNIT_H>(lane)) ^ (uint32_t(h) << 6), scales, next_row, 32u,
                            a.down.zeros ? ZEROS : 0u, a.bf16_scales != 0, [&](int i, int, int part) { return x[now][i][part]; },
                            [&](int g, int) { return *reinterpret_cast<const float4 *>(mine + h * 32 + g * 8 + 2 * t); },
                            a.h_blocks - (2 * s + h) * 4);
                    }
                }
                release(2);
                issue(round, early);
                if (++s == a.h_stages || s == (chunk + 1) * a.chunk) {
                    // The chunk's sums to their places, of the tile's pairs.
                    const int pair0 = r.tile_first[tile], n = r.tile_count[tile];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = 2 * t + i;
                        if (j < n) {
                            float *p = a.parts + (place + int(r.pair_slot[pair0 + j]) * a.chunks + chunk) * 32 + 2 * f;
                            const float pw = r.pair_weight[pair0 + j];
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                *reinterpret_cast<float2 *>(p + m * 16) = make_float2(__fmul_rn(pw, tot[m][0][i]), __fmul_rn(pw, tot[m][0][2 + i]));
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) tot[m][0][i] = 0.0f;
                    ++chunk;
                    if (s == a.h_stages) {
                        s = chunk = 0;
                        ++tile;
                        if (!AHEAD && u + 1 < u1) point(tile);
                    }
                }
                if (!AHEAD && u + 1 < u1) load(2 * s, 0);
            }
            __syncthreads();
            if (st.abort.flag) break;
            if (shares > 1) {  // the last share to end adds the chunks of all
                if (threadIdx.x == 0) {
                    __threadfence();
                    r.last = atomicAdd(a.counters + 2 + row_tile, 1u) == uint32_t(shares - 1);
                    __threadfence();
                }
                __syncthreads();
            }
            if (shares == 1 || r.last) {  // token by token, a lane a row, in the slots' order
                const int n = a.top_k * a.chunks;
                for (int o = threadIdx.x; o < a.tokens * 32; o += kMoeThreads) {
                    const float *p = a.parts + (place + (o >> 5) * n) * 32 + (o & 31);
                    float v = 0.0f;
                    for (int k = 0; k < n; k += 16) {  // (16 loads in flight)
                        float c[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) c[i] = k + i < n ? __ldcg(p + (k + i) * 32) : 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) v = __fadd_rn(v, c[i]);
                    }
                    const int row = row0 + (o & 31);
                    if (row < a.hidden) static_cast<X *>(a.y)[int64_t(o >> 5) * a.ldy + row] = from_float<X>(__fmul_rn(v, kS4Out));
                }
            }
        }
        if (threadIdx.x == 0 && item < first_items) r.ticket[later] = asked_ticket;
        __syncthreads();  // the tickets are there, and the sums are read
        while (issue(round, true)) {}  // (what the item's end left room for)
    }
    // After an abort copies in flight land before the CTA exits.
    for (; taken < asked; release(1)) mbar_wait(&st.full[warp][from], parity, nullptr, nullptr, a.wait_limit);
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxSize = 1 << 20;  // of hidden and inner
constexpr int64_t kMaxLdM = int64_t(1) << 36;
constexpr int kMaxDevM = 64;

int64_t up_to(int64_t v, int64_t n) { return (v + n - 1) / n * n; }
bool lies_on(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct MoeSpace {
    int64_t logits, xs, xps, hs, hps, parts, bytes;
    int chunk, chunks;
};

MoeSpace moe_space(int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int64_t top_k) {
    const int64_t stages = (hidden + 255) / 256, h_stages = (inner + 255) / 256, pairs = tokens * top_k;
    MoeSpace s;
    s.logits = up_to((2 + kMaxParts4) * 4, 256);
    s.xs = s.logits + up_to(tokens * experts * 4, 256);
    s.xps = s.xs + tokens * stages * 2 * kS4XBytes;
    s.hs = s.xps + up_to(tokens * stages * 8 * 8, 256);
    s.hps = s.hs + pairs * h_stages * 4 * kS4XBytes;
    s.parts = s.hps + up_to(pairs * h_stages * 8 * 8, 256);
    const int64_t most = std::min(h_stages, (kChunks + pairs - 1) / pairs);
    s.chunk = int((h_stages + most - 1) / most);
    s.chunks = int((h_stages + s.chunk - 1) / s.chunk);
    // (Never less than a set of the tokens' sums for every share, the size that small layers have.)
    const int64_t sets = std::min<int64_t>((hidden + 31) / 32, kPlaces) * top_k * s.chunks;
    s.bytes = s.parts + std::max<int64_t>(sets, kMaxParts4) * tokens * 32 * 4;
    return s;
}

template <typename... P, typename... A>
cudaError_t launch_moe(void (*fn)(P...), int64_t blocks, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    std::memset(&cfg, 0, sizeof(cfg));
    std::memset(attr, 0, sizeof(attr));
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(kMoeThreads, 1, 1);
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

template <typename X, int UNIT, bool ODD>
int launch_experts(MoeArgs a, const S4Weights &gu, const S4Weights &dn, int sms, cudaStream_t s) {
    constexpr int SG = 4 / UNIT;
    auto *fn = experts_kernel<X, UNIT, ODD>;
    a.scale_bytes = 2 * SG * 32 * (ODD ? 2 : 1) * (a.gate_up.zeros || a.down.zeros ? 2 : 1);
    // As many places as leave two CTAs on an SM, four where none do.
    const size_t sums = size_t(kMoeWarps) * 32 * kTile * 4;
    const size_t fixed = sums + sizeof(Routing) + sizeof(MoeTail) + kMoeWarps * 512 + 3 * 1024;  // (alignment, the system's 1 KB)
    const size_t place = size_t(kMoeWarps) * (kS4TileBytes + a.scale_bytes);
    a.places = kMaxRing;
    while (a.places > 0 && fixed + a.places * place > 114 * 1024) a.places -= 2;
    if (a.places == 0) a.places = 4;
    a.ring_bytes = kMoeWarps * a.places * kS4TileBytes;
    const size_t smem = a.places * place + sums + 1024;
    static std::atomic<int> ready[kMaxDevM];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_launch(e, "cudaGetDevice");
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 176 * 1024);
        // (An SM changes its split between shared memory and cache only when it is idle.)
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(router_kernel<X, UNIT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return fail_launch(e, "experts set-up");
        ready[dev].store(1, std::memory_order_release);
    }
    CUtensorMap up, down;
    int rc = encode_tmap_codes(&up, gu.codes, uint64_t(gu.cols + 1) / 2, uint64_t(gu.rows), uint64_t(gu.experts), uint64_t(gu.pitch),
                               uint64_t(gu.expert), 16);
    if (!rc)
        rc = encode_tmap_codes(&down, dn.codes, uint64_t(dn.cols + 1) / 2, uint64_t(dn.rows), uint64_t(dn.experts), uint64_t(dn.pitch),
                               uint64_t(dn.expert), 16);
    if (rc) return rc;
    const int64_t blocks = int64_t(a.tokens) * a.stages * 2 * SG, per_cta = kMoeWarps * (32 / (4 * UNIT));
    const int64_t makers = std::min<int64_t>((blocks + per_cta - 1) / per_cta, sms);  // CTAs that make the operands
    e = launch_moe(router_kernel<X, UNIT>, int64_t(a.tokens + kLogits - 1) / kLogits * a.experts + makers, 0, s, a);
    if (e == cudaSuccess) {
        const int per_sm = fixed + a.places * place <= 114 * 1024 ? 2 : 1;
        e = launch_moe(fn, std::min(sms * per_sm, kPlaces), smem, s, up, down, a);
    }
    return e == cudaSuccess ? PTC_OK : fail_launch(e, "experts launch");
}

template <typename X>
int run_moe(const MoeArgs &a, const S4Weights &gu, const S4Weights &dn, int sms, cudaStream_t s) {
    auto unit = [&](auto u) {
        constexpr int U = decltype(u)::value;
        return a.inner % 16 ? launch_experts<X, U, true>(a, gu, dn, sms, s) : launch_experts<X, U, false>(a, gu, dn, sms, s);
    };
    switch (s4_unit(gu.group)) {
        case 1: return unit(std::integral_constant<int, 1>());
        case 2: return unit(std::integral_constant<int, 2>());
        default: return unit(std::integral_constant<int, 4>());
    }
}

Experts experts_of(const S4Weights &w) {
    Experts e;
    e.scales = static_cast<const uint8_t *>(w.scales);
    e.zeros = static_cast<const uint8_t *>(w.zeros);
    e.groups = int(w.groups());
    e.tiles = int(w.tiles());
    return e;
}

}  // namespace

cudaError_t read_and_clear_moe_error_word(uint32_t *out) {
    uint32_t v = 0;
    const uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_moe_error, sizeof(v));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_moe_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace ptc

using namespace ptc;

extern "C" {

int64_t ptc_moe_a16_s4_workspace(int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int64_t top_k) {
    if (tokens <= 0 || hidden <= 0 || inner <= 0 || experts <= 0 || top_k <= 0 || tokens > kMaxTokens || hidden > kMaxSize ||
        inner > kMaxSize || experts > kMaxExperts || top_k > std::min<int64_t>(experts, kMaxTopK) || tokens * top_k > kMaxPairs)
        return 0;
    return moe_space(tokens, hidden, inner, experts, top_k).bytes;
}

int ptc_moe_a16_s4(int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int64_t top_k, int renormalize, int type,
                   const void *X, int64_t ldx, const void *router, int64_t ldr, int router_type, int64_t group, int scale_type,
                   const void *gate_up, int64_t ld_gate_up, int64_t expert_gate_up, const void *gate_up_scales,
                   const void *gate_up_zeros, const void *down, int64_t ld_down, int64_t expert_down, const void *down_scales,
                   const void *down_zeros, void *Y, int64_t ldy, int32_t *ids, float *weights, void *workspace,
                   int64_t workspace_bytes, void *stream) {
    set_message("");
    if (tokens < 0 || tokens > kMaxTokens || hidden < 1 || hidden > kMaxSize || inner < 1 || inner > kMaxSize || experts < 1 ||
        experts > kMaxExperts)
        return fail_status(PTC_ERR_INVALID, "sizes must satisfy 0 <= tokens <= 64, 1 <= hidden, inner <= 2^20, 1 <= experts <= 512");
    if (top_k < 1 || top_k > experts || top_k > kMaxTopK || tokens * top_k > kMaxPairs)
        return fail_status(PTC_ERR_INVALID, "top_k must be 1 .. min(experts, 32), and tokens * top_k at most 512");
    if (type != PTC_OUT_BF16 && type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "activations are PTC_OUT_BF16 or PTC_OUT_F16");
    if (router_type != type && router_type != PTC_OUT_F32)
        return fail_status(PTC_ERR_INVALID, "the router is of the activations' type or float32");
    if (scale_type != PTC_OUT_BF16 && scale_type != PTC_OUT_F16)
        return fail_status(PTC_ERR_INVALID, "scales are PTC_OUT_BF16 or PTC_OUT_F16");
    if (tokens == 0) return PTC_OK;
    if (!X || ldx < hidden || ldx > kMaxLdM || !Y || ldy < hidden || ldy > kMaxLdM || !router || ldr < hidden || ldr > kMaxLdM)
        return fail_status(PTC_ERR_INVALID, "X, Y or router is NULL, or its leading dimension is not hidden .. 2^36");
    // (One expert has no distance to the next; a tensor map wants one.)
    if (experts == 1) expert_gate_up = 2 * inner * ld_gate_up, expert_down = hidden * ld_down;
    const S4Weights gu{gate_up, ld_gate_up, expert_gate_up, gate_up_scales, gate_up_zeros, 2 * inner, hidden, group, experts};
    const S4Weights dn{down, ld_down, expert_down, down_scales, down_zeros, hidden, inner, group, experts};
    int rc = check_s4(gu);
    if (!rc) rc = check_s4(dn);
    if (rc) return rc;
    for (const S4Weights *w : {&gu, &dn})
        if (experts > 1 && (w->expert < (w->rows - 1) * w->pitch + (w->cols + 1) / 2 || w->expert > kMaxLdM))
            return fail_status(PTC_ERR_INVALID, "experts' matrices overlap, or lie over 2^36 bytes apart");
    const int64_t need = ptc_moe_a16_s4_workspace(tokens, hidden, inner, experts, top_k);
    if (!workspace || workspace_bytes < need) return fail_status(PTC_ERR_INVALID, "the workspace is too small");
    const int rs = router_type == PTC_OUT_F32 ? 4 : 2;
    if (!lies_on(X, 2) || !lies_on(Y, 2) || !lies_on(router, uintptr_t(rs)) || !lies_on(ids, 4) || !lies_on(weights, 4))
        return fail_status(PTC_ERR_ALIGN, "X, Y, router, ids and weights must be aligned to their elements");
    if (!lies_on(workspace, 256)) return fail_status(PTC_ERR_ALIGN, "the workspace must be 256-byte aligned");
    auto span = [&](const S4Weights &w) {
        return flat_bytes(w.codes, uint64_t(w.experts > 1 ? w.experts - 1 : 0) * uint64_t(w.expert) + uint64_t(w.rows - 1) * uint64_t(w.pitch) +
                                       uint64_t((w.cols + 1) / 2));
    };
    const ByteRows in[] = {elem_rows(X, tokens, hidden, ldx, 2), elem_rows(router, experts, hidden, ldr, rs), span(gu),
                           flat_bytes(gu.scales, gu.scale_bytes()), flat_bytes(gu.zeros, gu.scale_bytes()), span(dn),
                           flat_bytes(dn.scales, dn.scale_bytes()), flat_bytes(dn.zeros, dn.scale_bytes())};
    const ByteRows out[] = {elem_rows(Y, tokens, hidden, ldy, 2), flat_bytes(ids, uint64_t(tokens * top_k) * 4),
                            flat_bytes(weights, uint64_t(tokens * top_k) * 4), flat_bytes(workspace, uint64_t(need))};
    for (int i = 0; i < 4; ++i) {
        for (const ByteRows &b : in)
            if (rows_overlap(out[i], b)) return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
        for (int j = 0; j < i; ++j)
            if (rows_overlap(out[i], out[j])) return fail_status(PTC_ERR_OVERLAP, "an output overlaps another argument");
    }
    int sms;
    if ((rc = usable_device(&sms))) return rc;
    const MoeSpace at = moe_space(tokens, hidden, inner, experts, top_k);
    char *ws = static_cast<char *>(workspace);
    MoeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = X;
    a.ldx = ldx;
    a.router = router;
    a.ldr = ldr;
    a.router_f32 = router_type == PTC_OUT_F32;
    a.xvec = lies_on(X, 16) && (tokens == 1 || ldx % 8 == 0);
    a.rvec = lies_on(router, 16) && (experts == 1 || ldr * rs % 16 == 0);
    a.y = Y;
    a.ldy = ldy;
    a.ids = ids;
    a.weights = weights;
    a.tokens = int(tokens);
    a.hidden = int(hidden);
    a.inner = int(inner);
    a.experts = int(experts);
    a.top_k = int(top_k);
    a.renormalize = renormalize != 0;
    a.bf16_scales = scale_type == PTC_OUT_BF16;
    a.per_group = int(group >= 128 ? group / 128 : 1);
    a.gate_up = experts_of(gu);
    a.down = experts_of(dn);
    a.halves = int((hidden + kS4Half - 1) / kS4Half);
    a.stages = int((hidden + kS4Stage - 1) / kS4Stage);
    a.h_halves = int((inner + kS4Half - 1) / kS4Half);
    a.h_stages = int((inner + kS4Stage - 1) / kS4Stage);
    a.h_blocks = int((inner + 31) / 32);
    a.chunk = at.chunk;
    a.chunks = at.chunks;
    a.counters = reinterpret_cast<uint32_t *>(ws);
    a.logits = reinterpret_cast<float *>(ws + at.logits);
    a.xs = reinterpret_cast<uint8_t *>(ws + at.xs);
    a.xps = reinterpret_cast<float2 *>(ws + at.xps);
    a.hs = reinterpret_cast<uint8_t *>(ws + at.hs);
    a.hps = reinterpret_cast<float2 *>(ws + at.hps);
    a.parts = reinterpret_cast<float *>(ws + at.parts);
    a.stall = take_stall_tile();
    a.wait_limit = wait_limit_ns();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return type == PTC_OUT_BF16 ? run_moe<__nv_bfloat16>(a, gu, dn, sms, s) : run_moe<__half>(a, gu, dn, sms, s);
}

}  // extern "C"
