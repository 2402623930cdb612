// A whole routed MoE layer for a few tokens (T <= 16) in one kernel launch:
// router, selection, expert up projections, activation, expert down
// projections, weighted sum, shared expert and residual.
//
//   L = x . Wr^T;  s = sigmoid(L) or softmax(L);  picks = top-k of s + b;
//   w = s / (sum s + eps) * scale;  h_j = bf16(act(W1[e_j] x));
//   y = bf16(out_scale * sum_j w_j W2[e_j] h_j + W2s act(W1s x) + residual)
//
// At this size the layer is one pass over the picked experts' weights, so the
// kernel is built around that stream.  One CTA per SM, 16 consumer warps in 4
// groups of 4 and a producer warp per group.  A group has its own part of the
// work and its own slots of a shared-memory ring, which its producer fills by TMA
// (stream.cuh has the stage layout); its 4 warps share a tile's k and multiply
// with m16n8k16 MMAs -- the token count is at most the MMA's N, so tensor
// throughput does not matter; reading and converting weights does.  One producer
// for all groups measured 192 us where four take 82 (8 tokens, bf16, below).
//
//   up    The active experts' features (I per routed expert) form one list;
//         every group takes an equal contiguous part of it, in tiles of 8
//         features (SwiGLU: 8 gate and 8 up rows, which meet in one thread) or
//         16 (relu^2).  h goes to global memory, one row per routed pair.
//   down  Every CTA owns H / CTAs rows of y and runs them through all active
//         experts, so y needs no atomics and no second pass: partial sums
//         stay in shared memory and one fixed-order sum ends the row.  With few
//         rows and many experts, CTAs share blocks of 16 rows instead and the
//         last one of a block adds its parts up, in order.
//
// Two grid barriers (after the logits, after h) join the phases; the launch is
// cooperative, so all CTAs are resident and the waits end.  Neither stops the
// stream of weights for long: the producers fetch the shared expert's rows
// before the routing is known and the first down rows before h is.  (Consumers
// that do not wait at the second barrier, and logits polled by tags instead of
// the first, both measured slower: more fences and more polls on one line.)
//
// Router sums carry ~46 bits (fp32 pairs) and close scores are compared in 64: E * H * T
// is small here, and picks are then those of the real-number scores up to ties.
//
// Measured (calls in a row through DecodeLayer, weights rotated through more than
// L2; the device's own time is ~1.5 us less; floor = bytes at 6455 GB/s): 16 tokens,
// 32 experts, k = 4, 2048 x 1792, bf16: 91-101 us (floor 96 by the expected number of
// active experts; moe_forward's tcgen05 tiles take 83); 8 tokens 72-84 us (72;
// moe_forward 93); one token of relu^2 64 experts, k = 6, 2048 x 1024 with a shared
// expert 26 us (10.5); 4-bit 64 experts, k = 4, 2048 x 1536: one affine token 22.6 us
// (3.4), five NVFP4 tokens 45-48 us (15); one token of a tiny block 12.3 us.  Bound: HBM for bf16 from a few tokens on; the conversion of codes
// (integer instructions at half rate) and the per-tile work for 4 bits; for one
// token ~11 us of latency, a chain of a launch, two fenced grid barriers (~1.5 us
// each), three dependent memory round trips and the selection.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "stream.cuh"
#include "tmap_rows.h"

namespace moe {
namespace {

using namespace stream;

constexpr int kGroups = 4;                      // consumer groups, each on a tile of its own
constexpr int kGw = 4;                          // warps of a group: they share a tile's k
constexpr int kCw = kGroups * kGw;              // consumer warps
constexpr int kCThreads = kCw * 32;
constexpr int kThreads = kCThreads + kGroups * 32;   // + a producer warp per group
constexpr int kMaxE = 257;                      // 256 experts and the shared one
constexpr int kMaxK = 32;
constexpr int kMaxStages = 16;
constexpr int kMostCounted = 1 << 17;            // comparisons of a selection by counting
constexpr int kMaxYRows = 16 * 160;              // rows of y times the CTAs that share them
constexpr int kMaxParts = 4;                    // parts of a router row

struct WMat {                                   // one weight tensor of the experts
    CUtensorMap map;                            // (experts * rows) rows of codes
    CUtensorMap smap, bmap;                     // boxes of their scales and biases, when boxed
    bool flat;                                  // rows are not whole 128-byte chunks
    bool boxed;
    const unsigned char* w;
    const unsigned char* scale;
    const unsigned char* bias;
    const float* glob;
    int rows, K;                                // rows per expert, row length
};

// Division by a number the host knows: a runtime divide costs ~150 cycles of
// latency, and a one-token call has a dozen in a row.  m = floor(2^64 / n) + 1
// gives floor(v m / 2^64) = floor(v / n) for v, n < 2^32; m = 0 stands for n = 1.
struct Divisor {
    uint64_t m;
};
Divisor divisor(uint32_t n) { return Divisor{n == 1 ? 0 : ~0ull / n + 1}; }
MOE_DEV uint32_t div_by(uint32_t v, Divisor d) { return d.m ? (uint32_t)__umul64hi(v, d.m) : v; }

struct DecodeArgs {
    const uint16_t* x;
    const float* logits;
    const float* w_router;
    const float* ebias;
    const uint16_t* residual;
    WMat W1, W2, S1, S2;
    int T, H, E, k, I, Is;
    float eps, scale, out_scale, limit, limit_s;
    int softmax, no_norm;
    int32_t* idx;
    float* w;
    uint16_t* y;
    unsigned long long* sync;                   // barrier arrivals: a multiple of the grid size between calls
    float2* lg;                                 // (parts, T, E): logits (hi, lo), each part over H / parts of the row
    int parts;                                  // 1, 2 or 4
    int up_stages, i_stages, is_stages;         // stages of a row: H; I and Is in the down products
    Divisor by_grid, by_groups, by_I, by_E, by_i_stages;
    uint16_t* h;                                // (T k, I)
    uint16_t* hs;                               // (T, Is)
    int stages;                                 // ring slots per group
    StageDims sd, sd2;                          // stages of the up and the down products
    int stage_bytes;
    int ys_off;                                 // shared memory of the shared expert's y sums
    int ring_off;
    // > 1 (few rows of y, much work for each): ysplit CTAs share a block of 16 rows,
    // each runs a part of its work, and the last one to finish adds the parts up
    int ysplit;
    Divisor by_ysplit, by_yworkers;
    float2* ypart;                              // (ysplit, T, H): sums of the routed and the shared experts
    int* ydone;                                 // per block: CTAs that wrote theirs; zero between calls
    uint32_t wait_limit;                        // polls of a ring wait
    uint32_t grid_limit, missing;               // polls of a grid barrier; arrivals it waits for in vain (0 but in the expiry check)
    int* err;
};

template <int NT>
struct Layout {                                 // shared memory (byte offsets)
    static constexpr int kTok = 8 * NT;
    static constexpr int kMask = 0;                                   // kMaxE words: tokens of an expert
    static constexpr int kList = kMask + (kMaxE + kTok * (kMaxK + 1) + 3) / 4 * 16;   // (behind the masks: keys by rank) active expert ids
    static constexpr int kPick = kList + 1040;                        // [kTok][kMaxK] expert of a pick
    static constexpr int kSlot = kPick + kTok * kMaxK * 4;             // [kTok][256] bytes: pick number of an expert
    static constexpr int kMisc = kSlot + kTok * 256;                  // active count, abort flag; maxima and scales of the token rows
    static constexpr int kBar = kMisc + 16 + 2 * kCw * 4;
    static constexpr int kRed = kBar + 2 * kMaxStages * 8;            // group sums; later y sums per warp
    static constexpr int kRedBuf = kGw * kRows * kTok * 4;            // one buffer of one group
    static constexpr int kBufs = NT == 1 ? 2 : 1;                     // buffers of a group
    static constexpr int kRedBytes = kGroups * kBufs * kRedBuf;       // 16 KB
    static constexpr int kYw = kCw * kRows * kTok * 4;                // one set of y sums per warp
    static constexpr int kX = (kRed + kRedBytes + 127) & ~127;
    static_assert(kTok * 256 * 4 <= kRedBytes, "the score keys fit them too");
    static_assert((NT == 1 ? 2 : 1) * kYw <= kRedBytes, "y sums (16 columns: the routed experts' only) fit the group-sum buffers");
};

MOE_DEV uint64_t key64(double c) {              // order of c; NaN lowest (1), -0 == +0
    if (c != c) return 1ull;
    if (c == 0.0) c = 0.0;
    const uint64_t u = (uint64_t)__double_as_longlong(c);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

MOE_DEV uint32_t key32(float c) {               // the same order for fp32
    if (c != c) return 1u;
    if (c == 0.0f) c = 0.0f;
    const uint32_t u = __float_as_uint(c);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
MOE_DEV float unkey32(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

MOE_DEV double sigmoid64(double L) { return 1.0 / (1.0 + exp(-L)); }

// Unevaluated fp32 sums hi + lo (about 46 bits), for the router's dot products:
// double-precision arithmetic runs at a small fraction of the fp32 rate.  (The _rn
// functions are never contracted: a product fused into the next sum would no longer be
// the one whose error is kept.)
struct F2 {
    float hi, lo;
};
MOE_DEV void add_to(F2& a, float v) {           // a += v, error-free in hi
    const float s = __fadd_rn(a.hi, v), t = __fsub_rn(s, a.hi);
    a.lo += __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(v, t));
    a.hi = s;
}
MOE_DEV void add_to(F2& a, F2 b) {
    add_to(a, b.hi);
    a.lo += b.lo;
}
MOE_DEV void fma_to(F2& a, float x, float y) {  // a += x y, the product's rounding error kept
    const float p = __fmul_rn(x, y);
    const float e = fmaf(x, y, -p);
    add_to(a, p);
    a.lo += e;
}
// An infinite or NaN sum is hi alone (its error terms are NaN).
MOE_DEV double f2_value(F2 a) { return fabsf(a.hi) <= 3.402823466e38f ? (double)a.hi + (double)a.lo : (double)a.hi; }

// The logit of (token t, expert e): given, or the parts' sum in order.
MOE_DEV F2 logit_f2(const DecodeArgs& a, int t, int e) {
    if (a.logits) return F2{__ldg(a.logits + (size_t)t * a.E + e), 0.0f};
    float2 v[kMaxParts];
#pragma unroll
    for (int p = 0; p < kMaxParts; ++p)
        if (p < a.parts) v[p] = __ldcg(a.lg + ((size_t)p * a.T + t) * a.E + e);
    F2 sum{v[0].x, v[0].y};
#pragma unroll
    for (int p = 1; p < kMaxParts; ++p)
        if (p < a.parts) add_to(sum, F2{v[p].x, v[p].y});
    return sum;
}
MOE_DEV double logit_of(const DecodeArgs& a, int t, int e) { return f2_value(logit_f2(a, t, e)); }

// Softmax statistics of a token's logits, by one warp: max and sum of exp
// (NaN when a logit is NaN, which makes every score of the row NaN).
MOE_DEV void softmax_stats64(const DecodeArgs& a, int t, double& m, double& z) {
    const int lane = threadIdx.x & 31;
    double v[8];
    m = -INFINITY;
    z = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lane + 32 * i < a.E ? logit_of(a, t, lane + 32 * i) : -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmax(m, v[i]);
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 1
    for (int i = 0; i < (a.E + 31) / 32; ++i) {
        double w = v[0];
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j == i) w = v[j];
        if (lane + 32 * i < a.E) z += exp(w - m);
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}
MOE_DEV double score64(const DecodeArgs& a, double L, double m, double z) {
    return a.softmax ? (z == z ? exp(L - m) / z : z) : sigmoid64(L);
}

// Turns a token's logits into score keys (softmax), by one warp; returns the largest logit.
MOE_DEV float softmax_keys(const DecodeArgs& a, uint32_t* s_key) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, z = 0.0f;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, __uint_as_float(s_key[e]));
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int e = lane; e < a.E; e += 32) z += expf(__uint_as_float(s_key[e]) - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    for (int e = lane; e < a.E; e += 32) {
        const float s = z == z ? expf(__uint_as_float(s_key[e]) - m) / z : z;
        s_key[e] = key32(s + (a.ebias ? __ldg(a.ebias + e) : 0.0f));
    }
    return m;
}

// Picks of one token by one warp, from fp32 score keys: already ranked (counted)
// or by k + 1 rounds of a warp-wide maximum.  The fp32 scores are within 2e-6
// (1 + |c|) of the 64-bit ones, so where the first k + 1 of them are further
// apart than twice that, their order is the 64-bit order; else the token is
// ranked again from 64-bit scores.  `slack` is added to that distance: a softmax
// score also moves by up to 2 p (1 - p) |m| 2^-24 <= |m| 2^-25 through the rounding of
// computed logits to fp32 (m: the largest; far smaller logits have p = 0).
// (A round is ~500 cycles of latency, the count of a whole rank ~300 for 64
// experts but E^2 T work: it is used up to kMostCounted comparisons.)
MOE_DEV void select_token(const DecodeArgs& a, int t, bool counted, float slack, uint32_t* s_key,
                          const uint32_t* s_sorted, int* pick, unsigned char* slot, uint32_t* mask) {
    const int lane = threadIdx.x & 31;
    int my_e = 0;
    bool close = false;
    const int rounds = min(a.k + 1, a.E);
    if (counted) {
        if (lane < a.k) my_e = pick[lane];
        for (int j = lane; j + 1 < rounds; j += 32) {
            const uint32_t hi = s_sorted[j], lo = s_sorted[j + 1];
            const float c = unkey32(hi);
            close |= hi > 1u && lo > 1u && !(c - unkey32(lo) > 4e-6f * (1.0f + fabsf(c)) + slack);   // both numbers
        }
        close = __any_sync(0xffffffffu, close);
    } else {
        uint32_t last = 0;
        for (int j = 0; j < rounds; ++j) {
            uint32_t best = 0;
            int be = 0xffff;
            for (int e = lane; e < a.E; e += 32) {
                const uint32_t c = s_key[e];
                if (c > best) { best = c; be = e; }
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)be : 0xffffu);
            if (lane == (e & 31)) s_key[e] = 0u;    // picked: below every NaN
            if (lane == j) my_e = e;
            if (j > 0 && last > 1u && top > 1u) {
                const float c = unkey32(last);
                close |= !(c - unkey32(top) > 4e-6f * (1.0f + fabsf(c)) + slack);
            }
            last = top;
        }
    }
    if (close) {                                // warp-uniform
        double m = 0.0, z = 1.0;
        if (a.softmax) softmax_stats64(a, t, m, z);
        uint64_t key[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane + 32 * i;
            key[i] = e < a.E ? key64(score64(a, logit_of(a, t, e), m, z) + (a.ebias ? (double)__ldg(a.ebias + e) : 0.0))
                             : 0ull;
        }
        for (int j = 0; j < a.k; ++j) {
            uint64_t best = key[0];
            int bi = 0;
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (key[i] > best) { best = key[i]; bi = i; }
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
            const bool ch = (uint32_t)(best >> 32) == hi;
            const uint32_t lo = __reduce_max_sync(0xffffffffu, ch ? (uint32_t)best : 0u);
            const bool win = ch && (uint32_t)best == lo;
            const int e = (int)__reduce_min_sync(0xffffffffu, win ? (uint32_t)(lane + 32 * bi) : 0xffffu);
            if (lane == (e & 31)) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i == (e >> 5)) key[i] = 0ull;
            }
            if (lane == j) my_e = e;
        }
    }
    if (lane < a.k) {
        pick[lane] = my_e;
        slot[my_e] = (unsigned char)lane;
        atomicOr(mask + my_e, 1u << t);
    }
}

// Routing weights of one token's picks by one warp, 64-bit, rounded once.
MOE_DEV void weigh_token(const DecodeArgs& a, int t, const int* pick) {
    const int lane = threadIdx.x & 31;
    double m = 0.0, z = 1.0, s = 0.0, sum = 0.0;
    if (a.softmax) softmax_stats64(a, t, m, z);
    const int e = lane < a.k ? pick[lane] : 0;
    if (lane < a.k) s = score64(a, logit_of(a, t, e), m, z);
    for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, s, j);   // rank order
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = e;
        __stcg(a.w + (size_t)t * a.k + lane, (float)(a.no_norm ? s * a.scale : s / (sum + (double)a.eps) * a.scale));
    }
}

// The c-th set bit of m (c < popc(m)).
MOE_DEV int nth_bit(uint32_t m, int c) {
    for (int i = 0; i < c; ++i) m &= m - 1;
    return __ffs(m) - 1;
}

// A unit of work: rows of one expert against all its tokens.
struct Unit {
    int e;                                      // expert; a.E: the shared one
    int n;                                      // features (up) or rows (down): rows of both halves, or of each when dual
    int f0;                                     // first feature (up) or row of y (down)
    int row0, row1;                             // first weight row of either half of 8 rows
};

// Start of part i of d.n equal parts of v (v * i below 2^32: at most 256 experts
// of 16384 features times the groups of the grid, 592 on this part).
MOE_DEV int part(int v, int i, Divisor d) { return (int)div_by((uint32_t)v * (uint32_t)i, d); }

// Requests stage c of a unit's rows (and their scales).
template <int FMT>
MOE_DEV void issue_weights(const StageDims& sd, const WMat& m, const Unit& u, bool dual, int c, uint32_t dst,
                           uint64_t* bar, uint64_t pol) {
    using F = Fmt<FMT>;
    const int lane = threadIdx.x & 31;
    const bool two = dual || u.n > 8;           // else the second half's rows are nobody's
    uint32_t sb = 0, sdst = 0;
    size_t s0 = 0;
    if (FMT != kBf16 && !m.boxed) {
        // scale rows start anywhere: copy the 16-byte aligned span around them
        // (the arrays hold a multiple of 128 bytes, so it stays inside)
        const size_t SB = F::scale_bytes(m.K);
        size_t b = 0, e = 0;
        if (m.K <= kSpanMaxK) {                 // whole rows: one span per half
            const int n = dual ? u.n : lane == 0 ? min(u.n, 8) : u.n - 8;
            if (lane < 2 && n > 0) {
                b = (size_t)(lane ? u.row1 : u.row0) * SB;
                e = b + n * SB;
                sdst = lane * (sd.area / 2);
            }
        } else if (lane < kRows) {
            const int loc = lane & 7, n = dual || lane < 8 ? min(u.n, 8) : u.n - 8;
            if (loc < n) {
                const int k0 = c * sd.k;
                b = (size_t)((lane >= 8 ? u.row1 : u.row0) + loc) * SB + F::scale_bytes(k0);
                e = b + F::scale_bytes(min(sd.k, m.K - k0));
                sdst = lane * (sd.area / kRows);
            }
        }
        if (e > b) {
            s0 = b & ~size_t(15);
            sb = (uint32_t)(((e + 15) & ~size_t(15)) - s0);
        }
    }
    uint32_t total = (two ? 2u : 1u) * sd.half;
    if (FMT != kBf16)
        total += (FMT == kAffine ? 2u : 1u) *
                 (m.boxed ? (two ? 2u : 1u) * 8 * F::kScaleBox : __reduce_add_sync(0xffffffffu, sb));
    if (lane == 0) mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (lane < (two ? 2 : 1)) {
        const int row = lane ? u.row1 : u.row0;
        if (FMT != kBf16 && m.boxed) {
            const int x = c * (int)F::scale_bytes(sd.k);
            const uint32_t to = dst + sd.scales + lane * (sd.area / 2);
            tma_load_rows(to, &m.smap, x, row, bar, pol);
            if (FMT == kAffine) tma_load_rows(to + sd.area, &m.bmap, x, row, bar, pol);
        }
        if (!m.flat) {
            tma_load_3d(dst + lane * sd.half, &m.map, row, c * sd.chunks, bar, pol);
        } else {
            for (int i = 0; i < sd.chunks; ++i)
                tma_load_rows(dst + lane * sd.half + i * 1024, &m.map, (c * sd.chunks + i) * 128, row, bar, pol);
        }
    }
    if (FMT != kBf16 && sb) {
        bulk_load(dst + sd.scales + sdst, m.scale + s0, sb, bar, pol);
        if (FMT == kAffine) bulk_load(dst + sd.scales + sd.area + sdst, m.bias + s0, sb, bar, pol);
    }
}

// Where the scales of row `loc` of a half (first row: `base`) start at stage c,
// from the stage's scale area on (before the swizzle's term).
template <int FMT>
MOE_DEV uint32_t scale_off(int area, int stage_k, int K, bool boxed, uint32_t base, int half, int loc, int c) {
    using F = Fmt<FMT>;
    if (boxed) return half * (area / 2) + loc * F::kScaleBox;
    // only the low 4 bits of the global byte count: 32-bit products do
    const uint32_t SB = (uint32_t)F::scale_bytes(K), o = (uint32_t)F::scale_bytes(c * stage_k);
    if (K <= kSpanMaxK) return half * (area / 2) + ((base * SB) & 15) + loc * SB + o;
    return (half * 8 + loc) * (area / kRows) + (((base + loc) * SB + o) & 15);
}

template <int FMT, int NT, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1) k_decode(const __grid_constant__ DecodeArgs a) {
    using F = Fmt<FMT>;
    using L = Layout<NT>;
    constexpr int TT = L::kTok;
    constexpr int kFeat = DUAL ? 8 : kRows;     // features of an up tile
    extern __shared__ __align__(128) unsigned char sm[];
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(sm + L::kMask);
    int* s_list = reinterpret_cast<int*>(sm + L::kList);
    int* s_pick = reinterpret_cast<int*>(sm + L::kPick);
    unsigned char* s_slot = sm + L::kSlot;
    int* s_nact = reinterpret_cast<int*>(sm + L::kMisc);
    uint32_t* s_wmax = reinterpret_cast<uint32_t*>(sm + L::kMisc + 16);              // [kCw]
    float* s_xinv = reinterpret_cast<float*>(sm + L::kMisc + 16 + kCw * 4);           // [kCw]: 1 / the tokens' scales
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t* empty = full + kMaxStages;
    float* s_red = reinterpret_cast<float*>(sm + L::kRed);
    const int xstride = a.H * 2 + F::kXPad;
    const uint32_t xs = smem_u32(sm + L::kX);
    // affine: per group of 64 k and token (constant part of the products, sum of x)
    float2* s_tab = reinterpret_cast<float2*>(sm + L::kX + a.T * xstride);
    const uint32_t tab0 = xs + a.T * xstride;
    const uint32_t ring = (smem_u32(sm) + a.ring_off + 1023) & ~1023u;   // swizzled boxes start on 1 KB

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = gridDim.x, cta = blockIdx.x;
    const int Sg = a.stages;                    // ring slots of one group (its own: it alone fills and frees them in order)
    for (int i = tid; i < kMaxE; i += kThreads) s_mask[i] = 0;
    if (tid < kGroups * Sg) {
        mbar_init(&full[tid], 2);               // weights, token rows
        mbar_init(&empty[tid], kGw);
        fence_mbar_init();
    }
    if (tid == 0) *s_abort = 0;
    if (warp == kCw && lane < (a.Is > 0 ? 4 : 2))
        tma_prefetch_desc(lane == 0 ? &a.W1.map : lane == 1 ? &a.W2.map : lane == 2 ? &a.S1.map : &a.S2.map);
    __syncthreads();

    const int grp = warp < kCw ? warp / kGw : warp - kCw;
    const int ring0 = grp * Sg;                 // first ring slot of this warp's group

    // Work of this group: equal parts, over all groups of the grid, of the
    // shared expert's features and of the routed experts' list (once it is known).
    const int wk = cta * kGroups + grp;
    // This CTA's rows of y, in tiles of at most 16; each tile's list of
    // (expert, chunk of k) is dealt out to the groups in equal parts.
    int yr0 = part(a.H, cta, a.by_grid), yr1 = part(a.H, cta + 1, a.by_grid), ypart = 0;
    if (a.ysplit > 1) {
        const int block = (int)div_by(cta, a.by_ysplit);
        ypart = cta - block * a.ysplit;
        yr0 = min(a.H, block * kRows);
        yr1 = min(a.H, yr0 + kRows);
    }
    const int ytiles = max(1, (yr1 - yr0 + kRows - 1) / kRows);
    // phases: 0 the shared expert's features, 1 the routed experts', 2.. tiles of y
    auto rows_of_tile = [&](int tile, int& r0, int& n) {
        const int rows = yr1 - yr0;
        r0 = ytiles == 1 ? 0 : rows * tile / ytiles;
        n = (ytiles == 1 ? rows : rows * (tile + 1) / ytiles) - r0;
        r0 += yr0;
    };
    // Calls f(unit, of a routed expert, first stage, end stage) for the group's units
    // of a phase, in order; f returns false to stop.  A down unit is a run of chunks
    // of one expert: a tile's (expert, chunk) list is dealt out to the groups.
    auto walk = [&](int phase, int nact, auto&& f) {
        int p, end, li = 0, off = 0, r0 = 0, nr = 0;
        if (phase == 0) {
            p = off = part(a.Is, wk, a.by_groups);
            end = part(a.Is, wk + 1, a.by_groups);
        } else if (phase == 1) {
            p = part(nact * a.I, wk, a.by_groups);
            end = part(nact * a.I, wk + 1, a.by_groups);
            li = (int)div_by(p, a.by_I);
            off = p - li * a.I;
        } else {
            rows_of_tile(phase - 2, r0, nr);
            if (nr == 0) return;                // fewer rows than CTAs
            const int total = nact * a.i_stages + a.is_stages;
            p = part(total, ypart * kGroups + grp, a.by_yworkers);
            end = part(total, ypart * kGroups + grp + 1, a.by_yworkers);
            li = min((int)div_by(p, a.by_i_stages), nact);
            off = p - li * a.i_stages;
        }
        while (p < end) {
            const bool routed = phase != 0 && li < nact;
            Unit u;
            u.e = routed ? s_list[li] : a.E;
            int c0 = 0, c1, took;
            const int width = phase < 2 ? (routed ? a.I : a.Is) : (routed ? a.i_stages : a.is_stages);
            if (phase < 2) {
                took = u.n = min(min(kFeat, width - off), end - p);
                u.f0 = off;
                u.row0 = (routed ? u.e * a.W1.rows : 0) + off;
                u.row1 = u.row0 + (DUAL ? width : 8);
                c1 = a.up_stages;
            } else {
                took = min(width - off, end - p);
                u.n = nr;
                u.f0 = r0;
                u.row0 = (routed ? u.e * a.H : 0) + r0;
                u.row1 = u.row0 + 8;
                c0 = off;
                c1 = off + took;
            }
            if (!f(u, routed, c0, c1)) return;
            p += took;
            off += took;
            if (off == width) {
                off = 0;
                ++li;
            }
        }
    };
    // Row of the activations of column c of expert e (its tokens: mask).
    auto h_row = [&](int e, uint32_t mask, int c) -> const uint16_t* {
        const int t = nth_bit(mask, c);
        return e < a.E ? a.h + ((size_t)t * a.k + s_slot[t * 256 + e]) * a.I : a.hs + (size_t)t * a.Is;
    };

    if (warp >= kCw) {
        // -------------------------------------------------------- producer of one group
        const uint64_t pol = policy_evict_first(), pol_h = policy_evict_last();
        int slot = 0, fills = 0;                // next ring slot; stages issued
        uint32_t ph = 1;                        // parity of the slot's last release (fresh: passes)
        bool ok = true;
        // a stage's full barrier takes two arrivals: the weights', the token rows'
        auto weights = [&](const StageDims& sd, const WMat& m, const Unit& u, bool dual, int c) {
            const int s = ring0 + slot;
            const bool got = mbar_wait(&empty[s], ph, s_abort, a.wait_limit);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                return;
            }
            issue_weights<FMT>(sd, m, u, dual, c, ring + s * a.stage_bytes, &full[s], pol);
            ++fills;
            if (++slot == Sg) {
                slot = 0;
                ph ^= 1;
            }
        };
        int hslot = 0, hfills = 0;              // the same for the second arrival
        auto no_tokens = [&]() {                // up: the columns are read from xs
            if (lane == 0) mbar_arrive(&full[ring0 + hslot]);
            ++hfills;
            hslot = hslot + 1 == Sg ? 0 : hslot + 1;
        };
        auto tokens = [&](const Unit& u, int K, int c) {   // down: chunk c of the activations of u's tokens
            const uint32_t mask = s_mask[u.e];
            const int n = __popc(mask), s = ring0 + hslot;
            const int k0 = c * a.sd2.k, kc = min(a.sd2.k, K - k0);
            if (lane == 0) mbar_arrive_expect_tx(&full[s], n * kc * 2);
            __syncwarp();
            if (lane < n)
                bulk_load(ring + s * a.stage_bytes + a.sd2.tokens + lane * (a.sd2.k * 2 + F::kXPad),
                          h_row(u.e, mask, lane) + k0, kc * 2, &full[s], pol_h);
            ++hfills;
            hslot = hslot + 1 == Sg ? 0 : hslot + 1;
        };
        // the shared expert's first rows need no routing: fill the free slots with them
        int pre = 0;
        if (a.Is > 0) walk(0, 0, [&](const Unit& u, bool, int c0, int c1) {
            for (int c = c0; c < c1 && pre < Sg; ++c, ++pre) {
                weights(a.sd, a.S1, u, DUAL, c);
                no_tokens();
            }
            return pre < Sg;
        });
        __syncthreads();                        // routing tables ready
        const int nact = *s_nact;
        if (a.Is > 0) {
            int q = 0;
            walk(0, nact, [&](const Unit& u, bool, int c0, int c1) {
                for (int c = c0; c < c1 && ok; ++c)
                    if (q++ >= pre) {
                        weights(a.sd, a.S1, u, DUAL, c);
                        if (ok) no_tokens();
                    }
                return ok;
            });
        }
        walk(1, nact, [&](const Unit& u, bool, int c0, int c1) {
            for (int c = c0; c < c1 && ok; ++c) {
                weights(a.sd, a.W1, u, DUAL, c);
                if (ok) no_tokens();
            }
            return ok;
        });
        // Down: the first Sg stages' weights are requested before h is there.
        int ahead = 0;
        walk(2, nact, [&](const Unit& u, bool routed, int c0, int c1) {
            for (int c = c0; c < c1 && ahead < Sg && ok; ++c, ++ahead) weights(a.sd2, routed ? a.W2 : a.S2, u, false, c);
            return ahead < Sg && ok;
        });
        // CTA t weighs token t's picks for the grid: 64-bit arithmetic in every CTA
        // took longer than small layers' products, and the down products, which
        // need the weights first, are behind the grid barrier anyway
        if (grp == 0) {
            if (cta < a.T) weigh_token(a, cta, s_pick + cta * kMaxK);
            asm volatile("bar.arrive 7, %0;" ::"r"(kCThreads + 32) : "memory");
        }
        named_bar(6, kThreads);                 // every h is written
        fence_proxy_async_all();
        if (*s_abort) ok = false;
        for (int tile = 0; tile < ytiles; ++tile) {
            int q = tile ? ahead : 0;
            walk(2 + tile, nact, [&](const Unit& u, bool routed, int c0, int c1) {
                for (int c = c0; c < c1 && ok; ++c) {
                    if (q++ >= ahead) weights(a.sd2, routed ? a.W2 : a.S2, u, false, c);
                    if (ok) tokens(u, routed ? a.I : a.Is, c);
                }
                return ok;
            });
        }
        if (!ok) {
            if (lane == 0) report_error(a.err, kErrWaitExpired);
            *s_abort = 1;
            // stages whose token rows were never sent: let their barriers complete
            for (; hfills < fills; ++hfills, hslot = hslot + 1 == Sg ? 0 : hslot + 1)
                if (lane == 0) mbar_arrive(&full[ring0 + hslot]);
        }
        // every copy issued lands before the CTA can exit
        for (int i = max(0, fills - Sg); i < fills; ++i)
            mbar_wait(&full[ring0 + i % Sg], (uint32_t)((i / Sg) & 1), nullptr, a.wait_limit);
    } else {
        // -------------------------------------------------------- consumers
        const int gw = warp % kGw, gt = tid % (kGw * 32);
        const int g = lane >> 2, t4 = lane & 3;
        const int sg = F::sigma(g);             // the row of a half that MMA row g is
        const uint32_t x4 = FMT == kBf16 ? (t4 ^ sg) << 4 : (((t4 >> 1) ^ sg) << 4) | ((t4 & 1) << 3);
        bool dead = false;
        // Grid barrier: arrivals only ever add up, gridDim.x per barrier, so what
        // is there when a CTA looks, rounded down to a multiple of that, is where
        // the count stood before its next own arrival.  A CTA whose wait runs out goes
        // on to the end and arrives at every barrier: the counts are whole after it.
        unsigned long long seen = 0, target = 0;
        if (tid == 0) asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(a.sync) : "memory");
        // thread 0: the release covers what it and, through the CTA's barrier just
        // before, the other consumers wrote
        auto arrive = [&]() {
            asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(a.sync), "l"(1ull) : "memory");
            target = (target ? target : __umul64hi(seen, a.by_grid.m) * (uint32_t)G) + (uint32_t)G;
        };
        auto grid_wait = [&]() {                // thread 0
            bool ok = false;
            for (uint32_t i = 0; i < a.grid_limit && !ok; ++i) {
                unsigned long long v;
                asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(a.sync) : "memory");
                ok = v >= target + a.missing;
            }
            if (!ok) {
                report_error(a.err, kErrWaitExpired);
                *s_abort = 1;
            }
        };
        const int lw = a.T > 8 ? 0 : a.T > 4 ? 1 : a.T > 2 ? 2 : a.T > 1 ? 3 : 4;   // log2 of the warps per token
        const int t = warp >> lw, ws = warp & ((1 << lw) - 1);   // this warp's token, and its share
        // ---- router: work item (expert, part of H); a warp takes one token's
        // row, or a share of it when there are fewer tokens than warps
        if (!a.logits) {
            F2* s_d = reinterpret_cast<F2*>(s_red);              // [kCw]
            const int nq = a.parts == 4 ? a.H >> 4 : a.parts == 2 ? a.H >> 3 : a.H >> 2;                    // groups of 4 k in a part (H is a multiple of 64)
            for (int it = cta; it < a.E * a.parts; it += G) {
                const int e = a.parts == 4 ? it >> 2 : a.parts == 2 ? it >> 1 : it, p = it - e * a.parts;
                F2 acc{0.0f, 0.0f}, acc2{0.0f, 0.0f};
                if (t < a.T)
#pragma unroll 4
                    for (int q = ws * 32 + lane; q < nq; q += 32 << lw) {
                        const float4 w = __ldg(reinterpret_cast<const float4*>(a.w_router + (size_t)e * a.H) + p * nq + q);
                        const uint2 v = *(reinterpret_cast<const uint2*>(a.x + (size_t)t * a.H) + p * nq + q);
                        fma_to(acc, w.x, bf16lo(v.x));
                        fma_to(acc2, w.y, bf16hi(v.x));
                        fma_to(acc, w.z, bf16lo(v.y));
                        fma_to(acc2, w.w, bf16hi(v.y));
                    }
                add_to(acc, acc2);
                for (int o = 16; o > 0; o >>= 1)
                    add_to(acc, F2{__shfl_xor_sync(0xffffffffu, acc.hi, o), __shfl_xor_sync(0xffffffffu, acc.lo, o)});
                if (lane == 0) s_d[warp] = acc;
                named_bar(5, kCThreads);
                if (warp == 0) {                                 // the warps of a token, by shuffles among 16 lanes
                    acc = s_d[lane & 15];
                    for (int o = (1 << lw) >> 1; o > 0; o >>= 1)
                        add_to(acc, F2{__shfl_xor_sync(0xffffffffu, acc.hi, o), __shfl_xor_sync(0xffffffffu, acc.lo, o)});
                    const int tt = lane >> lw;
                    if (lane < 16 && tt << lw == lane && tt < a.T)
                        __stcg(a.lg + ((size_t)p * a.T + tt) * a.E + e, make_float2(acc.hi, acc.lo));
                }
                if (it + G < a.E * a.parts) named_bar(5, kCThreads);
            }
            __syncwarp();
            if (tid == 0) arrive();
        }
        // ---- token rows into shared memory (while the other CTAs' logits arrive);
        // 4-bit experts: in f16, scaled by a power of two that brings the row's
        // largest finite value to [2^14, 2^15) (values below 2^-31 of that, in affine's
        // odd pairs 2^-27, lose bits to f16's subnormals; infinities and NaN stay)
        float xscale = 1.0f;
        if (FMT != kBf16) {
            float m = 0.0f;
            if (t < a.T)
#pragma unroll 4
                for (int c = ws * 32 + lane; c < a.H / 8; c += 32 << lw) {
                    const uint4 v = *(reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H) + c);
                    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = fabsf(bf16lo(r[i])), q = fabsf(bf16hi(r[i]));
                        if (p < INFINITY) m = fmaxf(m, p);       // false for NaN
                        if (q < INFINITY) m = fmaxf(m, q);
                    }
                }
            const uint32_t mw = __reduce_max_sync(0xffffffffu, __float_as_uint(m));   // not negative: bits order as values
            if (lane == 0) s_wmax[warp] = mw;
            named_bar(5, kCThreads);
            uint32_t mt = 0;
            for (int i = 0; i < 1 << lw; ++i) mt = max(mt, s_wmax[(t << lw) + i]);
            const int field = mt ? min(253, 268 - (int)(mt >> 23)) : 127;
            xscale = __uint_as_float((uint32_t)field << 23);
            if (ws == 0 && lane == 0) s_xinv[t] = __uint_as_float((uint32_t)(254 - field) << 23);
        }
        if (t < a.T) {
            const int nc = a.H / 8;
#pragma unroll 2
            for (int c0 = ws * 32; c0 < nc; c0 += 32 << lw) {    // warp-uniform: lanes meet in shuffles below
                const int c = c0 + lane;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (c < nc) v = *(reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H) + c);
                if (FMT != kBf16) {
                    float f[8] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y),
                                  bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w)};
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= xscale;
                    if (FMT == kNvfp4) {
                        v = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                                       pack_f16x2(f[6], f[7]));
                    } else {
                        // pairs (j, j + 4); the odd pairs meet codes that count 16-fold
                        v = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f),
                                       pack_f16x2(f[2], f[6]), pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f));
                        const float e0 = (f[0] + f[4]) + (f[2] + f[6]), e1 = (f[1] + f[5]) + (f[3] + f[7]);
                        float big = fmaf(1024.0f, e0, 64.0f * e1), sum = e0 + e1;
#pragma unroll
                        for (int o = 4; o > 0; o >>= 1) {        // 8 lanes hold the 64 k of a group
                            big += __shfl_xor_sync(0xffffffffu, big, o);
                            sum += __shfl_xor_sync(0xffffffffu, sum, o);
                        }
                        if ((lane & 7) == 0 && c < nc) s_tab[(c >> 3) * a.T + t] = make_float2(big, sum);
                    }
                }
                if (c < nc) *reinterpret_cast<uint4*>(sm + L::kX + (size_t)t * xstride + c * 16) = v;
            }
        }
        if (!a.logits && tid == 0) grid_wait();
        named_bar(5, kCThreads);
        // ---- selection: every CTA picks for all tokens, a warp per token
        uint32_t* s_key = reinterpret_cast<uint32_t*>(s_red);          // [T][Ep], zeros behind the experts
        const int Ep = (a.E + 3) & ~3;
        for (int i = tid; i < a.T * a.E; i += kCThreads) {
            const int tt = (int)div_by(i, a.by_E), e = i - tt * a.E;
            const F2 l2 = logit_f2(a, tt, e);
            const float L = fabsf(l2.hi) <= 3.402823466e38f ? l2.hi + l2.lo : l2.hi;
            s_key[tt * Ep + e] = a.softmax ? __float_as_uint(L)
                                           : key32(1.0f / (1.0f + expf(-L)) + (a.ebias ? __ldg(a.ebias + e) : 0.0f));
            if (e == a.E - 1)
                for (int q = a.E; q < Ep; ++q) s_key[tt * Ep + q] = 0u;
        }
        named_bar(5, kCThreads);
        float slack = 0.0f;
        if (a.softmax) {
            if (warp < a.T) {
                const float m = softmax_keys(a, s_key + warp * Ep);
                if (!a.logits) slack = fabsf(m) * 0x1p-23f;      // two scores' share, doubled
            }
            named_bar(5, kCThreads);
        }
        uint32_t* s_sorted = s_mask + kMaxE;                           // [T][kMaxK + 1]: keys by rank
        const bool counted = a.T * a.E * a.E <= kMostCounted;
        if (counted) {
            // an expert's rank is the number of experts before it
            for (int i = tid; i < a.T * a.E; i += kCThreads) {
                const int tt = (int)div_by(i, a.by_E), e = i - tt * a.E;
                const uint32_t* row = s_key + tt * Ep;
                const uint32_t mine = row[e];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < Ep; j += 4) {
                    const uint4 q = *reinterpret_cast<const uint4*>(row + j);
                    rank += (q.x > mine - (j < e)) + (q.y > mine - (j + 1 < e)) + (q.z > mine - (j + 2 < e)) +
                            (q.w > mine - (j + 3 < e));
                }
                if (rank <= a.k) s_sorted[tt * (kMaxK + 1) + rank] = mine;
                if (rank < a.k) s_pick[tt * kMaxK + rank] = e;
            }
            named_bar(5, kCThreads);
        }
        if (warp < a.T)
            select_token(a, warp, counted, slack, s_key + warp * Ep, s_sorted + warp * (kMaxK + 1), s_pick + warp * kMaxK,
                         s_slot + warp * 256, s_mask);
        named_bar(5, kCThreads);
        if (warp * 32 < a.E) {                  // the active experts, ascending: a warp per 32
            int before = 0, n = 0;
            uint32_t mine = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j * 32 < a.E) {
                    const int e = j * 32 + lane;
                    const uint32_t bal = __ballot_sync(0xffffffffu, e < a.E && s_mask[e] != 0);
                    if (j < warp) before += __popc(bal);
                    if (j == warp) mine = bal;
                    n += __popc(bal);
                }
            if (mine >> lane & 1u) s_list[before + __popc(mine & ((1u << lane) - 1))] = warp * 32 + lane;
            if (tid == 0) {
                *s_nact = n;
                s_mask[a.E] = (1u << a.T) - 1;
            }
        }
        __syncthreads();                        // routing tables ready (producer too)
        const int nact = *s_nact;
        int slot = 0;                           // this group's next ring slot, and its parity
        uint32_t ph = 0;
        float* red = s_red + grp * L::kBufs * (L::kRedBuf / 4);
        int rbuf = 0;
        float* yw = s_red + warp * kRows * TT;                  // this warp's sums [row][token] of a tile of y
        float* s_ys = reinterpret_cast<float*>(sm + a.ys_off);   // and the shared expert's, of all warps
        float* ysw = s_ys + warp * kRows * TT;

#pragma unroll 1
        for (int phase = a.Is > 0 ? 0 : 1; phase < 2 + ytiles; ++phase) {
            const bool up = phase < 2;
            // (selected one by one: through a reference every use would be an indexed
            // constant load, ~50 cycles each in a row)
            const int sd_k = up ? a.sd.k : a.sd2.k, sd_half = up ? a.sd.half : a.sd2.half;
            const int sd_area = up ? a.sd.area : a.sd2.area, sd_scales = up ? a.sd.scales : a.sd2.scales;
            if (phase == 2) {                   // every h is written
                fence_proxy_async_all();        // (the down stages read it through the async proxy)
                named_bar(7, kCThreads + 32);   // with the producer warp that weighs
                if (tid == 0) arrive();
                if (tid == 0) grid_wait();
                named_bar(6, kThreads);
                if (*s_abort) dead = true;
            }
            float res = 0.0f;                   // this thread's element of the tile's residual
            if (!up) {
                for (int i = lane; i < kRows * TT; i += 32) {
                    yw[i] = 0.0f;
                    if (a.Is > 0) ysw[i] = 0.0f;
                }
                __syncwarp();
                int r0, nr;
                rows_of_tile(phase - 2, r0, nr);
                const int r = tid % kRows, t = tid / kRows;
                if (a.residual && r < nr && t < a.T) res = bf16f(a.residual[(size_t)t * a.H + r0 + r]);
            }
            walk(phase, nact, [&](const Unit& u, bool routed, int c0, int c1) {
                const int K = up ? a.H : routed ? a.I : a.Is;
                const bool boxed = FMT != kBf16 && (up ? a.W1.boxed : routed ? a.W2.boxed : a.S2.boxed);
                const uint32_t mask = s_mask[u.e];
                const int ncol = __popc(mask), ntn = (ncol + 7) / 8;
                float acc[NT][4];
                uint32_t col[NT];               // this lane's column of each block of 8: offset of its first k
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
                    const int c = n * 8 + g < ncol ? n * 8 + g : 0;
                    col[n] = (up ? xs + nth_bit(mask, c) * xstride : a.sd2.tokens + c * (a.sd2.k * 2 + F::kXPad)) +
                             t4 * (FMT == kBf16 ? 16 : 32);
                }
                float wcol[NT][2] = {};         // down: weights of this lane's result columns (ahead of the wait)
                if (!up && u.e < a.E)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int c = n * 8 + 2 * t4 + q;
                            if (c < ncol) {
                                const int t = nth_bit(mask, c);
                                wcol[n][q] = __ldcg(a.w + (size_t)t * a.k + s_slot[t * 256 + u.e]);
                            }
                        }
                uint32_t tcol[NT][2] = {};      // affine up: table entries of this lane's result columns
                if (FMT == kAffine && up)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int c = n * 8 + 2 * t4 + q;
                            tcol[n][q] = tab0 + nth_bit(mask, c < ncol ? c : 0) * 8;
                        }
                for (int c = c0; c < c1; ++c) {
                    const int s = ring0 + slot, steps = min(sd_k, K - c * sd_k) / kStep;
                    const uint32_t st = ring + s * a.stage_bytes;
                    const int s0 = (uint32_t)(steps * gw) / kGw, n = (uint32_t)(steps * (gw + 1)) / kGw - s0;
                    uint32_t xb[NT], sc0 = 0, sc1 = 0, sb = 0, sx = 0;
#pragma unroll
                    for (int i = 0; i < NT; ++i) xb[i] = col[i] + (up ? c * sd_k * 2 : st) + s0 * (kStep * 2);
                    if (FMT != kBf16) {
                        sb = s0 * (FMT == kAffine ? 2 : 4) + (FMT == kNvfp4 ? t4 : 0);
                        sx = !boxed ? 0 : FMT == kNvfp4 ? sg << 4 : (sg >> 1) << 4;
                        sc0 = st + sd_scales + scale_off<FMT>(sd_area, sd_k, K, boxed, u.row0, 0, sg, c);
                        sc1 = st + sd_scales + scale_off<FMT>(sd_area, sd_k, K, boxed, u.row1, 1, sg, c);
                    }
                    if (!dead) {
                        const bool got = mbar_wait(&full[s], ph, s_abort, a.wait_limit);
                        if (!__all_sync(0xffffffffu, got)) {
                            dead = true;
                            if (lane == 0) report_error(a.err, kErrWaitExpired);
                            *s_abort = 1;
                        }
                    }
                    if (!dead) {
                        if (FMT != kBf16 && up) {
                            uint32_t tab[NT][2] = {};
                            if (FMT == kAffine)
#pragma unroll
                                for (int i = 0; i < NT; ++i)
#pragma unroll
                                    for (int q = 0; q < 2; ++q) tab[i][q] = tcol[i][q] + (c * (sd_k / 64) + s0) * a.T * 8;
                            run_steps_f16<FMT, NT>(st + sg * 128, sd_half, x4, s0, n, sc0, sc1, sb, sx, sd_area, xb, tab, a.T * 8,
                                                   ntn, acc);
                        } else {
                            run_steps<FMT, NT>(st + sg * 128, sd_half, x4, s0, n, sc0, sc1, sb, sx, sd_area, xb, ntn, acc);
                        }
                    }
                    __syncwarp();
                    // (after a wait that ran out the slot's copies may still be under way: it
                    // is not released, and the producer, which then stops, fills it no more)
                    if (lane == 0 && !dead) mbar_arrive(&empty[s]);
                    if (++slot == Sg) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
                // NVFP4: the expert's global scale (bf16 products carry 2^-8)
                const float gl = FMT == kNvfp4 ? (up ? 1.0f : 256.0f) * __ldg((up ? (routed ? a.W1.glob : a.S1.glob) : (routed ? a.W2.glob : a.S2.glob)) +
                                                                              (routed ? u.e : 0))
                                               : 1.0f;
                if (up) {
                    // the group's four k shares meet in shared memory
                    float* r = red + rbuf * (L::kRedBuf / 4);
                    if (L::kBufs == 2) rbuf ^= 1;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n < ntn) {
                            float* p = r + (gw * kRows + sg) * TT + n * 8 + 2 * t4;
                            *reinterpret_cast<float2*>(p) = make_float2(acc[n][0], acc[n][1]);
                            *reinterpret_cast<float2*>(p + 8 * TT) = make_float2(acc[n][2], acc[n][3]);
                        }
                    named_bar(1 + grp, kGw * 32);
                    for (int i = gt; i < kFeat * ncol; i += kGw * 32) {
                        const int f = i % kFeat, c = i / kFeat;
                        if (f >= u.n || dead) continue;
                        float v = 0.0f, w = 0.0f;
#pragma unroll
                        for (int q = 0; q < kGw; ++q) {
                            v += r[(q * kRows + f) * TT + c];
                            if (DUAL) w += r[(q * kRows + 8 + f) * TT + c];
                        }
                        if (FMT != kBf16) {
                            const float sc = s_xinv[nth_bit(mask, c)] * (FMT == kNvfp4 ? gl : 1.0f);
                            v *= sc;
                            w *= sc;
                        }
                        if (DUAL) {
                            clamp_swiglu(v, w, u.e == a.E ? a.limit_s : a.limit);
                            // (fast exp and quotient, ~2^-19: the result is rounded to bf16)
                            v = __fdividef(v, 1.0f + __expf(-v)) * w;
                        } else {
                            v = act_relu2(v);
                        }
                        // the activation is rounded once to bf16, the down products' operand type
                        // and moe_experts' h.  Its rounding adds to y's own: y is off by 0.0020-
                        // 0.0025 of its size (rms) instead of 0.0016.  h as a sum of two bf16
                        // took that away for 5 NVFP4 tokens 45 -> 48 us, 8 bf16 tokens 82 -> 88,
                        // 16 tokens 93 -> 115 (token rows crowd the weights out of the ring)
                        const int pos = u.f0 + f;
                        __stcg(const_cast<uint16_t*>(h_row(u.e, mask, c)) + (FMT == kBf16 ? pos : pair_pos(pos)), f2bf16(v));
                    }
                    if (L::kBufs == 1) named_bar(1 + grp, kGw * 32);   // the buffer is read
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = n * 8 + 2 * t4 + i;
                            if (c < ncol) {
                                const int t = nth_bit(mask, c);
                                const float w = (routed ? wcol[n][i] : 1.0f) * gl;
                                float* y = routed ? yw : ysw;
                                y[sg * TT + t] += w * acc[n][i];
                                y[(sg + 8) * TT + t] += w * acc[n][2 + i];
                            }
                        }
                    __syncwarp();
                }
                return true;
            });
            if (!up) {
                int r0, nr;
                rows_of_tile(phase - 2, r0, nr);
                named_bar(5, kCThreads);
                const int r = tid % kRows, t = tid / kRows;
                const bool mine = tid < kRows * TT && r < nr && t < a.T;
                const size_t o = (size_t)t * a.H + r0 + r;
                float v = 0.0f, sh = 0.0f;
                if (mine) {
#pragma unroll
                    for (int w = 0; w < kCw; ++w) v += s_red[(w * kRows + r) * TT + t];
                    if (a.Is > 0)
                        for (int w = 0; w < kCw; ++w) sh += s_ys[(w * kRows + r) * TT + t];
                }
                bool finish = true;
                if (a.ysplit > 1 && nr > 0) {
                    if (mine) __stcg(a.ypart + (size_t)ypart * a.T * a.H + o, make_float2(v, sh));
                    __threadfence();
                    named_bar(5, kCThreads);
                    if (tid == 0) {
                        const int block = r0 / kRows;
                        *s_nact = atomicAdd(a.ydone + block, 1);     // (the active count is no longer needed)
                        if (*s_nact == a.ysplit - 1) a.ydone[block] = 0;
                        __threadfence();
                    }
                    named_bar(5, kCThreads);
                    finish = *s_nact == a.ysplit - 1;
                    if (finish && mine) {
                        v = sh = 0.0f;
                        for (int q = 0; q < a.ysplit; ++q) {
                            const float2 p = __ldcg(a.ypart + (size_t)q * a.T * a.H + o);
                            v += p.x;
                            sh += p.y;
                        }
                    }
                }
                if (mine && finish && !dead) {
                    v *= a.out_scale;           // once, on the finished sum
                    if (a.Is > 0) v += sh;
                    if (a.residual) v += res;
                    a.y[o] = f2bf16(v);
                }
                named_bar(5, kCThreads);
            }
        }
    }
}

// What moe_decode_prepare leaves in the caller's moe_decode_plan.
struct Plan {
    DecodeArgs a;
    uint64_t magic;
    size_t smem, ws_bytes, ws_lg, ws_h, ws_hs, ws_yp;
    int device, grid;
    cudaError_t (*launch)(const Plan&, const DecodeArgs&, cudaStream_t);
};
constexpr uint64_t kPlanMagic = 0x6d6f65646563ull;
static_assert(sizeof(Plan) + alignof(Plan) <= sizeof(moe_decode_plan), "moe_decode_plan holds a Plan at any address");

template <int FMT, int NT, bool DUAL>
cudaError_t launch(const Plan& p, const DecodeArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_decode<FMT, NT, DUAL>, a);
}

// Shared memory of a CTA that may have max_smem bytes: the ring's stages and what
// lies in front of it.  The bytes to ask for, or 0 where not one stage fits.
template <int FMT, int NT>
size_t lay_out(DecodeArgs& a, int max_smem) {
    using F = Fmt<FMT>;
    // + 1 KB: the ring starts on a multiple of that
    // token rows and (affine) their table; the shared expert's y sums lie in the
    // second half of the group-sum buffers, or for 16 columns over the token
    // rows, which the down products no longer read, where those are long enough
    using L = Layout<NT>;
    const int x_bytes = a.T * (a.H * 2 + F::kXPad + (FMT == kAffine ? a.H / 8 : 0));
    const bool over_x = NT == 2 && x_bytes >= L::kYw;
    a.ys_off = NT == 1 ? L::kRed + L::kYw : over_x ? L::kX : (L::kX + x_bytes + 15) & ~15;
    a.ring_off = NT == 1 || over_x ? L::kX + x_bytes : a.ys_off + L::kYw;
    const size_t fixed = (size_t)a.ring_off + 1024;
    const int room = fixed < (size_t)max_smem ? (int)(max_smem - fixed) : 0;
    // Two slots per group of 16 KB of weights each where they fit, smaller ones
    // (at last a single one) where the token rows leave less room.  Down stages
    // hold the columns' activations too: as many chunks as fit behind them.
    auto up = [&](int c) { return F::dims(c, a.H, 0, 0); };
    auto down = [&](int c) { return F::dims(c, a.I, a.Is, a.T); };
    int slots = 3, c1, c2;
    do {
        const int most = room / (--slots * kGroups);
        // (affine: even numbers, for scale boxes on 16-byte starts)
        for (c1 = 8; c1 > 1 && up(c1).bytes > most;) c1 -= FMT == kAffine && c1 > 2 ? 2 : 1;
        for (c2 = 8; c2 > 1 && down(c2).bytes > most;) c2 -= FMT == kAffine && c2 > 2 ? 2 : 1;
    } while (slots > 1 && (c1 == 1 || c2 == 1));
    a.sd = up(c1);
    a.sd2 = down(c2);
    a.stage_bytes = std::max(a.sd.bytes, a.sd2.bytes);
    a.stages = std::min(kMaxStages, room / a.stage_bytes) / kGroups;
    return a.stages < 1 ? 0 : fixed + (size_t)kGroups * a.stages * a.stage_bytes;
}

template <int FMT, int NT, bool DUAL>
cudaError_t plan(Plan& p) {
    DecodeArgs& a = p.a;
    const DeviceInfo& di = device_info();
    using F = Fmt<FMT>;
    const size_t smem = lay_out<FMT, NT>(a, di.max_smem_optin);
    if (!smem) return cudaErrorNotSupported;
    const int c1 = a.sd.chunks, c2 = a.sd2.chunks;
    const int n1 = a.E * a.W1.rows, n2 = a.E * a.W2.rows;
    auto map = [&](WMat& m, int rows, int chunks) {
        const uint64_t bytes = FMT == kBf16 ? (uint64_t)m.K * 2 : (uint64_t)m.K / 2;
        cudaError_t e = make_tmap_rows(&m.map, m.w, bytes, bytes, rows, 8, chunks, &m.flat);
        m.boxed = F::boxed(chunks, m.K);
        if (e == cudaSuccess && m.boxed)
            e = make_tmap_narrow(&m.smap, m.scale, F::scale_bytes(m.K), rows, F::kScaleBox);
        if (e == cudaSuccess && m.boxed && FMT == kAffine)
            e = make_tmap_narrow(&m.bmap, m.bias, F::scale_bytes(m.K), rows, F::kScaleBox);
        return e;
    };
    cudaError_t e = map(a.W1, n1, c1);
    if (e == cudaSuccess) e = map(a.W2, n2, c2);
    if (e == cudaSuccess && a.Is > 0) e = map(a.S1, a.S1.rows, c1);
    if (e == cudaSuccess && a.Is > 0) e = map(a.S2, a.S2.rows, c2);
    if (e != cudaSuccess) return e;
    // parts of the router's rows: work for all CTAs
    a.parts = di.sm_count >= 4 * a.E ? 4 : di.sm_count >= 2 * a.E ? 2 : 1;
    a.up_stages = (a.H + a.sd.k - 1) / a.sd.k;
    a.i_stages = (a.I + a.sd2.k - 1) / a.sd2.k;
    a.is_stages = (a.Is + a.sd2.k - 1) / a.sd2.k;
    a.by_grid = divisor(di.sm_count);
    a.by_groups = divisor(di.sm_count * kGroups);
    a.by_I = divisor(a.I);
    a.by_E = divisor(a.E);
    a.by_i_stages = divisor(a.i_stages);
    const int blocks = (a.H + kRows - 1) / kRows;
    // stages of a tile of y, when every pick goes to an expert of its own
    const int work = std::min(a.E, a.T * a.k) * a.i_stages + a.is_stages;
    // Adding the parts up costs ~2.5 us (2 x 128 x 256 x 8 experts, one token: 11.5
    // -> 14.0 us); a group's stage ~0.7 us (9 tokens, 20 experts of 320 x 1984,
    // affine: 60.5 -> 43.1 us): split where a group has 6 stages or more, into
    // parts of at least 2.
    if (work >= 6 * kGroups)
        a.ysplit = std::max(1, std::min(std::min(di.sm_count, kMaxYRows / kRows) / blocks, work / (2 * kGroups)));
    else
        a.ysplit = 1;
    a.by_ysplit = divisor(a.ysplit);
    a.by_yworkers = divisor(a.ysplit * kGroups);
    if ((uint64_t)a.E * a.I * (di.sm_count * kGroups + 1) >> 32) return cudaErrorNotSupported;   // part()
    p.smem = smem;
    p.grid = di.sm_count;
    p.launch = launch<FMT, NT, DUAL>;
    return ensure_smem(k_decode<FMT, NT, DUAL>, smem);
}

template <int FMT>
cudaError_t plan_fmt(Plan& p, bool dual) {
    if (p.a.T <= 8) return dual ? plan<FMT, 1, true>(p) : plan<FMT, 1, false>(p);
    return dual ? plan<FMT, 2, true>(p) : plan<FMT, 2, false>(p);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct DecodeWs {
    size_t lg, h, hs, yp, total;                // behind 1 KB of counts
};

DecodeWs ws_layout(const moe_dims* d, int Is) {
    DecodeWs L{};
    size_t off = 1024;
    L.lg = off;
    off = align256(off + (size_t)kMaxParts * d->T * d->E * 8);
    L.h = off;
    off = align256(off + (size_t)d->T * d->k * d->I * 2);
    L.hs = off;
    L.yp = off = align256(off + (size_t)d->T * Is * 2);
    L.total = align256(off + (size_t)d->T * kMaxYRows * 8);
    return L;
}

moe_status refuse(moe_status st, const char* msg) {
    set_last_error(msg);
    return st;
}

// Sizes of moe_decode: moe_dims' limits, few tokens, and token rows that fit
// shared memory beside the weight ring.
moe_status check_sizes(const moe_dims* d, int Is) {
    moe_status st = validate_dims(d);
    if (st != MOE_OK) return st;
    if (d->T > MOE_DECODE_MAX_T) return refuse(MOE_ERR_SHAPE, "moe_decode: T > 16 (use moe_forward)");
    if ((long long)d->T * d->H > 65536) return refuse(MOE_ERR_SHAPE, "moe_decode: T * H > 65536 (use moe_forward)");
    if (Is < 0 || Is > 16384 || Is % 64)
        return refuse(MOE_ERR_SHAPE, "moe_decode: Is must be 0 or a multiple of 64 up to 16384");
    return MOE_OK;
}

WMat mat(const void* w, const void* scale, const void* bias, const float* glob, int rows, int K) {
    WMat m{};
    m.w = static_cast<const unsigned char*>(w);
    m.scale = static_cast<const unsigned char*>(scale);
    m.bias = static_cast<const unsigned char*>(bias);
    m.glob = glob;
    m.rows = rows;
    m.K = K;
    return m;
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The layer and the sizes, on the host.
moe_status check_layer(const moe_layer* L, const moe_dims* d) {
    if (!L) return refuse(MOE_ERR_NULL, "layer is NULL");
    moe_status st = check_sizes(d, L->Is);
    if (st != MOE_OK) return st;
    if (L->router.score != MOE_SCORE_SIGMOID && L->router.score != MOE_SCORE_SOFTMAX)
        return refuse(MOE_ERR_UNSUPPORTED, "router score");
    if (L->router.norm_topk != 0 && L->router.norm_topk != 1) return refuse(MOE_ERR_UNSUPPORTED, "norm_topk");
    if (misaligned(L->w_router, 16)) return refuse(MOE_ERR_ALIGN, "w_router not 16-byte aligned");
    if (misaligned(L->expert_bias, 4)) return refuse(MOE_ERR_ALIGN, "expert_bias not 4-byte aligned");
    if ((st = validate_weights(&L->W)) != MOE_OK) return st;
    if (L->Is > 0) {
        if ((st = validate_weights(&L->Ws)) != MOE_OK) return st;
        if (L->Ws.fmt != L->W.fmt || L->Ws.act != L->W.act)
            return refuse(MOE_ERR_UNSUPPORTED, "the shared expert's format or activation differs from the routed experts'");
    }
    return MOE_OK;
}

// Whether n bytes at p and m at q share one.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + m && b < a + n;
}

// What a call of T tokens brings.
moe_status check_call(const void* x, const float* logits, const float* w_router, const void* residual,
                      const int32_t* topk_idx, const float* topk_w, const void* y, const void* ws, size_t ws_bytes,
                      size_t need, int T, int H, int E, int k) {
    if (!x || !y) return refuse(MOE_ERR_NULL, "x or y is NULL");
    if (!topk_idx || !topk_w) return refuse(MOE_ERR_NULL, "topk_idx or topk_w is NULL");
    if (!logits && !w_router) return refuse(MOE_ERR_NULL, "w_router is NULL (routing from x)");
    if (misaligned(x, 16) || misaligned(y, 16)) return refuse(MOE_ERR_ALIGN, "x or y not 16-byte aligned");
    if (misaligned(residual, 16)) return refuse(MOE_ERR_ALIGN, "residual not 16-byte aligned");
    if (misaligned(logits, 4) || misaligned(topk_idx, 4) || misaligned(topk_w, 4))
        return refuse(MOE_ERR_ALIGN, "logits, topk_idx or topk_w not 4-byte aligned");
    // (x and logits may lie anywhere in y: they are read before the second grid barrier, y is written behind it)
    const size_t rows = (size_t)T * H * 2, picks = (size_t)T * k * 4;
    if (residual != y && overlap(residual, rows, y, rows))
        return refuse(MOE_ERR_UNSUPPORTED, "moe_decode: y overlaps a part of residual (it may be residual itself)");
    if (!ws) return refuse(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (misaligned(ws, 256)) return refuse(MOE_ERR_ALIGN, "workspace not 256-byte aligned");
    if (ws_bytes < need) return refuse(MOE_ERR_WORKSPACE, "workspace smaller than moe_decode_workspace_bytes()");
    // the picks are written while other CTAs still read x and logits, topk_w is read back
    const void* outs[3] = {topk_idx, topk_w, y};
    for (int i = 0; i < 3; ++i) {
        const size_t n = i < 2 ? picks : rows;
        const bool in = i < 2 && (overlap(outs[i], n, x, rows) || overlap(outs[i], n, residual, rows) ||
                                  overlap(outs[i], n, logits, (size_t)T * E * 4));
        if (in || overlap(outs[i], n, outs[(i + 1) % 3], i == 1 ? rows : picks) || overlap(outs[i], n, ws, need))
            return refuse(MOE_ERR_UNSUPPORTED, "moe_decode: topk_idx, topk_w or y overlaps another argument");
    }
    return MOE_OK;
}

// A prepared call; polls > 0: with grid barriers that run out after that many.
moe_status run(const moe_decode_plan* plan, const void* x, const float* logits, const void* residual, int32_t* topk_idx,
               float* topk_w, void* y, void* ws, size_t ws_bytes, uint32_t polls, moe_stream_t stream) {
    if (!plan) return refuse(MOE_ERR_NULL, "plan is NULL");
    Plan p;
    memcpy(&p, plan, sizeof p);
    if (p.magic != kPlanMagic) return refuse(MOE_ERR_UNSUPPORTED, "not a plan of moe_decode_prepare");
    if (p.a.T == 0) return set_last_launch_count(0), MOE_OK;   // empty batch: nothing to do
    const moe_status st = check_call(x, logits, p.a.w_router, residual, topk_idx, topk_w, y, ws, ws_bytes, p.ws_bytes,
                                     p.a.T, p.a.H, p.a.E, p.a.k);
    if (st != MOE_OK) return st;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev != p.device)
        return refuse(MOE_ERR_UNSUPPORTED, "the plan was prepared for another device");
    if (polls) {
        p.a.grid_limit = polls;
        p.a.missing = 1;
    }
    char* b = static_cast<char*>(ws);
    p.a.x = static_cast<const uint16_t*>(x);
    p.a.logits = logits;
    p.a.residual = static_cast<const uint16_t*>(residual);
    p.a.idx = topk_idx;
    p.a.w = topk_w;
    p.a.y = static_cast<uint16_t*>(y);
    p.a.sync = reinterpret_cast<unsigned long long*>(b);
    p.a.lg = reinterpret_cast<float2*>(b + p.ws_lg);
    p.a.h = reinterpret_cast<uint16_t*>(b + p.ws_h);
    p.a.hs = reinterpret_cast<uint16_t*>(b + p.ws_hs);
    p.a.ypart = reinterpret_cast<float2*>(b + p.ws_yp);
    p.a.ydone = reinterpret_cast<int*>(b + 256);
    if (e == cudaSuccess) e = p.launch(p, p.a, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return refuse(MOE_ERR_CUDA, cudaGetErrorString(e));
    set_last_launch_count(1);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_decode_workspace_bytes(const moe_dims* d, int32_t Is) {
    return check_sizes(d, Is) == MOE_OK ? ws_layout(d, Is).total : 0;
}

moe_status moe_decode_smem_layout(const moe_dims* d, int32_t Is, int32_t fmt, int32_t smem_bytes, moe_decode_smem* out) {
    const moe_status st = check_sizes(d, Is);
    if (st != MOE_OK) return st;
    if (!out) return refuse(MOE_ERR_NULL, "out is NULL");
    if (fmt != MOE_W_BF16 && fmt != MOE_W_AFFINE4_G64 && fmt != MOE_W_NVFP4) return refuse(MOE_ERR_UNSUPPORTED, "fmt");
    if (d->T == 0) return refuse(MOE_ERR_SHAPE, "moe_decode_smem_layout: T = 0 launches nothing");
    DecodeArgs a{};
    a.T = d->T;
    a.H = d->H;
    a.I = d->I;
    a.Is = Is;
    const auto go = [&](auto f) {
        constexpr int F = decltype(f)::value;
        out->smem = (int64_t)(d->T <= 8 ? lay_out<F, 1>(a, smem_bytes) : lay_out<F, 2>(a, smem_bytes));
        out->boxed_up = Fmt<F>::boxed(a.sd.chunks, a.H);
        out->boxed_down = Fmt<F>::boxed(a.sd2.chunks, a.I);
        out->boxed_shared = Fmt<F>::boxed(a.sd2.chunks, Is);
    };
    if (fmt == MOE_W_BF16) go(std::integral_constant<int, kBf16>());
    else if (fmt == MOE_W_AFFINE4_G64) go(std::integral_constant<int, kAffine>());
    else go(std::integral_constant<int, kNvfp4>());
    out->ring = a.ring_off;
    out->slots = a.stages;
    out->stage_bytes = a.stage_bytes;
    const auto stage = [](const StageDims& s) {
        return moe_decode_stage{s.chunks, s.k, s.half, s.scales, s.area, s.tokens, s.bytes};
    };
    out->up = stage(a.sd);
    out->down = stage(a.sd2);
    return MOE_OK;
}

moe_status moe_decode_prepare(const moe_layer* L, const moe_dims* d, moe_decode_plan* out) {
    const moe_status st = check_layer(L, d);
    if (st != MOE_OK) return st;
    if (!out) return refuse(MOE_ERR_NULL, "plan is NULL");
    const DecodeWs wl = ws_layout(d, L->Is);
    const bool dual = L->W.act == MOE_ACT_SWIGLU;
    Plan p{};
    DecodeArgs& a = p.a;
    a.w_router = L->w_router;
    a.ebias = L->expert_bias;
    a.W1 = mat(L->W.w1, L->W.w1_scale, L->W.w1_bias, L->W.w1_global, dual ? 2 * d->I : d->I, d->H);
    a.W2 = mat(L->W.w2, L->W.w2_scale, L->W.w2_bias, L->W.w2_global, d->H, d->I);
    if (L->Is > 0) {
        a.S1 = mat(L->Ws.w1, L->Ws.w1_scale, L->Ws.w1_bias, L->Ws.w1_global, dual ? 2 * L->Is : L->Is, d->H);
        a.S2 = mat(L->Ws.w2, L->Ws.w2_scale, L->Ws.w2_bias, L->Ws.w2_global, d->H, L->Is);
        a.limit_s = L->Ws.swiglu_limit;
    }
    a.T = d->T;
    a.H = d->H;
    a.E = d->E;
    a.k = d->k;
    a.I = d->I;
    a.Is = L->Is;
    a.eps = L->eps;
    a.scale = L->router_scale;
    a.out_scale = L->out_scale;
    a.limit = L->W.swiglu_limit;
    a.softmax = L->router.score == MOE_SCORE_SOFTMAX;
    a.no_norm = L->router.norm_topk == 0;
    a.wait_limit = a.grid_limit = sm100::kWaitLimit;
    a.err = device_info().err_word;
    p.ws_bytes = wl.total;
    p.ws_lg = wl.lg;
    p.ws_h = wl.h;
    p.ws_hs = wl.hs;
    p.ws_yp = wl.yp;
    p.magic = kPlanMagic;
    cudaError_t e = cudaGetDevice(&p.device);
    if (e == cudaSuccess && d->T > 0)            // an empty batch launches nothing
        e = L->W.fmt == MOE_W_BF16          ? plan_fmt<kBf16>(p, dual)
            : L->W.fmt == MOE_W_AFFINE4_G64 ? plan_fmt<kAffine>(p, dual)
                                            : plan_fmt<kNvfp4>(p, dual);
    if (e == cudaErrorNotSupported) return refuse(MOE_ERR_UNSUPPORTED, "moe_decode: shared memory or driver of this device");
    if (e != cudaSuccess) return refuse(MOE_ERR_CUDA, cudaGetErrorString(e));
    memset(out, 0, sizeof *out);
    memcpy(out, &p, sizeof p);
    return MOE_OK;
}

moe_status moe_decode_run(const moe_decode_plan* plan, const void* x, const float* logits, const void* residual,
                          int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
    return run(plan, x, logits, residual, topk_idx, topk_w, y, ws, ws_bytes, 0, stream);
}

moe_status moe_decode_expiry_check(const moe_decode_plan* plan, const void* x, const float* logits,
                                   const void* residual, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                                   size_t ws_bytes, uint32_t polls, moe_stream_t stream) {
    if (polls < 1 || polls > (1u << 20))
        return refuse(MOE_ERR_SHAPE, "moe_decode_expiry_check: polls must be in [1, 2^20]");
    return run(plan, x, logits, residual, topk_idx, topk_w, y, ws, ws_bytes, polls, stream);
}

moe_status moe_decode(const moe_layer* L, const moe_dims* d, const void* x, const float* logits,
                      const void* residual, int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes,
                      moe_stream_t stream) {
    moe_status st = check_layer(L, d);
    if (st != MOE_OK) return st;
    if (d->T == 0) return set_last_launch_count(0), MOE_OK;   // empty batch: nothing to do
    st = check_call(x, logits, L->w_router, residual, topk_idx, topk_w, y, ws, ws_bytes, ws_layout(d, L->Is).total,
                    d->T, d->H, d->E, d->k);
    if (st != MOE_OK) return st;
    moe_decode_plan plan;
    st = moe_decode_prepare(L, d, &plan);
    return st != MOE_OK ? st
                        : moe_decode_run(&plan, x, logits, residual, topk_idx, topk_w, y, ws, ws_bytes, stream);
}

}  // extern "C"
