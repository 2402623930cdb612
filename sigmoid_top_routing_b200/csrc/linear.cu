// A linear layer with bias, activation and residual in the product's epilogue:
//
//   y[m, n] = act(sum_k x[m, k] W[n, k] + bias[n]) + residual[m, n]
//
// act none, relu(v)^2, or SwiGLU over W = [gate; up] (2N rows): silu(g) u.
// bf16 x and W, fp32 sums, one rounding at the store (none for fp32 y).
//
// Both kernels put weight rows on the MMA's M (A operand) and tokens on its N,
// so a few tokens cost a narrow MMA, and a TMEM lane is a feature: its bias is
// one register and the 32 lanes of a warp store 32 neighbouring features of a
// token, for any N and any alignment of the rows.  For SwiGLU a 128-row A tile
// holds 64 features: within each 32-lane quarter of TMEM, lanes 0-15 are gate
// rows and 16-31 the matching up rows (one TMA box of 16 rows x 2 halves per
// quarter), so gate and up meet by one warp shuffle.
//
//   k_linear_pair   persistent, 256 x BN tiles on SM pairs (cta_group::2), for
//                   products with enough tiles to fill the SMs.  Each CTA loads
//                   its 128 weight rows and half of the token rows, 128 k a round,
//                   into a ring of 192 KB; two TMEM accumulators let the epilogue
//                   of one tile overlap the next one's MMAs.
//   k_linear_split  one 128 x BN tile per cluster of ks CTAs that share its K,
//                   for few tokens or small products: partial sums meet through
//                   distributed shared memory in rank order, so no workspace, no
//                   atomics, and the same bits every time.
//
// Measured: 8192 x 7168 (SwiGLU: 14336 rows) x 2048 309 us = 1557 TFLOP/s in bursts,
// 366-373 us = 1300 call after call at the power limit; 8192 x 2048 x 7168 with bias and
// residual 162 us = 1484 and 192-195 us = 1250 (a library product of the same sizes,
// without epilogue, 365-430 and 182-231 us); 512 x 4096 x 2048 relu^2 10.6 us; 77 x 1537
// x 1795 with fp32 residual 7.8 us; 8 x 7168 (SwiGLU) x 2048 14.4 us = 4.1 TB/s; one token
// 2048 x 2048 4.8-5.6 us.  (The last four are device times; calls in a row from Python
// take 10.2-15 us, ~10 us of them on the host.)  Bound: the tensor cores at the large sizes (an SM takes ~75 GB/s of
// operands per tile: 32 KB per 64 k at BN = 256), latency and the sharing of a
// weight stream by uneven numbers of CTAs at the small ones.
//
// Rows and k past the ends are zero-filled by TMA on both operands.  Every wait
// is bounded; on expiry the kernel records device error 2, drains and returns.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {
namespace {

using namespace sm100;

constexpr int kBK = 64;                          // k per stage: one 128-byte swizzle row
constexpr int kAStage = 128 * kBK * 2;           // 16 KB of weight rows per CTA
constexpr int kLinThreads = 320;                 // producer, MMA issuer, 8 epilogue warps (two per TMEM quarter)
constexpr int kMaxStage = 8;
constexpr int kMaxKs = 8;                        // CTAs that share a tile's K

struct LinParams {
    const float* bias;
    const void* residual;
    void* y;
    long long ldr, ldy;                          // row strides in elements
    int M, N, nkb;                               // tokens, features, k-blocks
    int n_wt, n_tt, BN;                          // weight tiles, token tiles, tokens of a tile
    int stages, ks;
    int res_f32, y_f32;
    float limit;
    uint32_t hold;                               // > 0 (the expiry check): the MMA warp first waits this long for nothing
    int* err;
};

// Residual values of NC consecutive tokens of one feature (the column at t0),
// requested together; FULL: all of them exist.
template <int NC, bool FULL>
MOE_DEV void load_res(const LinParams& p, int f, int t0, int n, float (&q)[NC]) {
    if (p.res_f32) {
        const float* r = static_cast<const float*>(p.residual) + (size_t)t0 * p.ldr + f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            q[i] = FULL || i < n ? *r : 0.0f;
            r += p.ldr;
        }
    } else {
        const uint16_t* r = static_cast<const uint16_t*>(p.residual) + (size_t)t0 * p.ldr + f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            q[i] = __uint_as_float((FULL || i < n) ? (uint32_t)*r : 0u);   // widened in add_res
            r += p.ldr;
        }
    }
}
template <int NC>
MOE_DEV void add_res(const LinParams& p, const float (&q)[NC], float (&o)[NC]) {
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] += p.res_f32 ? q[i] : __uint_as_float(__float_as_uint(q[i]) << 16);
}
template <int NC, bool FULL>
MOE_DEV void store_out(const LinParams& p, int f, int t0, int n, const float (&o)[NC]) {
    if (p.y_f32) {
        float* y = static_cast<float*>(p.y) + (size_t)t0 * p.ldy + f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (FULL || i < n) *y = o[i];
            y += p.ldy;
        }
    } else {
        uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)t0 * p.ldy + f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (FULL || i < n) *y = f2bf16(o[i]);
            y += p.ldy;
        }
    }
}

// Epilogue of NC columns (tokens t0 .. t0 + NC - 1) of this lane's feature row.
// f: the lane's feature (SwiGLU: the same for lanes l and l + 16).
template <int ACT, int NC>
MOE_DEV void emit(const LinParams& p, const float (&v)[NC], int f, int t0, float b0, float b1) {
    constexpr int C = ACT == MOE_ACT_SWIGLU ? NC / 2 : NC;       // columns this lane stores
    const int lane = threadIdx.x & 31;
    const int t = ACT == MOE_ACT_SWIGLU && lane >= 16 ? t0 + C : t0;
    const int n = min(C, p.M - t);
    const bool live = f < p.N, full = t0 + NC <= p.M;            // full: warp-uniform
    float q[C], o[C];
    if (p.residual && live) {                    // requested first: the activation hides some of the latency
        if (full) load_res<C, true>(p, f, t, n, q);
        else load_res<C, false>(p, f, t, n, q);
    }
    if constexpr (ACT == MOE_ACT_SWIGLU) {
        // low lanes end up with gate and up of the first half of the columns, high lanes of the second
        const bool lo = lane < 16;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, lo ? v[C + i] : v[i], 16);
            float g = (lo ? v[i] : other) + b0, u = (lo ? other : v[C + i]) + b1;
            clamp_swiglu(g, u, p.limit);
            // bf16 results: exp and the quotient to ~2^-19, far below the store's 2^-8
            o[i] = p.y_f32 ? act_swiglu(g, u) : __fdividef(g, 1.0f + __expf(-g)) * u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = ACT == MOE_ACT_RELU2 ? act_relu2(v[i] + b0) : v[i] + b0;
    }
    if (live) {
        if (p.residual) add_res(p, q, o);
        if (full) store_out<C, true>(p, f, t, n, o);
        else store_out<C, false>(p, f, t, n, o);
    }
}

// Feature of TMEM lane `row` (0..127) of a CTA's tile that starts at feature f0.
template <int ACT>
MOE_DEV int feature_of(int f0, int row) {
    return ACT == MOE_ACT_SWIGLU ? f0 + 16 * (row >> 5) + (row & 15) : f0 + row;
}
template <int ACT>
MOE_DEV void bias_of(const LinParams& p, int f, float& b0, float& b1) {
    b0 = b1 = 0.0f;
    if (p.bias && f < p.N) {
        b0 = __ldg(p.bias + f);
        if (ACT == MOE_ACT_SWIGLU) b1 = __ldg(p.bias + p.N + f);
    }
}

// One lane of a converged warp.  Producer and MMA loops run on all 32 lanes with
// warp-uniform values and only their TMA, MMA and commit instructions under this
// predicate: inside an `if (lane == 0)` those instructions' operands are not
// uniform to the compiler, which then issues them lane by lane (~40 cycles each;
// a k-block of the pair kernel took 305 ns whatever its width).
MOE_DEV bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
MOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag, uint32_t limit) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, limit));
}

// 3D tiled load (SwiGLU weights: k, row, gate / up half).
MOE_DEV void tma_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
MOE_DEV void tma_load_3d_pair(void* dst, const CUtensorMap* m, int x, int y, int z, uint32_t cbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(cbar)
        : "memory");
}

MOE_DEV void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Tile t of the persistent order: weight tiles in groups of 8, token tiles
// within a group, so the tiles running at one time share operands in L2.
MOE_DEV void tile_of(const LinParams& p, int t, int& wt, int& tt) {
    const int per = 8 * p.n_tt, g = t / per, r = t - g * per;
    const int gw = min(8, p.n_wt - g * 8);
    tt = r / gw;
    wt = g * 8 + r - tt * gw;
}

// Pair stages hold two k-blocks: a round of the pipeline (wait, issue, commit)
// costs ~200 ns whatever it moves, which bounded narrow tiles at 64 k a round.
constexpr int kPairA = 2 * kAStage;              // 32 KB of weight rows per CTA
constexpr int kPairRing = 192 * 1024;
constexpr int kPairMaxStages = 5;
constexpr size_t kPairSmem = size_t(kPairRing) + 1024 + 256;

template <int ACT>
__global__ void __launch_bounds__(kLinThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, LinParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sA = sm;
    const int S = p.stages, bstage = p.BN * 128;             // two blocks of BN / 2 token rows
    unsigned char* sB = sm + S * kPairA;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kPairRing);
    uint64_t* empty = full + kPairMaxStages;
    uint64_t* tfull = empty + kPairMaxStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    constexpr int kF = ACT == MOE_ACT_SWIGLU ? 64 : 128;         // features of a CTA's 128 rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 16);            // the epilogue warps of both CTAs
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    cluster_sync();                              // both CTAs' barriers exist before either signals the other
    if (warp == 1) {
        tmem_alloc_pair(s_tmem, 512);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_trigger();
    const int total = p.n_wt * p.n_tt, tbeg = blockIdx.x >> 1, tstep = gridDim.x >> 1;
    // A wait ran out: neither CTA of the pair can go on without the other.
    auto give_up = [&]() {
        if (lane == 0) report_error(p.err, kErrWaitExpired);
        *s_abort = 1;
        st_cluster_u32(mapa_shared(smem_u32(const_cast<const int*>(s_abort)), rank ^ 1u), 1u);
    };
    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0, issued = 0, par = 0;
        bool ok = true;
        const uint32_t bytes = 2u * (kPairA + bstage);                   // of both CTAs
        for (int t = tbeg; t < total && ok; t += tstep) {
            int wt, tt;
            tile_of(p, t, wt, tt);
            const int f0 = (wt * 2 + (int)rank) * kF, row = tt * p.BN + (int)rank * (p.BN / 2);
            for (int kb = 0; kb < p.nkb; kb += 2) {      // k past the end is zero-filled
                if (!warp_wait(&empty[s], ph ^ 1, s_abort, kWaitLimit)) { ok = false; break; }
                if (elect_one()) {
                    // both CTAs' loads complete on the even CTA's barrier, which arrives once
                    const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        unsigned char* a = sA + s * kPairA + h * kAStage;
                        const int x = (kb + h) * kBK;
                        if (ACT == MOE_ACT_SWIGLU) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) tma_load_3d_pair(a + q * 4096, &tmA, x, f0 + 16 * q, 0, fb);
                        } else {
                            tma_load_2d_pair(a, &tmA, x, f0, fb);
                        }
                        tma_load_2d_pair(sB + s * bstage + h * (bstage / 2), &tmB, x, row, fb);
                    }
                }
                __syncwarp();
                issued |= 1u << s;
                par = (par & ~(1u << s)) | (ph << s);
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) give_up();
        if (rank == 0)                           // counts the odd CTA's bytes too
            for (int q = 0; q < S; ++q)
                if (issued >> q & 1u) mbar_wait(&full[q], par >> q & 1u, nullptr, kWaitLimit);
    } else if (warp == 1) {
        if (rank == 0) {
            int s = 0, it = 0;
            uint32_t ph = 0;
            bool ok = !p.hold || warp_wait(drain, 0, nullptr, p.hold);   // (nothing is committed to it yet)
            const uint32_t idesc = idesc_bf16(256, p.BN);
            for (int t = tbeg; t < total && ok; t += tstep, ++it) {
                const int buf = it & 1;
                if (!warp_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, s_abort, kWaitLimit)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + buf * 256;
                for (int kb = 0; kb < p.nkb; kb += 2) {
                    if (!warp_wait(&full[s], ph, s_abort, kWaitLimit)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = sdesc_sw128(smem_u32(sA + s * kPairA));
                    const uint64_t bd = sdesc_sw128(smem_u32(sB + s * bstage));
                    const uint64_t ad2 = ad + (kAStage >> 4), bd2 = bd + uint64_t(bstage >> 5);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk)
                            umma_bf16_pair(d, ad + uint64_t(kk * 2), bd + uint64_t(kk * 2), idesc, kb != 0 || kk != 0);
                        if (kb + 1 < p.nkb) {
#pragma unroll
                            for (int kk = 0; kk < kBK / 16; ++kk)
                                umma_bf16_pair(d, ad2 + uint64_t(kk * 2), bd2 + uint64_t(kk * 2), idesc, true);
                        }
                        umma_commit_pair_both(&empty[s]);
                        if (kb + 2 >= p.nkb) umma_commit_pair_both(&tfull[buf]);
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            if (!ok) give_up();
            if (elect_one()) umma_commit_pair_local(drain);
            __syncwarp();
            mbar_wait(drain, 0, nullptr, kWaitLimit);
        }
        __syncwarp();
    } else {
        const int sub = warp & 3, row = 32 * sub + lane;
        int it = 0;
        bool dead = false;
        for (int t = tbeg; t < total; t += tstep, ++it) {
            int wt, tt;
            tile_of(p, t, wt, tt);
            const int buf = it & 1, f = feature_of<ACT>((wt * 2 + (int)rank) * kF, row);
            float b0, b1;
            bias_of<ACT>(p, f, b0, b1);
            if (!dead) {
                const bool ok = mbar_wait(&tfull[buf], (it >> 1) & 1, s_abort, kWaitLimit);
                if (__any_sync(0xffffffffu, !ok)) {
                    give_up();
                    dead = true;
                }
            }
            tc_fence_after();
            if (!dead) {
                const uint32_t tb = tmem + (uint32_t(32 * sub) << 16) + buf * 256;
                const int nc = min(p.BN, p.M - tt * p.BN);
                for (int c = warp < 6 ? 0 : 16; c < nc; c += 32) {
                    float v[16];
                    tmem_ld16(tb + c, v);
                    emit<ACT, 16>(p, v, f, tt * p.BN + c, b0, b1);
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank != 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
                else mbar_arrive(&tempty[buf]);
            }
        }
    }
    __syncthreads();
    cluster_sync();                              // the pair's MMAs and both epilogues are done with TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

MOE_DEV float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

template <int ACT>
__global__ void __launch_bounds__(kLinThreads)
    k_linear_split(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, LinParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, bstage = p.BN * 128;
    unsigned char* sA = sm;
    unsigned char* sB = sm + S * kAStage;
    __shared__ uint64_t full[kMaxStage], empty[kMaxStage], done;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    constexpr int kF = ACT == MOE_ACT_SWIGLU ? 64 : 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.ks > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / p.ks, tt = tile / p.n_wt, wt = tile - tt * p.n_wt;
    const int kb0 = rank * p.nkb / p.ks, kb1 = (rank + 1) * p.nkb / p.ks;
    const int cols = p.BN <= 32 ? 32 : p.BN <= 64 ? 64 : p.BN <= 128 ? 128 : 256;   // TMEM columns
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(&s_tmem, cols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();
    const int f0 = wt * kF;
    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0, issued = 0, par = 0;
        bool ok = true;
        const uint64_t pol = policy_evict_first();               // weights of a single token tile are read once
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(&empty[s], ph ^ 1, &s_abort, kWaitLimit)) { ok = false; break; }
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], kAStage + bstage);
                unsigned char* a = sA + s * kAStage;
                if (ACT == MOE_ACT_SWIGLU) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tma_load_3d(a + q * 4096, &tmA, kb * kBK, f0 + 16 * q, 0, &full[s]);
                } else if (p.n_tt == 1) {
                    tma_load_2d_hint(a, &tmA, kb * kBK, f0, &full[s], pol);
                } else {
                    tma_load_2d(a, &tmA, kb * kBK, f0, &full[s]);
                }
                tma_load_2d(sB + s * bstage, &tmB, kb * kBK, tt * p.BN, &full[s]);
            }
            __syncwarp();
            issued |= 1u << s;
            par = (par & ~(1u << s)) | (ph << s);
            if (++s == S) { s = 0; ph ^= 1; }
        }
        if (!ok) {
            if (lane == 0) report_error(p.err, kErrWaitExpired);
            s_abort = 1;
        }
        for (int q = 0; q < S; ++q)
            if (issued >> q & 1u) mbar_wait(&full[q], par >> q & 1u, nullptr, kWaitLimit);
    } else if (warp == 1) {
        int s = 0;
        uint32_t ph = 0;
        bool ok = !p.hold || warp_wait(&done, 0, nullptr, p.hold);   // (nothing is committed to it yet)
        const uint32_t idesc = idesc_bf16(128, p.BN);
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
            if (!warp_wait(&full[s], ph, &s_abort, kWaitLimit)) { ok = false; break; }
            tc_fence_after();
            const uint64_t ad = sdesc_sw128(smem_u32(sA + s * kAStage));
            const uint64_t bd = sdesc_sw128(smem_u32(sB + s * bstage));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                    umma_bf16(tmem, ad + uint64_t(kk * 2), bd + uint64_t(kk * 2), idesc, kb != kb0 || kk != 0);
                umma_commit(&empty[s]);
                if (kb == kb1 - 1) umma_commit(&done);
            }
            __syncwarp();
            if (++s == S) { s = 0; ph ^= 1; }
        }
        if (!ok) {
            if (lane == 0) report_error(p.err, kErrWaitExpired);
            s_abort = 1;
            if (elect_one()) umma_commit(&done);                 // what was issued completes
            __syncwarp();
        }
    }
    __syncwarp();
    // The accumulator is complete, and with it every load has been consumed.
    const bool ok = mbar_wait(&done, 0, nullptr, kWaitLimit);
    if (!ok) s_abort = 1;
    __syncthreads();
    tc_fence_after();
    const bool dead = s_abort != 0;
    if (dead && threadIdx.x == 0) report_error(p.err, kErrWaitExpired);
    const int sub = warp & 3, row = 32 * sub + lane;
    const int f = feature_of<ACT>(f0, row), t0 = tt * p.BN;
    const int nc = min(p.BN, p.M - t0);          // tokens of this tile
    float b0, b1;
    bias_of<ACT>(p, f, b0, b1);
    const uint32_t tb = tmem + (uint32_t(32 * sub) << 16);
    const int half = warp < 6 ? 0 : 1;           // the two warps of a TMEM quarter share its columns
    if (p.ks == 1) {
        if (warp >= 2 && !dead)
            for (int c = half * 16; c < nc; c += 32) {
                float v[16];
                tmem_ld16(tb + c, v);
                emit<ACT, 16>(p, v, f, t0 + c, b0, b1);
                __syncwarp();
            }
    } else {
        float* part = reinterpret_cast<float*>(sm);              // [BN][128], over the stages
        if (warp >= 2)
            for (int c = half * 16; c < nc; c += 32) {
                float v[16];
                tmem_ld16(tb + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * 128 + row] = v[i];
            }
        cluster_sync();
        if (warp >= 2 && !dead) {
            // four columns at a time, dealt out to the ranks and halves; all ranks'
            // values are requested at once
            const uint32_t mine = smem_u32(part);
            for (int c = (rank * 2 + half) * 4; c < nc; c += p.ks * 8) {
                float q[kMaxKs][4], v[4] = {};
#pragma unroll
                for (int r = 0; r < kMaxKs; ++r)
                    if (r < p.ks) {
                        const uint32_t a = mapa_shared(mine + (c * 128 + row) * 4, r);
#pragma unroll
                        for (int i = 0; i < 4; ++i) q[r][i] = ld_cluster_f32(a + i * 512);
                    }
#pragma unroll
                for (int r = 0; r < kMaxKs; ++r)
                    if (r < p.ks) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] += q[r][i];
                    }
                emit<ACT, 4>(p, v, f, t0 + c, b0, b1);
                __syncwarp();
            }
        }
        cluster_sync();                          // nobody leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, cols);
    }
}

// ---------------------------------------------------------------------------- host side

// bf16 rows in the 128-byte swizzle; halves > 1 adds a third dimension of that
// many row blocks, `rows` rows apart.
cudaError_t make_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t ld, uint32_t box_rows,
                     uint32_t halves) {
    const cuuint64_t dims[3] = {K, rows, halves}, strides[2] = {ld * 2, rows * ld * 2};
    const cuuint32_t box[3] = {kBK, box_rows, halves};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, halves > 1 ? 3 : 2, base, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

struct LinCall {
    const void *x, *w;
    long long ldx, ldw;
    int K;
};

template <int ACT>
cudaError_t maps(const LinCall& c, const LinParams& p, uint32_t b_rows, CUtensorMap* ta, CUtensorMap* tb) {
    cudaError_t e = ACT == MOE_ACT_SWIGLU ? make_map(ta, c.w, c.K, p.N, c.ldw, 16, 2)
                                          : make_map(ta, c.w, c.K, p.N, c.ldw, 128, 1);
    return e != cudaSuccess ? e : make_map(tb, c.x, c.K, p.M, c.ldx, b_rows, 1);
}

// Tokens of a pair tile: the width that finishes all tiles soonest.  A k-block
// of a tile measured 225-250 ns at 128 tokens and 295-370 ns at 256 (one tile
// alone - all SMs busy), so a tile costs its width plus 160.
int pick_bn(int M, int n_wt, int pairs) {
    int best = 256;
    long long cost = -1;
    for (int bn = 256; bn >= 32; bn -= 16) {
        const long long tiles = (long long)n_wt * ((M + bn - 1) / bn);
        const long long c = (tiles + pairs - 1) / pairs * (bn + 160);
        if (cost < 0 || c < cost) {
            cost = c;
            best = bn;
        }
    }
    return best;
}

template <int ACT>
cudaError_t run_linear(const LinCall& c, LinParams p, cudaStream_t s) {
    const DeviceInfo& di = device_info();
    constexpr int kF = ACT == MOE_ACT_SWIGLU ? 64 : 128;
    const int pairs = di.sm_count / 2;
    CUtensorMap ta, tb;
    cudaError_t e;
    p.nkb = (c.K + kBK - 1) / kBK;
    const int wt2 = (p.N + 2 * kF - 1) / (2 * kF), bn2 = pick_bn(p.M, wt2, pairs);
    const long long tiles2 = (long long)wt2 * ((p.M + bn2 - 1) / bn2);
    // Pair tiles when they fill half of the SMs or more.
    if (p.M > 64 && tiles2 * 2 > pairs) {
        p.BN = bn2;
        p.n_wt = wt2;
        p.n_tt = (p.M + bn2 - 1) / bn2;
        p.stages = std::min(kPairMaxStages, kPairRing / (kPairA + bn2 * 128));
        if ((e = maps<ACT>(c, p, bn2 / 2, &ta, &tb)) != cudaSuccess) return e;
        auto kern = k_linear_pair<ACT>;
        if ((e = ensure_smem(kern, kPairSmem)) != cudaSuccess) return e;
        const int grid = (int)std::min<long long>(tiles2, pairs) * 2;
        return launch_k_pair(kern, dim3(grid), dim3(kLinThreads), kPairSmem, s, true, ta, tb, p);
    }
    p.BN = std::min(128, (p.M + 15) / 16 * 16);
    p.n_wt = (p.N + kF - 1) / kF;
    p.n_tt = (p.M + p.BN - 1) / p.BN;
    const long long tiles = (long long)p.n_wt * p.n_tt;
    p.ks = 1;
    while (p.ks < kMaxKs && tiles * p.ks * 2 <= 2 * di.sm_count && p.nkb >= p.ks * 4) p.ks *= 2;
    const int stage = kAStage + p.BN * 128;
    p.stages = std::max(2, std::min(std::min(kMaxStage, 100 * 1024 / stage), (p.nkb + p.ks - 1) / p.ks));
    const size_t smem = std::max((size_t)p.stages * stage, (size_t)p.BN * 512) + 1024;
    if ((e = maps<ACT>(c, p, p.BN, &ta, &tb)) != cudaSuccess) return e;
    auto kern = k_linear_split<ACT>;
    if ((e = ensure_smem(kern, smem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.ks));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.ks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ta, tb, p);
}

moe_status refuse(moe_status st, const char* msg) {
    set_last_error(msg);
    return st;
}
bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// A matrix in memory, in bytes.
struct Span {
    uintptr_t p;
    long long rows, row, pitch;
    Span(const void* q, long long rows, long long cols, long long ld, int es)
        : p(reinterpret_cast<uintptr_t>(q)), rows(rows), row(cols * es), pitch(rows > 1 ? ld * es : cols * es) {}
    uintptr_t end() const { return p + (uintptr_t)((rows - 1) * pitch + row); }
};
// Whether two of them share a byte.  Column blocks of one buffer (same pitch) do
// not; rows that interleave with another pitch count as shared.
bool overlap(const Span& a, const Span& b) {
    if (a.p >= b.end() || b.p >= a.end()) return false;
    const Span &lo = a.p <= b.p ? a : b, &hi = a.p <= b.p ? b : a;
    if (lo.rows > 1 && hi.rows > 1 && lo.pitch != hi.pitch) return true;
    if (lo.rows == 1 && hi.rows == 1) return true;
    const long long pitch = std::max(lo.rows > 1 ? lo.pitch : 0, hi.rows > 1 ? hi.pitch : 0);
    const long long off = (long long)(hi.p - lo.p) % pitch;
    return off < lo.row || off + hi.row > pitch;
}

// A call; hold > 0: whose first wait runs out after that many polls.
moe_status linear(const void* x, const void* w, const float* bias, const void* residual, const moe_linear_dims* d,
                  const moe_linear_cfg* cfg, void* y, uint32_t hold, moe_stream_t stream) {
    if (!d || !cfg) return refuse(MOE_ERR_NULL, "dims or cfg is NULL");
    if (d->M < 0 || d->N < 1 || d->K < 1) return refuse(MOE_ERR_SHAPE, "moe_linear: need M >= 0, N >= 1, K >= 1");
    constexpr int kMost = 1 << 24;
    if (d->M > kMost || d->N > kMost || d->K > kMost) return refuse(MOE_ERR_SHAPE, "moe_linear: a size above 2^24");
    if (cfg->act != MOE_ACT_NONE && cfg->act != MOE_ACT_RELU2 && cfg->act != MOE_ACT_SWIGLU)
        return refuse(MOE_ERR_UNSUPPORTED, "moe_linear: activation");
    if ((cfg->res_f32 | cfg->y_f32) & ~1) return refuse(MOE_ERR_UNSUPPORTED, "moe_linear: res_f32 and y_f32 are 0 or 1");
    if (!(cfg->swiglu_limit >= 0.0f) || cfg->swiglu_limit > 3.0e38f)
        return refuse(MOE_ERR_SHAPE, "swiglu_limit must be finite and >= 0 (0 = off)");
    const long long ldx = d->ldx ? d->ldx : d->K, ldw = d->ldw ? d->ldw : d->K;
    const long long ldr = d->ldr ? d->ldr : d->N, ldy = d->ldy ? d->ldy : d->N;
    constexpr long long kMostLd = 1ll << 31;
    if (ldx < d->K || ldw < d->K || ldr < d->N || ldy < d->N || ldx > kMostLd || ldw > kMostLd || ldr > kMostLd ||
        ldy > kMostLd)
        return refuse(MOE_ERR_SHAPE, "moe_linear: a row stride below the row length (or above 2^31)");
    if (ldx % 8 || ldw % 8) return refuse(MOE_ERR_ALIGN, "moe_linear: row strides of x and w must be multiples of 8 elements");
    if (d->M == 0) return set_last_launch_count(0), MOE_OK;
    if (!x || !w || !y) return refuse(MOE_ERR_NULL, "x, w or y is NULL");
    if (misaligned(x, 16) || misaligned(w, 16)) return refuse(MOE_ERR_ALIGN, "x or w not 16-byte aligned");
    if (misaligned(bias, 4) || misaligned(residual, cfg->res_f32 ? 4 : 2) || misaligned(y, cfg->y_f32 ? 4 : 2))
        return refuse(MOE_ERR_ALIGN, "bias, residual or y not aligned to its elements");
    // y is written while other tiles still read x and w; a residual element is read
    // by the thread that writes its place in y, and by no other
    const Span sy(y, d->M, d->N, ldy, cfg->y_f32 ? 4 : 2);
    const long long rows = (cfg->act == MOE_ACT_SWIGLU ? 2ll : 1ll) * d->N;
    const bool in_place = residual == y && cfg->res_f32 == cfg->y_f32 && (ldr == ldy || d->M == 1);
    if (overlap(sy, Span(x, d->M, d->K, ldx, 2)) || overlap(sy, Span(w, rows, d->K, ldw, 2)) ||
        (bias && overlap(sy, Span(bias, 1, rows, rows, 4))) ||
        (residual && !in_place && overlap(sy, Span(residual, d->M, d->N, ldr, cfg->res_f32 ? 4 : 2))))
        return refuse(MOE_ERR_UNSUPPORTED, "moe_linear: y overlaps an input (only the residual itself may be y)");
    LinCall c{x, w, ldx, ldw, d->K};
    LinParams p{};
    p.bias = bias;
    p.residual = residual;
    p.y = y;
    p.ldr = ldr;
    p.ldy = ldy;
    p.M = d->M;
    p.N = d->N;
    p.res_f32 = cfg->res_f32;
    p.y_f32 = cfg->y_f32;
    p.limit = cfg->swiglu_limit;
    p.hold = hold;
    p.err = device_info().err_word;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = cfg->act == MOE_ACT_NONE    ? run_linear<MOE_ACT_NONE>(c, p, s)
                          : cfg->act == MOE_ACT_RELU2 ? run_linear<MOE_ACT_RELU2>(c, p, s)
                                                      : run_linear<MOE_ACT_SWIGLU>(c, p, s);
    if (e != cudaSuccess) {
        set_last_error(cudaGetErrorString(e));
        return MOE_ERR_CUDA;
    }
    set_last_launch_count(1);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear(const void* x, const void* w, const float* bias, const void* residual, const moe_linear_dims* d,
                      const moe_linear_cfg* cfg, void* y, moe_stream_t stream) {
    return linear(x, w, bias, residual, d, cfg, y, 0, stream);
}

moe_status moe_linear_expiry_check(const void* x, const void* w, const float* bias, const void* residual,
                                   const moe_linear_dims* d, const moe_linear_cfg* cfg, void* y, uint32_t polls,
                                   moe_stream_t stream) {
    if (polls < 1 || polls > (1u << 20))
        return refuse(MOE_ERR_SHAPE, "moe_linear_expiry_check: polls must be in [1, 2^20]");
    return linear(x, w, bias, residual, d, cfg, y, polls, stream);
}

}  // extern "C"
