// Pieces of the weight-streaming kernels for a few token rows: TMA boxes of
// weight rows in a ring of shared-memory stages, and m16n8k16 products of 16
// weight rows with up to 8 NT token columns.
//
// Weights.  A stage holds two halves of 8 rows (SwiGLU: 8 gate and 8 up rows),
// each as `chunks` blocks of 8 rows x 128 bytes with the 128-byte swizzle, as a
// box of the tensor (128 bytes, rows, row bytes / 128) lands.  One TMA per half
// brings a whole stage; copies of single rows measured ~40 cycles each, too
// slow for rows of 1 KB and less.  A box always has 8 rows: where a unit has
// fewer, the others belong to a neighbouring CTA that loads them anyway, so
// they come from L2 and are ignored.
//
// Operands.  In one step (64 k) lane (g = lane / 4, t = lane % 4) reads k of
// row sigma(g) of both halves -- bf16: two runs of 8 k, 4-bit: one run of 16 --
// and feeds them to the k slots of four MMAs in the order they lie in memory;
// the token operand is read with the same assignment, so the sum over k is
// complete although the slots are permuted.  sigma orders the 8 rows so that
// the lanes of one shared-memory phase fall on distinct banks under the swizzle:
// bf16 reads 16 bytes a lane (2 rows x 4 lanes a phase: rows r and r + 4),
// 4-bit 8 bytes a lane (4 rows x 4 lanes: rows of equal parity).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace moe {
namespace stream {

using namespace sm100;

enum { kBf16 = 0, kAffine = 1, kNvfp4 = 2 };          // the library's weight format codes

constexpr int kRows = 16;                             // weight rows of a stage (the MMA's M)
constexpr int kStep = 64;                             // k per step
constexpr int kSpanMaxK = 2048;                       // 4-bit: longest row whose scales come as one span per half

// Layout of one stage for `chunks` 128-byte chunks of each row.
struct StageDims {
    int chunks, k;                                    // chunks and k of a row in one stage
    int half;                                         // bytes of a half's codes
    int area;                                         // 4-bit: bytes of one scale array (affine has two): a box or
                                                      // span per half at area / 2, or 16 row slots of area / 16
    int scales, tokens;                               // byte offsets of the scales and of the token rows
    int bytes;
};

template <int FMT>
struct Fmt {
    static constexpr int kChunkK = FMT == kBf16 ? 64 : 256;            // k of 128 bytes
    // Pad of token rows in shared memory (stride = 2 k + pad): bf16 reads 16 of
    // 64 consecutive bytes per lane, 4-bit two 16-byte pieces of 128.
    static constexpr int kXPad = FMT == kBf16 ? 64 : 16;
    static MOE_DEV __host__ int sigma(int g) { return FMT == kBf16 ? (g >> 1) | ((g & 1) << 2) : ((g & 3) << 1) | (g >> 2); }
    // bytes of the scales of k weights (each array)
    static MOE_DEV __host__ size_t scale_bytes(int k) { return FMT == kAffine ? (size_t)k / 32 : (size_t)k / 16; }
    // Scales of a stage arrive as one box per half (8 rows x 128 bytes NVFP4, 64
    // affine) in the swizzle of that width where their rows are whole 16-byte units
    // and a stage starts on one: the 8 rows of a load phase then fall on distinct
    // banks (as plain spans, rows of 64 or 128 bytes cost 4 or 8 wavefronts a load).
    static constexpr int kScaleBox = FMT == kAffine ? 64 : 128;
    static bool boxed(int chunks, int K) {
        if (K == 0) return false;
        return FMT == kNvfp4 ? K % 256 == 0 : FMT == kAffine && K % 512 == 0 && chunks % 2 == 0;
    }
    // Long unboxed rows: the scales of each of the 16 rows in a slot of its own.
    static bool row_slots(int chunks, int K) { return FMT != kBf16 && K > kSpanMaxK && !boxed(chunks, K); }
    // Bytes of one scale array of a stage, for rows of length K.
    static int scale_area(int chunks, int K) {
        if (FMT == kBf16 || K == 0) return 0;
        if (boxed(chunks, K)) return 2 * 8 * kScaleBox;
        if (K <= kSpanMaxK) return 2 * (int)((8 * scale_bytes(K) + 32 + 15) & ~size_t(15));
        return kRows * (int)((scale_bytes(chunks * kChunkK) + 32 + 15) & ~size_t(15));
    }
    // A stage for rows of length K1 or K2 with `cols` token rows behind the weights.
    static StageDims dims(int chunks, int K1, int K2, int cols) {
        StageDims d{};
        d.chunks = chunks;
        d.k = chunks * kChunkK;
        d.half = chunks * 1024;
        d.scales = 2 * d.half;
        const int a1 = scale_area(chunks, K1), a2 = scale_area(chunks, K2);
        d.area = a1 > a2 ? a1 : a2;
        // the larger area may be the other matrix's: 16 row slots still start on 16 bytes
        if (row_slots(chunks, K1) || row_slots(chunks, K2)) d.area = (d.area + 255) & ~255;
        // both halves' boxes (area / 2 apart) start on a swizzle period, 8 box rows
        if (boxed(chunks, K1) || boxed(chunks, K2)) d.area = (d.area + 16 * kScaleBox - 1) & ~(16 * kScaleBox - 1);
        d.tokens = d.scales + (FMT == kAffine ? 2 * d.area : d.area);
        d.bytes = (d.tokens + cols * (d.k * 2 + kXPad) + 1023) & ~1023;
        return d;
    }
};

// Box (128 bytes, 8 rows, chunks) at (0, row, chunk).
MOE_DEV void tma_load_3d(uint32_t dst, const CUtensorMap* m, int row, int chunk, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(row), "r"(chunk), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Box (128 bytes, 8 rows) of a 2D map whose rows are not whole chunks.
MOE_DEV void tma_load_rows(uint32_t dst, const CUtensorMap* m, int x, int row, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(row), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Untiled bulk copy global -> this CTA's shared memory (16-byte aligned
// addresses and size), completing on `bar`.
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Orders this thread's generic-proxy accesses with later async-proxy
// accesses, and the other way round.
MOE_DEV void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

MOE_DEV uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
MOE_DEV uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
MOE_DEV uint32_t lds_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
MOE_DEV uint32_t lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

MOE_DEV void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (v & m) | o in one instruction with both constants in registers (written as
// an expression, the two constants became two instructions: an affine f16 step
// took 475 instead of 360 cycles at 16 warps).
MOE_DEV uint32_t and_or(uint32_t v, uint32_t m, uint32_t o) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(m), "r"(o));
    return r;
}
// Affine codes: nibbles j and j + 4 of v as the bf16 pair (128 + q_j, 128 + q_{j+4}), exact.
MOE_DEV uint32_t nib_pair(uint32_t v, int j) { return and_or(v >> (4 * j), 0x000F000Fu, 0x43004300u); }

// e2m1 codes (nibbles j and j + 4 of w, j = 0..3) times a block scale, as bf16
// pairs.  A code's exponent and mantissa bits at bits 8..6 of a bf16 are its
// magnitude times 2^-126 (subnormals included); the scale comes times 2^118,
// so the exact product carries 2^-8.
MOE_DEV void e2m1_pairs(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
    constexpr uint32_t S = 0x80008000u, M = 0x01C001C0u;
    o[0] = ((w & 0x000F000Fu) * 0x1040u) & (S | M);
    o[1] = ((w << 8) & S) | ((w << 2) & M);
    o[2] = ((w << 4) & S) | ((w >> 2) & M);
    o[3] = (w & S) | ((w >> 6) & M);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 r =
            __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o[i]), *reinterpret_cast<const __nv_bfloat162*>(&scale));
        o[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
}
// An e4m3 byte times 2^118 as an equal bf16 pair (exact: at most 448 * 2^118; NaN stays NaN).
MOE_DEV uint32_t e4m3_to_bf16x2_118(uint32_t b) {
    const uint32_t h = e4m3x2_to_f16x2(b);
    const float f = __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu))) * 0x1p118f;
    return __float_as_uint(f) >> 16 | (__float_as_uint(f) & 0xFFFF0000u);
}

// The token operand of bf16 4-bit steps (and of affine f16 ones) holds, per 8
// consecutive k, the pairs (j, j + 4): element i of the 8 goes to position 2 (i % 4) + i / 4.
MOE_DEV int pair_pos(int k) { return (k & ~7) | (((k & 3) << 1) | ((k >> 2) & 1)); }

// The products of steps [s, s + n) of a stage, token operand in bf16.  w: this lane's row of half 0
// (stage + sigma 128), half 1 at + half; x4: the lane's 16-byte unit, XORed by
// the row; sc0, sc1: the scale rows of its two rows, read at byte sb ^ sx (sb: this
// step's, sx: the swizzle's term of the row); xb: this lane's k of its column, per block of 8 tokens, at the first step.
template <int FMT, int NT>
MOE_DEV void run_steps(uint32_t w, uint32_t half, uint32_t x4, int s, int n, uint32_t sc0, uint32_t sc1, uint32_t sb, uint32_t sx, uint32_t area,
                       uint32_t (&xb)[NT], int ntn, float (&acc)[NT][4]) {
    if constexpr (FMT == kBf16) {
        w += s * 1024;
#pragma unroll 2
        for (; n > 0; --n, w += 1024) {
            const uint4 p0 = lds128(w + x4), q0 = lds128(w + half + x4);
            const uint4 p1 = lds128(w + (x4 ^ 64)), q1 = lds128(w + half + (x4 ^ 64));
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    const uint4 x = lds128(xb[i]), y = lds128(xb[i] + 64);
                    xb[i] += 128;
                    mma_bf16(acc[i], p0.x, q0.x, p0.y, q0.y, x.x, x.y);
                    mma_bf16(acc[i], p0.z, q0.z, p0.w, q0.w, x.z, x.w);
                    mma_bf16(acc[i], p1.x, q1.x, p1.y, q1.y, y.x, y.y);
                    mma_bf16(acc[i], p1.z, q1.z, p1.w, q1.w, y.z, y.w);
                }
        }
    } else if constexpr (FMT == kAffine) {
        // sum_k w x = s sum_k (128 + q) x + (b - 128 s) sum_k x over the step,
        // which is one group of 64; sum_k x by MMAs against ones
#pragma unroll 1
        for (; n > 0; --n, ++s, sb += 2) {
            const uint32_t a = w + ((s & ~3) << 8) + (((s << 5) & 0x60) ^ x4);
            const uint2 p = lds64(a), q = lds64(a + half);
            const uint32_t o0 = sc0 + (sb ^ sx), o1 = sc1 + (sb ^ sx);
            const float s0 = bf16f(lds_u16(o0)), s1 = bf16f(lds_u16(o1));
            const float b0 = fmaf(-128.0f, s0, bf16f(lds_u16(o0 + area)));
            const float b1 = fmaf(-128.0f, s1, bf16f(lds_u16(o1 + area)));
            constexpr uint32_t one = 0x3F803F80u;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    const uint4 u = lds128(xb[i]), v = lds128(xb[i] + 16);
                    xb[i] += 128;
                    float c[4] = {}, x[4] = {};
                    mma_bf16(x, one, one, one, one, u.x, u.y);
                    mma_bf16(c, nib_pair(p.x, 0), nib_pair(q.x, 0), nib_pair(p.x, 1), nib_pair(q.x, 1), u.x, u.y);
                    mma_bf16(x, one, one, one, one, u.z, u.w);
                    mma_bf16(c, nib_pair(p.x, 2), nib_pair(q.x, 2), nib_pair(p.x, 3), nib_pair(q.x, 3), u.z, u.w);
                    mma_bf16(x, one, one, one, one, v.x, v.y);
                    mma_bf16(c, nib_pair(p.y, 0), nib_pair(q.y, 0), nib_pair(p.y, 1), nib_pair(q.y, 1), v.x, v.y);
                    mma_bf16(x, one, one, one, one, v.z, v.w);
                    mma_bf16(c, nib_pair(p.y, 2), nib_pair(q.y, 2), nib_pair(p.y, 3), nib_pair(q.y, 3), v.z, v.w);
                    acc[i][0] = fmaf(s0, c[0], fmaf(b0, x[0], acc[i][0]));
                    acc[i][1] = fmaf(s0, c[1], fmaf(b0, x[1], acc[i][1]));
                    acc[i][2] = fmaf(s1, c[2], fmaf(b1, x[0], acc[i][2]));
                    acc[i][3] = fmaf(s1, c[3], fmaf(b1, x[1], acc[i][3]));
                }
        }
    } else {
        // a lane's 16 k are one scale block: e2m1 * e4m3 exactly in bf16, times 2^-8
#pragma unroll 1
        for (; n > 0; --n, ++s, sb += 4) {
            const uint32_t a = w + ((s & ~3) << 8) + (((s << 5) & 0x60) ^ x4);
            const uint2 p = lds64(a), q = lds64(a + half);
            const uint32_t s0 = e4m3_to_bf16x2_118(lds_u8(sc0 + (sb ^ sx))), s1 = e4m3_to_bf16x2_118(lds_u8(sc1 + (sb ^ sx)));
            uint4 u[NT], v[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    u[i] = lds128(xb[i]);
                    v[i] = lds128(xb[i] + 16);
                    xb[i] += 128;
                }
            uint32_t f[4], h[4];
            e2m1_pairs(p.x, s0, f);
            e2m1_pairs(q.x, s1, h);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    mma_bf16(acc[i], f[0], h[0], f[1], h[1], u[i].x, u[i].y);
                    mma_bf16(acc[i], f[2], h[2], f[3], h[3], u[i].z, u[i].w);
                }
            e2m1_pairs(p.y, s0, f);
            e2m1_pairs(q.y, s1, h);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    mma_bf16(acc[i], f[0], h[0], f[1], h[1], v[i].x, v[i].y);
                    mma_bf16(acc[i], f[2], h[2], f[3], h[3], v[i].z, v[i].w);
                }
        }
    }
}

MOE_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 4-bit steps with the token operand in f16 (x after a power-of-two scale per
// token).  A step costs 75-90 issue cycles per warp instead of ~135 with bf16:
// integer and shift instructions issue at half rate, and f16 needs fewer.
//   NVFP4   the e2m1 pairs and block scales convert by instruction, their f16
//           product is exact; x in natural order.
//   affine  in f16, 1024 + q and 1024 + 16 q are exact for a nibble at bits 0-3
//           and 4-7 of a half: two pairs of codes per shift.  The second kind meets
//           x / 16, and the products start at minus their constant part:
//             sum_k q x = sum (1024 + q) x + sum (1024 + 16 q) (x / 16) - O,
//           O = 1024 (sum x + sum x / 16) over the respective k, from a table of
//           (O, sum x) per group of 64 and token.  O is up to ~100 times the
//           result, so a group's sum is good to ~1e-5 of itself: far inside the
//           bf16 rounding of the activations.
// tab: this lane's columns 2t and 2t + 1 of each block of 8 in the table at the
// first step; tstep: bytes from one group to the next.
template <int FMT, int NT>
MOE_DEV void run_steps_f16(uint32_t w, uint32_t half, uint32_t x4, int s, int n, uint32_t sc0, uint32_t sc1, uint32_t sb, uint32_t sx, uint32_t area,
                           uint32_t (&xb)[NT], uint32_t (&tab)[NT][2], uint32_t tstep, int ntn, float (&acc)[NT][4]) {
    if constexpr (FMT == kNvfp4) {
#pragma unroll 2
        for (; n > 0; --n, ++s, sb += 4) {
            const uint32_t a = w + ((s & ~3) << 8) + (((s << 5) & 0x60) ^ x4);
            const uint2 p = lds64(a), q = lds64(a + half);
            const uint32_t s0 = e4m3x2_to_f16x2(lds_u8(sc0 + (sb ^ sx)) * 0x0101u),
                           s1 = e4m3x2_to_f16x2(lds_u8(sc1 + (sb ^ sx)) * 0x0101u);
            uint32_t f[2][4], h[2][4];
            e2m1x8_to_f16(p.x, f[0]);
            e2m1x8_to_f16(q.x, h[0]);
            e2m1x8_to_f16(p.y, f[1]);
            e2m1x8_to_f16(q.y, h[1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j >> 2][j & 3] = hmul2_u32(f[j >> 2][j & 3], s0);
                h[j >> 2][j & 3] = hmul2_u32(h[j >> 2][j & 3], s1);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    const uint4 u = lds128(xb[i]), v = lds128(xb[i] + 16);
                    xb[i] += 128;
                    mma_f16(acc[i], f[0][0], h[0][0], f[0][1], h[0][1], u.x, u.y);
                    mma_f16(acc[i], f[0][2], h[0][2], f[0][3], h[0][3], u.z, u.w);
                    mma_f16(acc[i], f[1][0], h[1][0], f[1][1], h[1][1], v.x, v.y);
                    mma_f16(acc[i], f[1][2], h[1][2], f[1][3], h[1][3], v.z, v.w);
                }
        }
    } else {
        const auto lo = [](uint32_t v) { return and_or(v, 0x000F000Fu, 0x64006400u); };
        const auto hi = [](uint32_t v) { return and_or(v, 0x00F000F0u, 0x64006400u); };
        // (unrolled twice the loop is slower: 1 token, 4 of 64 experts of 2048 x 1536,
        // 21.9 us to 20.9; NVFP4's is faster, 5 tokens 44.9 us to 45.3)
#pragma unroll 1
        for (; n > 0; --n, ++s, sb += 2) {
            const uint32_t a = w + ((s & ~3) << 8) + (((s << 5) & 0x60) ^ x4);
            const uint2 p = lds64(a), q = lds64(a + half);
            const uint32_t o0 = sc0 + (sb ^ sx), o1 = sc1 + (sb ^ sx);
            const float s0 = bf16f(lds_u16(o0)), s1 = bf16f(lds_u16(o1));
            const float b0 = bf16f(lds_u16(o0 + area)), b1 = bf16f(lds_u16(o1 + area));
            const uint32_t px = p.x >> 8, qx = q.x >> 8, py = p.y >> 8, qy = q.y >> 8;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == 0 || i < ntn) {
                    const uint4 u = lds128(xb[i]), v = lds128(xb[i] + 16);
                    const uint2 t0 = lds64(tab[i][0]), t1 = lds64(tab[i][1]);   // (O, sum x) of the two columns
                    xb[i] += 128;
                    tab[i][0] += tstep;
                    tab[i][1] += tstep;
                    float c[4];
                    c[0] = c[2] = -__uint_as_float(t0.x);
                    c[1] = c[3] = -__uint_as_float(t1.x);
                    mma_f16(c, lo(p.x), lo(q.x), hi(p.x), hi(q.x), u.x, u.y);
                    mma_f16(c, lo(px), lo(qx), hi(px), hi(qx), u.z, u.w);
                    mma_f16(c, lo(p.y), lo(q.y), hi(p.y), hi(q.y), v.x, v.y);
                    mma_f16(c, lo(py), lo(qy), hi(py), hi(qy), v.z, v.w);
                    const float x0 = __uint_as_float(t0.y), x1 = __uint_as_float(t1.y);
                    acc[i][0] = fmaf(s0, c[0], fmaf(b0, x0, acc[i][0]));
                    acc[i][1] = fmaf(s0, c[1], fmaf(b0, x1, acc[i][1]));
                    acc[i][2] = fmaf(s1, c[2], fmaf(b1, x0, acc[i][2]));
                    acc[i][3] = fmaf(s1, c[3], fmaf(b1, x1, acc[i][3]));
                }
        }
    }
}

MOE_DEV uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace stream
}  // namespace moe
