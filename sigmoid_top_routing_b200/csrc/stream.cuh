// Pieces of the weight-streaming kernels for a few token rows (decode.cu,
// linear_few.cu): bulk copies of weight rows into a ring of shared-memory
// stages, and m16n8k16 products of 16 weight rows with up to 8 NT token columns.
//
// A stage holds a chunk of 16 rows (at most 1 KB of each: 512 k of bf16, 2048
// 4-bit codes).  The row stride is padded so that the lanes of one shared-memory
// load phase fall on distinct banks: bf16 rows are read 16 bytes a lane (a
// phase is 8 lanes: 2 rows x 64 bytes, stride = 64 mod 128), 4-bit rows 8
// bytes a lane (16 lanes: 4 rows x 32 bytes, stride = 32 mod 128).
//
// Within one step (32 k bf16, 64 k 4-bit) lane (g = lane / 4, t = lane % 4)
// holds consecutive k of rows g and g + 8 -- 8 k from k0 + 8 t, or 16 k from
// k0 + 16 t -- and feeds them to the k slots of two (four) MMAs in the order
// they lie in memory; the token operand is read with the same assignment, so
// the sum over k is complete although the slots are permuted.
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

// Sizes of one stage, for `chunk` k per row (a multiple of the step).
struct StageDims {
    int chunk;                                        // k of a row in one stage
    int row_stride;                                   // bytes between rows
    int codes;                                        // kRows * row_stride
    // 4-bit scales: one span per half when a stage holds whole rows (<= 8 rows
    // + 32 bytes per half), else one slot per row (its bytes + 32)
    int slot, area;                                   // bytes of a slot and of one array (affine has two)
    int bytes;                                        // of the whole stage
};

template <int FMT>
struct Fmt {
    static constexpr int kStep = FMT == kBf16 ? 32 : 64;          // k per step
    static constexpr int kRowPad = FMT == kBf16 ? 64 : 32;
    static StageDims dims(int chunk) {
        StageDims d{};
        d.chunk = chunk;
        d.row_stride = (FMT == kBf16 ? chunk * 2 : chunk / 2) + kRowPad;   // row bytes: a multiple of 128
        d.codes = kRows * d.row_stride;
        d.slot = FMT == kBf16 ? 0 : (FMT == kAffine ? chunk / 32 : chunk / 16) + 32;
        d.area = kRows * d.slot;
        d.bytes = d.codes + (FMT == kAffine ? 2 * d.area : d.area);
        return d;
    }
    // token rows in shared memory: stride pad in bytes (see the phases above;
    // 4-bit reads two 16-byte pieces of 32 consecutive bytes per lane)
    static constexpr int kXPad = FMT == kBf16 ? 64 : 16;
    // bytes of k weights of one row, and of their scales (each array)
    static MOE_DEV size_t row_bytes(int k) { return FMT == kBf16 ? (size_t)k * 2 : (size_t)k / 2; }
    static MOE_DEV size_t scale_bytes(int k) { return FMT == kAffine ? (size_t)k / 32 : (size_t)k / 16; }
};

// Untiled bulk copy global -> this CTA's shared memory (16-byte aligned
// addresses and size), completing on `bar`.
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

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

// Affine codes: nibbles j and j + 4 of v as the bf16 pair (128 + q_j, 128 + q_{j+4}), exact.
MOE_DEV uint32_t nib_pair(uint32_t v, int j) { return ((v >> (4 * j)) & 0x000F000Fu) | 0x43004300u; }

// The token operand of affine steps holds, per 8 consecutive k, the pairs
// (j, j + 4): element i of the 8 goes to position 2 (i % 4) + i / 4.
MOE_DEV int affine_pos(int k) { return (k & ~7) | (((k & 3) << 1) | ((k >> 2) & 1)); }

}  // namespace stream
}  // namespace moe
