// Tensor maps of row-major rows of bytes, cut into 128-byte chunks, for TMA
// boxes of several rows and chunks in the 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// `rows` rows of `row_bytes` bytes, `stride` bytes apart (a multiple of 16).
// Whole chunks (row_bytes % 128 == 0): *flat = false and the map is 3D, (byte in
// chunk, row, chunk) with boxes of (128, box_rows, box_chunks), so one load
// brings several chunks, each as box_rows x 128 bytes.  Else *flat = true and
// the map is 2D, (byte in row, row) with boxes of (128, box_rows), zero-filled
// past the row's end.  cudaErrorNotSupported without the driver entry point,
// cudaErrorInvalidValue when the driver rejects the description.
cudaError_t make_tmap_rows(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t stride, uint64_t rows,
                           uint32_t box_rows, uint32_t box_chunks, bool* flat);

// 2D map of the same rows for boxes of 8 rows x box_bytes (64 or 128) bytes in
// the swizzle of that width; row_bytes and stride are multiples of 16.
cudaError_t make_tmap_narrow(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_bytes);

}  // namespace moe
