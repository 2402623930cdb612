// Tensor maps: the driver's encoder and plain 2D maps (tmap.h), row-major weight rows as
// 128-byte chunks (tmap_rows.h).
#include "tmap_rows.h"

#include "tmap.h"

#include <mutex>

namespace moe {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

}  // namespace

cudaError_t encode_tiled(CUtensorMap* m, CUtensorMapDataType dtype, uint32_t rank, const void* base,
                         const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                         CUtensorMapSwizzle swizzle) {
    EncodeFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    static constexpr cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    auto go = [&] {
        return enc(m, dtype, rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = go();
    if (r != CUDA_SUCCESS) {
        // a driver call, unlike the runtime's, does not make the device's context
        // current: a new thread whose first call this is has none
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = go();
    }
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_tmap_2d(CUtensorMap* m, CUtensorMapDataType dtype, uint32_t elem_bytes, const void* base,
                         uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows, bool swizzle128) {
    const cuuint64_t dims[2] = {inner, rows}, strides[1] = {inner * elem_bytes};
    const cuuint32_t box[2] = {box_inner, box_rows};
    return encode_tiled(m, dtype, 2, base, dims, strides, box,
                        swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

cudaError_t make_tmap_rows(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t stride, uint64_t rows,
                           uint32_t box_rows, uint32_t box_chunks, bool* flat) {
    *flat = row_bytes % 128 != 0;
    const cuuint64_t dims3[3] = {128, rows, row_bytes / 128}, dims2[2] = {row_bytes, rows};
    const cuuint64_t strides[2] = {stride, 128};
    const cuuint32_t box[3] = {128, box_rows, box_chunks};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, *flat ? 2 : 3, base, *flat ? dims2 : dims3, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t make_tmap_narrow(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_bytes) {
    const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {row_bytes};
    const cuuint32_t box[2] = {box_bytes, 8};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                        box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace moe
