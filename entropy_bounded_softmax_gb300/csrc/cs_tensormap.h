// Host side of tensor copies: the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <string.h>

#include "cs_internal.h"

namespace cs {

// cuTensorMapEncodeTiled, from the CUDA driver through the runtime (no link
// against the driver library); null if unavailable.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A map of four dimensions of 16-bit elements with 128-byte swizzling; elements
// outside the tensor read as zeros.
inline bool encode_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* data,
                       CUtensorMapDataType type, const cuuint64_t* dim, const cuuint64_t* bytes,
                       const cuuint32_t* box, const cuuint32_t* step) {
    auto encode = [&] {
        return enc(map, type, 4, const_cast<void*>(data), dim, bytes, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // The encoder is a driver call, which wants the thread's context bound;
    // the runtime binds it with the first call that needs it, and on a thread
    // of its own (autograd's) none may have come yet.  Setting the device that
    // is set binds it.
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// The map of a [B, heads, length, D] bf16 tensor (element strides of its first
// three dimensions in stride, the head dimension contiguous), copied in boxes
// of 64 head elements x box_rows rows with 128-byte swizzling; elements outside
// the tensor read as zeros.  A dimension of one element has no stride that
// matters, and gets one the encoder takes.  A tensor without elements gets an
// all-zero map, which no kernel uses.
inline bool encode_heads_map(CUtensorMap* map, const void* data, const FattnTask& t,
                             int heads, int length, const int64_t* stride, int box_rows) {
    memset(map, 0, sizeof(*map));
    if (length == 0) return true;
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dim[4] = {static_cast<cuuint64_t>(t.d_head),
                               static_cast<cuuint64_t>(length),
                               static_cast<cuuint64_t>(heads),
                               static_cast<cuuint64_t>(t.batch)};
    cuuint64_t bytes[3];
    for (int i = 0; i < 3; ++i)   // length, heads, batch
        bytes[i] = dim[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(stride[2 - i]) * 2;
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode_map(enc, map, data, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dim, bytes, box, step);
}

// The map of a cache's pages, [num_pages, page_size, kv_heads, D] 16-bit
// elements (strides of its first three dimensions, all of which are there), in
// boxes of 64 head elements of one head x box_rows slots of a page, swizzled as
// above; pages outside the cache read as zeros.  False, too, where the strides
// are none that tensor copies take.
inline bool encode_pages_map(CUtensorMap* map, const void* data, const TreeTask& t,
                             const int64_t* stride, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dim[4] = {static_cast<cuuint64_t>(t.d_head),
                               static_cast<cuuint64_t>(t.kv_heads),
                               static_cast<cuuint64_t>(t.page_size),
                               static_cast<cuuint64_t>(t.num_pages)};
    cuuint64_t bytes[3];
    for (int i = 0; i < 3; ++i) {   // head, slot, page
        bytes[i] = dim[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(stride[2 - i]) * 2;
        if (bytes[i] == 0 || bytes[i] >> 40) return false;
    }
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode_map(enc, map, data,
                      t.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      dim, bytes, box, step);
}

// The map of the queries of those pages' call, in boxes of 64 elements of the
// heads of one key head x as many tokens as make 128 rows; tokens past the last
// read as zeros.  False where they make none, or the strides are none that
// tensor copies take.
inline bool encode_queries_map(CUtensorMap* map, const TreeTask& t) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc || 128 % t.group != 0) return false;
    const cuuint64_t dim[4] = {static_cast<cuuint64_t>(t.d_head),
                               static_cast<cuuint64_t>(t.heads),
                               static_cast<cuuint64_t>(t.new_tokens),
                               static_cast<cuuint64_t>(t.batch)};
    cuuint64_t bytes[3];
    for (int i = 0; i < 3; ++i) {   // head, token, sequence
        bytes[i] = dim[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(t.q_stride[2 - i]) * 2;
        if (bytes[i] == 0 || bytes[i] >> 40) return false;
    }
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(t.group),
                               static_cast<cuuint32_t>(128 / t.group), 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode_map(enc, map, t.q,
                      t.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      dim, bytes, box, step);
}

}  // namespace cs
