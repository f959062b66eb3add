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
    auto encode = [&] {
        return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(data), dim, bytes,
                   box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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

}  // namespace cs
