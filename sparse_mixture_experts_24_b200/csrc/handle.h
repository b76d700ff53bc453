// handle.h -- the part of a moe_handle that the feed-forward block and the
// MXFP4 product (ffn_api.cu) use; moe_api.cu owns the handle and its forward
// workspace.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/moe.h"

namespace moe {

// Workspace of the feed-forward block.  Buffers grow, but a buffer that a
// larger one replaces stays allocated until moe_destroy: kernels in flight and
// captured graphs may still use it.  The status word never moves.
struct FfnWorkspace {
    int* status = nullptr;
    void* maps = nullptr;      // device tensor maps of the weight gradients
    void* h = nullptr;         // [rows][F]
    int64_t h_rows = 0;
    void* da = nullptr;        // [grad_rows][F]
    void* db = nullptr;
    int64_t grad_rows = 0;
    void* chunks = nullptr;    // scales of the MXFP4 product, turned over
    int64_t chunk_bytes = 0;
    std::vector<void*> allocations;
};

}  // namespace moe

namespace moe_api_detail {

struct HandleView {
    int n, d, F;
    bool bf16;
    int num_sms;
    int64_t* launches;
    moe::FfnWorkspace* ffn;
};

// Checks the device as every call does and describes the handle.
moe_status open_handle(moe_handle* h, HandleView* v);
// bf16 tensor map with 128-byte swizzle: dims and box from the contiguous axis
// outwards, strides of the axes after the first in bytes.
bool encode_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                 const uint32_t* box);
// The same with 64-byte swizzle, for bf16 and fp32.
bool encode_bf16_64(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box);
bool encode_f32_64(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                   const uint32_t* box);
// Unswizzled, for 32-bit words.
bool encode_words(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                  const uint32_t* box);
// 128-byte swizzle, for bytes.
bool encode_bytes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                  const uint32_t* box);
moe_status failed(moe_status s, const char* fmt, ...);  // sets moe_last_error()
moe_status done();

}  // namespace moe_api_detail
