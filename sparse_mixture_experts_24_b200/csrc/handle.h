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

// A buffer of the workspace.  It grows on demand: what a larger one replaces is
// freed (which waits for the device), unless a captured call used it -- a graph
// may replay with it, so it stays until moe_destroy.
struct FfnBuffer {
    void* p = nullptr;
    int64_t bytes = 0;
    bool captured = false;
};

// Workspace of the feed-forward block and the MXFP4 product.
struct FfnWorkspace {
    FfnBuffer fixed;   // status word, then the tensor maps of the weight gradients; never grows
    FfnBuffer hidden;  // h [rows][F]
    FfnBuffer grads;   // da, db [rows][F]
    FfnBuffer chunks;  // scales of the MXFP4 product, turned over
    std::vector<void*> kept;  // replaced, but used by captured calls
    int* status() const { return static_cast<int*>(fixed.p); }
    void* maps() const { return fixed.p ? static_cast<uint8_t*>(fixed.p) + 256 : nullptr; }
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

// Zeros `bytes` at p, complete on return.  cudaMemset would enqueue them on the legacy
// stream and return: nothing orders that with a caller's non-blocking stream, whose
// kernels may use the memory first and have it wiped behind them.
cudaError_t zero_now(void* p, size_t bytes);
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
