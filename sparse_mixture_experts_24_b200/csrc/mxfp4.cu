// mxfp4.cu -- microscaled 4-bit floating point (MXFP4): E2M1 values with one
// power-of-two scale (E8M0) per 32 consecutive elements of the reduction.
//
// A block of 32 elements v with m = max|v|:
//   scale code  c = clamp(floor(log2 m) - 2 + 127, 0, 254), 0 for m = 0; the
//               scale is 2^(c - 127).  m / 2^(c-127) lies in [4, 8): the largest
//               E2M1 magnitude is 6, its exponent 2.
//   element     E2M1(v / 2^(c-127)), to nearest, ties to even, saturating at 6
//   a block that holds a NaN or an infinity: c = 255 (NaN), all elements 0
// Codes pack element 2j into the low nibble of byte j, 2j+1 into the high one.
// Multiplying by a power of two is exact, so one rounding is made per element.
//
// mx_rows_kernel     blocks along the contiguous axis: the whole array is a
//                    run of blocks, 4 lanes per block (8 elements each), the
//                    maximum over two shuffles.
// mx_weights_kernel  [in][out] matrices with blocks along `in`: a block of
//                    threads takes 128 x 32 inputs, a thread one column of one
//                    block of 32, and turns the tile over in shared memory, so
//                    both the reads along `out` and the writes along `in` are
//                    whole sectors.
// Both are bound by memory: each input is read once, each output written once.
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Scale code of a block from the largest fp32 bit pattern of its magnitudes.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    if (top < 0x00800000u) return 0u;  // zero, or below 2^-126: the smallest scale
    const int c = static_cast<int>(top >> 23) - 2;
    return c < 0 ? 0u : static_cast<uint32_t>(c);
}

// 2^(127 - c) for c in [0, 253]: a normal fp32 number but for c = 253, 2^-126.
__device__ __forceinline__ float mx_inverse_scale(uint32_t c) { return __uint_as_float((254u - c) << 23); }

__device__ __forceinline__ float mx_scale(uint32_t c) {
    return __uint_as_float(c == 0u ? 0x00400000u : c << 23);  // c = 0: 2^-127, a subnormal
}

// E2M1 codes of two values (a in the low four bits) and what two codes stand for
// (exact in fp16).
__device__ __forceinline__ uint32_t mx_codes2(float a, float b) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest));
}
__device__ __forceinline__ float2 mx_values2(uint32_t codes) {
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(codes & 0xFFu), __NV_E2M1);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight elements of a block: codes, and in place the values.
__device__ __forceinline__ uint32_t mx_pack8(float (&v)[8], uint32_t c, bool values) {
    uint32_t packed = 0u;
    if (c != 255u) {
        const float inverse = mx_inverse_scale(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) packed |= mx_codes2(v[2 * i] * inverse, v[2 * i + 1] * inverse) << (8 * i);
    }
    if (values) {
        const float scale = c == 255u ? __uint_as_float(0x7FC00000u) : mx_scale(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 q = mx_values2(packed >> (8 * i));
            v[2 * i] = q.x * scale;
            v[2 * i + 1] = q.y * scale;
        }
    }
    return packed;
}

// kAhead pieces per thread and round, loaded together: one 16-byte load in
// flight per thread does not cover the latency of memory at its bandwidth.
template <bool kBf16, int kAhead>
__global__ void __launch_bounds__(256) mx_rows_kernel(const void* __restrict__ src, int64_t pieces,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                      void* __restrict__ values) {
    // piece = 8 elements; 4 neighbouring lanes hold one block.  `pieces` is a
    // multiple of 4, so a block is never cut by the end of the array.
    const int64_t step = static_cast<int64_t>(gridDim.x) * (256 * kAhead);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kAhead) + threadIdx.x; first - threadIdx.x < pieces;
         first += step) {
        uint4 raw[kAhead][kBf16 ? 1 : 2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t p = first + 256 * u;
#pragma unroll
            for (int h = 0; h < (kBf16 ? 1 : 2); ++h)
                raw[u][h] = p < pieces ? __ldg(static_cast<const uint4*>(src) + (kBf16 ? p : 2 * p + h))
                                       : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t p = first + 256 * u;
            float v[8];
            if (kBf16) {
                const uint4 q = raw[u][0];
                unpack_bf16x2(q.x, v[0], v[1]);
                unpack_bf16x2(q.y, v[2], v[3]);
                unpack_bf16x2(q.z, v[4], v[5]);
                unpack_bf16x2(q.w, v[6], v[7]);
            } else {
#pragma unroll
                for (int h = 0; h < (kBf16 ? 1 : 2); ++h) {
                    const uint4 q = raw[u][h];
                    v[4 * h] = __uint_as_float(q.x), v[4 * h + 1] = __uint_as_float(q.y);
                    v[4 * h + 2] = __uint_as_float(q.z), v[4 * h + 3] = __uint_as_float(q.w);
                }
            }
            uint32_t top = 0u;  // magnitudes order like their bit patterns, NaN and infinity above all
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t c = mx_scale_code(top);
            const uint32_t packed = mx_pack8(v, c, values != nullptr);
            if (p < pieces) {
                reinterpret_cast<uint32_t*>(codes)[p] = packed;
                if ((p & 3) == 0) scales[p >> 2] = static_cast<uint8_t>(c);
                if (values) {
                    if (kBf16) {
                        static_cast<uint4*>(values)[p] = pack_bf16x8(v);
                    } else {
                        static_cast<float4*>(values)[2 * p] = make_float4(v[0], v[1], v[2], v[3]);
                        static_cast<float4*>(values)[2 * p + 1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
        }
    }
}

constexpr int kMxTileK = 128, kMxTileN = 32;

template <bool kBf16>
__global__ void __launch_bounds__(128) mx_weights_kernel(const void* __restrict__ w, int rows, int cols,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                         void* __restrict__ values) {
    __shared__ uint4 s_codes[kMxTileN][kMxTileK / 32];
    __shared__ float s_values[kMxTileN][kMxTileK + 1];
    __shared__ uint8_t s_scales[kMxTileN][kMxTileK / 32];
    const int lane = threadIdx.x & 31, kb = threadIdx.x >> 5;
    const int k0 = blockIdx.x * kMxTileK, c0 = blockIdx.y * kMxTileN;
    const int64_t e = blockIdx.z;
    const int k = k0 + 32 * kb, col = c0 + lane;
    const int64_t base = (e * rows + k) * cols + col;
    const bool in = k < rows && col < cols;
    float v[32];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (!in)
            v[i] = 0.f;
        else if (kBf16)
            v[i] = bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(w) + base + static_cast<int64_t>(i) * cols));
        else
            v[i] = __ldg(static_cast<const float*>(w) + base + static_cast<int64_t>(i) * cols);
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    const uint32_t c = mx_scale_code(top);
    uint32_t packed[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = v[8 * q + i];
        packed[q] = mx_pack8(u, c, values != nullptr);
        if (values) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s_values[lane][32 * kb + 8 * q + i] = u[i];
        }
    }
    s_codes[lane][kb] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    s_scales[lane][kb] = static_cast<uint8_t>(c);
    __syncthreads();
    const int blocks = min(kMxTileK, rows - k0) / 32;  // `rows` is a multiple of 32
    {
        const int n = threadIdx.x >> 2, b = threadIdx.x & 3;
        if (c0 + n < cols && b < blocks) {
            const int64_t at = (e * cols + c0 + n) * (rows / 32) + k0 / 32 + b;
            reinterpret_cast<uint4*>(codes)[at] = s_codes[n][b];
            scales[at] = s_scales[n][b];
        }
    }
    if (values) {
        for (int i = threadIdx.x; i < kMxTileN * kMxTileK / 2; i += 128) {
            const int n = i / (kMxTileK / 2), kk = 2 * (i % (kMxTileK / 2));
            if (c0 + n >= cols || kk >= 32 * blocks) continue;
            const int64_t at = (e * cols + c0 + n) * rows + k0 + kk;
            const float a = s_values[n][kk], b = s_values[n][kk + 1];
            if (kBf16)
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(values) + at) = pack_bf16x2(a, b);
            else
                *reinterpret_cast<float2*>(static_cast<float*>(values) + at) = make_float2(a, b);
        }
    }
}

cudaError_t launch_mx_rows(const void* src, bool bf16, int64_t rows, int cols, uint8_t* codes, uint8_t* scales,
                           void* values, int num_sms, cudaStream_t st) {
    const int64_t pieces = rows * (cols / 8);
    // four pieces per thread once that still fills every SM with blocks
    const bool many = pieces >= static_cast<int64_t>(num_sms) * 8 * 256 * 4;
    const int64_t per = many ? 256 * 4 : 256;
    const int64_t blocks = std::min<int64_t>((pieces + per - 1) / per, static_cast<int64_t>(num_sms) * 32);
    auto kernel = bf16 ? (many ? mx_rows_kernel<true, 4> : mx_rows_kernel<true, 1>)
                       : (many ? mx_rows_kernel<false, 4> : mx_rows_kernel<false, 1>);
    kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(src, pieces, codes, scales, values);
    return cudaGetLastError();
}

cudaError_t launch_mx_weights(const void* w, bool bf16, int n, int rows, int cols, uint8_t* codes, uint8_t* scales,
                              void* values, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((rows + kMxTileK - 1) / kMxTileK),
                    static_cast<unsigned>((cols + kMxTileN - 1) / kMxTileN), static_cast<unsigned>(n));
    if (bf16)
        mx_weights_kernel<true><<<grid, 128, 0, st>>>(w, rows, cols, codes, scales, values);
    else
        mx_weights_kernel<false><<<grid, 128, 0, st>>>(w, rows, cols, codes, scales, values);
    return cudaGetLastError();
}

}  // namespace moe
