// gemm_mxfp4.cu -- grouped products of MXFP4 rows with the MXFP4 matrices of
// their expert:
//   out[r] = A[r] . W_e^T                              (plain)
//   out[r] = silu(A[r] . W1_e^T) (*) (A[r] . W3_e^T)   (pair)
// A [R][K] and W [n][N][K] as codes [..][K/2] and scales [..][K/32] (mxfp4.cu).
//
// A block owns 64 rows x 64 columns (of both matrices for a pair), decodes one
// block of 32 reduction elements at a time into shared memory and multiplies
// in fp32: 256 threads, 4 x 4 outputs each.
#include "ffn.cuh"
#include "kernels.h"

namespace moe {

namespace mxg {
constexpr int kM = 64, kN = 64, kThreads = 256;
struct Smem {
    SegmentPlan plan;
    float a[32][kM + 4];
    float b[2][32][kN + 4];
};
__device__ __forceinline__ float value(uint32_t code) {
    const uint32_t ex = (code >> 1) & 3u, man = code & 1u;
    const float mag = ex == 0u ? 0.5f * man : __uint_as_float(((ex + 126u) << 23) | (man << 22));
    return (code & 8u) ? -mag : mag;
}
__device__ __forceinline__ float scale(uint32_t c) {
    return c == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(c == 0u ? 0x00400000u : c << 23);
}
}  // namespace mxg

using namespace mxg;

template <bool kPair, bool kBf16Out>
__global__ void __launch_bounds__(kThreads) mx_gemm_simt_kernel(const MxGemmArgs g) {
    __shared__ Smem sm;
    load_plan(sm.plan, g.offsets, g.n, g.R, kM, g.status);
    if (static_cast<int>(blockIdx.x) >= sm.plan.blk[g.n]) return;
    const int e = plan_expert(sm.plan, g.n, blockIdx.x);
    const int row0 = sm.plan.off[e] + (static_cast<int>(blockIdx.x) - sm.plan.blk[e]) * kM;
    const int rows = min(kM, sm.plan.off[e + 1] - row0);
    const int col0 = blockIdx.y * kN;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int nb = g.K / 32;
    float acc[kPair ? 2 : 1][4][4] = {};
    for (int kb = 0; kb < nb; ++kb) {
        // 4 threads per row, 4 bytes (8 codes) each
        const int r = tid >> 2, q = tid & 3;
#pragma unroll
        for (int m = 0; m < (kPair ? 3 : 2); ++m) {
            const uint8_t* codes = m == 0 ? g.a_codes : (m == 1 ? g.b_codes : g.b2_codes);
            const uint8_t* scales = m == 0 ? g.a_scales : (m == 1 ? g.b_scales : g.b2_scales);
            const bool in = m == 0 ? r < rows : col0 + r < g.N;
            const int64_t line = m == 0 ? static_cast<int64_t>(row0) + r : static_cast<int64_t>(e) * g.N + col0 + r;
            uint32_t w = 0u;
            float s = 0.f;
            if (in) {
                w = __ldg(reinterpret_cast<const uint32_t*>(codes + (line * nb + kb) * 16) + q);
                s = scale(__ldg(scales + line * nb + kb));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = value((w >> (4 * i)) & 0xFu) * s;
                if (m == 0)
                    sm.a[8 * q + i][r] = v;
                else
                    sm.b[m - 1][8 * q + i][r] = v;
            }
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int p = 0; p < (kPair ? 2 : 1); ++p)
                        acc[p][i][j] = fmaf(sm.a[k][ty * 4 + i], sm.b[p][k][tx * 4 + j], acc[p][i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = col0 + tx * 4 + j;
            if (c >= g.N) continue;
            float v = acc[0][i][j];
            if (kPair) v = v / (1.f + expf(-v)) * acc[kPair ? 1 : 0][i][j];
            const int64_t at = (static_cast<int64_t>(row0) + r) * g.N + c;
            if (kBf16Out)
                static_cast<uint16_t*>(g.out)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
            else
                static_cast<float*>(g.out)[at] = v;
        }
    }
}

cudaError_t launch_mx_gemm(const MxGemmArgs& a, bool bf16_out, int num_sms, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((a.R + kM - 1) / kM + a.n), static_cast<unsigned>((a.N + kN - 1) / kN));
    if (a.b2_codes) {
        if (bf16_out)
            mx_gemm_simt_kernel<true, true><<<grid, kThreads, 0, st>>>(a);
        else
            mx_gemm_simt_kernel<true, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (bf16_out)
            mx_gemm_simt_kernel<false, true><<<grid, kThreads, 0, st>>>(a);
        else
            mx_gemm_simt_kernel<false, false><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace moe
