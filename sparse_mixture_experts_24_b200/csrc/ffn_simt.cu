// ffn_simt.cu -- the gated feed-forward block over expert segments, forward
// and backward, in fp32 on the CUDA cores (tensor cores have no fp32 x fp32
// kind that keeps full fp32 products).
//
// Five products share one kernel (ffn.cuh has the formulas):
//   kFfnUp    [a | b] = x . [w1 | w3] -> h (and a, b when they are kept)
//   kFfnDown  y = h . w2
//   kFfnGrad  dh = dy . w2^T -> da, db and h from a, b
//   kFfnDx    dx = da . w1^T + db . w3^T (one sum over both)
//   kFfnDw    [dw1 | dw3] = x^T . [da | db] and dw2 = h^T . dy, all in one launch
//
// A block owns 64 x 128 outputs, 128 threads hold 8 x 8 each: per reduction
// step a thread reads 16 values from shared memory for 64 multiply-adds.  The
// 128 columns are two halves of 64 (thread columns 4 tx .. 4 tx + 3 of either),
// so that the pairs a, b and da, db of one hidden column meet in one thread.
// The reduction runs in chunks of 16 through three shared-memory buffers, the
// next two chunks' asynchronous copies in flight while one is multiplied.
// One warp per scheduler issues a multiply-add every other cycle at best, and
// small batches have fewer tiles than SMs: a row product is then split along
// its reduction over a cluster of up to 8 blocks, whose partial sums meet in
// distributed shared memory and are added in rank order.
#include <algorithm>
#include <cstddef>

#include "ffn.cuh"
#include "kernels.h"

namespace moe {

namespace ffn_simt {

constexpr int kM = 64, kN = 128, kK = 16, kThreads = 128;
constexpr int kBuffers = 3;

__device__ __forceinline__ const float* at(const void* p, int64_t i) { return static_cast<const float*>(p) + i; }

// Asynchronous copies into shared memory; zeros instead where `in` is false (the
// source is not read then).
__device__ __forceinline__ void copy4(float* dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
}
// Two fp32 multiply-adds in one instruction, each rounded as fmaf: the loop is
// bound by issue slots, and this halves them.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

__device__ __forceinline__ void store4(void* p, int64_t i, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
}

struct Tiles {
    float a[kBuffers][kK][kM + 4];  // rows of both arrays stay 16-byte aligned: they are read as float4
    float b[kBuffers][kK][kN + 4];
};
struct __align__(16) Smem {
    union {
        Tiles t;
        float part[64][kThreads];  // a split reduction's accumulators: [value of the thread][thread]
    };
    SegmentPlan plan;
};
static_assert((kM + 4) % 4 == 0 && (kN + 4) % 4 == 0 && offsetof(Tiles, b) % 16 == 0, "float4 alignment");

}  // namespace ffn_simt

using namespace ffn_simt;

template <int kOp>
__global__ void __launch_bounds__(kThreads, kOp == kFfnGrad || kOp == kFfnDx ? 4 : 3)
    ffn_simt_kernel(const FfnArgs g, const int splits) {
    griddep_wait();
    __shared__ Smem sm;
    load_plan(sm.plan, g.offsets, g.n, g.R, kM, g.status);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int d = g.d, F = g.F;

    // the tile: expert, first output row (row ops: a row of the batch) and the
    // rows inside it, the column half starts, and the reduction
    int e, row0, rows, col[2];
    int64_t K;
    bool dw2 = false;
    if (kOp == kFfnDw) {
        e = blockIdx.y;
        const int t13 = (d / kM) * (F / 64), t = blockIdx.x;
        dw2 = t >= t13;
        const int nc = dw2 ? (d + kN - 1) / kN : F / 64;
        const int local = dw2 ? t - t13 : t;
        row0 = (local / nc) * kM;
        rows = kM;
        const int c = local % nc;
        col[0] = dw2 ? c * kN : c * 64;
        col[1] = dw2 ? c * kN + 64 : c * 64;
        K = sm.plan.off[e + 1] - sm.plan.off[e];
    } else {
        // x: row block and, fastest, the split of its reduction (one cluster)
        const int b = static_cast<int>(blockIdx.x) / splits;
        if (b >= sm.plan.blk[g.n]) return;
        e = plan_expert(sm.plan, g.n, b);
        row0 = sm.plan.off[e] + (b - sm.plan.blk[e]) * kM;
        rows = min(kM, sm.plan.off[e + 1] - row0);
        const int c = blockIdx.y;
        col[0] = kOp == kFfnUp ? c * 64 : c * kN;
        col[1] = kOp == kFfnUp ? c * 64 : c * kN + 64;
        K = kOp == kFfnUp || kOp == kFfnGrad ? d : (kOp == kFfnDown ? F : 2 * F);
    }
    const int cols = kOp == kFfnUp || kOp == kFfnGrad ? F : (kOp == kFfnDw && !dw2 ? F : d);
    const int64_t w_at = static_cast<int64_t>(e) * d * F;
    const int64_t seg0 = kOp == kFfnDw ? sm.plan.off[e] : 0;

    // Copies of chunk c (16 of the reduction) into buffer `buf`: 16 bytes where the
    // operand lies along the tile's rows or columns, element by element where it
    // lies along the reduction and has to be turned over; zeros past the segment.
    auto issue = [&](int64_t c, int buf) {
        int64_t k0 = c * kK;
        const bool second = kOp == kFfnDx && k0 >= F;  // F is a multiple of 16
        if (second) k0 -= F;
        if (kOp == kFfnDw) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int p = tid + i * kThreads, k = p >> 4, m = (p & 15) * 4;
                const bool in = k0 + k < K;
                const int64_t row = seg0 + (in ? k0 + k : 0);
                copy16(&sm.t.a[buf][k][m], dw2 ? at(g.h, row * F + row0 + m) : at(g.x, row * d + row0 + m), in);
            }
        } else {
            const int k = tid & 15, ld = kOp == kFfnUp || kOp == kFfnGrad ? d : F;
            const void* base = kOp == kFfnUp     ? g.x
                               : kOp == kFfnDown ? g.h
                               : kOp == kFfnGrad ? g.dy
                                                 : (second ? g.db : g.da);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (tid >> 4) + 8 * i;
                const bool in = r < rows;
                copy4(&sm.t.a[buf][k][r], at(base, (static_cast<int64_t>(row0) + (in ? r : 0)) * ld + k0 + k), in);
            }
        }
        if (kOp == kFfnGrad || kOp == kFfnDx) {  // B(n, k): the weights' rows, k contiguous
            const int k = tid & 15, ld = kOp == kFfnGrad ? d : F;
            const void* base = kOp == kFfnGrad ? g.w2 : (second ? g.w3 : g.w1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int n = (tid >> 4) + 8 * i, c0 = col[0] + n;  // the halves adjoin
                const bool in = c0 < cols;
                copy4(&sm.t.b[buf][k][n], at(base, w_at + static_cast<int64_t>(in ? c0 : 0) * ld + k0 + k), in);
            }
        } else {  // n contiguous
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = tid + i * kThreads, n = (p & 31) * 4, half = n >> 6;
                const int64_t k = k0 + (p >> 5);
                const int c0 = col[half] + (n & 63);
                const bool in = c0 < cols && k < K;
                const int64_t kk = in ? k : 0, cc = in ? c0 : 0;
                const float* src = kOp == kFfnUp     ? at(half ? g.w3 : g.w1, w_at + kk * F + cc)
                                   : kOp == kFfnDown ? at(g.w2, w_at + kk * d + cc)
                                   : dw2             ? at(g.dy, (seg0 + kk) * d + cc)
                                                     : at(half ? g.db : g.da, (seg0 + kk) * F + cc);
                copy16(&sm.t.b[buf][p >> 5][n], src, in);
            }
        }
    };

    uint64_t acc2[8][4];  // two neighbouring columns each
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc2[i][j] = 0ull;

    const int rank = kOp == kFfnDw ? 0 : static_cast<int>(blockIdx.x) % splits;
    const int64_t all = (K + kK - 1) / kK, c0 = kOp == kFfnDw ? 0 : all * rank / splits;
    const int64_t chunks = kOp == kFfnDw ? all : all * (rank + 1) / splits - c0;
    // kBuffers - 1 chunks ahead; an empty group keeps the count where there is none
#pragma unroll
    for (int i = 0; i < kBuffers - 1; ++i) {
        if (i < chunks) issue(c0 + i, i);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int buf = 0;
    for (int64_t c = 0; c < chunks; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kBuffers - 2) : "memory");
        __syncthreads();  // chunk c is there for all, and all have done with chunk c - 1
        if (c + kBuffers - 1 < chunks) issue(c0 + c + kBuffers - 1, buf == 0 ? kBuffers - 1 : buf - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const float4 a0 = *reinterpret_cast<const float4*>(&sm.t.a[buf][k][ty * 8]);
            const float4 a1 = *reinterpret_cast<const float4*>(&sm.t.a[buf][k][ty * 8 + 4]);
            const float4 b0 = *reinterpret_cast<const float4*>(&sm.t.b[buf][k][tx * 4]);
            const float4 b1 = *reinterpret_cast<const float4*>(&sm.t.b[buf][k][64 + tx * 4]);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const uint64_t bv[4] = {pair2(b0.x, b0.y), pair2(b0.z, b0.w), pair2(b1.x, b1.y), pair2(b1.z, b1.w)};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t a2 = pair2(av[i], av[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) fma2(acc2[i][j], a2, bv[j]);
            }
        }
        if (++buf == kBuffers) buf = 0;
    }
    __syncthreads();  // the buffers hold the partial sums next

    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i][2 * j]), "=f"(acc[i][2 * j + 1]) : "l"(acc2[i][j]));
    if (kOp != kFfnDw && splits > 1) {
        // rank q finishes rows i = q, q + splits, ... of every thread's eight
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sm.part[i * 8 + j][tid] = acc[i][j];
        cluster_sync();
        const uint32_t mine = smem_u32(&sm.part[0][tid]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i % splits != rank) continue;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < splits; ++q) {
                const uint32_t from = mapa_shared(mine + i * 8 * kThreads * 4, q);
                float u[8];  // eight loads in flight
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u[j]) : "r"(from + j * kThreads * 4) : "memory");
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += u[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = v[j];
        }
        cluster_sync();  // the partial sums stay until every block has read them
    }

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty * 8 + i;
        if (r >= rows || (kOp != kFfnDw && i % splits != rank)) continue;
        const int64_t row = static_cast<int64_t>(row0) + r;
        const float* v = acc[i];
        if (kOp == kFfnUp) {
            const int64_t at = row * F + col[0] + tx * 4;
            float h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = v[j] / (1.f + expf(-v[j])) * v[4 + j];
            store4(g.h, at, h[0], h[1], h[2], h[3]);
            if (g.gate) {
                store4(g.gate, at, v[0], v[1], v[2], v[3]);
                store4(g.up, at, v[4], v[5], v[6], v[7]);
            }
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int c = col[half] + tx * 4;
                if (c >= cols) continue;
                const float* u = v + 4 * half;
                if (kOp == kFfnGrad) {
                    const int64_t at = row * F + c;
                    const float4 a4 = load4(g.gate, at), b4 = load4(g.up, at);
                    const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
                    float da[4], db[4], h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float s = 1.f / (1.f + expf(-a[j]));
                        h[j] = a[j] * s * b[j];
                        db[j] = u[j] * a[j] * s;
                        da[j] = u[j] * b[j] * s * (1.f + a[j] * (1.f - s));
                    }
                    store4(g.da, at, da[0], da[1], da[2], da[3]);
                    store4(g.db, at, db[0], db[1], db[2], db[3]);
                    store4(g.h, at, h[0], h[1], h[2], h[3]);
                } else if (kOp == kFfnDw) {
                    void* out = dw2 ? g.dw2 : (half ? g.dw3 : g.dw1);
                    store4(out, w_at + row * cols + c, u[0], u[1], u[2], u[3]);
                } else {
                    store4(kOp == kFfnDown ? g.y : g.dx, row * d + c, u[0], u[1], u[2], u[3]);
                }
            }
        }
    }
    griddep_launch_dependents();
}

template <int kOp>
static cudaError_t launch_row_op(const FfnArgs& a, int column_tiles, int K, int num_sms, cudaStream_t st) {
    const int64_t blocks = (a.R + kM - 1) / kM + a.n;  // at most
    const int64_t likely = std::max<int64_t>((a.R + kM - 1) / kM, std::min<int64_t>(a.n, a.R));
    // 3 or 4 blocks per SM run together; twice as many even out over the SMs
    int splits = 1;
    while (splits < 8 && likely * column_tiles * splits * 2 <= 8 * num_sms && K / kK >= 8 * splits) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * splits), static_cast<unsigned>(column_tiles));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (g_chain_started && pdl_enabled()) ? 2 : 1;
    g_chain_started = true;
    return cudaLaunchKernelEx(&cfg, ffn_simt_kernel<kOp>, a, splits);
}

cudaError_t launch_ffn_simt(int op, const FfnArgs& a, int num_sms, cudaStream_t st) {
    const int fd = (a.d + kN - 1) / kN, ff = (a.F + kN - 1) / kN;
    switch (op) {
        case kFfnUp: return launch_row_op<kFfnUp>(a, a.F / 64, a.d, num_sms, st);
        case kFfnDown: return launch_row_op<kFfnDown>(a, fd, a.F, num_sms, st);
        case kFfnGrad: return launch_row_op<kFfnGrad>(a, ff, a.d, num_sms, st);
        case kFfnDx: return launch_row_op<kFfnDx>(a, fd, 2 * a.F, num_sms, st);
        case kFfnDw: {
            const unsigned tiles = static_cast<unsigned>(a.d / kM) * (a.F / 64) + static_cast<unsigned>(a.F / kM) * fd;
            return launch_k(ffn_simt_kernel<kFfnDw>, dim3(tiles, a.n), dim3(kThreads), 0, st, a, 1);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
