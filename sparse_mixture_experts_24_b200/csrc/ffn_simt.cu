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
// With 3 blocks (12 warps) per SM the multiply-adds keep their pipe 57% (kFfnGrad) to
// 72% (kFfnUp, kFfnDw) busy (2,048 rows, 1,024 x 1,024; counters): 40 to 50 TFLOP/s
// over 4,096 rows.
// One warp per scheduler issues a multiply-add every other cycle at best, and
// small batches have fewer tiles than SMs: a product is then split along its
// reduction over a cluster of up to 8 blocks, whose partial sums meet in
// distributed shared memory and are added in rank order.  A tile of at most 32
// rows is split over the block's own warps too.  One expert of 256 x 768, 10 rows:
// forward 14.5 us (22.2 with whole tiles and the epilogue unrolled), backward 25.3
// (39.2); two rows of 8 experts of 640 x 1,216: 25.8 (44.8) and 54.5 (81.2).
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
__device__ __forceinline__ void copy4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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

// Operands are kept as [k][position].  The weights of kFfnGrad and kFfnDx, which lie
// along the reduction, keep that order: 16 values per column, four columns to a line
// whose padding spreads a warp's 16-byte reads over the banks.
constexpr int kLinesB = kN / 4, kLineB = 4 * kK + 4;
struct Tiles {
    float a[kBuffers][kK][kM + 4];
    union {
        float b[kBuffers][kK][kN + 4];
        float bk[kBuffers][kLinesB][kLineB];
    };
};
struct __align__(16) Smem {
    union {
        Tiles t;
        float4 part[16][kThreads];  // every thread's accumulators: four columns, [2 * row + half][thread]
    };
    SegmentPlan plan;
};
static_assert((kM + 4) % 4 == 0 && (kN + 4) % 4 == 0 && kLineB % 4 == 0 && sizeof(Tiles::a) % 16 == 0,
              "float4 alignment");

}  // namespace ffn_simt

using namespace ffn_simt;

template <int kOp>
__global__ void __launch_bounds__(kThreads, 3)
    ffn_simt_kernel(const FfnArgs g, const int splits) {
    griddep_wait();
    __shared__ Smem sm;
    load_plan(sm.plan, g.offsets, g.n, g.R, kM, g.status);
    const int tid = threadIdx.x;
    const int d = g.d, F = g.F;

    // the tile: expert, first output row (row ops: a row of the batch) and the
    // rows inside it, the column half starts, and the reduction
    int e, row0, rows, col[2];
    int64_t K;
    bool dw2 = false;
    if (kOp == kFfnDw) {
        e = blockIdx.y;
        const int t13 = (d / kM) * (F / 64), t = static_cast<int>(blockIdx.x) / splits;
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
    // A tile of at most 16 (32) rows needs one (two) of the four warps: all four then
    // take the same rows and a quarter (half) of every chunk each.
    const int groups = kOp == kFfnDw || rows > 32 ? 1 : (rows > 16 ? 2 : 4);
    const int per = kThreads / groups, group = tid / per, base = tid % per;
    const int tx = base & 15, ty = base >> 4;

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
            const int k = tid & 15, ld = kOp == kFfnGrad || kOp == kFfnUp ? d : F;
            const void* src = kOp == kFfnUp     ? g.x
                              : kOp == kFfnDown ? g.h
                              : kOp == kFfnGrad ? g.dy
                                                : (second ? g.db : g.da);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (tid >> 4) + 8 * i;
                if (r < rows)  // a row past the last only meets its own sums
                    copy4(&sm.t.a[buf][k][r], at(src, (static_cast<int64_t>(row0) + r) * ld + k0 + k));
            }
        }
        if (kOp == kFfnGrad || kOp == kFfnDx) {  // B(n, k): the weights' rows, k contiguous
            const int ld = kOp == kFfnGrad ? d : F;
            const void* src = kOp == kFfnGrad ? g.w2 : (second ? g.w3 : g.w1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = tid + i * kThreads, n = p >> 2, k = (p & 3) * 4, c0 = col[0] + n;  // the halves adjoin
                const bool in = c0 < cols;
                copy16(&sm.t.bk[buf][n >> 2][(n & 3) * kK + k],
                       at(src, w_at + static_cast<int64_t>(in ? c0 : 0) * ld + k0 + k), in);
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

    // Pairs of outputs: of neighbouring columns (a row's value twice), or of neighbouring
    // rows where B is read along the reduction (a column's value twice).  Turning B over
    // on its way in instead takes four times the copies: as fast for many rows, slower
    // for few (32 rows, 1,024 x 4,096, backward: 118 us against 139).
    constexpr bool kRowPairs = kOp == kFfnGrad || kOp == kFfnDx;
    uint64_t acc2[8][4];  // [row][column pair] or [column][row pair]
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc2[i][j] = 0ull;

    const int rank = static_cast<int>(blockIdx.x) % splits;
    const int64_t all = (K + kK - 1) / kK, c0 = all * rank / splits, chunks = all * (rank + 1) / splits - c0;
    auto multiply = [&](int buf, int kq) {  // four of the reduction
        if (kRowPairs) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[j] = *reinterpret_cast<const float4*>(&sm.t.bk[buf][half * 16 + tx][j * kK + kq * 4]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 a0 = *reinterpret_cast<const float4*>(&sm.t.a[buf][kq * 4 + k][ty * 8]);
                    const float4 a1 = *reinterpret_cast<const float4*>(&sm.t.a[buf][kq * 4 + k][ty * 8 + 4]);
                    const uint64_t av[4] = {pair2(a0.x, a0.y), pair2(a0.z, a0.w), pair2(a1.x, a1.y), pair2(a1.z, a1.w)};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = k == 0 ? b[j].x : (k == 1 ? b[j].y : (k == 2 ? b[j].z : b[j].w));
                        const uint64_t b2 = pair2(v, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) fma2(acc2[half * 4 + j][i], av[i], b2);
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = kq * 4; k < kq * 4 + 4; ++k) {
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
        }
    };
    // The copies run kBuffers - 1 chunks ahead; an empty group keeps the count where
    // there is none.  One loop from the first copy on: each copy of this code that
    // a block meets for the first time costs it a microsecond of instruction fetches.
    int buf = 0, into = 0;
    for (int64_t c = 1 - kBuffers; c < chunks; ++c) {
        if (c >= 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kBuffers - 2) : "memory");
            __syncthreads();  // chunk c is there for all, and all have done with chunk c - 1
        }
        if (c + kBuffers - 1 < chunks) issue(c0 + c + kBuffers - 1, into);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++into == kBuffers) into = 0;
        if (c < 0) continue;
        if (groups == 1) {
#pragma unroll
            for (int kq = 0; kq < kK / 4; ++kq) multiply(buf, kq);
        } else {
            for (int kq = group * (kK / 4 / groups); kq < (group + 1) * (kK / 4 / groups); ++kq) multiply(buf, kq);
        }
        if (++buf == kBuffers) buf = 0;
    }
    __syncthreads();  // the buffers hold the sums next

    // The sums go through shared memory, also where nothing is added to them: the
    // rest is then a loop over the thread's rows rather than eight copies of it.
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t p = kRowPairs ? acc2[4 * h + j][i >> 1] : acc2[i][2 * h + (j >> 1)];
                float lo, hi;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
                v[j] = (kRowPairs ? i & 1 : j & 1) ? hi : lo;
            }
            sm.part[2 * i + h][tid] = make_float4(v[0], v[1], v[2], v[3]);
        }
    if (groups > 1) {  // the block's own groups first
        __syncthreads();
        for (int v = group * (16 / groups); v < (group + 1) * (16 / groups); ++v) {
            float4 sum = sm.part[v][base];
            for (int q = 1; q < groups; ++q) {
                const float4 u = sm.part[v][base + q * per];
                sum.x += u.x, sum.y += u.y, sum.z += u.z, sum.w += u.w;
            }
            sm.part[v][base] = sum;
        }
        if (splits == 1) __syncthreads();
    }
    if (splits > 1) cluster_sync();
    const uint32_t part = smem_u32(&sm.part[0][base]);

    // rank and group finish every (splits * groups)th of the thread's eight rows
    for (int i = rank + splits * group; i < 8; i += splits * groups) {
        const int r = ty * 8 + i;
        if (r >= rows) break;
        float v[8];
        {
            const float4 lo = sm.part[2 * i][base], hi = sm.part[2 * i + 1][base];
            v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
            v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        }
        if (splits > 1) {
            float u[8][8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q >= splits) break;
                const uint32_t from = mapa_shared(part + 2 * i * kThreads * 16, q);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(u[q][4 * h]), "=f"(u[q][4 * h + 1]), "=f"(u[q][4 * h + 2]), "=f"(u[q][4 * h + 3])
                                 : "r"(from + h * kThreads * 16)
                                 : "memory");
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = u[0][j];
#pragma unroll
            for (int q = 1; q < 8; ++q) {
                if (q >= splits) break;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += u[q][j];
            }
        }
        const int64_t row = static_cast<int64_t>(row0) + r;
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
    if (splits > 1) cluster_sync();  // the sums stay until every block has read them
    griddep_launch_dependents();
}

// tiles: blocks that are likely to have work; chunks: of 16, in each one's reduction.
// It is split while that many blocks and a few more run together (3 per SM do, and
// more even out over them) and each keeps 8 chunks: backward of 480 rows, one expert of
// 192 x 384, with the weight gradients in one piece 63 us, split 44; 8,000 rows, 64 x
// 128, 508 and 104.
static int splits_for(int64_t tiles, int64_t chunks, int num_sms) {
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= 8 * num_sms && chunks >= 8 * splits) splits *= 2;
    return splits;
}

template <int kOp>
static cudaError_t launch_op(const FfnArgs& a, dim3 grid, int splits, cudaStream_t st) {
    grid.x *= static_cast<unsigned>(splits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
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

template <int kOp>
static cudaError_t launch_row_op(const FfnArgs& a, int column_tiles, int K, int num_sms, cudaStream_t st) {
    const int64_t blocks = a.R / kM + std::min<int64_t>(a.n, a.R);  // at most
    const int64_t likely = std::max<int64_t>((a.R + kM - 1) / kM, std::min<int64_t>(a.n, a.R));
    return launch_op<kOp>(a, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(column_tiles)),
                          splits_for(likely * column_tiles, K / kK, num_sms), st);
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
            return launch_op<kFfnDw>(a, dim3(tiles, a.n),
                                     splits_for(static_cast<int64_t>(tiles) * a.n, a.R / a.n / kK, num_sms), st);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
