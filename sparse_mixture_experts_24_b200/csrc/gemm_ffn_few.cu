// gemm_ffn_few.cu -- the products of the gated feed-forward block (gemm_ffn.cu) in
// bf16 where its 256 x 256 tiles would be too few or mostly empty: few rows per
// expert, where the call is bound by reading the weights once, and outputs so
// narrow that the reduction has to be shared out.
//
// The row products (kFfnUp, kFfnDown, kFfnGrad, kFfnDx) are turned over: 128 weight
// columns are the MMA's M and kT rows of the batch its N, so a tile needs no
// padding to 256 rows and there are enough tiles to keep all SMs loading; where
// there are not (one dense expert's 14,336 x 4,096 output projection has 32), the
// reduction is split over a cluster of up to 8 CTAs, whose partial sums meet in
// distributed shared memory, added in rank order.  Both operands keep their
// layouts: the weights are M-major for kFfnUp and kFfnDown (their rows are the
// reduction) and K-major for the other two, the rows are K-major.  kFfnDw takes 128
// x 128 outputs the same way, da, db or dy M-major and x or h N-major, over the
// expert's rows.
//
// 192 threads, one CTA per SM (the ring takes its shared memory):
//   warp 0     TMA, 64 of K per step: 128 weight columns (kFfnUp: of both
//              matrices) and kT rows;
//   warp 1     tcgen05.mma M 128, N kT, K 16 (kFfnUp: two accumulators);
//   warps 2-5  bring the accumulators to shared memory, one column per thread;
//              then every warp finishes whole rows, 4 columns per lane (128 rows of
//              1,024 x 4,096: forward 36 us when a thread kept its column, 24 so).
// The weights do not depend on the kernel before: their copies for the whole
// ring start before the programmatic-launch wait, under its last tiles.
// Every wait is bounded (common.cuh).
#include <algorithm>

#include "ffn.cuh"
#include "kernels.h"

namespace moe {

namespace ffn_few {

constexpr int kBM = 128, kBK = 64;
constexpr int kWBytes = kBM * kBK * 2;   // 16 KB: 128 columns of one matrix
constexpr int kChunk = 64 * kBK * 2;     // 8 KB: 64 columns, M-major
constexpr int kThreads = 192;
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 216 * 1024;

template <int kOp, int kT>
struct Cfg {
    static constexpr int kMats = kOp == kFfnUp ? 2 : 1;
    static constexpr int kStageBytes = kMats * kWBytes + kT * kBK * 2;
    static constexpr int kStages = kRingBytes / kStageBytes < kMaxStages ? kRingBytes / kStageBytes : kMaxStages;
    static constexpr int kTmemCols = kMats * kT < 32 ? 32 : kMats * kT;
    // the ring holds the partial sums of a split reduction afterwards
    static_assert(kOp != kFfnDw || kT == kBM, "two blocks of 128 columns");
    static_assert(kMats * kT * kBM * 4 <= kStages * kStageBytes, "partial sums");
};

struct __align__(128) Tail {
    CUtensorMap map[4];  // kFfnGrad: a map under construction per epilogue warp
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t accum_full;
    uint32_t tmem_base;
    SegmentPlan plan;
};
constexpr int kTailBytes = (static_cast<int>(sizeof(Tail)) + 127) / 128 * 128;

template <int kOp, int kT>
constexpr int smem_bytes() {
    return Cfg<kOp, kT>::kStages * Cfg<kOp, kT>::kStageBytes + kTailBytes + 1024;
}

__device__ __forceinline__ float sigmoid(float a) { return __fdividef(1.f, 1.f + __expf(-a)); }

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The sum of 16 bytes at `addr` over the cluster's CTAs, in rank order, with all
// loads in flight together.
__device__ __forceinline__ float4 sum_cluster(uint32_t addr, int splits) {
    float4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < splits) v[q] = load_cluster(mapa_shared(addr, q));
#pragma unroll
    for (int q = 1; q < 8; ++q)
        if (q < splits) v[0].x += v[q].x, v[0].y += v[q].y, v[0].z += v[q].z, v[0].w += v[q].w;
    return v[0];
}

__device__ __forceinline__ void put4(void* base, int64_t at, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void get4(const void* base, int64_t at, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}

// Weight columns col .. col + 3 (d and ffn are multiples of 64) of row `row` of the
// batch: accumulators v (and u, kFfnUp).
template <int kOp>
__device__ __forceinline__ void finish4(const FfnArgs& f, int64_t row, int col, const float4& v4, const float4& u4) {
    const float v[4] = {v4.x, v4.y, v4.z, v4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
    if (kOp == kFfnUp) {
        const int64_t at = row * f.F + col;
        if (f.gate) {
            put4(f.gate, at, v);
            put4(f.up, at, u);
        }
        float h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = v[j] * sigmoid(v[j]) * u[j];
        put4(f.h, at, h);
    } else if (kOp == kFfnGrad) {
        const int64_t at = row * f.F + col;
        float a[4], b[4], da[4], db[4], h[4];
        get4(f.gate, at, a);
        get4(f.up, at, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s = sigmoid(a[j]), as = a[j] * s;
            h[j] = as * b[j];
            db[j] = v[j] * as;
            da[j] = v[j] * b[j] * (s + as * (1.f - s));
        }
        put4(f.h, at, h);
        put4(f.db, at, db);
        put4(f.da, at, da);
    } else {
        put4(kOp == kFfnDown ? f.y : f.dx, row * f.d + col, v);
    }
}

}  // namespace ffn_few

using namespace ffn_few;

template <int kOp, int kT>
__global__ void __launch_bounds__(ffn_few::kThreads, 1)
    ffn_few_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                   const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
                   const __grid_constant__ FfnSideMaps<kOp> dw, const FfnArgs f, const int steps, const int splits) {
    using C = Cfg<kOp, kT>;
    constexpr bool kWMn = kOp == kFfnUp || kOp == kFfnDown || kOp == kFfnDw;  // the MMA's A is M-major
    constexpr bool kRMn = kOp == kFfnDw;                                      // and its B N-major
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    ffn_few::Tail* tail = reinterpret_cast<ffn_few::Tail*>(smem + C::kStages * C::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    load_plan(tail->plan, f.offsets, f.n, f.R, kT, f.status);
    const SegmentPlan& plan = tail->plan;
    griddep_launch_dependents();
    // the tensor maps of kFfnDw are written by warps 2 .. 5 of all CTAs
    auto write_maps = [&]() {
        if constexpr (kOp == kFfnGrad) {
            if (dw.out && warp >= 2)
                write_dw_maps(dw.m, dw.out, &tail->map[warp - 2], plan, f.n,
                              static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x) * 4 + warp - 2,
                              static_cast<int>(gridDim.x * gridDim.y) * 4);
        }
    };
    // x: weight column tile and, fastest, the split of its reduction; y: row block
    if (kOp != kFfnDw && static_cast<int>(blockIdx.y) >= plan.blk[f.n]) {
        griddep_wait();
        write_maps();
        return;  // the whole cluster: its CTAs share blockIdx.y
    }
    const int rank = static_cast<int>(blockIdx.x) % splits, tile = static_cast<int>(blockIdx.x) / splits;
    // row0, rows: the tile's rows of the batch, or (kFfnDw) of the weight gradient
    int e, row0, rows, col0, which = 0, reduce = steps;
    if (kOp == kFfnDw) {  // y: expert; x: dw1, dw3, dw2, as many tiles each
        e = blockIdx.y;
        const int nf = (f.F + kBM - 1) / kBM, nd = (f.d + kBM - 1) / kBM;
        which = tile / (nf * nd);
        const int local = tile - which * nf * nd, nc = which == 2 ? nd : nf;
        row0 = local / nc * kT;
        col0 = (local - local / nc * nc) * kBM;
        rows = min(kT, (which == 2 ? f.F : f.d) - row0);
        reduce = (plan.off[e + 1] - plan.off[e] + kBK - 1) / kBK;
    } else {
        e = plan_expert(plan, f.n, blockIdx.y);
        row0 = plan.off[e] + (static_cast<int>(blockIdx.y) - plan.blk[e]) * kT;
        rows = min(kT, plan.off[e + 1] - row0);
        col0 = tile * kBM;
    }
    const int k0 = static_cast<int>(static_cast<int64_t>(reduce) * rank / splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(reduce) * (rank + 1) / splits);
    int* status = f.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&tail->full[s]), 1);
            mbar_init(smem_u32(&tail->empty[s]), 1);
        }
        mbar_init(smem_u32(&tail->accum_full), 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem_base), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tail->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA ----------------
            const CUtensorMap *ma = nullptr, *mb = nullptr;
            if constexpr (kOp == kFfnDw) {  // maps [5][n]: x, h, da, db, dy
                griddep_wait();
                ma = dw.maps + (which == 2 ? 4 : 2 + which) * f.n + e;
                mb = dw.maps + (which == 2 ? 1 : 0) * f.n + e;
                acquire_map(ma);
                acquire_map(mb);
            }
            auto weights = [&](int kb, int stage) {
                const uint32_t fb = smem_u32(&tail->full[stage]);
                mbar_arrive_expect_tx(fb, C::kStageBytes);
                const uint32_t dst = smem_u32(smem + stage * C::kStageBytes);
                int k = kb * kBK;
                if (kOp == kFfnUp) {
                    tma_load_4d(dst, &tm_b0, fb, 0, k, tile * 2, e);
                    tma_load_4d(dst + kWBytes, &tm_b1, fb, 0, k, tile * 2, e);
                } else if (kOp == kFfnDown) {
                    tma_load_4d(dst, &tm_b0, fb, 0, k, tile * 2, e);
                } else if (kOp == kFfnGrad) {
                    tma_load_3d(dst, &tm_b0, fb, k, col0, e);
                } else if (kOp == kFfnDw) {
                    tma_load_3d(dst, ma, fb, 0, plan.off[e] + k, col0 / 64);
                } else {
                    const bool second = k >= f.F;
                    tma_load_3d(dst, second ? &tm_b1 : &tm_b0, fb, second ? k - f.F : k, col0, e);
                }
            };
            auto batch = [&](int kb, int stage) {
                const uint32_t fb = smem_u32(&tail->full[stage]);
                const uint32_t dst = smem_u32(smem + stage * C::kStageBytes) + C::kMats * kWBytes;
                const int k = kb * kBK;
                if (kOp == kFfnDw) {
                    tma_load_3d(dst, mb, fb, 0, plan.off[e] + k, row0 / 64);
                    return;
                }
                const bool second = kOp == kFfnDx && k >= f.F;
                tma_load_2d(dst, second ? &tm_a1 : &tm_a0, fb, second ? k - f.F : k, row0);
            };
            const int ahead = min(C::kStages, k1 - k0);
            for (int i = 0; i < ahead; ++i) weights(k0 + i, i);
            griddep_wait();
            for (int i = 0; i < ahead; ++i) batch(k0 + i, i);
            bool ok = true;
            for (int i = ahead; i < k1 - k0; ++i) {
                const int stage = i % C::kStages;
                const uint32_t use = static_cast<uint32_t>(i / C::kStages);
                if (!mbar_wait(smem_u32(&tail->empty[stage]), (use & 1u) ^ 1u, status, kStatusTimeoutEmpty)) {
                    ok = false;
                    break;
                }
                weights(k0 + i, stage);
                batch(k0 + i, stage);
            }
            if (!ok)  // give every armed copy its time to land before the CTA leaves
                for (int s = 0; s < C::kStages; ++s)
                    mbar_wait(smem_u32(&tail->full[s]), 0, status, kStatusTimeoutDrain);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA ----------------
            constexpr uint32_t idesc = make_idesc_bf16(kBM, kT, kWMn ? 1 : 0, kRMn ? 1 : 0);
            bool ok = true;
            for (int i = 0; i < k1 - k0; ++i) {
                const int stage = i % C::kStages;
                const uint32_t use = static_cast<uint32_t>(i / C::kStages);
                if (!mbar_wait(smem_u32(&tail->full[stage]), use & 1u, status, kStatusTimeoutFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = smem_u32(smem + stage * C::kStageBytes);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                    const uint32_t b = base + C::kMats * kWBytes;
                    const uint64_t bd = kRMn ? make_smem_desc(b + kk * 2048, kChunk, 1024, 2)
                                             : make_smem_desc(b + kk * 32, 16, 1024, 2);
#pragma unroll
                    for (int m = 0; m < C::kMats; ++m) {
                        const uint32_t a = base + m * kWBytes;
                        const uint64_t ad = kWMn ? make_smem_desc(a + kk * 2048, kChunk, 1024, 2)
                                                 : make_smem_desc(a + kk * 32, 16, 1024, 2);
                        tc_mma_f16(tmem_base + static_cast<uint32_t>(m * kT), ad, bd, idesc, (i | kk) != 0 ? 1u : 0u);
                    }
                }
                tc_commit(smem_u32(&tail->empty[stage]));
            }
            (void)ok;
            tc_commit(smem_u32(&tail->accum_full));
            mbar_wait(smem_u32(&tail->accum_full), 0, status, kStatusTimeoutDrain);
        }
    } else {
        // ---------------- accumulators ----------------
        const int quad = warp & 3;  // TMEM lanes 32 * quad .. + 31
        const int c = quad * 32 + lane;
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        if (kOp == kFfnGrad) {
            griddep_wait();
            write_maps();
        }
        const bool done = mbar_wait(smem_u32(&tail->accum_full), 0, status, kStatusTimeoutAccum);
        __syncwarp();
        tc_fence_after();
        float* part = reinterpret_cast<float*>(smem);  // [matrix][row][128 columns]
        if (done) {
#pragma unroll 1
            for (int t0 = 0; t0 < rows; t0 += 16) {
                uint32_t v[16], u[16];
                tmem_ld_32x32b_x16(tbase + t0, v);
                if (kOp == kFfnUp) tmem_ld_32x32b_x16(tbase + kT + t0, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // (kFfnDw: a share, or an expert, without rows multiplies nothing)
                    const float vf = kOp == kFfnDw && k0 == k1 ? 0.f : __uint_as_float(v[i]), uf = kOp == kFfnUp ? __uint_as_float(u[i]) : 0.f;
                    part[(t0 + i) * kBM + c] = vf;
                    if (kOp == kFfnUp) part[(kT + t0 + i) * kBM + c] = uf;
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    {
        // every CTA of the cluster finishes its share of the rows, a warp one at a time
        const int cols = kOp == kFfnUp || kOp == kFfnGrad || (kOp == kFfnDw && which != 2) ? f.F : f.d;
        const uint32_t part = smem_u32(smem);
        const int col = lane * 4;
        if (col0 + col < cols)
            for (int t = rank + splits * warp; t < rows; t += splits * (ffn_few::kThreads / 32)) {
                const float4 v = sum_cluster(part + (t * kBM + col) * 4, splits);
                const float4 u = kOp == kFfnUp ? sum_cluster(part + ((kT + t) * kBM + col) * 4, splits)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
                if (kOp == kFfnDw) {
                    const float out[4] = {v.x, v.y, v.z, v.w};
                    put4(which == 0 ? f.dw1 : (which == 1 ? f.dw3 : f.dw2),
                         static_cast<int64_t>(e) * f.d * f.F + static_cast<int64_t>(row0 + t) * cols + col0 + col, out);
                } else {
                    finish4<kOp>(f, static_cast<int64_t>(row0) + t, col0 + col, v, u);
                }
            }
        __syncwarp();
    }
    if (splits > 1) cluster_sync();  // the partial sums stay until every CTA has read them
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

// The most rows that an expert is likely to have (ragged experts: up to about 1.4
// times the average), and the blocks of `height` rows that all of them make, rather
// too many than too few: one more than run together costs a whole round.  The offsets
// are on the device, so a router more skewed than that gets the same results from a
// choice made for the average: 8 experts of 4,096 x 14,336, 180 rows forward, 505 us
// spread evenly, 628 with 44% of them at one expert (whose weights three blocks of 32
// rows then read), 398 with all of them there (143 for that expert alone, n = 1).  At 44%
// all else from 64 to 8,192 rows, both passes, was within 5% of even, but for 8,192 rows
// backward (4.1 and 4.8 ms).
static int64_t most_rows(const FfnArgs& f) { return f.n == 1 ? f.R : (7 * f.R + 5 * f.n - 1) / (5 * f.n); }
static int64_t likely_blocks(const FfnArgs& f, int height) {
    const int64_t used = std::min<int64_t>(f.n, f.R);
    if (f.n == 1) return (f.R + height - 1) / height;
    return most_rows(f) <= height ? used : f.R / height + used;
}
static int out_cols(int op, const FfnArgs& f) { return op == kFfnUp || op == kFfnGrad ? f.F : f.d; }
static int out_steps(int op, const FfnArgs& f) {
    if (op == kFfnDw) return static_cast<int>(std::max<int64_t>(1, most_rows(f) / kBK));
    return (op == kFfnUp || op == kFfnGrad ? f.d : (op == kFfnDown ? f.F : 2 * f.F)) / kBK;
}
static int64_t out_tiles(int op, const FfnArgs& f, int height) {
    if (op == kFfnDw) return static_cast<int64_t>(f.n) * 3 * ((f.d + kBM - 1) / kBM) * ((f.F + kBM - 1) / kBM);
    return (out_cols(op, f) + kBM - 1) / kBM * likely_blocks(f, height);
}
// The reduction is split while all CTAs run together and keep 8 steps.
static int out_splits(int op, const FfnArgs& f, int height, int num_sms) {
    const int64_t tiles = out_tiles(op, f, height);
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= num_sms && out_steps(op, f) >= 8 * splits) splits *= 2;
    return splits;
}

template <int kOp, int kT>
static cudaError_t launch_few(const CUtensorMap* m, const FfnArgs& f, const FfnSideMaps<kOp>& dw, int num_sms,
                              cudaStream_t st) {
    constexpr int smem = smem_bytes<kOp, kT>();
    static_assert(smem <= 232448, "shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(ffn_few_kernel<kOp, kT>), smem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = kOp == kFfnDw ? out_tiles(kOp, f, kT) / f.n : (out_cols(kOp, f) + kBM - 1) / kBM;
    const int64_t blocks = kOp == kFfnDw ? f.n : f.R / kT + std::min<int64_t>(f.n, f.R);  // at most
    const int splits = out_splits(kOp, f, kT, num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(ffn_few::kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, ffn_few_kernel<kOp, kT>, m[0], m[1], m[2], m[3], dw, f, out_steps(kOp, f), splits);
}

template <int kT>
static cudaError_t launch_few_op(int op, const CUtensorMap* m, const FfnArgs& f, const FfnDwMaps& dw, int num_sms,
                                 cudaStream_t st) {
    switch (op) {
        case kFfnUp: return launch_few<kFfnUp, kT>(m, f, {}, num_sms, st);
        case kFfnDown: return launch_few<kFfnDown, kT>(m, f, {}, num_sms, st);
        case kFfnGrad: return launch_few<kFfnGrad, kT>(m, f, dw, num_sms, st);
        case kFfnDx: return launch_few<kFfnDx, kT>(m, f, {}, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

// Which kernel takes a row product: this one in tiles of the returned rows, or
// (0) the other one in tiles of 256 x 256 by pairs of CTAs.
//   kFfnUp    in tiles of 32 rows wherever they hold an expert's rows (128 experts of
//             2,048 x 768, 1,024 rows, with the output projection: 225 us against 256);
//   kFfnDown  wherever one tile holds them and the reduction is 48 steps or longer (8
//             experts of 4,096 x 14,336, 400 rows, the whole block: 508 against 541);
//   else, and for the backward products, what two estimates say, in steps of 64 (about
//             0.35 us).  A tile here takes its share of the steps (kFfnUp, two matrices:
//             1.4 times as long) and 10 more, the other kernel's last tile 18 more;
//             the rows' output and (kFfnGrad) elementwise part is counted by the row
//             here and by the tile there, where the next tile's product hides half of
//             it.  The reduction over a cluster decides most: one expert of 640 x 3,584,
//             512 rows, backward 34 us against 58, 1,024 rows 43 against 59, 2,048 rows
//             75 either way; 8 experts of 384 x 7,808, 2,000 rows, 123 against 157;
//             kFfnGrad too for 128 rows, 21 against 29; forward, 90 rows over two
//             experts of 2,048 x 5,632, both products 38 us, kFfnDown alone 46,
//             neither 66.
//   kFfnDw    the same, a tile here costing a tenth more per step and 14: one expert of
//             256 x 512, 8,192 rows, with the hidden gradient 34 us against 61; 640 x
//             448, 8,021 rows, 48 against 63; 1 row of the first 13 against 16.
int ffn_few_rows(int op, const FfnArgs& f, int num_sms) {
    if (op == kFfnDw) {
        const int steps = out_steps(op, f), splits = out_splits(op, f, 128, num_sms);
        const int64_t rounds = (out_tiles(op, f, 128) * splits + num_sms - 1) / num_sms, pairs = num_sms / 2;
        const int64_t d2 = (f.d + 255) / 256, F2 = (f.F + 255) / 256;
        const int64_t others = (f.n * (d2 * ((f.F + 127) / 128) + F2 * d2) + pairs - 1) / pairs;
        return rounds * (steps / splits * 11 / 10 + 14) < others * steps + 18 ? 128 : 0;
    }
    const int64_t most = most_rows(f);
    const int height = most <= 32 ? 32 : 128;
    const int64_t cols = out_cols(op, f), tiles = out_tiles(op, f, height);
    const int steps = out_steps(op, f);
    if (op == kFfnUp && most <= 32) return 32;
    if (op == kFfnDown && most <= height && steps >= 48) return height;
    const int rows = static_cast<int>(std::min<int64_t>(most, height));
    const int splits = out_splits(op, f, height, num_sms), share = steps / splits;
    const int64_t rounds = (tiles * splits + num_sms - 1) / num_sms, pairs = num_sms / 2;
    const int64_t pair_cols = op == kFfnUp ? 128 : 256;
    const int64_t others = (likely_blocks(f, 256) * ((cols + pair_cols - 1) / pair_cols) + pairs - 1) / pairs;
    int64_t here, there = others * steps + 18;
    if (op == kFfnUp) {
        here = rounds * (share * 7 / 5 + 10 + 20 * rows / 128);
    } else if (op == kFfnGrad) {
        here = rounds * (share + 20 + 15 * rows / 128) * 20 / 19;  // as good is not enough
        there = others * (steps + 18) + 19;
    } else {
        here = rounds * (share + 10 + 10 * rows / 128);
    }
    return here < there ? height : 0;
}

cudaError_t launch_ffn_few(int op, int rows, const CUtensorMap* maps, const FfnArgs& f, const FfnDwMaps& dw,
                           int num_sms, cudaStream_t st) {
    if (op == kFfnDw) return launch_few<kFfnDw, 128>(maps, f, {dw.out}, num_sms, st);
    return rows == 32 ? launch_few_op<32>(op, maps, f, dw, num_sms, st)
                      : launch_few_op<128>(op, maps, f, dw, num_sms, st);
}

}  // namespace moe
