// gemm_ffn.cu -- the products of the gated feed-forward block over expert
// segments, forward and backward, in bf16 on the sm_100a tensor cores
// (tcgen05.mma on CTA pairs, accumulators in tensor memory, operands by TMA).
//
// ffn.cuh has the formulas.  Five products share one kernel; M x N is one
// pair's 256 x 256 tile, K runs in steps of 64:
//   op        M        N                      K          operands in shared memory
//   kFfnUp    rows     128 a | 128 b columns  d          x K-major, w1 | w3 N-major
//   kFfnDown  rows     256 of d               F          h K-major, w2 N-major
//   kFfnGrad  rows     256 of F               d          dy K-major, w2 K-major
//   kFfnDx    rows     256 of d               F, then F  da, db K-major; w1, w3 K-major
//   kFfnDw    d (dw1, dw3) or F (dw2)         e's rows   x or h M-major; da | db, or dy, N-major
// The matrices are read where they lie, in the layout of the forward layer:
// which of an operand's two axes is contiguous only changes its descriptor.
//
// Roles, 320 threads in each of a pair's two CTAs (one CTA per SM):
//   warp 0     TMA of this CTA's 128 rows of A and 128 columns of B, 32 KB per
//              step into a ring of six; the bytes of both CTAs are counted on
//              the leader's barrier (no multicast);
//   warp 1     of the leader: tcgen05.mma.cta_group::2 (M 256, N 256, K 16);
//   warps 2-9  epilogue, two per 32 accumulator rows, each on half the columns:
//              the block's elementwise part on the fp32 accumulators, bf16
//              rows through the warp's exchange blocks (ffn.cuh), by TMA where
//              all 32 rows are stored.  128 experts of 2,048 x 768 with 128 rows
//              each: storing 16 bytes per lane straight from registers, dw took
//              628 us; 64-byte segments through the blocks 442 us, by
//              TMA 286 us, as 128-byte rows of both blocks together 270 us.  Two accumulators (512 TMEM columns): a tile's epilogue
//              runs under the next tile's products.
// kFfnDx adds both of its products in one accumulator: K simply runs over da
// with w1 and then db with w3.  kFfnDw does all three weight gradients in one
// launch; its reduction runs over an expert's rows, which end anywhere, so each
// expert has tensor maps of its own whose row extent is the segment's end (the
// copies read zeros past it, whatever lies there); kFfnGrad's epilogue warps write
// them while they wait for their first accumulator.
// Row tiles that reach past a segment's end compute rows of the next expert
// and do not store them.
//
// Every wait is bounded (common.cuh); both CTAs of a pair leave together.
#include <algorithm>

#include "ffn.cuh"
#include "kernels.h"

namespace moe {

namespace ffn_tc {

constexpr int kBM = 256, kBN = 256, kBK = 64;
constexpr int kStages = 6;
constexpr int kABytes = 128 * kBK * 2;   // 16 KB: this CTA's rows
constexpr int kBBytes = 128 * kBK * 2;   // 16 KB: this CTA's columns
constexpr int kChunk = 64 * kBK * 2;     // 8 KB: 64 columns of an M- or N-major operand
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;

struct __align__(16) Tail {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t accum_full[2];
    uint64_t accum_empty[2];
    uint64_t done;
    uint32_t tmem_base;
    SegmentPlan plan;
};
// Shared memory, 1 KB aligned: barriers and plan, the ring, two exchange blocks
// per epilogue warp.
constexpr int kTailBytes = (static_cast<int>(sizeof(Tail)) + 1023) / 1024 * 1024;
constexpr int kSmemBytes = kTailBytes + kStages * kStageBytes + 2 * kEpiWarps * kExchangeBytes;
static_assert(kSmemBytes <= 232448, "shared memory");

struct Tile {
    int e;
    int row0;    // first row of the batch (row ops) or first output row (kFfnDw)
    int rows;    // rows of the tile to store
    int n_tile;
    int k0;      // kFfnDw: first row of the segment
    int steps;   // 64-deep K steps
    bool dw2;
};

// Row ops: tile t -> (expert, column tile, 256-row block); an expert's row
// blocks are cut into bands whose A rows fit in L2, the row block fastest
// inside a band, so that a band stays there while the expert's weight columns
// stream past it.  kFfnDw: all tiles of dw1 and dw3, then dw2, expert by
// expert, the output row block fastest.
template <int kOp>
__device__ __forceinline__ Tile tile_at(int t, const SegmentPlan& p, const FfnTcArgs& a) {
    Tile ti;
    if (kOp == kFfnDw) {
        const int per = a.dw_tiles13 + a.dw_tiles2;
        ti.e = t / per;
        int local = t - ti.e * per;
        ti.dw2 = local >= a.dw_tiles13;
        if (ti.dw2) local -= a.dw_tiles13;
        const int height = ti.dw2 ? a.F : a.d;
        const int mb = (height + kBM - 1) / kBM;
        ti.n_tile = local / mb;
        ti.row0 = (local - ti.n_tile * mb) * kBM;
        ti.rows = min(kBM, height - ti.row0);
        ti.k0 = p.off[ti.e];
        ti.steps = (p.off[ti.e + 1] - ti.k0 + kBK - 1) / kBK;
        return ti;
    }
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.blk[mid] * a.n_tiles <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int local = t - p.blk[lo] * a.n_tiles;
    const int count = p.blk[lo + 1] - p.blk[lo];
    const int band = min(count, a.band);
    const int whole = count / band * band;
    int m;
    if (local < whole * a.n_tiles) {
        const int b = local / (band * a.n_tiles);
        const int r = local - b * band * a.n_tiles;
        ti.n_tile = r / band;
        m = b * band + (r - ti.n_tile * band);
    } else {
        const int rem = count - whole;
        const int r = local - whole * a.n_tiles;
        ti.n_tile = r / rem;
        m = whole + (r - ti.n_tile * rem);
    }
    ti.e = lo;
    ti.row0 = p.off[lo] + m * kBM;
    ti.rows = min(kBM, p.off[lo + 1] - ti.row0);
    ti.steps = a.steps;
    ti.k0 = 0;
    ti.dw2 = false;
    return ti;
}

__device__ __forceinline__ float sigmoid(float a) { return __fdividef(1.f, 1.f + __expf(-a)); }

// Hand an accumulator back to the leader's MMA thread.  Relaxed: what has to
// come before it are the warp's tensor-memory loads, which tcgen05.wait::ld has
// completed.  A release at cluster scope would also wait for the warp's global
// stores of the tile.
__device__ __forceinline__ void hand_back_to(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// 32 accumulators as 16 words of bf16 pairs.
__device__ __forceinline__ void pack32(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
}

}  // namespace ffn_tc

using namespace ffn_tc;

template <int kOp>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_tc_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                  const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
                  const __grid_constant__ FfnOutMaps tm_out, const __grid_constant__ FfnSideMaps<kOp> dw,
                  const FfnTcArgs args) {
    constexpr bool kAMn = kOp == kFfnDw;                      // A is M-major in shared memory
    constexpr bool kBMn = kOp != kFfnGrad && kOp != kFfnDx;   // B is N-major
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Tail* tail = reinterpret_cast<Tail*>(smem_raw);
    uint8_t* smem = smem_raw + kTailBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(nclusters_x());
    int* status = args.f.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&tail->full[s]), 1);
            mbar_init(smem_u32(&tail->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tail->accum_full[b]), 1);
            mbar_init(smem_u32(&tail->accum_empty[b]), 2 * kEpiWarps);
        }
        mbar_init(smem_u32(&tail->done), 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0 && kOp != kFfnDw) {
        tma_prefetch_desc(&tm_a0);
        tma_prefetch_desc(&tm_b0);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&tail->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    griddep_wait();
    load_plan(tail->plan, args.f.offsets, args.n, args.f.R, kBM, status);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = tail->tmem_base;
    const SegmentPlan& plan = tail->plan;
    const int total = kOp == kFfnDw ? args.n * (args.dw_tiles13 + args.dw_tiles2) : plan.blk[args.n] * args.n_tiles;
    // this pair's tiles: runs of `run` tiles, dealt round robin
    const int run = kOp == kFfnDw ? args.dw_run : 1;
    auto tile_index = [&](int i) { return (i / run * ncl + cid) * run + i % run; };

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int stage = 0;
            uint32_t phase = 0;
            int armed[kStages];
            for (int s = 0; s < kStages; ++s) armed[s] = -1;
            bool ok = true;
            const CUtensorMap *ma = &tm_a0, *mb = &tm_b0;
            int held = -1;  // kFfnDw: (expert, matrix) whose maps are acquired
            const int r = static_cast<int>(rank);
            for (int i = 0, t = cid * run; t < total && ok; t = tile_index(++i)) {
                const Tile ti = tile_at<kOp>(t, plan, args);
                if constexpr (kOp == kFfnDw) {
                    if (ti.steps > 0 && held != 2 * ti.e + (ti.dw2 ? 1 : 0)) {
                        held = 2 * ti.e + (ti.dw2 ? 1 : 0);
                        // maps [5][n]: x, h, da, db, dy; the peer's columns are db's
                        ma = dw.maps + (ti.dw2 ? 1 : 0) * args.n + ti.e;
                        mb = dw.maps + (ti.dw2 ? 4 : 2 + r) * args.n + ti.e;
                        acquire_map(ma);
                        acquire_map(mb);
                    }
                }
                for (int kb = 0; kb < ti.steps; ++kb) {
                    if (!mbar_wait(smem_u32(&tail->empty[stage]), phase ^ 1u, status, kStatusTimeoutEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_local = smem_u32(&tail->full[stage]);
                    if (rank == 0) {
                        mbar_arrive_expect_tx(full_local, 2 * kStageBytes);
                        armed[stage] = static_cast<int>(phase);
                    }
                    const uint32_t full = mapa_shared(full_local, 0);
                    const uint32_t a_dst = smem_u32(smem + stage * kStageBytes);
                    const uint32_t b_dst = a_dst + kABytes;
                    int k = kb * kBK;
                    if (kOp == kFfnUp) {
                        tma_load_2d_pair(a_dst, ma, full, k, ti.row0 + 128 * r);
                        tma_load_4d_pair(b_dst, r == 0 ? &tm_b0 : &tm_b1, full, 0, k, ti.n_tile * 2, ti.e);
                    } else if (kOp == kFfnDown) {
                        tma_load_2d_pair(a_dst, ma, full, k, ti.row0 + 128 * r);
                        tma_load_4d_pair(b_dst, mb, full, 0, k, ti.n_tile * 4 + 2 * r, ti.e);
                    } else if (kOp == kFfnGrad) {
                        tma_load_2d_pair(a_dst, ma, full, k, ti.row0 + 128 * r);
                        tma_load_3d_pair(b_dst, mb, full, k, ti.n_tile * kBN + 128 * r, ti.e);
                    } else if (kOp == kFfnDx) {
                        const bool second = k >= args.F;
                        if (second) k -= args.F;
                        tma_load_2d_pair(a_dst, second ? &tm_a1 : &tm_a0, full, k, ti.row0 + 128 * r);
                        tma_load_3d_pair(b_dst, second ? &tm_b1 : &tm_b0, full, k, ti.n_tile * kBN + 128 * r, ti.e);
                    } else {
                        tma_load_3d_pair(a_dst, ma, full, 0, ti.k0 + k, ti.row0 / 64 + 2 * r);
                        tma_load_3d_pair(b_dst, mb, full, 0, ti.k0 + k,
                                         ti.dw2 ? ti.n_tile * 4 + 2 * r : ti.n_tile * 2);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the leader's barriers count both CTAs' copies: nothing may still be
            // landing when the pair exits
            if (rank == 0)
                for (int s = 0; s < kStages; ++s)
                    if (armed[s] >= 0)
                        mbar_wait(smem_u32(&tail->full[s]), static_cast<uint32_t>(armed[s]), status,
                                  kStatusTimeoutDrain);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer (leader) ----------------
            constexpr uint32_t idesc = make_idesc_bf16(kBM, kBN, kAMn ? 1 : 0, kBMn ? 1 : 0);
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            for (int t = cid * run; t < total && ok; t = tile_index(++local)) {
                const Tile ti = tile_at<kOp>(t, plan, args);
                const int buf = local & 1;
                const uint32_t bph = static_cast<uint32_t>(local >> 1) & 1u;
                if (!mbar_wait(smem_u32(&tail->accum_empty[buf]), bph ^ 1u, status, kStatusTimeoutAccum)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kBN);
                for (int kb = 0; kb < ti.steps; ++kb) {
                    if (!mbar_wait(smem_u32(&tail->full[stage]), phase, status, kStatusTimeoutFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_base = smem_u32(smem + stage * kStageBytes);
                    const uint32_t b_base = a_base + kABytes;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        // K-major: 16 of K are 32 bytes inside the 128-byte swizzle row;
                        // M- or N-major: 16 of K are two groups of 8 rows of 128 bytes,
                        // and the operand's two 64-column chunks lie 8 KB apart
                        const uint64_t ad = kAMn ? make_smem_desc(a_base + kk * 2048, kChunk, 1024, 2)
                                                 : make_smem_desc(a_base + kk * 32, 16, 1024, 2);
                        const uint64_t bd = kBMn ? make_smem_desc(b_base + kk * 2048, kChunk, 1024, 2)
                                                 : make_smem_desc(b_base + kk * 32, 16, 1024, 2);
                        tc_mma_f16_pair(d_tmem, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
                    }
                    const uint32_t eb = smem_u32(&tail->empty[stage]);
                    tc_commit_pair(mapa_shared(eb, 0));
                    tc_commit_pair(mapa_shared(eb, 1));
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) {
                    const uint32_t fb = smem_u32(&tail->accum_full[buf]);
                    tc_commit_pair(mapa_shared(fb, 0));
                    tc_commit_pair(mapa_shared(fb, 1));
                }
            }
            tc_commit_pair(mapa_shared(smem_u32(&tail->done), 0));
            mbar_wait(smem_u32(&tail->done), 0, status, kStatusTimeoutDrain);
        }
    } else {
        // ---------------- epilogue (warps 2..9 of both CTAs) ----------------
        const int quad = warp & 3;         // TMEM lanes 32 * quad .. + 31
        const int half = (warp - 2) >> 2;  // accumulator columns 128 * half .. + 127
        const uint32_t hand_back[2] = {mapa_shared(smem_u32(&tail->accum_empty[0]), 0),
                                       mapa_shared(smem_u32(&tail->accum_empty[1]), 0)};
        const FfnArgs& f = args.f;
        uint8_t* block = smem + kStages * kStageBytes + (warp - 2) * (2 * kExchangeBytes);
        int turn = 0;
        if constexpr (kOp == kFfnGrad)
            if (dw.out)
                write_dw_maps(dw.m, dw.out, block, plan, args.n, static_cast<int>(blockIdx.x) * kEpiWarps + warp - 2,
                              static_cast<int>(gridDim.x) * kEpiWarps);
        // 32 columns of this warp's rows to one output: through its tensor map where
        // all 32 rows are stored, else row by row
        auto store = [&](const uint32_t* w, int which, void* out, int64_t row, int cols, int col, int valid) {
            if (valid == 32) {
                exchange_send_2d(block, turn, w, lane, &tm_out.m[which], col, static_cast<int>(row));
            } else {
                if (lane == 0) exchange_drain_reads();
                __syncwarp();
                exchange_store(block, w, lane, valid, static_cast<uint16_t*>(out) + row * cols + col, cols * 2LL);
            }
        };
        int local = 0;
        for (int t = cid * run; t < total; t = tile_index(++local)) {
            const Tile ti = tile_at<kOp>(t, plan, args);
            const int buf = local & 1;
            const uint32_t bph = static_cast<uint32_t>(local >> 1) & 1u;
            uint4 gate_next[4], up_next[4];
            if (kOp == kFfnGrad) {
                const int r0 = 128 * static_cast<int>(rank) + 32 * quad;
                const int col = ti.n_tile * kBN + half * 128;
                const int64_t o = ((static_cast<int64_t>(ti.row0) + r0) * args.F + col) * 2;
                const int valid = col < args.F ? ti.rows - r0 : 0;
                exchange_fetch(gate_next, lane, valid, static_cast<const uint8_t*>(f.gate) + o, args.F * 2LL);
                exchange_fetch(up_next, lane, valid, static_cast<const uint8_t*>(f.up) + o, args.F * 2LL);
            }
            if (!mbar_wait(smem_u32(&tail->accum_full[buf]), bph, status, kStatusTimeoutAccum)) break;
            tc_fence_after();
            const uint32_t tbase =
                tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(buf * kBN);
            const int r0 = 128 * static_cast<int>(rank) + 32 * quad;  // this warp's 32 rows of the tile
            const int valid = min(32, ti.rows - r0);                 // warp-uniform, like every column test
            const int64_t row = static_cast<int64_t>(ti.row0) + r0;
            bool returned = false;  // the accumulator
            if (valid <= 0) {
                // nothing of this warp's to store
            } else if (kOp == kFfnUp) {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    const int at = half * 64 + c * 32;  // hidden columns of the tile
                    const int col = ti.n_tile * 128 + at;
                    if (col >= args.F) break;
                    uint32_t a[32], b[32], w[16];
                    tmem_ld_32x32b_x32(tbase + at, a);
                    tmem_ld_32x32b_x32(tbase + 128 + at, b);
                    tmem_wait_ld();
                    if (f.gate) {
                        pack32(a, w);
                        store(w, 1, f.gate, row, args.F, col, valid);
                        pack32(b, w);
                        store(w, 2, f.up, row, args.F, col, valid);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float h[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float av = __uint_as_float(a[2 * j + i]);
                            h[i] = av * sigmoid(av) * __uint_as_float(b[2 * j + i]);
                        }
                        w[j] = pack_bf16x2(h[0], h[1]);
                    }
                    store(w, 0, f.h, row, args.F, col, valid);
                }
            } else if (kOp == kFfnGrad) {
                // the first chunk of gate and up was fetched before the wait for the
                // accumulator; chunk c + 1 is in flight while chunk c is computed
                const int64_t ld = static_cast<int64_t>(args.F) * 2;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const int at = half * 128 + c * 32;
                    const int col = ti.n_tile * kBN + at;
                    if (col >= args.F) break;
                    const int64_t o = (row * args.F + col) * 2;
                    uint32_t ga[16], gb[16], dh[32];
                    tmem_ld_32x32b_x32(tbase + at, dh);
                    if (lane == 0) exchange_drain_reads();
                    __syncwarp();
                    exchange_turn(block, gate_next, lane, ga);
                    exchange_turn(block, up_next, lane, gb);
                    if (c < 3 && col + 32 < args.F) {
                        exchange_fetch(gate_next, lane, valid, static_cast<const uint8_t*>(f.gate) + o + 64, ld);
                        exchange_fetch(up_next, lane, valid, static_cast<const uint8_t*>(f.up) + o + 64, ld);
                    }
                    tmem_wait_ld();
                    uint32_t hw[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a[2], b[2], x[2], y[2], h[2];
                        unpack_bf16x2(ga[j], a[0], a[1]);
                        unpack_bf16x2(gb[j], b[0], b[1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float s = sigmoid(a[i]), g = __uint_as_float(dh[2 * j + i]);
                            const float as = a[i] * s;
                            h[i] = as * b[i];
                            y[i] = g * as;
                            x[i] = g * b[i] * (s + as * (1.f - s));
                        }
                        ga[j] = pack_bf16x2(x[0], x[1]);
                        gb[j] = pack_bf16x2(y[0], y[1]);
                        hw[j] = pack_bf16x2(h[0], h[1]);
                    }
                    store(ga, 0, f.da, row, args.F, col, valid);
                    store(gb, 1, f.db, row, args.F, col, valid);
                    store(hw, 2, f.h, row, args.F, col, valid);
                }
            } else {
                // Down, Dx: columns of y or dx.  Dw: half 0 of a dw1 | dw3 tile is
                // dw1's columns, half 1 dw3's; dw2 tiles are 256 columns wide, and
                // every warp has 32 rows or none (d and F are multiples of 64).
                const int cols = kOp == kFfnDw && !ti.dw2 ? args.F : args.d;
                const int col0 = kOp == kFfnDw && !ti.dw2 ? ti.n_tile * 128 : ti.n_tile * kBN + half * 128;
                // all columns at once, so that the four loads wait once
                uint32_t w[4][16];
                if (ti.steps > 0) {
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tbase + half * 128 + c * 32, v[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) pack32(v[c], w[c]);
                } else {  // an expert without rows
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[c][j] = 0u;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) hand_back_to(hand_back[buf]);
                returned = true;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int col = col0 + c * 32;
                    if (col >= cols) break;
                    if (kOp == kFfnDw) {
                        if (c % 2 == 0)
                            exchange_send_wide_3d(block, w[c], w[c + 1], lane, &tm_out.m[ti.dw2 ? 2 : half], col,
                                                  static_cast<int>(row), ti.e);
                    } else
                        store(w[c], 0, kOp == kFfnDown ? f.y : f.dx, row, args.d, col, valid);
                }
            }
            if (!returned) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) hand_back_to(hand_back[buf]);
            }
        }
        if (lane == 0) exchange_drain();
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();  // no remote arrive or commit may target a CTA that has left
    griddep_launch_dependents();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

template <int kOp>
static cudaError_t launch_op(const CUtensorMap* m, const FfnOutMaps& out, const FfnSideMaps<kOp>& dw,
                             const FfnTcArgs& a, int64_t max_tiles, int num_sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(ffn_tc_kernel<kOp>), kSmemBytes, done);
    if (e != cudaSuccess) return e;
    int64_t pairs = num_sms / 2;
    if (max_tiles < pairs) pairs = max_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (g_chain_started && pdl_enabled()) ? 2 : 1;
    g_chain_started = true;
    return cudaLaunchKernelEx(&cfg, ffn_tc_kernel<kOp>, m[0], m[1], m[2], m[3], out, dw, a);
}

cudaError_t launch_ffn_tc(int op, const CUtensorMap* maps, const FfnOutMaps& out, const FfnArgs& f,
                          const FfnDwMaps& dw, int num_sms, cudaStream_t st) {
    FfnTcArgs a{};
    a.f = f;
    a.n = f.n;
    a.d = f.d;
    a.F = f.F;
    auto up = [](int64_t v, int64_t by) { return static_cast<int>((v + by - 1) / by); };
    if (op == kFfnDw) {
        a.dw_tiles13 = up(f.d, kBM) * up(f.F, 128);
        a.dw_tiles2 = up(f.F, kBM) * up(f.d, kBN);
        // Runs of four tiles where every next tile would be another expert's (fewer
        // tiles per expert than pairs) and tiles are short (up to three steps): the
        // change, two tensor maps to fetch, costs as much as the tile.  128 experts of
        // 2,048 x 768, with the hidden gradient: 8,192 rows 341 us against 386 one by
        // one, 16,384 rows 400 against 425, 24,576 rows 463 against 474; 8 experts of
        // 4,096 x 14,336, 768 rows: 913 against 778.
        a.dw_run = a.dw_tiles13 + a.dw_tiles2 <= num_sms / 2 && f.R <= 192 * static_cast<int64_t>(f.n) ? 4 : 1;
        return launch_op<kFfnDw>(maps, out, {dw.out}, a, static_cast<int64_t>(f.n) * (a.dw_tiles13 + a.dw_tiles2), num_sms, st);
    }
    const int k = op == kFfnUp || op == kFfnGrad ? f.d : (op == kFfnDown ? f.F : 2 * f.F);
    a.steps = k / kBK;
    a.n_tiles = op == kFfnUp ? up(f.F, 128) : (op == kFfnGrad ? up(f.F, kBN) : up(f.d, kBN));
    // bands of 32 MB of A rows (the forward layer's measured budget)
    const int64_t band = (static_cast<int64_t>(32) << 20) / (static_cast<int64_t>(kBM) * k * 2);
    a.band = static_cast<int>(band < 1 ? 1 : band);
    const int64_t tiles = (f.R / kBM + std::min<int64_t>(f.n, f.R)) * static_cast<int64_t>(a.n_tiles);
    switch (op) {
        case kFfnUp: return launch_op<kFfnUp>(maps, out, {}, a, tiles, num_sms, st);
        case kFfnDown: return launch_op<kFfnDown>(maps, out, {}, a, tiles, num_sms, st);
        case kFfnGrad: return launch_op<kFfnGrad>(maps, out, dw, a, tiles, num_sms, st);
        case kFfnDx: return launch_op<kFfnDx>(maps, out, {}, a, tiles, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
