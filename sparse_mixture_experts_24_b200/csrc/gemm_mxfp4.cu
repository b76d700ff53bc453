// gemm_mxfp4.cu -- grouped products of MXFP4 rows with the MXFP4 matrices of
// their expert on the sm_100a block-scaled tensor cores:
//   out[r] = A[r] . W_e^T                              (plain)
//   out[r] = silu(A[r] . W_e^T) (*) (A[r] . P_e^T)     (pair)
// A [R][K] and W, P [n][N][K] as codes [..][K/2] and scales [..][K/32]
// (mxfp4.cu).  tcgen05.mma kind::mxf4 multiplies the E2M1 codes with their
// power-of-two scales (one per 32 of K) and accumulates in fp32.
//
// Three kernels:
//   mx_scales_kernel     turns the scales over.  The format keeps a row's scales
//                        contiguous; the tensor core takes, per 128 rows and 128 of
//                        K, 512 bytes with row r's four at 16 (r % 32) + 4 (r / 32).
//                        It writes them as chunks of 1 KB per block of up to 128 rows
//                        (or columns) and step of 256 of K into scratch: a 16th of the
//                        codes' bytes where blocks and steps are whole.  Turned
//                        over by warps of the product kernel instead, from the rows 8
//                        to 16 bytes at a time, they bound it: 8,192 rows over 8
//                        experts, 4,096 x 14,336 twice, 597 to 1,641 us by five ways
//                        of fetching them against 406 + 15 us.
//   mx_gemm_kernel       one CTA per SM, tiles of kTM rows x kBN columns
//   mx_gemm_pair_kernel  CTA pairs, 256 x 256 tiles, for many rows per expert
//
// mx_gemm_kernel, 352 threads, K in steps of 256 (a pair's tile: 128 columns of W
// beside the same 128 of P):
//   warp 0       TMA: codes of the tile's rows and columns (128 bytes per row and
//                step, 128-byte swizzle; past K, N or R the copy reads zeros) and
//                their scale chunks;
//   warp 10      one thread copies a step's scales into tensor memory (tcgen05.cp
//                32x128b.warpx4); a copy holds the scales of two MMAs, told apart
//                by the descriptor's scale id;
//   warp 1       one thread issues the step's four MMAs (M 128, K 64);
//   warps 2-9    epilogue, two per 32 accumulator rows, each on half the columns:
//                the accumulators go to registers and are handed back first.
// kTM = 64 loads only 64 rows of A per tile (batches of few rows per expert); the
// MMA's other 64 rows read whatever follows and are never stored.
// Every wait is bounded (common.cuh).
#include <algorithm>

#include "ffn.cuh"
#include "kernels.h"

namespace moe {

namespace mxg {

constexpr int kBK = 256;                    // K per step: 128 bytes of codes
constexpr int kBBlockBytes = 128 * 128;     // 128 columns
constexpr int kSfBytes = 2 * 512;           // a step's scales of 128 rows
constexpr int kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kCopyWarp = 2 + kEpiWarps;
constexpr int kThreads = (kCopyWarp + 1) * 32;
constexpr int kMaxStages = 7;
constexpr int kPairRows = 256;              // rows of a tile of mx_gemm_pair_kernel

template <int kBN, int kTM>
struct Cfg {
    static constexpr int kBlocks = kBN / 128;
    static constexpr int kABytes = kTM * 128;
    static constexpr int kCodeBytes = kABytes + kBlocks * kBBlockBytes;
    static constexpr int kStageBytes = kCodeBytes + (1 + kBlocks) * kSfBytes;
    static constexpr int kStages = kBN == 128 ? (kTM == 64 ? 7 : 6) : 4;
    static constexpr int kAccBufs = kBN == 128 ? 2 : 1;
    static constexpr int kSfCols = 8 * (1 + kBlocks);  // per stage
    static constexpr int kSfBase = kAccBufs * kBN;
    static_assert(kSfBase + kStages * kSfCols <= kTmemCols && kStages <= kMaxStages, "tensor memory");
    static_assert(kStageBytes % 1024 == 0, "the codes' swizzle");
};

struct __align__(16) Tail {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t scales[kMaxStages];  // in tensor memory
    uint64_t copied;
    uint64_t accum_full[2];
    uint64_t accum_empty[2];
    uint64_t done;
    uint32_t tmem_base;
    SegmentPlan plan;
};
constexpr int kTailBytes = (static_cast<int>(sizeof(Tail)) + 1023) / 1024 * 1024;

// Shared memory, 1 KB aligned: barriers and plan, the ring, an exchange block per
// epilogue warp.
template <int kBN, int kTM>
constexpr int smem_bytes() {
    return kTailBytes + Cfg<kBN, kTM>::kStages * Cfg<kBN, kTM>::kStageBytes + kEpiWarps * kExchangeBytes;
}

struct Tile {
    int e, n_tile, row0, rows;
};

// Tile t -> (expert, column tile, row block), the row block fastest: the
// expert's rows (K / 2 bytes each) stay in L2 while its columns stream past.
template <int kTM>
__device__ __forceinline__ Tile tile_at(int t, const SegmentPlan& p, int n, int n_tiles) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.blk[mid] * n_tiles <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int local = t - p.blk[lo] * n_tiles, count = p.blk[lo + 1] - p.blk[lo];
    Tile ti;
    ti.e = lo;
    ti.n_tile = local / count;
    ti.row0 = p.off[lo] + (local - ti.n_tile * count) * kTM;
    ti.rows = min(kTM, p.off[lo + 1] - ti.row0);
    return ti;
}

// D[tmem] (+)= A x B, E2M1 operands with a power-of-two scale per 32 of K.
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// E2M1 A and B (code 1), E8M0 scales (scale format 1), both K-major; `id`: the
// byte of each 32-bit scale word where this MMA's two scales start.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24) | (id << 29);
}

// fp32 outputs keep the library exponential (2 ulp); the fast division adds 2
// ulp and gives 0 for a below -87, where silu is under 1e-35.
template <bool kBf16Out>
__device__ __forceinline__ float silu(float a) {
    return __fdividef(a, 1.f + (kBf16Out ? __expf(-a) : expf(-a)));
}

// Columns col .. col+31 of 32 rows of out (a lane its row, `valid` of them).
// Rows that are whole vectors go through the warp's exchange block, others
// element by element.
template <bool kBf16>
__device__ __forceinline__ void store_rows(uint8_t* block, void* out, int64_t row0, int valid, int lane, int N,
                                           int col, const uint32_t (&v)[32]) {
    if (kBf16) {
        uint16_t* o = static_cast<uint16_t*>(out) + row0 * N + col;
        if (N % 8 == 0 && col + 32 <= N) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            exchange_store(block, w, lane, valid, o, static_cast<int64_t>(N) * 2);
        } else if (lane < valid) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col + j < N)
                    o[static_cast<int64_t>(lane) * N + j] =
                        static_cast<uint16_t>(pack_bf16x2(__uint_as_float(v[j]), 0.f));
        }
    } else {
        float* o = static_cast<float*>(out) + row0 * N + col;
        if (N % 4 == 0 && col + 32 <= N) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                exchange_store(block, v + 16 * h, lane, valid, o + 16 * h, static_cast<int64_t>(N) * 4);
        } else if (lane < valid) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col + j < N) o[static_cast<int64_t>(lane) * N + j] = __uint_as_float(v[j]);
        }
    }
}

}  // namespace mxg

using namespace mxg;

template <bool kPair, bool kBf16Out, int kBN, int kTM>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_b2, const __grid_constant__ CUtensorMap tm_chunks,
                   const MxGemmArgs args, const MxChunks ch) {
    using C = Cfg<kBN, kTM>;
    static_assert(!kPair || kBN == 256, "a pair's tile is one block of each matrix");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Tail* tail = reinterpret_cast<Tail*>(smem_raw);
    uint8_t* smem = smem_raw + kTailBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kColsOut = kPair ? 128 : kBN;  // output columns of a tile
    const int n_tiles = (args.N + kColsOut - 1) / kColsOut;
    const int steps = ch.steps;
    int* status = args.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&tail->full[s]), 1);
            mbar_init(smem_u32(&tail->empty[s]), 1);
            mbar_init(smem_u32(&tail->scales[s]), 1);
        }
        mbar_init(smem_u32(&tail->copied), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tail->accum_full[b]), 1);
            mbar_init(smem_u32(&tail->accum_empty[b]), kEpiWarps);
        }
        mbar_init(smem_u32(&tail->done), 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_chunks);
        if (kPair) tma_prefetch_desc(&tm_b2);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    load_plan(tail->plan, args.offsets, args.n, args.R, kTM, status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tail->tmem_base;
    const SegmentPlan& plan = tail->plan;
    const int total = plan.blk[args.n] * n_tiles;
    const int first = blockIdx.x, stride = gridDim.x;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            auto codes = [&](const Tile& ti, int ks, int stage) {
                const uint32_t fb = smem_u32(&tail->full[stage]);
                mbar_arrive_expect_tx(fb, C::kStageBytes);
                const uint32_t base = smem_u32(smem + stage * C::kStageBytes);
                tma_load_2d(base, &tm_a, fb, ks * 128, ti.row0);
#pragma unroll
                for (int b = 0; b < C::kBlocks; ++b)
                    tma_load_3d(base + C::kABytes + b * kBBlockBytes, kPair && b == 1 ? &tm_b2 : &tm_b, fb, ks * 128,
                                kPair ? ti.n_tile * 128 : ti.n_tile * kBN + b * 128, ti.e);
            };
            // The ring's first codes do not depend on the kernel before, which turns the
            // scales over: they are on their way while it runs.
            const int ahead = first < total ? min(C::kStages, steps) : 0;
            for (int ks = 0; ks < ahead; ++ks) codes(tile_at<kTM>(first, plan, args.n, n_tiles), ks, ks);
            griddep_wait();
            int stage = 0;
            uint32_t phase = 0;
            int armed[kMaxStages];
            for (int s = 0; s < kMaxStages; ++s) armed[s] = -1;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride) {
                const Tile ti = tile_at<kTM>(t, plan, args.n, n_tiles);
                // chunks of the tile's rows, and of its blocks of 128 columns
                const int sa = (plan.blk[ti.e] + (ti.row0 - plan.off[ti.e]) / kTM) * steps;
                const int cols = ch.a_blocks + ti.e * ch.col_blocks;
                const int c0 = kPair ? ti.n_tile : C::kBlocks * ti.n_tile;
                for (int ks = 0; ks < steps; ++ks) {
                    if (t != first || ks >= ahead) {
                        if (!mbar_wait(smem_u32(&tail->empty[stage]), phase ^ 1u, status, kStatusTimeoutEmpty)) {
                            ok = false;
                            break;
                        }
                        codes(ti, ks, stage);
                    }
                    armed[stage] = static_cast<int>(phase);
                    const uint32_t fb = smem_u32(&tail->full[stage]);
                    const uint32_t sf = smem_u32(smem + stage * C::kStageBytes) + C::kCodeBytes;
                    tma_load_2d(sf, &tm_chunks, fb, 0, sa + ks);
#pragma unroll
                    for (int b = 0; b < C::kBlocks; ++b) {
                        // a last, lone block of columns: the second one's outputs are not stored
                        const int c = kPair ? c0 + b * args.n * ch.col_blocks : min(c0 + b, ch.col_blocks - 1);
                        tma_load_2d(sf + (1 + b) * kSfBytes, &tm_chunks, fb, 0, (cols + c) * steps + ks);
                    }
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // nothing may still be landing when the CTA exits
            for (int s = 0; s < C::kStages; ++s)
                if (armed[s] >= 0)
                    mbar_wait(smem_u32(&tail->full[s]), static_cast<uint32_t>(armed[s]), status, kStatusTimeoutDrain);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride, ++local) {
                const int buf = C::kAccBufs == 2 ? (local & 1) : 0;
                const uint32_t use = static_cast<uint32_t>(C::kAccBufs == 2 ? local >> 1 : local);
                if (!mbar_wait(smem_u32(&tail->accum_empty[buf]), (use & 1u) ^ 1u, status, kStatusTimeoutAccum)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kBN);
                for (int ks = 0; ks < steps; ++ks) {
                    // the stage's scales are in tensor memory, so its codes have landed too
                    if (!mbar_wait(smem_u32(&tail->scales[stage]), phase, status, kStatusTimeoutFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = smem_u32(smem + stage * C::kStageBytes);
                    const uint32_t sf = tmem_base + static_cast<uint32_t>(C::kSfBase + stage * C::kSfCols);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int c = kk >> 1;
                        const uint64_t ad = make_smem_desc(base + kk * 32, 16, 1024, 2);
                        const uint64_t bd = make_smem_desc(base + C::kABytes + kk * 32, 16, 1024, 2);
                        mma_mxf4(d_tmem, ad, bd, (kk & 1) ? idesc_mxf4(128, kBN, 2) : idesc_mxf4(128, kBN, 0),
                                 sf + 4 * c, sf + 8 + 4 * C::kBlocks * c, (ks | kk) != 0 ? 1u : 0u);
                    }
                    tc_commit(smem_u32(&tail->empty[stage]));
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) tc_commit(smem_u32(&tail->accum_full[buf]));
            }
            // every MMA is done before tensor memory is freed
            tc_commit(smem_u32(&tail->done));
            mbar_wait(smem_u32(&tail->done), 0, status, kStatusTimeoutDrain);
        }
    } else if (warp == kCopyWarp) {
        if (lane == 0) {
            // ---------------- scales into tensor memory ----------------
            // Tensor memory: A's two chunks, then for either chunk the blocks of B.  A
            // stage's columns are written again only after its next full barrier, which
            // follows the MMAs that read them.
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride) {
                for (int ks = 0; ks < steps; ++ks) {
                    if (!mbar_wait(smem_u32(&tail->full[stage]), phase, status, kStatusTimeoutFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf_smem = smem_u32(smem + stage * C::kStageBytes) + C::kCodeBytes;
                    const uint32_t sf = tmem_base + static_cast<uint32_t>(C::kSfBase + stage * C::kSfCols);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tc_cp_32x128b_warpx4(sf + 4 * c, make_smem_desc(sf_smem + c * 512, 0, 128, 0));
#pragma unroll
                        for (int b = 0; b < C::kBlocks; ++b)
                            tc_cp_32x128b_warpx4(sf + 8 + 4 * (c * C::kBlocks + b),
                                                 make_smem_desc(sf_smem + (1 + b) * kSfBytes + c * 512, 0, 128, 0));
                    }
                    tc_commit(smem_u32(&tail->scales[stage]));
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            tc_commit(smem_u32(&tail->copied));
            mbar_wait(smem_u32(&tail->copied), 0, status, kStatusTimeoutDrain);
        }
    } else {
        // ---------------- epilogue (warps 2..9) ----------------
        const int quad = warp & 3;         // TMEM lanes 32 * quad .. + 31
        const int half = (warp - 2) >> 2;  // half of the columns
        constexpr int kChunks = kBN / 64;  // 32-column chunks per warp
        uint8_t* block = smem + C::kStages * C::kStageBytes + (warp - 2) * kExchangeBytes;
        int local = 0;
        for (int t = first; t < total; t += stride, ++local) {
            const Tile ti = tile_at<kTM>(t, plan, args.n, n_tiles);
            const int buf = C::kAccBufs == 2 ? (local & 1) : 0;
            const uint32_t use = static_cast<uint32_t>(C::kAccBufs == 2 ? local >> 1 : local);
            if (!mbar_wait(smem_u32(&tail->accum_full[buf]), use & 1u, status, kStatusTimeoutAccum)) break;
            tc_fence_after();
            const uint32_t tbase =
                tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(buf * kBN);
            const int valid = min(32, ti.rows - quad * 32);  // warp-uniform
            const bool any = valid > 0;
            const int64_t row0 = static_cast<int64_t>(ti.row0) + quad * 32;
            uint32_t acc[kChunks][32];
            if (any) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    // pair: chunks of W (0, 2) and the same of P (1, 3)
                    tmem_ld_32x32b_x32(tbase + (kPair ? half * 64 + (i >> 1) * 32 + (i & 1) * 128
                                                      : (half * kChunks + i) * 32),
                                       acc[i]);
                tmem_wait_ld();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&tail->accum_empty[buf]));
            if (any) {
#pragma unroll
                for (int i = 0; i < (kPair ? kChunks / 2 : kChunks); ++i) {
                    const int col = kPair ? ti.n_tile * 128 + half * 64 + i * 32
                                          : ti.n_tile * kBN + (half * kChunks + i) * 32;
                    if (col < args.N) {
                        uint32_t(&v)[32] = acc[kPair ? 2 * i : i];
                        if (kPair) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint(silu<kBf16Out>(__uint_as_float(v[j])) *
                                                       __uint_as_float(acc[(2 * i + 1) % kChunks][j]));
                        }
                        store_rows<kBf16Out>(block, args.out, row0, valid, lane, args.N, col, v);
                    }
                }
            }
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    griddep_launch_dependents();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// The same on CTA pairs (cta_group::2) for many rows per expert: 256 x 256
// tiles, each CTA its own 128 rows and 128 of the columns.
// ---------------------------------------------------------------------------
// A 128 x 256 tile brings 48 KB of codes for the 510 cycles of its four MMAs,
// more than an SM gets from L2 in that time; a pair's CTA brings 32 KB for the
// same products.  What differs from mx_gemm_kernel:
//   - the leader's MMA thread issues the pair's copies and MMAs; a copy moves
//     either CTA's own shared memory into its own tensor memory: the scales of
//     its rows, and of all 256 columns;
//   - outputs leave by TMA through the warps' exchange blocks where all 32 rows
//     are stored and a row of out is a multiple of 16 bytes.
namespace mxp {

constexpr int kStages = 5;
constexpr int kCodeBytes = 2 * 128 * 128;             // 128 rows, 128 columns
constexpr int kStageBytes = kCodeBytes + 3 * kSfBytes;  // scales of 128 rows, 256 columns
constexpr int kSfCols = 24, kSfBase = 256;

struct __align__(16) Tail {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t scales[kStages];  // in tensor memory
    uint64_t copied;
    uint64_t accum_full;
    uint64_t accum_empty;
    uint64_t done;
    uint32_t tmem_base;
    SegmentPlan plan;
};
// Shared memory, 1 KB aligned: barriers and plan, the ring, two exchange blocks
// per epilogue warp.
constexpr int kTailBytes = (static_cast<int>(sizeof(Tail)) + 1023) / 1024 * 1024;
constexpr int kSmemBytes = kTailBytes + kStages * kStageBytes + 2 * kEpiWarps * kExchangeBytes;
static_assert(kSmemBytes <= 232448 && kStageBytes % 1024 == 0 && kSfBase + kStages * kSfCols <= kTmemCols, "budget");

__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

}  // namespace mxp

template <bool kPair, bool kBf16Out>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_b2, const __grid_constant__ CUtensorMap tm_out,
                        const __grid_constant__ CUtensorMap tm_chunks, const MxGemmArgs args, const MxChunks ch,
                        const int out_by_map) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    mxp::Tail* tail = reinterpret_cast<mxp::Tail*>(smem_raw);
    uint8_t* smem = smem_raw + mxp::kTailBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    constexpr int kColsOut = kPair ? 128 : 256;  // output columns of a tile
    const int n_tiles = (args.N + kColsOut - 1) / kColsOut;
    const int steps = ch.steps;
    int* status = args.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < mxp::kStages; ++s) {
            mbar_init(smem_u32(&tail->full[s]), 1);
            mbar_init(smem_u32(&tail->empty[s]), 1);
            mbar_init(smem_u32(&tail->scales[s]), 1);
        }
        mbar_init(smem_u32(&tail->copied), 1);
        mbar_init(smem_u32(&tail->accum_full), 1);
        mbar_init(smem_u32(&tail->accum_empty), 2 * kEpiWarps);
        mbar_init(smem_u32(&tail->done), 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        if (kPair) tma_prefetch_desc(&tm_b2);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&tail->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    load_plan(tail->plan, args.offsets, args.n, args.R, kPairRows, status);
    griddep_wait();  // the scales' chunks
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = tail->tmem_base;
    const SegmentPlan& plan = tail->plan;
    const int total = plan.blk[args.n] * n_tiles;
    const int first = static_cast<int>(cluster_id_x()), stride = static_cast<int>(nclusters_x());
    const int r128 = 128 * static_cast<int>(rank);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int stage = 0;
            uint32_t phase = 0;
            int armed[mxp::kStages];
            for (int s = 0; s < mxp::kStages; ++s) armed[s] = -1;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride) {
                const Tile ti = tile_at<kPairRows>(t, plan, args.n, n_tiles);
                // this CTA's 128 rows, and the tile's two blocks of 128 columns
                const int m = (ti.row0 - plan.off[ti.e]) / kPairRows;
                const int sa = ((plan.blk[ti.e] + m) * 2 + static_cast<int>(rank)) * steps;
                const int cols = ch.a_blocks + ti.e * ch.col_blocks;
                const int c0 = kPair ? ti.n_tile : 2 * ti.n_tile;
                const int sb0 = (cols + c0) * steps;
                // a last, lone block of columns: the second one's outputs are not stored
                const int sb1 = (kPair ? cols + args.n * ch.col_blocks + c0
                                       : cols + min(c0 + 1, ch.col_blocks - 1)) * steps;
                for (int ks = 0; ks < steps; ++ks) {
                    if (!mbar_wait(smem_u32(&tail->empty[stage]), phase ^ 1u, status, kStatusTimeoutEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_local = smem_u32(&tail->full[stage]);
                    if (rank == 0) {
                        mbar_arrive_expect_tx(full_local, 2 * mxp::kStageBytes);
                        armed[stage] = static_cast<int>(phase);
                    }
                    const uint32_t full = mapa_shared(full_local, 0);
                    const uint32_t base = smem_u32(smem + stage * mxp::kStageBytes);
                    tma_load_2d_pair(base, &tm_a, full, ks * 128, ti.row0 + r128);
                    tma_load_3d_pair(base + kBBlockBytes, kPair && rank ? &tm_b2 : &tm_b, full, ks * 128,
                                     kPair ? ti.n_tile * 128 : ti.n_tile * 256 + r128, ti.e);
                    const uint32_t sf = base + mxp::kCodeBytes;
                    tma_load_2d_pair(sf, &tm_chunks, full, 0, sa + ks);
                    tma_load_2d_pair(sf + kSfBytes, &tm_chunks, full, 0, sb0 + ks);
                    tma_load_2d_pair(sf + 2 * kSfBytes, &tm_chunks, full, 0, sb1 + ks);
                    if (++stage == mxp::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the leader's barriers count both CTAs' copies: nothing may still be
            // landing when the pair exits
            if (rank == 0)
                for (int s = 0; s < mxp::kStages; ++s)
                    if (armed[s] >= 0)
                        mbar_wait(smem_u32(&tail->full[s]), static_cast<uint32_t>(armed[s]), status,
                                  kStatusTimeoutDrain);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer (leader) ----------------
            int stage = 0;
            uint32_t phase = 0, use = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride, ++use) {
                if (!mbar_wait(smem_u32(&tail->accum_empty), (use & 1u) ^ 1u, status, kStatusTimeoutAccum)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int ks = 0; ks < steps; ++ks) {
                    // the stage's scales are in tensor memory, so its codes have landed too
                    if (!mbar_wait(smem_u32(&tail->scales[stage]), phase, status, kStatusTimeoutFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = smem_u32(smem + stage * mxp::kStageBytes);
                    const uint32_t sf = tmem_base + static_cast<uint32_t>(mxp::kSfBase + stage * mxp::kSfCols);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int c = kk >> 1;
                        const uint64_t ad = make_smem_desc(base + kk * 32, 16, 1024, 2);
                        const uint64_t bd = make_smem_desc(base + kBBlockBytes + kk * 32, 16, 1024, 2);
                        mxp::mma(tmem_base, ad, bd, (kk & 1) ? idesc_mxf4(256, 256, 2) : idesc_mxf4(256, 256, 0),
                                 sf + 4 * c, sf + 8 + 8 * c, (ks | kk) != 0 ? 1u : 0u);
                    }
                    const uint32_t eb = smem_u32(&tail->empty[stage]);
                    tc_commit_pair(mapa_shared(eb, 0));
                    tc_commit_pair(mapa_shared(eb, 1));
                    if (++stage == mxp::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) {
                    const uint32_t fb = smem_u32(&tail->accum_full);
                    tc_commit_pair(mapa_shared(fb, 0));
                    tc_commit_pair(mapa_shared(fb, 1));
                }
            }
            tc_commit_pair(mapa_shared(smem_u32(&tail->done), 0));
            mbar_wait(smem_u32(&tail->done), 0, status, kStatusTimeoutDrain);
        }
    } else if (warp == kCopyWarp) {
        if (lane == 0 && rank == 0) {
            // ---------------- scales into tensor memory (leader) ----------------
            // A stage's columns are written again only after its next full barrier,
            // which follows the MMAs that read them.
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride) {
                for (int ks = 0; ks < steps; ++ks) {
                    if (!mbar_wait(smem_u32(&tail->full[stage]), phase, status, kStatusTimeoutFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf_smem = smem_u32(smem + stage * mxp::kStageBytes) + mxp::kCodeBytes;
                    const uint32_t sf = tmem_base + static_cast<uint32_t>(mxp::kSfBase + stage * mxp::kSfCols);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        mxp::copy_scales(sf + 4 * c, make_smem_desc(sf_smem + c * 512, 0, 128, 0));
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            mxp::copy_scales(sf + 8 + 4 * (2 * c + b),
                                             make_smem_desc(sf_smem + (1 + b) * kSfBytes + c * 512, 0, 128, 0));
                    }
                    tc_commit_pair(mapa_shared(smem_u32(&tail->scales[stage]), 0));
                    if (++stage == mxp::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            tc_commit_pair(mapa_shared(smem_u32(&tail->copied), 0));
            mbar_wait(smem_u32(&tail->copied), 0, status, kStatusTimeoutDrain);
        }
    } else {
        // ---------------- epilogue (warps 2..9 of both CTAs) ----------------
        const int quad = warp & 3;         // TMEM lanes 32 * quad .. + 31
        const int half = (warp - 2) >> 2;  // accumulator columns 128 * half .. (a pair: 64 * half of either)
        uint8_t* block = smem + mxp::kStages * mxp::kStageBytes + (warp - 2) * (2 * kExchangeBytes);
        const uint32_t hand_back = mapa_shared(smem_u32(&tail->accum_empty), 0);
        int turn = 0;
        uint32_t use = 0;
        for (int t = first; t < total; t += stride, ++use) {
            const Tile ti = tile_at<kPairRows>(t, plan, args.n, n_tiles);
            if (!mbar_wait(smem_u32(&tail->accum_full), use & 1u, status, kStatusTimeoutAccum)) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
            const int valid = min(32, ti.rows - r128 - quad * 32);  // warp-uniform
            const int64_t row0 = static_cast<int64_t>(ti.row0) + r128 + quad * 32;
            uint32_t acc[4][32];
            if (valid > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmem_ld_32x32b_x32(
                        tbase + (kPair ? half * 64 + (i >> 1) * 32 + (i & 1) * 128 : half * 128 + i * 32), acc[i]);
                tmem_wait_ld();
            }
            // relaxed: the loads above are complete, and nothing else has to be
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(hand_back)
                             : "memory");
            if (valid > 0) {
#pragma unroll
                for (int i = 0; i < (kPair ? 2 : 4); ++i) {
                    const int col = kPair ? ti.n_tile * 128 + half * 64 + i * 32 : ti.n_tile * 256 + half * 128 + i * 32;
                    if (col >= args.N) break;
                    uint32_t(&v)[32] = acc[kPair ? 2 * i : i];
                    if (kPair) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(silu<kBf16Out>(__uint_as_float(v[j])) *
                                                   __uint_as_float(acc[(2 * i + 1) & 3][j]));
                    }
                    if (out_by_map && valid == 32) {
                        if (kBf16Out) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                v[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                            exchange_send_2d(block, turn, v, lane, &tm_out, col, static_cast<int>(row0));
                        } else {
                            exchange_send_2d(block, turn, v, lane, &tm_out, col, static_cast<int>(row0));
                            if (col + 16 < args.N)
                                exchange_send_2d(block, turn, v + 16, lane, &tm_out, col + 16, static_cast<int>(row0));
                        }
                    } else {
                        if (lane == 0) exchange_drain_reads();
                        __syncwarp();
                        store_rows<kBf16Out>(block, args.out, row0, valid, lane, args.N, col, v);
                    }
                }
            }
            __syncwarp();
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

// Scales [rows][nb] -> chunks [block][step][1024].  One block of threads per
// chunk row: the row blocks of A in the order of the product's tiles (ch.tile_rows
// rows each, 256 as two blocks of 128), then the 128-column blocks of W, then of P.
// kWords: words of a row taken at a time, a power of two, so that short rows leave no
// lane idle (128 blocks of 213 rows and 1,912 columns, K 480: 27 us with 32 words for all).
template <int kWords>
__global__ void __launch_bounds__(256) mx_scales_kernel(const MxGemmArgs args, const MxChunks ch) {
    __shared__ SegmentPlan plan;
    __shared__ uint32_t slab[128][kWords + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int nb = args.K / 32, steps = ch.steps;
    int64_t block = blockIdx.x;
    uint8_t* dst = ch.base + block * steps * kSfBytes;
    const uint8_t* src;  // the block's first row, and how many it has
    int rows;
    if (block < ch.a_blocks) {
        load_plan(plan, args.offsets, args.n, args.R, ch.tile_rows, args.status);
        const int halves = ch.tile_rows == kPairRows ? 2 : 1, height = ch.tile_rows / halves;
        const int tile = static_cast<int>(block / halves);
        if (tile >= plan.blk[args.n]) return;
        const int e = plan_expert(plan, args.n, tile);
        const int64_t row = static_cast<int64_t>(plan.off[e]) +
                            static_cast<int64_t>(tile - plan.blk[e]) * ch.tile_rows + height * (block % halves);
        rows = static_cast<int>(min(static_cast<int64_t>(height), plan.off[e + 1] - row));
        src = args.a_scales + row * nb;
    } else {
        block -= ch.a_blocks;
        const int64_t own = static_cast<int64_t>(args.n) * ch.col_blocks;
        const bool second = block >= own;
        if (second) block -= own;
        const int64_t e = block / ch.col_blocks;
        // an expert without rows has no tile that reads these (8 experts of 14,336 x 4,096,
        // gated pairs, one row: 33.7 us with them, 20.8 without)
        if (args.offsets && __ldg(args.offsets + e) == __ldg(args.offsets + e + 1)) return;
        const int64_t col = (block - e * ch.col_blocks) * 128;
        rows = static_cast<int>(min(static_cast<int64_t>(128), args.N - col));
        src = (second ? args.b2_scales : args.b_scales) + (e * args.N + col) * nb;
    }
    // Slabs of kWords / 2 steps through shared memory: reads of up to 128 bytes of a
    // row, 512 contiguous bytes written by a warp.
    constexpr int kAtOnce = 256 / kWords, kTurns = 128 / kAtOnce, kSlab = kWords / 2;
    const int q = threadIdx.x % kWords, r0 = threadIdx.x / kWords;
    for (int s0 = 0; s0 < steps; s0 += kSlab) {
        const int n_steps = min(kSlab, steps - s0), have = nb - 8 * s0;
        uint32_t v[kTurns];  // all in flight together; past the row's end the smallest scale
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            const int r = r0 + kAtOnce * j;
            const uint8_t* p = src + static_cast<int64_t>(r) * nb + 8 * s0 + 4 * q;
            v[j] = 0u;
            if (r < rows && 4 * q < have) {
                if (ch.words) {
                    v[j] = __ldg(reinterpret_cast<const uint32_t*>(p));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * q + i < have) v[j] |= static_cast<uint32_t>(__ldg(p + i)) << (8 * i);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kTurns; ++j) slab[r0 + kAtOnce * j][q] = v[j];
        __syncthreads();
        // 16 bytes: rows i, i + 32, i + 64, i + 96 of one word
        for (int u = threadIdx.x; u < n_steps * 64; u += 256) {
            const int i = u & 31, w = u >> 5;
            reinterpret_cast<uint4*>(dst + static_cast<int64_t>(s0) * kSfBytes)[u] =
                make_uint4(slab[i][w], slab[i + 32][w], slab[i + 64][w], slab[i + 96][w]);
        }
        __syncthreads();
    }
}

int64_t mx_gemm_most_chunks(int64_t R, int n, int N, int K, int pair) {
    // any tile height, for R rows or fewer: 64-row tiles have the most blocks
    const int64_t rows = (R + 63) / 64 + 2 * static_cast<int64_t>(n);
    return (rows + static_cast<int64_t>(n) * ((N + 127) / 128) * (1 + pair)) * ((K + kBK - 1) / kBK);
}

MxChunks mx_gemm_chunks(const MxGemmArgs& a, int num_sms) {
    MxChunks ch{};
    const int64_t pair_cols = a.b2_codes ? 128 : 256;
    // By the average alone: the offsets are on the device.  However skewed the rows are,
    // the results are the same; only the choice may then be the slower one.
    // CTA pairs where the experts average at least 256 rows and the tiles fill the
    // pairs (4,096 rows over 8 experts of 14,336 x 4,096: 137 us against 148 for
    // 128-row tiles; 1,024 rows: 65 against 64); 64-row tiles where they average at
    // most 48, so that ragged experts mostly end in their first tile (one row, a
    // gated pair of that size: 18.9 against 21.7 us; 4,099 rows over 128 experts of
    // 2,048 x 768 the same; 8,192 rows 50 against 45).
    if (a.R >= 256 * static_cast<int64_t>(a.n) && (a.R / 256) * ((a.N + pair_cols - 1) / pair_cols) >= num_sms / 2)
        ch.tile_rows = kPairRows;
    else
        ch.tile_rows = a.R <= 48 * static_cast<int64_t>(a.n) ? 64 : 128;
    const int halves = ch.tile_rows == kPairRows ? 2 : 1;
    ch.steps = (a.K + kBK - 1) / kBK;
    ch.a_blocks = static_cast<int>(halves * (a.R / ch.tile_rows + std::min<int64_t>(a.n, a.R)));
    ch.col_blocks = (a.N + 127) / 128;
    ch.blocks = ch.a_blocks + static_cast<int64_t>(a.n) * ch.col_blocks * (a.b2_codes ? 2 : 1);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.a_scales) | reinterpret_cast<uintptr_t>(a.b_scales) |
                         reinterpret_cast<uintptr_t>(a.b2_scales) | static_cast<uintptr_t>(a.K / 32);
    ch.words = at % 4 == 0 ? 1 : 0;
    return ch;
}

template <bool kPair, bool kBf16Out>
static cudaError_t launch_pairs(const CUtensorMap* m, const MxGemmArgs& a, const MxChunks& ch, int num_sms,
                                cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(mx_gemm_pair_kernel<kPair, kBf16Out>), mxp::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = mxp::kSmemBytes;
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
    return cudaLaunchKernelEx(&cfg, mx_gemm_pair_kernel<kPair, kBf16Out>, m[0], m[1], m[2], m[3], m[4], a, ch,
                              a.N % (kBf16Out ? 8 : 4) == 0 ? 1 : 0);
}

template <bool kPair, bool kBf16Out, int kBN, int kTM>
static cudaError_t launch(const CUtensorMap* m, const MxGemmArgs& a, const MxChunks& ch, int num_sms,
                          cudaStream_t st) {
    constexpr int smem = smem_bytes<kBN, kTM>();
    static_assert(smem <= 232448, "shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(mx_gemm_kernel<kPair, kBf16Out, kBN, kTM>), smem, done);
    if (e != cudaSuccess) return e;
    const int64_t n_tiles = (a.N + (kPair ? 128 : kBN) - 1) / (kPair ? 128 : kBN);
    int64_t g = (a.R / kTM + std::min<int64_t>(a.n, a.R)) * n_tiles;
    if (g > num_sms) g = num_sms;
    return launch_k(mx_gemm_kernel<kPair, kBf16Out, kBN, kTM>, dim3(static_cast<unsigned>(g)), dim3(kThreads), smem,
                    st, m[0], m[1], m[2], m[4], a, ch);
}

template <bool kBf16Out, int kTM>
static cudaError_t launch_single(const CUtensorMap* m, const MxGemmArgs& a, const MxChunks& ch, int num_sms,
                                 cudaStream_t st) {
    if (a.b2_codes) return launch<true, kBf16Out, 256, kTM>(m, a, ch, num_sms, st);
    // 256-column tiles halve the reads of A (300 rows over 8 experts of 14,336 x
    // 4,096: 51.3 us against 52.9); 128-column ones are taken when the wide ones would
    // leave SMs without a tile (one row, one such expert: 14.4 against 16.5)
    const int64_t tiles = std::max<int64_t>((a.R + kTM - 1) / kTM, std::min<int64_t>(a.n, a.R)) * ((a.N + 255) / 256);
    return tiles >= num_sms ? launch<false, kBf16Out, 256, kTM>(m, a, ch, num_sms, st)
                            : launch<false, kBf16Out, 128, kTM>(m, a, ch, num_sms, st);
}

template <bool kBf16Out>
static cudaError_t launch_product(const CUtensorMap* m, const MxGemmArgs& a, const MxChunks& ch, int num_sms,
                                  cudaStream_t st) {
    if (ch.tile_rows == kPairRows)
        return a.b2_codes ? launch_pairs<true, kBf16Out>(m, a, ch, num_sms, st)
                          : launch_pairs<false, kBf16Out>(m, a, ch, num_sms, st);
    return ch.tile_rows == 64 ? launch_single<kBf16Out, 64>(m, a, ch, num_sms, st)
                              : launch_single<kBf16Out, 128>(m, a, ch, num_sms, st);
}

cudaError_t launch_mx_gemm(const CUtensorMap* m, const MxGemmArgs& a, bool bf16_out, const MxChunks& ch, int num_sms,
                           cudaStream_t st) {
    const dim3 blocks(static_cast<unsigned>(ch.blocks)), threads(256);
    cudaError_t e = ch.steps <= 2   ? launch_k(mx_scales_kernel<4>, blocks, threads, 0, st, a, ch)
                    : ch.steps <= 4 ? launch_k(mx_scales_kernel<8>, blocks, threads, 0, st, a, ch)
                    : ch.steps <= 8 ? launch_k(mx_scales_kernel<16>, blocks, threads, 0, st, a, ch)
                                    : launch_k(mx_scales_kernel<32>, blocks, threads, 0, st, a, ch);
    if (e != cudaSuccess) return e;
    return bf16_out ? launch_product<true>(m, a, ch, num_sms, st) : launch_product<false>(m, a, ch, num_sms, st);
}

}  // namespace moe
