// ffn.cuh -- what the kernels of the gated feed-forward block over expert
// segments (ffn_simt.cu, gemm_ffn.cu) and of the grouped MXFP4 product share:
// the segment plan that every block derives from the caller's offsets, and the
// block's formulas.
//
//   a = x . w1_e, b = x . w3_e, s = 1 / (1 + e^-a), h = a s b, y = h . w2_e
//   dh = dy . w2_e^T, db = dh a s, da = dh b s (1 + a (1 - s))
//   dx = da . w1_e^T + db . w3_e^T, dw1 = x^T . da, dw3 = x^T . db, dw2 = h^T . dy
//
// Source of the forward: SwiGLU_i(x) = (silu(x.w1_i) (*) x.w3_i) . w2_i
// ("Mixtral of Experts" section 2.1, flash-card page); the backward is its
// derivative.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFfnMaxExperts = 256;

// Segment plan in shared memory: expert e holds rows off[e] .. off[e+1]-1, cut
// into blocks of block_rows rows; blk is the exclusive prefix of the blocks.
struct SegmentPlan {
    int32_t off[kFfnMaxExperts + 1];
    int32_t blk[kFfnMaxExperts + 1];
};

// Every thread of the block (a multiple of 32, at least 32) calls this.
// Offsets come from the caller's device memory: unless they ascend within
// [0, R], every segment is taken as empty and kStatusOffsets is set, so no
// kernel ever addresses a row outside the caller's buffers.  A null `offsets`
// means one segment of all R rows (n = 1).
__device__ __forceinline__ void load_plan(SegmentPlan& p, const int32_t* offsets, int n, int64_t R, int block_rows,
                                          int* status) {
    const int tid = threadIdx.x, nt = blockDim.x;
    for (int i = tid; i <= n; i += nt)
        p.off[i] = offsets ? __ldg(offsets + i) : (i == 0 ? 0 : static_cast<int32_t>(R));
    __syncthreads();
    int bad = 0;
    for (int i = tid; i <= n; i += nt) {
        const int32_t v = p.off[i];
        if (v < 0 || v > R || (i > 0 && v < p.off[i - 1])) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        for (int i = tid; i <= n; i += nt) p.off[i] = p.blk[i] = 0;
        if (tid == 0 && status) atomicOr(status, kStatusOffsets);
        __syncthreads();
        return;
    }
    if (tid < 32) {
        int base = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + tid;
            const int own = i < n ? (p.off[i + 1] - p.off[i] + block_rows - 1) / block_rows : 0;
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += u;
            }
            if (i < n) p.blk[i] = base + incl - own;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (tid == 0) p.blk[n] = base;
    }
    __syncthreads();
}

// The tensor maps of kFfnDw: for every expert a copy of the given ones whose row
// extent (dimension 1) is the end of the expert's segment, so that copies read
// zeros past it.  Called by whole warps, each with 128 bytes of shared memory of
// its own (128-byte aligned); warp `first` of `stride` writes its share.
template <int kMaps>
__device__ __forceinline__ void write_dw_maps(const CUtensorMap (&maps)[kMaps], CUtensorMap* out, void* scratch,
                                              const SegmentPlan& plan, int n, int first, int stride) {
    static_assert(sizeof(CUtensorMap) == 128, "32 words");
    const int lane = threadIdx.x & 31;
    for (int j = first; j < kMaps * n; j += stride) {
        const int which = j / n, e = j - which * n;
        static_cast<uint32_t*>(scratch)[lane] = reinterpret_cast<const uint32_t*>(&maps[which])[lane];
        __syncwarp();
        if (lane == 0)
            asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_u32(scratch)),
                         "r"(max(1, plan.off[e + 1]))
                         : "memory");
        __syncwarp();
        asm volatile(
            "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
                reinterpret_cast<uint64_t>(out + j)),
            "r"(smem_u32(scratch))
            : "memory");
        __syncwarp();
    }
}

// Before a copy by a map that the device wrote.
__device__ __forceinline__ void acquire_map(const CUtensorMap* map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map))
                 : "memory");
}

// Expert that owns row block `b` (b < blk[n]).
__device__ __forceinline__ int plan_expert(const SegmentPlan& p, int n, int b) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.blk[mid] <= b)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A warp's exchange block: 32 rows of 64 bytes in shared memory, the four
// 16-byte pieces of row r at (piece ^ (r / 2 % 4)), free of bank conflicts both
// by rows (a lane its row) and across them (four lanes a row).  The epilogues
// hold one accumulator row per lane; written straight from registers, every
// 16-byte store of a warp touches 32 lines of memory, half a sector each.
// Through the block a store covers 8 rows of 64 contiguous bytes.
constexpr int kExchangeBytes = 32 * 64;

__device__ __forceinline__ uint4* exchange_at(uint8_t* block, int row, int piece) {
    return reinterpret_cast<uint4*>(block + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}

// w: this lane's row, 16 words.  Row r < valid goes to out + r * ld_bytes
// (16-byte aligned).  Every lane of the warp calls this.
__device__ __forceinline__ void exchange_store(uint8_t* block, const uint32_t* w, int lane, int valid,
                                               void* out, int64_t ld_bytes) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *exchange_at(block, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = j * 8 + (lane >> 2), q = lane & 3;
        if (r < valid)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + r * ld_bytes + q * 16) = *exchange_at(block, r, q);
    }
    __syncwarp();
}

// The same through the tensor map of the output (32 x 32 boxes, 64-byte swizzle:
// the block's own layout), for warps whose 32 rows are all to be stored: a
// tenth of the load-store unit's work.  Two blocks take turns; `turn` counts
// the warp's stores.  c0, c1 (, c2): column, row (and expert).
__device__ __forceinline__ uint8_t* exchange_put(uint8_t* blocks, int& turn, const uint32_t* w, int lane) {
    uint8_t* block = blocks + (turn++ & 1) * kExchangeBytes;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the block is free again
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) *exchange_at(block, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    return block;
}
__device__ __forceinline__ void exchange_send_2d(uint8_t* blocks, int& turn, const uint32_t* w, int lane,
                                                 const CUtensorMap* map, int c0, int c1) {
    const uint32_t src = smem_u32(exchange_put(blocks, turn, w, lane));
    if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
            "r"(c0), "r"(c1), "r"(src)
            : "memory");
}
// 64 columns through both blocks together, as 32 rows of 128 bytes (128-byte swizzle).
__device__ __forceinline__ void exchange_send_wide_3d(uint8_t* blocks, const uint32_t* lo, const uint32_t* hi, int lane,
                                                      const CUtensorMap* map, int c0, int c1, int c2) {
    static_assert(2 * kExchangeBytes == 32 * 128, "32 rows of 128 bytes");
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t* w = (q < 4 ? lo : hi) + 4 * (q & 3);
        *reinterpret_cast<uint4*>(blocks + lane * 128 + ((q ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
            "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(blocks))
            : "memory");
}
// Before another use of the blocks, and before the warp ends: every store that
// this lane has sent is complete.
__device__ __forceinline__ void exchange_drain() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void exchange_drain_reads() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The two halves of a load: fetch (in flight until its registers are used) and
// the turn to one row per lane.  Rows past `valid` read zeros.
__device__ __forceinline__ void exchange_fetch(uint4 (&v)[4], int lane, int valid, const void* src, int64_t ld_bytes) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = j * 8 + (lane >> 2), q = lane & 3;
        v[j] = r < valid ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + r * ld_bytes + q * 16)
                         : make_uint4(0u, 0u, 0u, 0u);
    }
}
__device__ __forceinline__ void exchange_turn(uint8_t* block, const uint4 (&v)[4], int lane, uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *exchange_at(block, j * 8 + (lane >> 2), lane & 3) = v[j];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 u = *exchange_at(block, lane, q);
        w[4 * q] = u.x, w[4 * q + 1] = u.y, w[4 * q + 2] = u.z, w[4 * q + 3] = u.w;
    }
    __syncwarp();
}

}  // namespace moe
