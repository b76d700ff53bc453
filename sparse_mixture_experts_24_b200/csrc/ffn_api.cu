// ffn_api.cu -- the C ABI of the gated feed-forward block over expert segments
// (forward, backward) and of MXFP4 (quantisation, grouped product), declared in
// include/moe.h: argument checks, workspace, launch sequences.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/moe.h"
#include "handle.h"
#include "kernels.h"

using moe_api_detail::done;
using moe_api_detail::failed;
using moe_api_detail::HandleView;
using moe_api_detail::open_handle;

namespace {

moe_status cuda_failed(cudaError_t e, const char* what) {
    return failed(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define FFN_REQUIRE_PTR(p)                                                                      \
    do {                                                                                        \
        if (!(p)) return failed(MOE_ERR_INVALID_ARG, "%s is NULL", #p);                         \
        if (!aligned16(p)) return failed(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
    } while (0)

moe_status check_rows(int64_t R, const char* name = "R") {
    if (R < 0) return failed(MOE_ERR_INVALID_ARG, "%s = %lld < 0", name, static_cast<long long>(R));
    if (R > 2147483647LL - 256)
        return failed(MOE_ERR_INVALID_ARG, "%s = %lld exceeds 2^31 - 257", name, static_cast<long long>(R));
    return MOE_OK;
}

// offsets may be left out for one expert only; 4-byte integers, so their own
// alignment is what is asked of them.
moe_status check_offsets(int n, const int32_t* offsets) {
    if (!offsets && n != 1) return failed(MOE_ERR_INVALID_ARG, "offsets is NULL with n = %d experts", n);
    if (reinterpret_cast<uintptr_t>(offsets) & 3u)
        return failed(MOE_ERR_INVALID_ARG, "offsets is not 4-byte aligned");
    return MOE_OK;
}

// Whether `st` is being captured (a reservation is not on a stream).
moe_status capturing(cudaStream_t st, bool on_stream, bool* yes) {
    *yes = false;
    if (!on_stream) return MOE_OK;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cap);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_failed(e, "cudaStreamIsCapturing");
    }
    *yes = cap != cudaStreamCaptureStatusNone;
    return MOE_OK;
}

// At least `bytes` in b.
moe_status room(moe::FfnWorkspace* w, moe::FfnBuffer* b, int64_t bytes, bool capture) {
    if (bytes > b->bytes) {
        if (capture)
            return failed(MOE_ERR_INVALID_ARG,
                          "the workspace is too small and cannot grow while the stream is captured: call "
                          "moe_reserve_ffn or moe_reserve_matmul_mxfp4 first");
        if (b->p) {
            if (b->captured) {
                try {
                    w->kept.push_back(b->p);
                } catch (...) {  // no exception leaves a C entry point
                    return failed(MOE_ERR_ALLOC, "out of host memory");
                }
            } else {
                cudaFree(b->p);
            }
            *b = moe::FfnBuffer{};
        }
        cudaError_t e = cudaMalloc(&b->p, static_cast<size_t>(bytes));
        if (e != cudaSuccess) {
            cudaGetLastError();
            *b = moe::FfnBuffer{};
            return failed(MOE_ERR_ALLOC, "cudaMalloc(%lld bytes) for the workspace failed: %s",
                          static_cast<long long>(bytes), cudaGetErrorString(e));
        }
        b->bytes = bytes;
    }
    b->captured |= capture;
    return MOE_OK;
}

// The status word and the tensor maps; then room for `rows` hidden rows and, for
// the backward pass, their gradients; and for `chunks` KB of turned-over scales.
moe_status need(const HandleView& v, int64_t rows, bool backward, int64_t chunks, cudaStream_t st, bool on_stream) {
    moe::FfnWorkspace* w = v.ffn;
    bool capture = false;
    moe_status s = capturing(st, on_stream, &capture);
    if (s != MOE_OK) return s;
    if (!w->fixed.p) {
        s = room(w, &w->fixed, 256 + static_cast<int64_t>(sizeof(CUtensorMap)) * moe::kFfnDwMaps * v.n, capture);
        if (s != MOE_OK) return s;
        cudaError_t e = moe_api_detail::zero_now(w->fixed.p, 256);
        if (e != cudaSuccess) {  // no later call may take the word as it is
            cudaFree(w->fixed.p);
            w->fixed = moe::FfnBuffer{};
            return cuda_failed(e, "zeroing the status word");
        }
    }
    const int64_t row = static_cast<int64_t>(v.F) * (v.bf16 ? 2 : 4);
    if (rows > 0) s = room(w, &w->hidden, row * rows, capture);
    if (s == MOE_OK && rows > 0 && backward) s = room(w, &w->grads, 2 * row * rows, capture);
    if (s == MOE_OK && chunks > 0) s = room(w, &w->chunks, chunks * 1024, capture);
    return s;
}

moe::FfnArgs ffn_args(const HandleView& v, int64_t R, const int32_t* offsets) {
    moe::FfnArgs a{};
    a.offsets = offsets;
    a.n = v.n;
    a.R = R;
    a.d = v.d;
    a.F = v.F;
    a.h = v.ffn->hidden.p;
    a.da = v.ffn->grads.p;
    a.db = static_cast<uint8_t*>(v.ffn->grads.p) + v.ffn->grads.bytes / 2;
    a.status = v.ffn->status();
    return a;
}

using moe_api_detail::encode_bf16;

// Row operand [rows][cols]: box_rows rows x 64 columns per copy.
bool map_rows(CUtensorMap* m, const void* p, int64_t rows, int cols, int box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
    return encode_bf16(m, p, 2, dims, strides, box);
}

// Rows [rows][cols] read along their columns: two 64-column chunks of 64 rows.
bool map_rows_across(CUtensorMap* m, const void* p, int64_t rows, int cols) {
    const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols) / 64};
    const uint64_t strides[2] = {static_cast<uint64_t>(cols) * 2, 128};
    const uint32_t box[3] = {64, 64, 2};
    return encode_bf16(m, p, 3, dims, strides, box);
}

// Weights [n][rows][cols] whose rows are the reduction: two 64-column chunks of
// 64 rows; or whose columns are: 128 rows x 64 columns.
bool map_weights_across(CUtensorMap* m, const void* p, int n, int rows, int cols) {
    const uint64_t r = rows, c = cols;
    const uint64_t dims[4] = {64, r, c / 64, static_cast<uint64_t>(n)};
    const uint64_t strides[3] = {c * 2, 128, r * c * 2};
    const uint32_t box[4] = {64, 64, 2, 1};
    return encode_bf16(m, p, 4, dims, strides, box);
}
bool map_weights(CUtensorMap* m, const void* p, int n, int rows, int cols) {
    const uint64_t r = rows, c = cols;
    const uint64_t dims[3] = {c, r, static_cast<uint64_t>(n)};
    const uint64_t strides[2] = {c * 2, r * c * 2};
    const uint32_t box[3] = {64, 128, 1};
    return encode_bf16(m, p, 3, dims, strides, box);
}

// Outputs: 32 rows x 32 columns per store, of rows [rows][cols]; or x 64 columns of
// weight gradients [n][rows][cols].
bool map_out(CUtensorMap* m, const void* p, int64_t rows, int cols) {
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
    const uint32_t box[2] = {32, 32};
    return moe_api_detail::encode_bf16_64(m, p, 2, dims, strides, box);
}
bool map_out_weights(CUtensorMap* m, const void* p, int n, int rows, int cols) {
    const uint64_t r = rows, c = cols;
    const uint64_t dims[3] = {c, r, static_cast<uint64_t>(n)};
    const uint64_t strides[2] = {c * 2, r * c * 2};
    const uint32_t box[3] = {64, 32, 1};
    return encode_bf16(m, p, 3, dims, strides, box);
}

moe_status run(const HandleView& v, int op, const moe::FfnArgs& a, cudaStream_t st, const char* what,
               const moe::FfnDwMaps& dw = {}) {
    cudaError_t e;
    if (v.bf16) {
        CUtensorMap m[4] = {};
        const int n = v.n, d = v.d, F = v.F;
        const int few = moe::ffn_few_rows(op, a, v.num_sms), box = few ? few : 128;
        bool ok = true;
        if (op == moe::kFfnUp)
            ok = map_rows(&m[0], a.x, a.R, d, box) && map_weights_across(&m[2], a.w1, n, d, F) &&
                 map_weights_across(&m[3], a.w3, n, d, F);
        else if (op == moe::kFfnDown)
            ok = map_rows(&m[0], a.h, a.R, F, box) && map_weights_across(&m[2], a.w2, n, F, d);
        else if (op == moe::kFfnGrad)
            ok = map_rows(&m[0], a.dy, a.R, d, box) && map_weights(&m[2], a.w2, n, F, d);
        else if (op == moe::kFfnDx)
            ok = map_rows(&m[0], a.da, a.R, F, box) && map_rows(&m[1], a.db, a.R, F, box) &&
                 map_weights(&m[2], a.w1, n, d, F) && map_weights(&m[3], a.w3, n, d, F);
        moe::FfnOutMaps out = {};
        if (few || !ok)
            ;  // no output maps
        else if (op == moe::kFfnUp)
            ok = map_out(&out.m[0], a.h, a.R, F) &&
                 (!a.gate || (map_out(&out.m[1], a.gate, a.R, F) && map_out(&out.m[2], a.up, a.R, F)));
        else if (op == moe::kFfnGrad)
            ok = map_out(&out.m[0], a.da, a.R, F) && map_out(&out.m[1], a.db, a.R, F) &&
                 map_out(&out.m[2], a.h, a.R, F);
        else if (op == moe::kFfnDw)
            ok = map_out_weights(&out.m[0], a.dw1, n, d, F) && map_out_weights(&out.m[1], a.dw3, n, d, F) &&
                 map_out_weights(&out.m[2], a.dw2, n, F, d);
        else
            ok = map_out(&out.m[0], op == moe::kFfnDown ? a.y : a.dx, a.R, d);
        if (!ok) return failed(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%s)", what);
        e = few ? moe::launch_ffn_few(op, few, m, a, dw, v.num_sms, st)
                : moe::launch_ffn_tc(op, m, out, a, dw, v.num_sms, st);
    } else {
        e = moe::launch_ffn_simt(op, a, v.num_sms, st);
    }
    if (e != cudaSuccess) return cuda_failed(e, what);
    *v.launches += 1;
    return MOE_OK;
}

// The operands of the weight gradients, whose per-expert maps kFfnGrad writes.
moe_status dw_maps(const HandleView& v, const moe::FfnArgs& a, moe::FfnDwMaps* dw) {
    if (!map_rows_across(&dw->m[0], a.x, a.R, v.d) || !map_rows_across(&dw->m[1], a.h, a.R, v.F) ||
        !map_rows_across(&dw->m[2], a.da, a.R, v.F) || !map_rows_across(&dw->m[3], a.db, a.R, v.F) ||
        !map_rows_across(&dw->m[4], a.dy, a.R, v.d))
        return failed(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (weight gradients)");
    dw->out = static_cast<CUtensorMap*>(v.ffn->maps());
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_reserve_ffn(moe_handle* h, int64_t R_max, int backward) {
    if (!h) return failed(MOE_ERR_INVALID_ARG, "null handle");
    moe_status s = check_rows(R_max, "R_max");
    if (s != MOE_OK) return s;
    if (backward != 0 && backward != 1)
        return failed(MOE_ERR_INVALID_ARG, "backward = %d is neither 0 nor 1", backward);
    if (R_max == 0) return done();
    HandleView v;
    s = open_handle(h, &v);
    if (s != MOE_OK) return s;
    s = need(v, R_max, backward == 1, 0, nullptr, false);
    return s == MOE_OK ? done() : s;
}

moe_status moe_ffn_forward(moe_handle* h, int64_t R, const int32_t* offsets, const void* x, const void* w1,
                           const void* w3, const void* w2, void* gate, void* up, void* y, moe_stream_t stream) {
    if (!h) return failed(MOE_ERR_INVALID_ARG, "null handle");
    moe_status s = check_rows(R);
    if (s != MOE_OK) return s;
    if (R == 0) return done();
    FFN_REQUIRE_PTR(x);
    FFN_REQUIRE_PTR(w1);
    FFN_REQUIRE_PTR(w3);
    FFN_REQUIRE_PTR(w2);
    FFN_REQUIRE_PTR(y);
    if ((gate == nullptr) != (up == nullptr))
        return failed(MOE_ERR_INVALID_ARG, "gate and up must both be given or both be null");
    if (gate) {
        FFN_REQUIRE_PTR(gate);
        FFN_REQUIRE_PTR(up);
    }
    HandleView v;
    s = open_handle(h, &v);
    if (s != MOE_OK) return s;
    s = check_offsets(v.n, offsets);
    if (s != MOE_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    s = need(v, R, false, 0, st, true);
    if (s != MOE_OK) return s;
    moe::FfnArgs a = ffn_args(v, R, offsets);
    a.x = x;
    a.w1 = w1;
    a.w3 = w3;
    a.w2 = w2;
    a.gate = gate;
    a.up = up;
    a.y = y;
    moe::chain_begin();
    s = run(v, moe::kFfnUp, a, st, "feed-forward projections launch");
    if (s != MOE_OK) return s;
    s = run(v, moe::kFfnDown, a, st, "feed-forward output launch");
    return s == MOE_OK ? done() : s;
}

moe_status moe_ffn_backward(moe_handle* h, int64_t R, const int32_t* offsets, const void* x, const void* w1,
                            const void* w3, const void* w2, const void* gate, const void* up, const void* dy,
                            void* dx, void* dw1, void* dw3, void* dw2, moe_stream_t stream) {
    if (!h) return failed(MOE_ERR_INVALID_ARG, "null handle");
    moe_status s = check_rows(R);
    if (s != MOE_OK) return s;
    if ((dw1 == nullptr) != (dw3 == nullptr) || (dw1 == nullptr) != (dw2 == nullptr))
        return failed(MOE_ERR_INVALID_ARG, "dw1, dw3 and dw2 must all be given or all be null");
    if (!dx && !dw1) return failed(MOE_ERR_INVALID_ARG, "neither dx nor the weight gradients are asked for");
    if (dw1) {
        FFN_REQUIRE_PTR(dw1);
        FFN_REQUIRE_PTR(dw3);
        FFN_REQUIRE_PTR(dw2);
    }
    if (R > 0) {
        if (dx) FFN_REQUIRE_PTR(dx);
        FFN_REQUIRE_PTR(x);
        FFN_REQUIRE_PTR(w1);
        FFN_REQUIRE_PTR(w3);
        FFN_REQUIRE_PTR(w2);
        FFN_REQUIRE_PTR(gate);
        FFN_REQUIRE_PTR(up);
        FFN_REQUIRE_PTR(dy);
    }
    HandleView v;
    s = open_handle(h, &v);
    if (s != MOE_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (R == 0) {  // no rows: the weight gradients are zero
        const size_t bytes = static_cast<size_t>(v.n) * v.d * v.F * (v.bf16 ? 2 : 4);
        for (void* p : {dw1, dw3, dw2}) {
            cudaError_t e = p ? cudaMemsetAsync(p, 0, bytes, st) : cudaSuccess;
            if (e != cudaSuccess) return cuda_failed(e, "cudaMemsetAsync(weight gradients)");
        }
        return done();
    }
    s = check_offsets(v.n, offsets);
    if (s != MOE_OK) return s;
    s = need(v, R, true, 0, st, true);
    if (s != MOE_OK) return s;
    moe::FfnArgs a = ffn_args(v, R, offsets);
    a.x = x;
    a.dy = dy;
    a.w1 = w1;
    a.w3 = w3;
    a.w2 = w2;
    a.gate = const_cast<void*>(gate);
    a.up = const_cast<void*>(up);
    a.dx = dx;
    a.dw1 = dw1;
    a.dw3 = dw3;
    a.dw2 = dw2;
    moe::chain_begin();
    moe::FfnDwMaps dw = {};
    if (dw1 && v.bf16) s = dw_maps(v, a, &dw);
    if (s == MOE_OK) s = run(v, moe::kFfnGrad, a, st, "feed-forward hidden gradient launch", dw);
    if (s == MOE_OK && dx) s = run(v, moe::kFfnDx, a, st, "feed-forward input gradient launch");
    if (s == MOE_OK && dw1) s = run(v, moe::kFfnDw, a, st, "feed-forward weight gradient launch", dw);
    return s == MOE_OK ? done() : s;
}

namespace {
// N and K of the MXFP4 product.
moe_status check_mx_shape(int N, int K) {
    if (N < 1 || N > 1048576) return failed(MOE_ERR_INVALID_ARG, "N = %d outside [1, 1048576]", N);
    if (K < 32 || K % 32 != 0 || K > 1048576)
        return failed(MOE_ERR_INVALID_ARG, "K = %d is not a multiple of 32 in [32, 1048576]", K);
    return MOE_OK;
}

// SM count of the current device; what a device is never changes, so it is
// asked for once per device.
moe_status device_of_call(int* sms) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_failed(e, "cudaGetDevice");
    if (dev < kDevices && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return MOE_OK;
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_failed(e, "cudaDeviceGetAttribute");
    if (major != 10 || minor != 0) return failed(MOE_ERR_UNSUPPORTED, "device %d is not sm_100", dev);
    if (dev < kDevices) known[dev].store(*sms, std::memory_order_relaxed);
    return MOE_OK;
}
}  // namespace

moe_status moe_quantize_mxfp4(int64_t rows, int cols, const void* x, moe_dtype dtype, uint8_t* codes,
                              uint8_t* scales, void* values, moe_stream_t stream) {
    moe_status s = check_rows(rows, "rows");
    if (s != MOE_OK) return s;
    if (cols < 32 || cols % 32 != 0)
        return failed(MOE_ERR_INVALID_ARG, "cols = %d is not a positive multiple of 32", cols);
    if (dtype != MOE_F32 && dtype != MOE_BF16)
        return failed(MOE_ERR_INVALID_ARG, "dtype = %d is not MOE_F32 or MOE_BF16", static_cast<int>(dtype));
    if (rows == 0) return done();
    FFN_REQUIRE_PTR(x);
    FFN_REQUIRE_PTR(codes);
    if (!scales) return failed(MOE_ERR_INVALID_ARG, "scales is NULL");
    if (values) FFN_REQUIRE_PTR(values);
    int sms = 0;
    s = device_of_call(&sms);
    if (s != MOE_OK) return s;
    cudaError_t e = moe::launch_mx_rows(x, dtype == MOE_BF16, rows, cols, codes, scales, values, sms,
                                        reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_failed(e, "MXFP4 quantisation launch");
    return done();
}

moe_status moe_quantize_weights_mxfp4(int n, int rows, int cols, const void* w, moe_dtype dtype, uint8_t* codes,
                                      uint8_t* scales, void* values, moe_stream_t stream) {
    if (n < 1 || n > 65535) return failed(MOE_ERR_INVALID_ARG, "n = %d outside [1, 65535]", n);
    if (rows < 32 || rows % 32 != 0)
        return failed(MOE_ERR_INVALID_ARG, "rows = %d is not a positive multiple of 32", rows);
    if (cols < 1 || cols > 1048576) return failed(MOE_ERR_INVALID_ARG, "cols = %d outside [1, 1048576]", cols);
    if (dtype != MOE_F32 && dtype != MOE_BF16)
        return failed(MOE_ERR_INVALID_ARG, "dtype = %d is not MOE_F32 or MOE_BF16", static_cast<int>(dtype));
    FFN_REQUIRE_PTR(w);
    FFN_REQUIRE_PTR(codes);
    if (!scales) return failed(MOE_ERR_INVALID_ARG, "scales is NULL");
    if (values) FFN_REQUIRE_PTR(values);
    int sms = 0;
    moe_status s = device_of_call(&sms);
    if (s != MOE_OK) return s;
    cudaError_t e = moe::launch_mx_weights(w, dtype == MOE_BF16, n, rows, cols, codes, scales, values,
                                           reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_failed(e, "MXFP4 weight quantisation launch");
    return done();
}

moe_status moe_reserve_matmul_mxfp4(moe_handle* h, int64_t R_max, int N, int K, int pair) {
    if (!h) return failed(MOE_ERR_INVALID_ARG, "null handle");
    moe_status s = check_rows(R_max, "R_max");
    if (s != MOE_OK) return s;
    s = check_mx_shape(N, K);
    if (s != MOE_OK) return s;
    if (pair != 0 && pair != 1) return failed(MOE_ERR_INVALID_ARG, "pair = %d is neither 0 nor 1", pair);
    if (R_max == 0) return done();
    HandleView v;
    s = open_handle(h, &v);
    if (s != MOE_OK) return s;
    s = need(v, 0, false, moe::mx_gemm_most_chunks(R_max, v.n, N, K, pair), nullptr, false);
    return s == MOE_OK ? done() : s;
}

moe_status moe_matmul_mxfp4(moe_handle* h, int64_t R, int N, int K, const int32_t* offsets, const uint8_t* a_codes,
                            const uint8_t* a_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                            const uint8_t* pair_codes, const uint8_t* pair_scales, void* out, moe_stream_t stream) {
    if (!h) return failed(MOE_ERR_INVALID_ARG, "null handle");
    moe_status s = check_rows(R);
    if (s != MOE_OK) return s;
    s = check_mx_shape(N, K);
    if (s != MOE_OK) return s;
    if ((pair_codes == nullptr) != (pair_scales == nullptr))
        return failed(MOE_ERR_INVALID_ARG, "pair_codes and pair_scales must both be given or both be null");
    if (R == 0) return done();
    FFN_REQUIRE_PTR(a_codes);
    FFN_REQUIRE_PTR(w_codes);
    if (pair_codes) FFN_REQUIRE_PTR(pair_codes);
    FFN_REQUIRE_PTR(out);
    if (!a_scales) return failed(MOE_ERR_INVALID_ARG, "a_scales is NULL");
    if (!w_scales) return failed(MOE_ERR_INVALID_ARG, "w_scales is NULL");
    HandleView v;
    s = open_handle(h, &v);
    if (s != MOE_OK) return s;
    s = check_offsets(v.n, offsets);
    if (s != MOE_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    moe::MxGemmArgs a{offsets,  v.n,      R,          N,           K,   a_codes, a_scales,
                      w_codes,  w_scales, pair_codes, pair_scales, out, nullptr};
    moe::MxChunks ch = moe::mx_gemm_chunks(a, v.num_sms);
    s = need(v, 0, false, ch.blocks * ch.steps, st, true);
    if (s != MOE_OK) return s;
    a.status = v.ffn->status();
    ch.base = static_cast<uint8_t*>(v.ffn->chunks.p);
    const uint64_t k2 = static_cast<uint64_t>(K) / 2, cols = static_cast<uint64_t>(N);
    const uint64_t a_dims[2] = {k2, static_cast<uint64_t>(R)}, a_strides[1] = {k2};
    const uint32_t a_box[2] = {128, ch.tile_rows < 128 ? static_cast<uint32_t>(ch.tile_rows) : 128u};
    const uint64_t w_dims[3] = {k2, cols, static_cast<uint64_t>(v.n)}, w_strides[2] = {k2, k2 * cols};
    const uint32_t w_box[3] = {128, 128, 1};
    const uint64_t o_dims[2] = {cols, static_cast<uint64_t>(R)}, o_strides[1] = {cols * (v.bf16 ? 2 : 4)};
    const uint32_t o_box[2] = {v.bf16 ? 32u : 16u, 32};
    const uint64_t c_dims[2] = {256, static_cast<uint64_t>(ch.blocks * ch.steps)}, c_strides[1] = {1024};
    const uint32_t c_box[2] = {256, 1};
    CUtensorMap m[5] = {};
    using namespace moe_api_detail;
    bool mapped = encode_bytes(&m[0], a_codes, 2, a_dims, a_strides, a_box) &&
                  encode_bytes(&m[1], w_codes, 3, w_dims, w_strides, w_box) &&
                  encode_words(&m[4], ch.base, 2, c_dims, c_strides, c_box);
    if (pair_codes) mapped = mapped && encode_bytes(&m[2], pair_codes, 3, w_dims, w_strides, w_box);
    if (ch.tile_rows > 128 && N % (v.bf16 ? 8 : 4) == 0)
        mapped = mapped && (v.bf16 ? encode_bf16_64(&m[3], out, 2, o_dims, o_strides, o_box)
                                   : encode_f32_64(&m[3], out, 2, o_dims, o_strides, o_box));
    if (!mapped) return failed(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (MXFP4 product)");
    moe::chain_begin();
    cudaError_t e = moe::launch_mx_gemm(m, a, v.bf16, ch, v.num_sms, st);
    if (e != cudaSuccess) return cuda_failed(e, "MXFP4 product launch");
    *v.launches += 2;
    return done();
}

}  // extern "C"
