// linear_api.cu -- the extern "C" entry points of the grouped linear operators and the
// 8-bit activation checkpoint (declared in include/moe.h).
//
// As in moe_api.cu: arguments are checked on the host before anything is queued, and
// nothing allocates, frees or synchronises (except in MOE_DEBUG_SYNC=1 mode).
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxLinearRows = 1 << 30;
constexpr int kMaxLinearDim = 1 << 30;  // of K and N: sizes are rounded up to tiles in 32 bits

moe_status check_linear(int rows, int K, int N, int E, moe_dtype dt) {
    if (rows < 0 || K <= 0 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || K % 8 != 0 || N % 8 != 0 || rows > kMaxLinearRows ||
        K > kMaxLinearDim || N > kMaxLinearDim)
        return MOE_ERR_UNSUPPORTED;
    // 32-bit coordinates inside one expert's weights and one array of rows; element
    // offsets are 64-bit
    if (static_cast<long long>(E) * N >= (1LL << 31) || static_cast<long long>(E) * K >= (1LL << 31))
        return MOE_ERR_UNSUPPORTED;
    const long long widest = K > N ? K : N;
    if (rows * widest >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;  // tile counts in 32 bits
    return MOE_OK;
}

bool valid_act(moe_act act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_SILU; }
bool valid_dt(moe_dtype dt) { return dt == MOE_F32 || dt == MOE_BF16; }
bool optional_ok(const void* p) { return aligned16(p); }  // null is aligned

// Workspace regions (1 KiB aligned).  The status word and the counters, which are zero between
// calls, come first and have the same place for every shape and for both directions: one
// workspace may serve them all in turn.
struct LinearWs {
    size_t status, counters, db_counters, partials, dz, dz_tail, x_tail, db_part, total;
};
LinearWs linear_ws(int rows, int K, int N, int E, moe_dtype dt, bool backward) {
    LinearWs L{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 1024);
        return at;
    };
    L.status = take(256);
    L.counters = take(kLinearCounters * 4);
    L.db_counters = take(kLinearDbCounters * 4);
    L.partials = take(dt == MOE_BF16 ? linear_partial_floats(rows) * 4 : 0);
    const size_t b = backward ? 1 : 0, tail = b * E * kTailRows;
    L.dz = take(b * rows * N * 2);
    L.dz_tail = take(tail * N * 2);
    L.x_tail = take(tail * K * 2);
    L.db_part = take(b * linear_chunks(rows, E) * N * 4);
    L.total = o;
    return L;
}

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Short calls overlap the launch of one kernel with the end of the one before (PdlScope):
// 637 x 2 rows, K = 104, N = 5328, backward 49.7 -> 42.6 us.  Long ones gain nothing.
bool short_call(int rows, int K, int N) {
    return rows <= 256 || static_cast<double>(rows) * K * N < 8e9;
}

moe_status finish_linear(cudaError_t err, cudaStream_t s, uint32_t* status) {
    if (err == cudaErrorInvalidValue) return MOE_ERR_INVALID_ARG;  // tensor map refused
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    if (!debug_sync_enabled()) return MOE_OK;
    if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
    uint32_t flags = 0;
    if (status && cudaMemcpy(&flags, status, 4, cudaMemcpyDeviceToHost) != cudaSuccess)
        return MOE_ERR_CUDA;
    return (flags & MOE_DEV_FLAG_TIMEOUT) ? MOE_ERR_TIMEOUT : MOE_OK;
}

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

moe_status linear_impl(const char* name, bool train, const void* x, const int32_t* offsets,
                       const void* W, const void* bias, const void* residual, int rows, int K,
                       int N, int E, moe_act act, moe_dtype dt, moe_dtype y_dt, void* y,
                       int8_t* codes, float* scales, void* ws, size_t ws_bytes,
                       cudaStream_t stream) {
    const moe_status st = check_linear(rows, K, N, E, dt);
    if (st != MOE_OK) return st;
    if (!valid_act(act) || !valid_dt(y_dt)) return MOE_ERR_INVALID_ARG;
    if ((train && dt != MOE_BF16) || (dt == MOE_F32 && y_dt != MOE_F32)) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!ptrs_ok({x, W, y, ws}) || !optional_ok(bias) || !optional_ok(residual) ||
        !optional_ok(offsets) || (offsets == nullptr && E != 1))
        return MOE_ERR_INVALID_ARG;
    if (train && !ptrs_ok({codes, scales})) return MOE_ERR_INVALID_ARG;
    const LinearWs L = linear_ws(rows, K, N, E, dt, false);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    Range range(name);
    PdlScope pdl(short_call(rows, K, N));
    LinearArgs a{};
    a.x = x;
    a.offsets = offsets;
    a.W = W;
    a.bias = bias;
    a.residual = residual;
    a.rows = rows;
    a.K = K;
    a.N = N;
    a.E = E;
    a.act = act;
    a.dt = dt;
    a.y_dt = y_dt;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    a.status = at<uint32_t>(ws, L.status);
    a.counters = at<uint32_t>(ws, L.counters);
    a.partials = at<float>(ws, L.partials);
    a.stream = stream;
    return finish_linear(launch_linear(a), stream, a.status);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_linear_workspace_bytes(int rows, int K, int N, int E, moe_dtype dt) {
    if (check_linear(rows, K, N, E, dt) != MOE_OK) return 0;
    return linear_ws(rows, K, N, E, dt, false).total;
}

moe_status moe_grouped_linear(const void* x, const int32_t* offsets, const void* W,
                              const void* bias, const void* residual, int rows, int K, int N,
                              int E, moe_act act, moe_dtype dt, moe_dtype y_dt, void* y, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
    return linear_impl("moe_grouped_linear", false, x, offsets, W, bias, residual, rows, K, N, E,
                       act, dt, y_dt, y, nullptr, nullptr, ws, ws_bytes, stream);
}

moe_status moe_grouped_linear_train(const void* x, const int32_t* offsets, const void* W,
                                    const void* bias, const void* residual, int rows, int K,
                                    int N, int E, moe_act act, moe_dtype dt, moe_dtype y_dt,
                                    void* y, int8_t* codes, float* scales, void* ws,
                                    size_t ws_bytes, cudaStream_t stream) {
    return linear_impl("moe_grouped_linear_train", true, x, offsets, W, bias, residual, rows, K, N,
                       E, act, dt, y_dt, y, codes, scales, ws, ws_bytes, stream);
}

moe_status moe_checkpoint_save(const void* v, int rows, int N, moe_dtype dt, int8_t* codes,
                               float* scales, cudaStream_t stream) {
    const moe_status st = check_linear(rows, 8, N, 1, dt);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!ptrs_ok({v, codes, scales})) return MOE_ERR_INVALID_ARG;
    PdlScope pdl(short_call(rows, 8, N));
    return finish_linear(launch_checkpoint_save(v, rows, N, dt, codes, scales, stream), stream,
                         nullptr);
}

moe_status moe_checkpoint_restore(const int8_t* codes, const float* scales, int rows, int N,
                                  moe_act act, moe_dtype out_dt, void* out, cudaStream_t stream) {
    const moe_status st = check_linear(rows, 8, N, 1, out_dt);
    if (st != MOE_OK) return st;
    if (!valid_act(act)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!ptrs_ok({codes, scales, out})) return MOE_ERR_INVALID_ARG;
    PdlScope pdl(short_call(rows, 8, N));
    return finish_linear(
        launch_checkpoint_restore(codes, scales, rows, N, act, out_dt, out, stream), stream,
        nullptr);
}

size_t moe_grouped_linear_backward_workspace_bytes(int rows, int K, int N, int E, moe_dtype dt) {
    if (check_linear(rows, K, N, E, dt) != MOE_OK || dt != MOE_BF16) return 0;
    return linear_ws(rows, K, N, E, dt, true).total;
}

moe_status moe_grouped_linear_backward(const void* dy, const void* x, const int32_t* offsets,
                                       const void* W, const int8_t* codes, const float* scales,
                                       int rows, int K, int N, int E, moe_act act, moe_dtype dt,
                                       moe_dtype dw_dt, void* dx, void* dW, float* db, void* ws,
                                       size_t ws_bytes, cudaStream_t stream) {
    const moe_status st = check_linear(rows, K, N, E, dt);
    if (st != MOE_OK) return st;
    if (!valid_act(act) || !valid_dt(dw_dt)) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (!optional_ok(dx) || !optional_ok(dW) || !optional_ok(db) || !optional_ok(offsets) ||
        (offsets == nullptr && E != 1))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) {  // no rows: the sums over rows are zero
        const size_t n = static_cast<size_t>(E) * N;
        const size_t el = dw_dt == MOE_BF16 ? 2 : 4;
        if ((dW && cudaMemsetAsync(dW, 0, n * K * el, stream) != cudaSuccess) ||
            (db && cudaMemsetAsync(db, 0, n * 4, stream) != cudaSuccess))
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!ptrs_ok({dy, x, W, ws})) return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_NONE && !ptrs_ok({codes, scales})) return MOE_ERR_INVALID_ARG;
    const LinearWs L = linear_ws(rows, K, N, E, dt, true);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    Range range("moe_grouped_linear_backward");
    PdlScope pdl(short_call(rows, K, N));
    LinearBwdArgs a{};
    a.dy = dy;
    a.x = x;
    a.offsets = offsets;
    a.W = W;
    a.codes = act == MOE_ACT_NONE ? nullptr : codes;
    a.scales = scales;
    a.rows = rows;
    a.K = K;
    a.N = N;
    a.E = E;
    a.act = act;
    a.dw_dt = dw_dt;
    a.dx = dx;
    a.dW = dW;
    a.db = db;
    a.dz = at<void>(ws, L.dz);
    a.dz_tail = at<void>(ws, L.dz_tail);
    a.x_tail = at<void>(ws, L.x_tail);
    a.db_part = at<float>(ws, L.db_part);
    a.db_counters = at<uint32_t>(ws, L.db_counters);
    a.status = at<uint32_t>(ws, L.status);
    a.counters = at<uint32_t>(ws, L.counters);
    a.partials = at<float>(ws, L.partials);
    a.stream = stream;
    return finish_linear(launch_linear_backward(a), stream, a.status);
}

}  // extern "C"
