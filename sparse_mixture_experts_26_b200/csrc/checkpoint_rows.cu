// checkpoint_rows.cu -- the 8-bit activation checkpoint by itself: rows in, codes and
// block scales out, and back through an activation.
//
// A block is 32 consecutive values of a row: s = max|v| / 128, q = floor(v / s), and q
// stands for (q + 1/2) s.  Half a step of offset instead of rounding to whole steps uses
// all 256 codes symmetrically (error <= max / 256 instead of max / 254 with a wasted
// code) and keeps the sign of every value.
//
// Both directions are bound by their bytes.  A thread owns eight consecutive values
// (16- or 32-byte loads, 8-byte code stores), so four neighbouring lanes own a block and
// two shuffles give its largest magnitude.
#include <cuda_bf16.h>

#include "act_checkpoint.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

// Rows are cut into whole blocks of 32 (four lanes each, so that a block never crosses a
// warp); lanes past N hold nothing.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    checkpoint_save_kernel(const T* __restrict__ v, int rows, int N, int8_t* __restrict__ codes,
                           float* __restrict__ scales) {
    const int nb = ckpt_blocks(N);
    const size_t n = static_cast<size_t>(rows) * nb * 4;
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (size_t base = blockIdx.x * static_cast<size_t>(blockDim.x); base < n; base += step) {
        const size_t i = base + threadIdx.x;
        const size_t blk = i >> 2;
        const size_t r = blk / nb;
        const int b = static_cast<int>(blk - r * nb);
        const int c = b * kCkptBlock + static_cast<int>(i & 3) * 8;
        const bool have = i < n && c < N;
        float x[8] = {};
        if (have) load8(v + r * N + c, x);
        uint32_t mag = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) mag = max(mag, ckpt_mag(x[k]));
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
        const float s = ckpt_scale(mag);
        if (have) {
            *reinterpret_cast<uint2*>(codes + r * N + c) = ckpt_pack8(x, s);
            if ((i & 3) == 0) scales[blk] = s;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    checkpoint_restore_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                              int rows, int N, int act, T* __restrict__ out) {
    const int n8 = N >> 3;
    const int nb = ckpt_blocks(N);
    const size_t n = static_cast<size_t>(rows) * n8;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const size_t r = i / n8;
        const int c = static_cast<int>(i - r * n8) * 8;
        float x[8];
        ckpt_unpack8(*reinterpret_cast<const uint2*>(codes + r * N + c),
                     scales[r * nb + c / kCkptBlock], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = act_value(act, x[k]);
        store8(out + r * N + c, x);
    }
}

int row_grid(size_t items) {
    const size_t blocks = (items + kRowThreads - 1) / kRowThreads;
    const size_t most = static_cast<size_t>(device_sm_count()) * 8;
    return static_cast<int>(blocks < 1 ? 1 : (blocks < most ? blocks : most));
}

}  // namespace

cudaError_t launch_checkpoint_save(const void* v, int rows, int N, moe_dtype dt, int8_t* codes,
                                   float* scales, cudaStream_t s) {
    const int grid = row_grid(static_cast<size_t>(rows) * ckpt_blocks(N) * 4);
    if (dt == MOE_BF16)
        return launch_k(checkpoint_save_kernel<__nv_bfloat16>, grid, kRowThreads, 0, s,
                        static_cast<const __nv_bfloat16*>(v), rows, N, codes, scales);
    return launch_k(checkpoint_save_kernel<float>, grid, kRowThreads, 0, s,
                    static_cast<const float*>(v), rows, N, codes, scales);
}

cudaError_t launch_checkpoint_restore(const int8_t* codes, const float* scales, int rows, int N,
                                      int act, moe_dtype out_dt, void* out, cudaStream_t s) {
    const int grid = row_grid(static_cast<size_t>(rows) * (N / 8));
    if (out_dt == MOE_BF16)
        return launch_k(checkpoint_restore_kernel<__nv_bfloat16>, grid, kRowThreads, 0, s, codes,
                        scales, rows, N, act, static_cast<__nv_bfloat16*>(out));
    return launch_k(checkpoint_restore_kernel<float>, grid, kRowThreads, 0, s, codes, scales, rows,
                    N, act, static_cast<float*>(out));
}

}  // namespace moe
