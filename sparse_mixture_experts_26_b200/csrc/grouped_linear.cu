// grouped_linear.cu -- the grouped linear operators on CUDA cores: plain tiled kernels
// that are right for every shape.
//
// A block computes a 64 x 64 tile of the output of one group with 256 threads, 4 x 4
// values each, over steps of 16 of the reduction staged in shared memory as fp32.
#include <cuda_bf16.h>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kT = 64;       // tile side
constexpr int kStep = 16;    // reduction per step
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    return static_cast<float>(v);
}

// Tile `y` of the row tiles of all groups -> group e, first row, end row.
__device__ __forceinline__ bool row_tile(const int* off, int E, int y, int& e, int& row0,
                                         int& row_end) {
    for (int g = 0; g < E; ++g) {
        const int t = (off[g + 1] - off[g] + kT - 1) / kT;
        if (y < t) {
            e = g;
            row0 = off[g] + y * kT;
            row_end = off[g + 1];
            return true;
        }
        y -= t;
    }
    return false;
}

// acc[i][j] += sum_c A(m0 + .., c) B(n0 + .., c): fa / fb read one operand value, 0
// outside.
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(int C, FA fa, FB fb, float (&acc)[4][4]) {
    __shared__ float sa[kStep][kT + 1], sb[kStep][kT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int c0 = 0; c0 < C; c0 += kStep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kStep * kT; i += kThreads) {
            const int c = i % kStep, m = i / kStep;
            sa[c][m] = c0 + c < C ? fa(m, c0 + c) : 0.f;
            sb[c][m] = c0 + c < C ? fb(m, c0 + c) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kStep; ++c) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[c][ty * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = sb[c][tx + 16 * j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
    }
}

template <typename T, typename TY>
__global__ void __launch_bounds__(kThreads) linear_kernel(const LinearArgs a) {
    __shared__ int off[kMaxExperts + 1];
    __shared__ float sz[kT][kT + 1];
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) load_group_bounds(a.offsets, a.E, a.rows, off);
    __syncthreads();
    int e, row0, row_end;
    if (!row_tile(off, a.E, blockIdx.y, e, row0, row_end)) return;
    const int n0 = blockIdx.x * kT;
    const T* x = static_cast<const T*>(a.x);
    const T* W = static_cast<const T*>(a.W) + static_cast<size_t>(e) * a.N * a.K;
    float acc[4][4] = {};
    tile_product(
        a.K,
        [&](int m, int c) {
            return row0 + m < row_end ? to_f32(x[static_cast<size_t>(row0 + m) * a.K + c]) : 0.f;
        },
        [&](int n, int c) {
            return n0 + n < a.N ? to_f32(W[static_cast<size_t>(n0 + n) * a.K + c]) : 0.f;
        },
        acc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sz[ty * 4 + i][tx + 16 * j] = acc[i][j];
    __syncthreads();
    // eight consecutive outputs per thread: 8 threads a row, 32 rows at a time
    const int f = (threadIdx.x & 7) * 8, n = n0 + f;
    for (int m = threadIdx.x >> 3; m < kT; m += kThreads / 8) {
        const int row = row0 + m;
        const bool valid = row < row_end && n < a.N;
        float z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = valid ? sz[m][f + k] : 0.f;
        if (valid && a.bias) {
            float b[8];
            load8(static_cast<const T*>(a.bias) + static_cast<size_t>(e) * a.N + n, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] += b[k];
        }
        if (!valid) continue;
        act_value8(a.act, z);
        if (a.residual) {
            float r[8];
            load8(static_cast<const T*>(a.residual) + static_cast<size_t>(row) * a.N + n, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] += r[k];
        }
        store8(static_cast<TY*>(a.y) + static_cast<size_t>(row) * a.N + n, z);
    }
}

unsigned blocks(int n) { return static_cast<unsigned>((n + kT - 1) / kT); }

}  // namespace

cudaError_t launch_linear(const LinearArgs& a) {
    if (a.dt == MOE_BF16) return launch_linear_bf16(a, /*transposed=*/false);
    const dim3 grid(blocks(a.N), blocks(a.rows) + a.E);
    return launch_k(linear_kernel<float, float>, grid, kThreads, 0, a.stream, a);
}

cudaError_t launch_linear_backward(const LinearBwdArgs& a) {
    cudaError_t err = launch_linear_dz(a);
    if (err == cudaSuccess && a.dx) {
        LinearArgs g{};
        g.x = a.codes ? a.dz : a.dy;
        g.offsets = a.offsets;
        g.W = a.W;
        g.rows = a.rows;
        g.K = a.N;  // the reduction
        g.N = a.K;
        g.E = a.E;
        g.dt = g.y_dt = MOE_BF16;
        g.y = a.dx;
        g.status = a.status;
        g.counters = a.counters;
        g.partials = a.partials;
        g.stream = a.stream;
        err = launch_linear_bf16(g, /*transposed=*/true);
    }
    if (err == cudaSuccess && a.dW) err = launch_linear_wgrad(a);
    return err;
}

}  // namespace moe
