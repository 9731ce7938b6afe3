// grouped_linear.cu -- the grouped linear operators' launches, and the fp32 forward on CUDA
// cores (fp32 throughout, no TF32: y_r = act(x_r W_e^T + b_e) + residual_r).
//
// The fp32 kernel: 128 threads, 16 (rows) x 8 (features), each with RM x RN sums in
// registers.  Steps of 32 of the reduction go through shared memory in rows of 36 floats, so
// that every read is 16 bytes (RM + RN reads for 4 RM RN multiply-adds); the next step's
// global loads are in flight meanwhile.  Small problems are chains of latencies and want
// many small tiles, large ones the better ratio of multiply-adds to reads:
// 32 x 32 tiles (2 x 4 sums) while 128 x 64 ones (8 x 8) would leave SMs without work.
#include <cuda_bf16.h>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 32;            // reduction per step
constexpr int kPitch = kStep + 4;    // floats

template <int RM, int RN>
__global__ void __launch_bounds__(kThreads) linear_f32_kernel(const LinearArgs a, int ftiles) {
    constexpr int kRowTile = 16 * RM, kFTile = 8 * RN;
    constexpr int kX = kRowTile * kStep / 4 / kThreads;  // 16-byte loads a thread and step
    constexpr int kW = kFTile * kStep / 4 / kThreads;
    __shared__ int off[kMaxExperts + 1];
    __shared__ __align__(16) float sx[kRowTile * kPitch], sw[kFTile * kPitch];
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) load_group_bounds(a.offsets, a.E, a.rows, off);
    __syncthreads();
    int ft;
    int y = divide(blockIdx.x, ftiles, ft), e = 0;  // row tile y of all groups'
    for (; e < a.E; ++e) {
        const int t = (off[e + 1] - off[e] + kRowTile - 1) / kRowTile;
        if (y < t) break;
        y -= t;
    }
    if (e == a.E) return;
    const int row0 = off[e] + y * kRowTile, row_end = off[e + 1], f0 = ft * kFTile;
    const float* __restrict__ x = static_cast<const float*>(a.x);
    const float* __restrict__ W =
        static_cast<const float*>(a.W) + static_cast<size_t>(e) * a.N * a.K;
    const int part = threadIdx.x & 7, line = threadIdx.x >> 3;  // loads: 8 threads a row
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;

    float4 px[kX], pw[kW];
    auto fetch = [&](int k0) {
        const int k = k0 + part * 4;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int r = row0 + line + 16 * i;
            px[i] = r < row_end && k < a.K
                        ? *reinterpret_cast<const float4*>(x + static_cast<size_t>(r) * a.K + k)
                        : zero;
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int f = f0 + line + 16 * i;
            pw[i] = f < a.N && k < a.K
                        ? *reinterpret_cast<const float4*>(W + static_cast<size_t>(f) * a.K + k)
                        : zero;
        }
    };
    float acc[RM][RN] = {};
    fetch(0);
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kX; ++i)
            *reinterpret_cast<float4*>(sx + (line + 16 * i) * kPitch + part * 4) = px[i];
#pragma unroll
        for (int i = 0; i < kW; ++i)
            *reinterpret_cast<float4*>(sw + (line + 16 * i) * kPitch + part * 4) = pw[i];
        __syncthreads();
        if (k0 + kStep < a.K) fetch(k0 + kStep);
#pragma unroll
        for (int k = 0; k < kStep; k += 4) {
            float4 xv[RM], wv[RN];
#pragma unroll
            for (int i = 0; i < RM; ++i)
                xv[i] = *reinterpret_cast<const float4*>(sx + (ty + 16 * i) * kPitch + k);
#pragma unroll
            for (int j = 0; j < RN; ++j)
                wv[j] = *reinterpret_cast<const float4*>(sw + (tx + 8 * j) * kPitch + k);
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < RN; ++j) {
                    acc[i][j] = fmaf(xv[i].x, wv[j].x, acc[i][j]);
                    acc[i][j] = fmaf(xv[i].y, wv[j].y, acc[i][j]);
                    acc[i][j] = fmaf(xv[i].z, wv[j].z, acc[i][j]);
                    acc[i][j] = fmaf(xv[i].w, wv[j].w, acc[i][j]);
                }
        }
    }
    // eight of a thread's outputs at a time; features 8 apart, so eight lanes write 32 bytes
    const float* bias = static_cast<const float*>(a.bias);
    const float* residual = static_cast<const float*>(a.residual);
    float* out = static_cast<float*>(a.y);
    constexpr int kRowsAtOnce = RN >= 8 ? 1 : 8 / RN;
#pragma unroll
    for (int i = 0; i < RM; i += kRowsAtOnce) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int f = f0 + tx + 8 * (k % RN);
            v[k] = acc[i + k / RN][k % RN] +
                   (bias && f < a.N ? bias[static_cast<size_t>(e) * a.N + f] : 0.f);
        }
        act_value8(a.act, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int f = f0 + tx + 8 * (k % RN), r = row0 + ty + 16 * (i + k / RN);
            if (f >= a.N || r >= row_end) continue;
            const size_t at = static_cast<size_t>(r) * a.N + f;
            out[at] = residual ? v[k] + residual[at] : v[k];
        }
    }
}

template <int RM, int RN>
cudaError_t launch_f32(const LinearArgs& a, long long& blocks, bool go) {
    const int ftiles = (a.N + 8 * RN - 1) / (8 * RN);
    const int groups = a.rows < a.E ? a.rows : a.E;
    blocks = (a.rows / (16 * RM) + groups) * static_cast<long long>(ftiles);
    if (!go) return cudaSuccess;
    return launch_k(linear_f32_kernel<RM, RN>, static_cast<unsigned>(blocks), kThreads, 0, a.stream,
                    a, ftiles);
}

cudaError_t launch_linear_f32(const LinearArgs& a) {
    long long blocks;
    launch_f32<8, 8>(a, blocks, false);
    return blocks >= 2LL * device_sm_count() ? launch_f32<8, 8>(a, blocks, true)
                                             : launch_f32<2, 4>(a, blocks, true);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a) {
    return a.dt == MOE_BF16 ? launch_linear_bf16(a, /*transposed=*/false) : launch_linear_f32(a);
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
