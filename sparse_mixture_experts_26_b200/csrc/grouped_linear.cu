// grouped_linear.cu -- the grouped linear operators' launches, and the fp32 forward on CUDA
// cores (fp32 throughout, no TF32: y_r = act(x_r W_e^T + b_e) + residual_r).
//
// The fp32 kernel: 128 threads, 16 (rows) x 8 (features), each with RM x RN sums in registers,
// one over the even and one over the odd k of the reduction: a 16-byte read of either operand
// then is two operands of an instruction that does two multiply-adds, with nothing to
// rearrange.  Steps of 32 of the reduction come asynchronously into three stages of shared
// memory, in rows of 36 floats, so that no read meets a bank twice; one barrier a step.
// Small problems are chains of latencies and want many small tiles, large ones the better ratio
// of multiply-adds to reads (launch_linear_f32).  Measured: 4096^3 47.6 TFLOP/s, two thirds
// of the multiply-add rate (cuBLAS 57), 8192 x 1024 -> 1024 45.8 (cuBLAS 51),
// 512 x 1024 -> 1024 38.6 us (scalar sums and two barriers a step: 34.5 TFLOP/s, 88 us).
#include <cuda_bf16.h>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 32;            // reduction per stage
constexpr int kPitch = kStep + 4;    // floats
constexpr int kStages = 3;

template <int RM, int RN>
struct F32Tile {
    static constexpr int kRows = 16 * RM, kF = 8 * RN;
    static constexpr int kStageFloats = (kRows + kF) * kPitch;
    static constexpr int kSmem = kStages * kStageFloats * 4;
};

// 16 bytes global -> shared, asynchronously; zeros if !have.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(have ? 16 : 0)
                 : "memory");
}

// act(z) in fp32, relative to itself: the approximations of act_value8 (1e-7 absolute) are made
// for epilogues that round to bf16.  Here the products take longer than CUDA's functions
// (8192 x 1024 -> 1024: 375 us without an activation, 386 with SiLU, 401 with GELU; 380 and 382
// with the approximations; small calls show no difference).  Infinities give the limits
// (Phi(-16) is zero, and e^-200).
__device__ __forceinline__ float act_f32(int act, float z) {
    if (act == MOE_ACT_GELU) return max_nan(z, -16.f) * normcdff(z);
    if (act == MOE_ACT_SILU) {
        const float t = expf(-fabsf(z));
        return __fdividef(max_nan(z, -200.f) * (z < 0.f ? t : 1.0f), 1.0f + t);
    }
    return act == MOE_ACT_RELU && z <= 0.f ? 0.f : z;
}

template <int RM, int RN>
__global__ void __launch_bounds__(kThreads) linear_f32_kernel(const LinearArgs a, int ftiles) {
    using Tile = F32Tile<RM, RN>;
    extern __shared__ __align__(16) float smem_f32[];
    __shared__ int off[kMaxExperts + 1];
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) load_group_bounds(a.offsets, a.E, a.rows, off);
    __syncthreads();
    int ft;
    int y = divide(blockIdx.x, ftiles, ft), e = 0;  // row tile y of all groups'
    for (; e < a.E; ++e) {
        const int t = (off[e + 1] - off[e] + Tile::kRows - 1) / Tile::kRows;
        if (y < t) break;
        y -= t;
    }
    if (e == a.E) return;
    const int row0 = off[e] + y * Tile::kRows, row_end = off[e + 1], f0 = ft * Tile::kF;
    const float* __restrict__ x = static_cast<const float*>(a.x);
    const float* __restrict__ W =
        static_cast<const float*>(a.W) + static_cast<size_t>(e) * a.N * a.K;
    const int part = threadIdx.x & 7, line = threadIdx.x >> 3;  // loads: 8 threads a row
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;

    const int steps = (a.K + kStep - 1) / kStep;
    auto fetch = [&](int step) {
        if (step < steps) {
            const int k = step * kStep + part * 4;
            float* sx = smem_f32 + step % kStages * Tile::kStageFloats + line * kPitch + part * 4;
            float* sw = sx + Tile::kRows * kPitch;
#pragma unroll
            for (int i = 0; i < Tile::kRows / 16; ++i) {
                const int r = row0 + line + 16 * i;
                const bool have = r < row_end && k < a.K;
                copy16(sx + 16 * i * kPitch, have ? x + static_cast<size_t>(r) * a.K + k : x, have);
            }
#pragma unroll
            for (int i = 0; i < Tile::kF / 16; ++i) {
                const int f = f0 + line + 16 * i;
                const bool have = f < a.N && k < a.K;
                copy16(sw + 16 * i * kPitch, have ? W + static_cast<size_t>(f) * a.K + k : W, have);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    F2 pair[RM][RN] = {};  // sums over even and over odd k
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s);
    for (int step = 0; step < steps; ++step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();  // this step's values are there, the last step's have been read
        fetch(step + kStages - 1);
        const float* sx = smem_f32 + step % kStages * Tile::kStageFloats + ty * kPitch;
        const float* sw = smem_f32 + step % kStages * Tile::kStageFloats +
                          (Tile::kRows + tx) * kPitch;
#pragma unroll
        for (int k = 0; k < kStep; k += 4) {
            ulonglong2 xv[RM];
#pragma unroll
            for (int i = 0; i < RM; ++i)
                xv[i] = *reinterpret_cast<const ulonglong2*>(sx + 16 * i * kPitch + k);
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const ulonglong2 wv = *reinterpret_cast<const ulonglong2*>(sw + 8 * j * kPitch + k);
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    pair[i][j] = f2_fma(xv[i].x, wv.x, pair[i][j]);
                    pair[i][j] = f2_fma(xv[i].y, wv.y, pair[i][j]);
                }
            }
        }
    }
    float acc[RM][RN];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) {
            float even, odd;
            f2_get(pair[i][j], even, odd);
            acc[i][j] = even + odd;
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
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act_f32(a.act, v[k]);
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
long long f32_blocks(const LinearArgs& a) {
    using Tile = F32Tile<RM, RN>;
    const int groups = a.rows < a.E ? a.rows : a.E;
    return (a.rows / Tile::kRows + groups) *
           static_cast<long long>((a.N + Tile::kF - 1) / Tile::kF);
}

template <int RM, int RN>
cudaError_t launch_f32(const LinearArgs& a) {
    using Tile = F32Tile<RM, RN>;
    static PerDeviceOnce once;
    if (const cudaError_t err = opt_in_smem(once, linear_f32_kernel<RM, RN>, Tile::kSmem);
        err != cudaSuccess)
        return err;
    return launch_k(linear_f32_kernel<RM, RN>, static_cast<unsigned>(f32_blocks<RM, RN>(a)), kThreads,
                    Tile::kSmem, a.stream, a, (a.N + Tile::kF - 1) / Tile::kF);
}

// Clocks of a step: a block's own latency, or its SM's throughput.
template <int RM, int RN>
float f32_clocks(const LinearArgs& a, float latency, float throughput) {
    using Tile = F32Tile<RM, RN>;
    const int groups = a.rows < a.E ? a.rows : a.E;
    const int n = (a.rows + groups - 1) / groups;
    const long long blocks = static_cast<long long>(groups) *
                             ((n + Tile::kRows - 1) / Tile::kRows) *
                             ((a.N + Tile::kF - 1) / Tile::kF);
    const long long sms = device_sm_count();
    const float busy = static_cast<float>((blocks + sms - 1) / sms) * throughput;
    return latency > busy ? latency : busy;
}

// Measured (us; tiles of 32 x 32, 64 x 32 and 128 x 64; the clocks are fitted to these):
//   1 group, 1 row, K 1024, N 1024         17    26    57
//   1 group, 256 rows, K 1024, N 1024      27    28    61
//   1 group, 512 rows, K 1024, N 1024      75    39    62
//   8 groups, 1024 rows, K 1024, N 1024    83    68   109
//   32 groups, 1000 rows, K 512, N 768     43    51    81
//   1 group, 4096 rows, K 4096, N 4096   4980  3480  2890
cudaError_t launch_linear_f32(const LinearArgs& a) {
    const float small = f32_clocks<2, 4>(a, 985.f, 670.f);
    const float middle = f32_clocks<4, 4>(a, 1550.f, 930.f);
    const float large = f32_clocks<8, 8>(a, 6500.f, 3100.f);
    if (small <= middle && small <= large) return launch_f32<2, 4>(a);
    return middle <= large ? launch_f32<4, 4>(a) : launch_f32<8, 8>(a);
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
