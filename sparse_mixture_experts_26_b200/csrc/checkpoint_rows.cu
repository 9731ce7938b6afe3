// checkpoint_rows.cu -- the 8-bit activation checkpoint by itself: rows in, codes and
// block scales out, and back through an activation.
//
// A block is 32 consecutive values of a row: s = max|v| / 128, q = floor(v / s), and q
// stands for (q + 1/2) s.  Half a step of offset instead of rounding to whole steps uses
// all 256 codes symmetrically (error <= max / 256 instead of max / 254 with a wasted
// code) and keeps the sign of every value.
//
// Both directions are bound by their bytes.  A thread owns eight consecutive values of a
// row (16- or 32-byte accesses, 8 bytes of codes), so four neighbouring lanes own a block
// and two shuffles give its largest magnitude; it walks down the rows with kRows of them
// in flight.  A block of threads is 2^lg column groups wide, to fit narrow rows too.
// Measured, restoring 8192 x 14336 to bf16 (367 MB; us): plain 60, SiLU 69 (the special function
// unit, 80 % busy), GELU 80 to 87 (17 instructions a value: 72 % of the issue slots and 65 % of
// the copy bandwidth, since a thread loads its rows and then computes them).  To fp32 (602 MB):
// 98 to 100.  Saving (us): bf16 65 to 68, fp32 93 to 96.
#include <cuda_bf16.h>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows in flight per thread

struct Walk {
    int c;           // first of this thread's eight columns
    int row, step;   // its first row, and the distance to the next
    __device__ __forceinline__ Walk(int lg, int strips) {
        const int by = static_cast<int>(blockIdx.x) / strips;
        const int bx = static_cast<int>(blockIdx.x) - by * strips;
        c = ((bx << lg) + static_cast<int>(threadIdx.x & ((1u << lg) - 1))) * 8;
        const int per = kThreads >> lg;
        row = by * per + static_cast<int>(threadIdx.x >> lg);
        step = static_cast<int>(gridDim.x) / strips * per;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
    checkpoint_save_kernel(const T* __restrict__ v, int rows, int N, int lg, int strips,
                           int8_t* __restrict__ codes, float* __restrict__ scales) {
    pdl_wait();
    pdl_launch_dependents();
    const Walk w(lg, strips);
    const int nb = ckpt_blocks(N);
    const bool have = w.c < N;
    // the warp's lanes leave together: rows differ inside a warp only for narrow blocks, so
    // the loop runs on the smallest row of the warp
    const int lead = __shfl_sync(0xffffffffu, w.row, 0);
    for (int d = 0; lead + d < rows; d += kRows * w.step) {
        float x[kRows][8];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = w.row + d + k * w.step;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = 0.f;
            if (have && r < rows) load8_global(v + static_cast<size_t>(r) * N + w.c, x[k]);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = w.row + d + k * w.step;
            const float s = ckpt_scale(ckpt_amax_block(ckpt_amax8(x[k])));
            if (have && r < rows) {
                *reinterpret_cast<uint2*>(codes + static_cast<size_t>(r) * N + w.c) =
                    sizeof(T) == 2 ? ckpt_pack8_bf16(x[k], s) : ckpt_pack8(x[k], s);
                if ((w.c & (kCkptBlock - 1)) == 0)
                    scales[static_cast<size_t>(r) * nb + w.c / kCkptBlock] = s;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6)
    checkpoint_restore_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                              int rows, int N, int lg, int strips, int act, T* __restrict__ out) {
    pdl_wait();
    pdl_launch_dependents();
    const Walk w(lg, strips);
    const int nb = ckpt_blocks(N);
    if (w.c >= N) return;
    for (int row = w.row; row < rows; row += kRows * w.step) {
        uint2 q[kRows];
        float s[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = row + k * w.step;
            if (r >= rows) continue;
            q[k] = *reinterpret_cast<const uint2*>(codes + static_cast<size_t>(r) * N + w.c);
            s[k] = scales[static_cast<size_t>(r) * nb + w.c / kCkptBlock];
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = row + k * w.step;
            if (r >= rows) continue;
            float x[8];
            ckpt_unpack8(q[k], s[k], x);
            act_value8(act, x);
            store8_global(out + static_cast<size_t>(r) * N + w.c, x);
        }
    }
}

// Blocks of 2^lg column groups x (256 >> lg) rows; up to 16 blocks an SM, each walking down.
struct Layout {
    int lg, strips, grid;
    Layout(int rows, int N) {
        const int groups = (N + 7) / 8;
        lg = 2;
        while (lg < 8 && (1 << lg) < groups) ++lg;
        strips = (groups + (1 << lg) - 1) >> lg;
        // one walk of kRows rows each, unless that leaves SMs without a block
        const long long per = kThreads >> lg;
        long long down = (rows + per * kRows - 1) / (per * kRows);
        if (down * strips < device_sm_count()) down = (rows + per - 1) / per;
        long long most = static_cast<long long>(device_sm_count()) * 16 / strips;
        if (most < 1) most = 1;
        grid = static_cast<int>((down < most ? down : most) * strips);
    }
};

}  // namespace

cudaError_t launch_checkpoint_save(const void* v, int rows, int N, moe_dtype dt, int8_t* codes,
                                   float* scales, cudaStream_t s) {
    const Layout l(rows, N);
    if (dt == MOE_BF16)
        return launch_k(checkpoint_save_kernel<__nv_bfloat16>, l.grid, kThreads, 0, s,
                        static_cast<const __nv_bfloat16*>(v), rows, N, l.lg, l.strips, codes,
                        scales);
    return launch_k(checkpoint_save_kernel<float>, l.grid, kThreads, 0, s,
                    static_cast<const float*>(v), rows, N, l.lg, l.strips, codes, scales);
}

cudaError_t launch_checkpoint_restore(const int8_t* codes, const float* scales, int rows, int N,
                                      int act, moe_dtype out_dt, void* out, cudaStream_t s) {
    const Layout l(rows, N);
    if (out_dt == MOE_BF16)
        return launch_k(checkpoint_restore_kernel<__nv_bfloat16>, l.grid, kThreads, 0, s, codes,
                        scales, rows, N, l.lg, l.strips, act, static_cast<__nv_bfloat16*>(out));
    return launch_k(checkpoint_restore_kernel<float>, l.grid, kThreads, 0, s, codes, scales, rows,
                    N, l.lg, l.strips, act, static_cast<float*>(out));
}

}  // namespace moe
