// act_checkpoint.cuh -- activations of the grouped linear operators, their slopes, and
// the 8-bit checkpoint format (include/moe.h, MOE_CHECKPOINT_BLOCK).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_internal.h"
#include "sm100_ptx.cuh"

namespace moe {

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Phi(-|z|), Phi the normal distribution, and e = exp(-z^2 / 2), by Abramowitz and Stegun
// 7.1.26 (erf x = 1 - (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x), off by at most
// 1.5e-7) at x = |z| / sqrt 2, with the exponent taken in base 2 of w = |z| sqrt(log2(e) / 2).
// No branch, so that eight of them overlap: erff's two ranges, taken in turn by a warp, made
// the epilogue the bound (K = 2048, GELU: 44,000 cycles a tile against 16,400 of tensor core
// time).  11 instructions and 2 of the special function unit.
__device__ __forceinline__ float normal_tail(float z, float& e) {
    const float w = fabsf(z) * 0.84932180f;       // sqrt(log2(e) / 2)
    e = ex2_approx(-w * w);
    const float t = rcp_approx(fmaf(0.27273749f, w, 1.0f));  // 0.3275911 / sqrt(log2(e))
    float p = fmaf(0.5307027145f, t, -0.726576013f);         // the coefficients, halved
    p = fmaf(p, t, 0.7107068705f);
    p = fmaf(p, t, -0.142248368f);
    p = fmaf(p, t, 0.127414796f);
    return p * t * e;
}
__device__ __forceinline__ float sigmoid(float z) {
    return rcp_approx(1.0f + ex2_approx(-1.44269504f * z));
}

// v = act(v).  A NaN stays one; an infinity gives an infinity or NaN.
//   GELU: z Phi(z) = max(z, 0) - |z| Phi(-|z|)
__device__ __forceinline__ void act_value8(int act, float (&v)[8]) {
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float e;
            const float tail = normal_tail(v[i], e);
            v[i] = fmaf(-fabsf(v[i]), tail, fmaxf(v[i], 0.f));
        }
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sigmoid(v[i]);
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i];
    }
}

// g *= act'(z); the slope of ReLU at 0 is 0.
//   GELU: Phi(z) + z phi(z), phi the normal density
//   SiLU: s (1 + z (1 - s)), s = 1 / (1 + e^-z)
__device__ __forceinline__ void act_slope8(int act, const float (&z)[8], float (&g)[8]) {
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float e;
            const float tail = normal_tail(z[i], e);
            const float phi = fmaf(0.39894228f * z[i], e, 0.5f);
            g[i] *= phi + copysignf(0.5f - tail, z[i]);
        }
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = sigmoid(z[i]);
            g[i] *= s * fmaf(z[i], 1.0f - s, 1.0f);
        }
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= z[i] <= 0.f ? 0.f : (z[i] > 0.f ? 1.f : z[i]);
    }
}

constexpr int kCkptBlock = MOE_CHECKPOINT_BLOCK;
inline __host__ __device__ int ckpt_blocks(int n) { return (n + kCkptBlock - 1) / kCkptBlock; }

// Largest magnitude of eight values; a NaN is larger than all, so that it reaches the scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ckpt_amax8(const float (&v)[8]) {
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
    return m;
}
// .. and of the block that four neighbouring lanes hold.  The whole warp calls this.
__device__ __forceinline__ float ckpt_amax_block(float m) {
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// s = amax / 128 (exact); 0 below 2^-100, where 1 / s could overflow.
__device__ __forceinline__ float ckpt_scale(float amax) {
    return amax < 0x1p-100f ? 0.f : amax * 0.0078125f;
}

__device__ __forceinline__ float ckpt_inverse(float s) { return s > 0.f ? rcp_approx(s) : 0.f; }

// floor(v / s) clamped to [-128, 127], as the low byte of the result.  v times the rounded
// reciprocal, rounded to the nearest whole number (by adding and taking off 1.5 2^23), is
// the answer or one more or less; the signs of v - q s and v - (q + 1) s (each one
// rounding, so the sign is that of the exact number) say which.  That is exact for bf16
// values, which often lie on a step, and keeps the sign of the smallest.  No conversion
// instruction: those run at a quarter of the rate.
__device__ __forceinline__ uint32_t ckpt_code(float v, float s, float inv) {
    constexpr float kMagic = 12582912.f;
    float q = fmaf(v, inv, kMagic) - kMagic;
    q += fmaf(-q, s, v) < 0.f ? -1.f : (fmaf(-(q + 1.f), s, v) >= 0.f ? 1.f : 0.f);
    q = fminf(fmaxf(q, -128.f), 127.f);
    return s > 0.f ? __float_as_uint(q + kMagic) : 0u;
}

__device__ __forceinline__ uint2 ckpt_bytes8(const uint32_t (&c)[8]) {
    auto four = [](uint32_t a, uint32_t b, uint32_t d, uint32_t e) {
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(d, e, 0x0040), 0x5410);
    };
    return make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
}
// Eight codes of consecutive values as two words.
__device__ __forceinline__ uint2 ckpt_pack8(const float (&v)[8], float s) {
    const float inv = ckpt_inverse(s);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = ckpt_code(v[i], s, inv);
    return ckpt_bytes8(c);
}
// The same for fp32 sums, whose last bits are rounding anyway: one multiply-add that rounds
// down is the floor, and a reciprocal short of 1 / s by about 2^-22 keeps |v / s| below 128
// without a clamp.  A value within 2^-15 of a step may take the code below it; the sign is
// kept.  (15 instructions a value the exact way, 2 this way: training's epilogue at K = 2048
// is bound by them.)
__device__ __forceinline__ uint2 ckpt_pack8_sums(const float (&v)[8], float s) {
    const float inv = ckpt_inverse(s) * (1.0f - 0x1p-22f);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(__fmaf_rd(v[i], inv, 12582912.f));
    return ckpt_bytes8(c);
}
// (q + 1/2) s = q s + s/2 in one rounding.  A byte with its sign bit flipped is q + 128;
// put below the exponent of 2^23 it is the float 2^23 + 128 + q.
__device__ __forceinline__ void ckpt_unpack8(uint2 c, float s, float (&v)[8]) {
    const float half = 0.5f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = (i < 4 ? c.x : c.y) ^ 0x80808080u;
        const float q =
            __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 | (i & 3))) - 8388736.f;
        v[i] = fmaf(q, s, half);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Group bounds, clamped to [0, rows] and never falling; offsets == nullptr: one group of
// all rows.  One whole warp fills off[0 .. E]; the loads go out together.
__device__ __forceinline__ void load_group_bounds(const int32_t* offsets, int E, int rows,
                                                  int* off) {
    const int lane = threadIdx.x & 31;
    auto bound = [&](int g) {
        if (offsets == nullptr) return g == 0 ? 0 : rows;
        const int v = offsets[g];
        return v < 0 ? 0 : (v > rows ? rows : v);
    };
    int v = lane <= E ? bound(lane) : 0;
    int last = E == 32 ? bound(32) : 0;  // the 33rd bound has no lane of its own
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = max(v, below);
    }
    if (lane <= E) off[lane] = v;
    if (E == 32 && lane == 31) off[32] = max(v, last);
    __syncwarp();
}

}  // namespace moe
