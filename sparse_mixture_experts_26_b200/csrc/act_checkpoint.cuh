// act_checkpoint.cuh -- activations of the grouped linear operators, their slopes, and
// the 8-bit checkpoint format (include/moe.h, MOE_CHECKPOINT_BLOCK).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_internal.h"
#include "sm100_ptx.cuh"

namespace moe {

__device__ __forceinline__ float rcp_approx(float v) {  // one step of v's reciprocal
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The normal distribution Phi(z), with e = exp(-z^2 / 2), by Abramowitz and Stegun 7.1.26
// (erf x = 1 - (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x), off by at most 1.5e-7),
// for x = |z| / sqrt 2.  No branch, so that eight of them overlap: erff's two ranges, taken
// in turn by a warp, made the epilogue the bound (K = 2048, GELU: 44,000 cycles a tile
// against 16,400 of tensor core time).
__device__ __forceinline__ float normal_cdf(float z, float e) {
    const float t = rcp_approx(fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.0f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float tail = 0.5f * p * t * e;  // Phi(-|z|)
    return z < 0.f ? tail : 1.0f - tail;
}

// act(z).  A NaN stays a NaN in every form.
__device__ __forceinline__ float act_value(int act, float z) {
    if (act == MOE_ACT_RELU) return z <= 0.f ? 0.f : z;
    if (act == MOE_ACT_GELU) return z * normal_cdf(z, __expf(-0.5f * z * z));
    if (act == MOE_ACT_SILU) return z * rcp_approx(1.0f + __expf(-z));
    return z;
}

// act'(z); the slope of ReLU at 0 is 0.
//   GELU: Phi(z) + z phi(z), phi the normal density
//   SiLU: s (1 + z (1 - s)), s = 1 / (1 + e^-z)
__device__ __forceinline__ float act_slope(int act, float z) {
    if (act == MOE_ACT_RELU) return z <= 0.f ? 0.f : (z > 0.f ? 1.f : z);
    if (act == MOE_ACT_GELU) {
        const float e = __expf(-0.5f * z * z);
        return fmaf(0.39894228f * z, e, normal_cdf(z, e));
    }
    if (act == MOE_ACT_SILU) {
        const float s = rcp_approx(1.0f + __expf(-z));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.f;
}

constexpr int kCkptBlock = MOE_CHECKPOINT_BLOCK;
inline __host__ __device__ int ckpt_blocks(int n) { return (n + kCkptBlock - 1) / kCkptBlock; }

// Largest magnitude of a block as its bit pattern: magnitudes order like their bits, and
// an infinity or NaN is the largest of all, so that it survives into the scale.
__device__ __forceinline__ uint32_t ckpt_mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// s = amax / 128 (exact); 0 below 2^-100, where 1 / s could overflow.
__device__ __forceinline__ float ckpt_scale(uint32_t mag) {
    const float amax = __uint_as_float(mag);
    return amax < 0x1p-100f ? 0.f : amax * 0.0078125f;
}

// floor(v / s) clamped to [-128, 127].  The product with the rounded reciprocal can land
// on the wrong side of a step; the signs of v - q s and v - (q + 1) s (each one rounding,
// so the sign is that of the exact number) put it back, which matters for bf16 values that
// lie on the steps and for the sign of the smallest ones.
__device__ __forceinline__ int ckpt_code(float v, float s, float inv) {
    float q = floorf(v * inv);
    q += fmaf(-q, s, v) < 0.f ? -1.f : (fmaf(-(q + 1.f), s, v) >= 0.f ? 1.f : 0.f);
    q = fminf(fmaxf(q, -128.f), 127.f);
    return s > 0.f ? static_cast<int>(q) : 0;
}
__device__ __forceinline__ float ckpt_inverse(float s) { return s > 0.f ? __frcp_rn(s) : 0.f; }

__device__ __forceinline__ float ckpt_value(int q, float s) {
    return (static_cast<float>(q) + 0.5f) * s;
}

// Eight codes of consecutive values as two words, and back.
__device__ __forceinline__ uint2 ckpt_pack8(const float (&v)[8], float s) {
    const float inv = ckpt_inverse(s);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i >> 2] |= (static_cast<uint32_t>(ckpt_code(v[i], s, inv)) & 0xffu) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void ckpt_unpack8(uint2 c, float s, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = i < 4 ? c.x : c.y;
        v[i] = ckpt_value(static_cast<int8_t>((w >> (8 * (i & 3))) & 0xffu), s);
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

// Group bounds, clamped and monotone; offsets == nullptr: one group of all rows.  One
// thread fills off[0 .. E].
__device__ __forceinline__ void load_group_bounds(const int32_t* offsets, int E, int rows,
                                                  int* off) {
    if (offsets == nullptr) {
        off[0] = 0;
        off[1] = rows;
        return;
    }
    int prev = 0;
    for (int g = 0; g <= E; ++g) {
        int v = offsets[g];
        v = v < prev ? prev : (v > rows ? rows : v);
        off[g] = v;
        prev = v;
    }
}

}  // namespace moe
