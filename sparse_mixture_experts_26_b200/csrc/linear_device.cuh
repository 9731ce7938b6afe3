// linear_device.cuh -- device code the grouped linear operators share: activations and their
// slopes, the 8-bit checkpoint format (include/moe.h, MOE_CHECKPOINT_BLOCK), group bounds.
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

// The larger one, the smaller one, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two floats in a 64-bit register: one instruction works on both.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_get(F2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_all(float a) { return f2(a, a); }

// Phi(-x) of two x in [0, 24], Phi the normal distribution, and e = exp(-x^2 / 2), by
// Abramowitz and Stegun 7.1.26 (erf u = 1 - (a1 t + .. + a5 t^5) exp(-u^2), t = 1 / (1 + p u),
// off by at most 1.5e-7) at u = x / sqrt 2.  The error shrinks with exp(-u^2): less than a
// bf16 half step relative to Phi(-x) up to x = 6.  No branch (erff's two ranges, taken in
// turn by a warp, made a GELU epilogue the bound), and one reciprocal for both values: the
// special function unit does 16 a clock, an eighth of the others.
__device__ __forceinline__ F2 normal_tails(float x0, float x1, F2& e) {
    const F2 x = f2(x0, x1);
    float m0, m1, d0, d1;
    f2_get(f2_mul(f2_mul(x, x), f2_all(-0.72134752f)), m0, m1);   // -log2(e) / 2
    e = f2(ex2_approx(m0), ex2_approx(m1));
    f2_get(f2_fma(x, f2_all(0.23164189f), f2_all(1.0f)), d0, d1);  // p / sqrt 2
    const float r = rcp_approx(d0 * d1);
    const F2 t = f2(r * d1, r * d0);
    F2 p = f2_fma(f2_all(0.5307027145f), t, f2_all(-0.726576013f));  // a5 .. a1, halved
    p = f2_fma(p, t, f2_all(0.7107068705f));
    p = f2_fma(p, t, f2_all(-0.142248368f));
    p = f2_fma(p, t, f2_all(0.127414796f));
    return f2_mul(f2_mul(p, t), e);
}
// SiLU z / (1 + e^-z), relative to itself as far down as e^z is a normal number, zero below; one
// reciprocal a value, so that nothing has to be held inside fp32 and a NaN stays with its own.
__device__ __forceinline__ float silu(float z) {
    return max_nan(z, -200.f) * rcp_approx(1.0f + ex2_approx(-1.44269504f * z));
}

// v = act(v), also far out: a NaN stays one (and leaves its neighbour alone), infinities give
// the limits.
//   GELU: z Phi(z) = max(z, 0) - |z| Phi(-|z|), |z| at most 24, where Phi is zero
__device__ __forceinline__ void act_value8(int act, float (&v)[8]) {
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            F2 e;
            float t0, t1;
            const float x0 = fminf(fabsf(v[i]), 24.f), x1 = fminf(fabsf(v[i + 1]), 24.f);
            f2_get(normal_tails(x0, x1, e), t0, t1);
            v[i] = fmaf(-x0, t0, max_nan(v[i], 0.f));
            v[i + 1] = fmaf(-x1, t1, max_nan(v[i + 1], 0.f));
        }
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu(v[i]);
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i];
    }
}

// g *= act'(z); the slope of ReLU at 0 is 0.
//   GELU: Phi(z) + z phi(z), phi the normal density: with x = |z| and d = x phi(x) - Phi(-x),
//   1 + d, or -d for z < 0, where Phi(-x) is all there is and keeps its bits
//   SiLU: s (1 + z (1 - s)), s = 1 / (1 + e^-z), where z (1 - s) is taken as z e^-z s for z > 0,
//   so that it vanishes for large z
__device__ __forceinline__ void act_slope8(int act, const float (&z)[8], float (&g)[8]) {
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            F2 e;
            const float x0 = min_nan(fabsf(z[i]), 24.f), x1 = min_nan(fabsf(z[i + 1]), 24.f);
            const F2 t = normal_tails(x0, x1, e);
            float d[2];
            f2_get(f2_fma(f2_mul(f2(x0, x1), f2_all(0.39894228f)), e, f2_mul(t, f2_all(-1.0f))),
                   d[0], d[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) g[i + k] *= z[i + k] < 0.f ? -d[k] : 1.0f + d[k];
        }
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = ex2_approx(-1.44269504f * z[i]), s = rcp_approx(1.0f + e);
            const float rest = z[i] > 0.f ? e * s : 1.0f - s;
            g[i] *= s * fmaf(max_nan(min_nan(z[i], 200.f), -200.f), rest, 1.0f);
        }
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = z[i] <= 0.f ? 0.f : g[i];
    }
}

// a / b and the remainder, 0 <= a < 2^31, b > 0: the quotient of the rounded floats is off by
// one, or by 2^-21 of a large quotient.  (A tile's decode stands between two tiles; integer divisions there cost
// the tensor cores about 1000 cycles a tile.)
__device__ __forceinline__ int divide(int a, int b, int& remainder) {
    int q = __float2int_rd(static_cast<float>(a) * rcp_approx(static_cast<float>(b)));
    int r = a - q * b;
    while (r < 0) --q, r += b;
    while (r >= b) ++q, r -= b;
    remainder = r;
    return q;
}

constexpr int kCkptBlock = MOE_CHECKPOINT_BLOCK;
inline __host__ __device__ int ckpt_blocks(int n) { return (n + kCkptBlock - 1) / kCkptBlock; }

// Largest magnitude of eight values; a NaN is larger than all, so that it reaches the scale.
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
// The same for bf16 values, in a third of the instructions.  Quotients of two 8-bit
// significands are whole or at least 2^-8 away from the next whole number above, except for
// small negative ones below zero: so 2^-10 on top of the product makes up for its rounding,
// and the sign is put right by hand (the same minimum holds the largest value at 127).
__device__ __forceinline__ uint2 ckpt_pack8_bf16(const float (&v)[8], float s) {
    constexpr float kMagic = 12582912.f;
    const float inv = ckpt_inverse(s);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = __fadd_rd(fmaf(v[i], inv, 0x1p-10f), kMagic);
        c[i] = __float_as_uint(fminf(q, v[i] < 0.f ? kMagic - 1.f : kMagic + 127.f));
    }
    const uint2 w = ckpt_bytes8(c);
    return s == 0.f ? make_uint2(0u, 0u) : w;
}
// The same for fp32 sums, whose last bits are rounding anyway: one multiply-add that rounds
// down is the floor, and a reciprocal short of 1 / s by about 2^-22 keeps |v / s| below 128
// without a clamp.  Of a value on a step or less than 2^-14 beyond it, seen from zero, the code
// may be the neighbour nearer zero, and the value off by (1/2 + 2^-14) s; the sign is kept.
// (15 instructions a value the exact way, 2 this way: training's epilogue at K = 2048 is bound
// by them.)
// BELOW_ZERO: a zero takes the code below it, so that q >= 0 says z > 0: rounded up from one less
// instead of down, which differs only at whole products (others' codes are short of theirs anyway).
template <bool BELOW_ZERO>
__device__ __forceinline__ uint2 ckpt_pack8_sums(const float (&v)[8], float s) {
    const float inv = ckpt_inverse(s) * (1.0f - 0x1p-22f);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = __float_as_uint(BELOW_ZERO ? __fmaf_ru(v[i], inv, 12582911.f)
                                          : __fmaf_rd(v[i], inv, 12582912.f));
    return ckpt_bytes8(c);
}
// (q + 1/2) s = q s + s/2 in one rounding.  A byte with its sign bit flipped is q + 128;
// put below the exponent of 2^23 it is the float 2^23 + 128 + q.
__device__ __forceinline__ void ckpt_unpack8(uint2 c, float s, float (&v)[8]) {
    const F2 scale = f2_all(s), half = f2_all(0.5f * s);
    const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t q = w[i >> 2];
        const F2 u = f2(__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7650 | (i & 3))),
                        __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7651 + (i & 3))));
        f2_get(f2_fma(f2_add(u, f2_all(-8388736.f)), scale, half), v[i], v[i + 1]);
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

// The same for global memory: eight floats of a thread are one 32-byte access where the buffer
// starts on a 32-byte boundary, which the 16 bytes that callers promise may not be.  (Two
// 16-byte stores write every sector in halves: 600 x 7168 restored to fp32 8.5 us, now 5.0.)
__device__ __forceinline__ bool aligned32(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}
__device__ __forceinline__ void load8_global(const float* p, float (&v)[8]) {
    if (!aligned32(p)) return load8(p, v);
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void store8_global(float* p, const float (&v)[8]) {
    if (!aligned32(p)) return store8(p, v);
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void load8_global(const __nv_bfloat16* p, float (&v)[8]) { load8(p, v); }
__device__ __forceinline__ void store8_global(__nv_bfloat16* p, const float (&v)[8]) {
    store8(p, v);
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
