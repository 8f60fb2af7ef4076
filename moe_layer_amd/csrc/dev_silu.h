// The SiLU-gated multiply of 8 columns, device code shared by the operators
// that make it (act.hip, quant_int8.hip).
#pragma once

#include "dense.h"

namespace moe {

namespace {

// silu(g) without overflow on either side: z = exp(-|g|) = h^2, h = 2^(c |g|)
// with c = -log2(e) / 2 in two parts.  c_hi has 16 bits, so its product with a
// bf16 |g| is exact; 2^(c_lo |g|) is 1 + c_lo ln(2) |g| to 2^-24.  r = 1 / (1 + z)
// with one Newton step, silu = g r for g >= 0 and g r h h else (z itself would
// be subnormal where silu is not).  Without the Newton step one of the 65280
// finite gates (5.9375) rounds to the wrong bf16.
__device__ __forceinline__ float silu_f32(float g, float below) {
    constexpr float kHi = -0.721343994140625f;                      // -log2(e) / 2 in 16 bits
    constexpr float kLo = -2.444247576e-06f;                   // ln(2) times the rest
    // min(|g|, 1000), where z and silu(-a) have long been 0: the middle of three
    // is one instruction, a minimum makes its operand canonical first
    const float a = __builtin_amdgcn_fmed3f(__builtin_fabsf(g), below, 1000.0f);
    float h = __builtin_amdgcn_exp2f(a * kHi);
    h = __builtin_fmaf(h, a * kLo, h);
    const float d = __builtin_fmaf(h, h, 1.0f);
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    return g < 0.0f ? -a * r * h * h : g * r;
}

// a = bf16(bf16(silu(g)) * u) of 8 gates and ups in packed bf16, after the clamp
template <bool kClamp>
__device__ __forceinline__ i32x4 silu_mul8(const i32x4& gw, const i32x4& uw, float limit) {
    float g[8], u[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        g[2 * q] = bf16_lo(gw[q]);
        g[2 * q + 1] = bf16_hi(gw[q]);
        u[2 * q] = bf16_lo(uw[q]);
        u[2 * q + 1] = bf16_hi(uw[q]);
    }
    if constexpr (kClamp) {
        // comparisons that a NaN fails: it stays (the middle of three alone would take
        // it for the lowest; NaN-keeping minima 39.4 us at 20011 x 2048, these 37.7)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            g[q] = g[q] > limit ? limit : g[q];
            u[q] = u[q] == u[q] ? __builtin_amdgcn_fmed3f(u[q], -limit, limit) : u[q];
        }
    }
    float below = 0.0f;                              // not known as a constant, which would undo the choice of fmed3
    asm("" : "+v"(below));
    i32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t sl = pack_bf16(silu_f32(g[2 * q], below), silu_f32(g[2 * q + 1], below));
        o[q] = int(pack_bf16(__fmul_rn(bf16_lo(sl), u[2 * q]), __fmul_rn(bf16_hi(sl), u[2 * q + 1])));
    }
    return o;
}

}  // namespace

}  // namespace moe
