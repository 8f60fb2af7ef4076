// SiLU-gated multiply of a product's gate and up halves (+ fp8 quantisation):
// the fused kernel of P2 section 1.2 as an operator of its own, with the
// rounding points of the fused epilogue,
//   a = bf16(bf16(silu(g)) * u),  silu(g) = g / (1 + exp(-g)),
// the optional clamp of the bf16 gate and up values before it, and codes and
// scales by moe_quant_act's rule.
//
// g is a bf16 value, so bf16(silu(g)) is a function of 16 bits; silu_f32 below
// gives its correct rounding for every finite g (a test compares all of them
// with 64-bit arithmetic), so the outputs are the definition's bit for bit.
//
// A thread makes 8 columns from 16 bytes of gate and 16 of up; a 128-column
// quantisation group is 16 neighbouring lanes.  HBM-bound: 4 bytes read per
// output, 1 + 4/128 (or 2) written; 20011 x 2048 to fp8 44.5 us, 4.64 TB/s (a
// 1 GiB copy 5.15 TB/s).  Two or four vectors a thread, or loads and stores
// past the caches' replacement, were no faster.  16 x 2048 2.8 us, of which an
// empty kernel takes 2.2.
#include "dense.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// silu(g) without overflow on either side: z = exp(-|g|) = 2^n 2^f with n whole
// and |f| <= 1/2 (f from an fma, so it keeps its low bits), r = 1 / (1 + z)
// with one Newton step, silu = g r for g >= 0 and g r z else.  Without the
// Newton step one of the 65280 finite gates (5.9375) rounds to the wrong bf16.
__device__ __forceinline__ float silu_f32(float g) {
    constexpr float kL = 1.44269504088896341f;             // log2(e) rounded to fp32
    const float a = fminf(__builtin_fabsf(g), 1000.0f);    // z and silu(-a) are 0 long before
    const float n = __builtin_rintf(a * -kL);
    const float f = __builtin_fmaf(-a, kL, -n);
    const float ex = __builtin_amdgcn_exp2f(f);
    const int ni = int(n);
    const float d = __fadd_rn(1.0f, __builtin_amdgcn_ldexpf(ex, ni));
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    return g < 0.0f ? __builtin_amdgcn_ldexpf(-a * r * ex, ni) : g * r;
}

template <int kQuant>
__global__ __launch_bounds__(kThreads) void silu_mul_kernel(const uint16_t* __restrict__ h, int rows, int cols,
                                                           float limit, uint16_t* __restrict__ yout,
                                                           uint8_t* __restrict__ codes, void* __restrict__ scales) {
    const int per_row = cols >> 3;
    const int64_t total = int64_t(rows) * per_row;
    const int64_t mine = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
    const bool live = mine < total;                  // a quantisation group is live as a whole
    const int64_t i = min(mine, total - 1);
    const int64_t at = i * 8;                        // first output column, over all rows
    const uint16_t* src = h + at + i / per_row * cols;
    const i32x4 gw = *reinterpret_cast<const i32x4*>(src);
    const i32x4 uw = *reinterpret_cast<const i32x4*>(src + cols);
    float g[8], u[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        g[2 * q] = bf16_lo(gw[q]);
        g[2 * q + 1] = bf16_hi(gw[q]);
        u[2 * q] = bf16_lo(uw[q]);
        u[2 * q + 1] = bf16_hi(uw[q]);
    }
    if (limit > 0.0f) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            g[q] = fminf(g[q], limit);
            u[q] = fminf(fmaxf(u[q], -limit), limit);
        }
    }
    i32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t sl = pack_bf16(silu_f32(g[2 * q]), silu_f32(g[2 * q + 1]));
        o[q] = int(pack_bf16(__fmul_rn(bf16_lo(sl), u[2 * q]), __fmul_rn(bf16_hi(sl), u[2 * q + 1])));
    }
    if (live && yout) *reinterpret_cast<i32x4*>(yout + at) = o;
    if constexpr (kQuant != 0) {
        constexpr int kLanes = kQuant == 1 ? 16 : 4;
        uint32_t lo, hi;
        const float s = quant8<kLanes>(o, lo, hi);
        if (live) {
            *reinterpret_cast<uint2*>(codes + at) = uint2{lo, hi};
            if ((threadIdx.x & (kLanes - 1)) == 0) {
                const int64_t group = at / (8 * kLanes);
                if constexpr (kQuant == 1) static_cast<float*>(scales)[group] = s;
                else static_cast<uint8_t*>(scales)[group] = uint8_t(__float_as_uint(s) >> 23);
            }
        }
    }
}

}  // namespace

hipError_t launch_silu_mul(const uint16_t* h, int rows, int cols, float clamp_limit, int quant, uint16_t* y,
                           uint8_t* codes, void* scales, hipStream_t s) {
    const int64_t n = int64_t(rows) * (cols >> 3);
    void (*kern)(const uint16_t*, int, int, float, uint16_t*, uint8_t*, void*) =
        quant == 0 ? silu_mul_kernel<0> : quant == 1 ? silu_mul_kernel<1> : silu_mul_kernel<2>;
    return start(kern, grid_of((n + kThreads - 1) / kThreads), kThreads, s, h, rows, cols, clamp_limit, y, codes,
                 scales);
}

}  // namespace moe
