// Launchers and shared device code of the operators around the fused layer:
// the quantising RMSNorm (norm.hip), the quantising SiLU-gated multiply
// (act.hip) and the dense and grouped products (gemm_pick.hip,
// gemm_split.hip, gemm_tile.hip).
#pragma once

#include "common.h"

namespace moe {

// ---------------------------------------------------------------------------
// gfx950's conversions, two values per instruction, round to nearest even
// ---------------------------------------------------------------------------

// two fp32 -> packed bf16 (a in the low half); the bits of f32_to_bf16_rne
// except that a NaN keeps its own quiet form
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// four fp32 within [-448, 448] -> packed E4M3FN codes (the codes of f32_to_e4m3_rne)
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return uint32_t(w);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Codes and scale of 8 consecutive bf16 values of a quantisation group held by
// `kLanes` neighbouring lanes (16: a 128-column group, 4: a 32-column one),
// which call it together: moe_quant_act's rule.  Returns the scale.
template <int kLanes>
__device__ __forceinline__ float quant8(const float (&v)[8], uint32_t& lo, uint32_t& hi) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, __builtin_fabsf(v[i]));
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
    const float s = fp8_group_scale(amax);
    // 1 / s of a power of two: mirror the exponent (s >= 2^-42, so 1 / s is normal)
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(__fmul_rn(v[i], inv), -448.0f), 448.0f);
    lo = pack_e4m3(q[0], q[1], q[2], q[3]);
    hi = pack_e4m3(q[4], q[5], q[6], q[7]);
    return s;
}

// A grid of at least n workgroups (n >= 1) numbered blockIdx.y * gridDim.x +
// blockIdx.x: a grid dimension holds less than 2^32 threads.
inline dim3 grid_of(int64_t n) {
    constexpr int64_t kMost = 1 << 21;
    const int64_t y = (n + kMost - 1) / kMost;
    return dim3(unsigned(y == 1 ? n : kMost), unsigned(y));
}

// ---------------------------------------------------------------------------
// launchers; kQuant: 0 none, 1 fp32 scale per 128 columns, 2 E8M0 per 32
// ---------------------------------------------------------------------------
struct NormArgs {
    const uint16_t* x;         // bf16 [rows, cols]
    const uint16_t* residual;  // bf16 [rows, cols] or null
    const uint16_t* weight;    // bf16 [cols]
    uint16_t* residual_out;    // or null
    uint16_t* y;               // or null
    uint8_t* codes;            // or null
    void* scales;
    int rows, cols;
    float eps;
};
int norm_max_cols();
hipError_t launch_norm(const NormArgs& a, int quant, hipStream_t s);

hipError_t launch_silu_mul(const uint16_t* h, int rows, int cols, float clamp_limit, int quant, uint16_t* y,
                           uint8_t* codes, void* scales, hipStream_t s);

// out[r, n] = bf16(sum_k a[r, k] w[e, n, k]) for the rows r of group e
struct RowsGemmArgs {
    const uint8_t* a;          // [rows, K] bf16 or e4m3
    const float* a_scale;      // [rows, K / 128] (fp8)
    const uint8_t* w;          // [E, N, K]
    const float* w_scale;      // [E, ceil(N / 128), K / 128] (fp8)
    const int32_t* offsets;    // [E + 1] device, or null: one group of all rows
    uint16_t* out;             // bf16 [rows, N]
    int rows, E, N, K;
};
hipError_t launch_rows_gemm(const RowsGemmArgs& g, bool fp8, hipStream_t s);
// its two forms, `shape` one of gemm_pick.hip's tiles
hipError_t launch_rows_split(const RowsGemmArgs& g, bool fp8, int shape, hipStream_t s);
hipError_t launch_rows_tile(const RowsGemmArgs& g, bool fp8, int shape, hipStream_t s);

}  // namespace moe
