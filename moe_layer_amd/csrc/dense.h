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

// maximum of the two 16-bit halves of each word
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_u16(uint32_t v) {
    return pk_max_u16(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, false)));
}

// Codes and scale of 8 consecutive bf16 values (packed, w) of a quantisation
// group held by kLanes neighbouring lanes (16: a 128-column group, 4: a
// 32-column one), which call it together: moe_quant_act's rule, whose scale
// never saturates a finite value.  The maximum is taken over the bits without
// their sign, which order as the magnitudes do.  Returns the scale.
template <int kLanes>
__device__ __forceinline__ float quant8(const i32x4& w, uint32_t& lo, uint32_t& hi) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t m = pk_max_u16(pk_max_u16(uint32_t(w[0]) & kAbs, uint32_t(w[1]) & kAbs),
                            pk_max_u16(uint32_t(w[2]) & kAbs, uint32_t(w[3]) & kAbs));
    m = dpp_max_u16<0xb1>(m);                              // quad_perm [1,0,3,2]
    m = dpp_max_u16<0x4e>(m);                              // quad_perm [2,3,0,1]
    if constexpr (kLanes == 16) {
        m = dpp_max_u16<0x141>(m);                         // row_half_mirror
        m = dpp_max_u16<0x140>(m);                         // row_mirror
    }
    const float s = fp8_group_scale(__uint_as_float(max(m & 0xffffu, m >> 16) << 16));
    // 1 / s of a power of two: mirror the exponent (s >= 2^-42, so 1 / s is normal)
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[2 * i] = __fmul_rn(bf16_lo(w[i]), inv);
        q[2 * i + 1] = __fmul_rn(bf16_hi(w[i]), inv);
    }
    lo = pack_e4m3(q[0], q[1], q[2], q[3]);
    hi = pack_e4m3(q[4], q[5], q[6], q[7]);
    return s;
}

// inclusive sum over the wave's lanes, in lane order
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast 31 into rows 2 and 3
    return v;
}

// Launch one kernel with its arguments (what <<<>>> does, in one runtime call
// instead of three; these launches stand between kernels of a few us).
template <typename... P, typename... A>
hipError_t start(void (*kern)(P...), dim3 grid, int threads, hipStream_t s, A... args) {
    static_assert(sizeof...(P) == sizeof...(A), "kernel arguments");
    return [&](P... p) {
        void* list[] = {static_cast<void*>(&p)...};
        return hipLaunchKernel(reinterpret_cast<const void*>(kern), grid, dim3(threads), list, 0, s);
    }(args...);
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
    double inv_cols;   // 1 / cols
};
hipError_t launch_norm(const NormArgs& a, int quant, hipStream_t s);

hipError_t launch_silu_mul(const uint16_t* h, int rows, int cols, float clamp_limit, int quant, uint16_t* y,
                           uint8_t* codes, void* scales, hipStream_t s);

// out[r, n] = bf16(sum_k a[r, k] w[e, n, k]) for the rows r of group e
enum RowsKind { kRowsBf16, kRowsFp8, kRowsInt8 };
struct RowsGemmArgs {
    const uint8_t* a;          // [rows, K] bf16, e4m3 or int8
    const float* a_scale;      // [rows, K / 128] (fp8), [rows] (int8)
    const uint8_t* w;          // [E, N, K]
    const float* w_scale;      // [E, ceil(N / 128), K / 128] (fp8), [E, N] (int8)
    const int32_t* offsets;    // [E + 1] device, or null: one group of all rows
    uint16_t* out;             // bf16 [rows, N]
    int rows, E, N, K;
};
hipError_t launch_rows_gemm(const RowsGemmArgs& g, RowsKind kind, hipStream_t s);
// the kernel that it takes: the form, its tile (gemm_pick.hip) and whether the
// weights go past the caches' replacement.  Reads sizes only, of offsets whether
// they are there.
struct RowsPlan {
    bool split;
    int shape, bw, bt, per_cu;
    bool one_pass;
};
RowsPlan plan_rows_gemm(const RowsGemmArgs& g, RowsKind kind);
hipError_t launch_rows_split(const RowsGemmArgs& g, RowsKind kind, int shape, bool one_pass, hipStream_t s);
hipError_t launch_rows_tile(const RowsGemmArgs& g, RowsKind kind, int shape, bool one_pass, hipStream_t s);

}  // namespace moe
