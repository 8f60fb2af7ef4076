// C ABI of the operators around the fused layer: argument checks and launches
// of moe_rmsnorm, moe_silu_mul, moe_gemm_fp8, moe_gemm_int8 and
// moe_grouped_gemm (documented in include/moe.h).
#include "moe.h"

#include <cmath>

#include "api_checks.h"
#include "dense.h"

using namespace moe;

namespace {

// columns per scale of a quantised row, 0 for none, -1 for an unknown format
int quant_group(int32_t quant) {
    switch (quant) {
        case MOE_WDTYPE_BF16: return 0;
        case MOE_WDTYPE_FP8_E4M3: return MOE_QUANT_GROUP;
        case MOE_WDTYPE_MXFP8: return MOE_MX_BLOCK;
        default: return -1;
    }
}
int quant_kind(int group) { return group == 0 ? 0 : group == MOE_QUANT_GROUP ? 1 : 2; }
int64_t scale_bytes(int64_t elems, int group) {
    return group == 0 ? 0 : elems / group * (group == MOE_QUANT_GROUP ? 4 : 1);
}

// codes and scales: both for a quantised format, neither else
int check_codes(const uint8_t* codes, const void* scales, int group) {
    if (group == 0) return codes || scales ? MOE_ERR_INVALID_ARG : MOE_OK;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_product(const void* a, const float* a_scale, const void* w, const float* w_scale, const void* out,
                  bool scaled) {
    if (!a || !w || !out || !aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
    if (scaled ? !a_scale || !w_scale || !aligned(a_scale, 4) || !aligned(w_scale, 4) : a_scale || w_scale)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// the operands of a weight type; false for an unknown one
bool rows_kind(int32_t wdtype, RowsKind& kind) {
    switch (wdtype) {
        case MOE_WDTYPE_BF16: kind = kRowsBf16; return true;
        case MOE_WDTYPE_FP8_E4M3: kind = kRowsFp8; return true;
        case MOE_WDTYPE_INT8: kind = kRowsInt8; return true;
        default: return false;
    }
}
// whether the products take rows of K elements
bool fits_k(RowsKind kind, int32_t K) {
    switch (kind) {
        case kRowsBf16: return K % 64 == 0 && K <= kMaxCols;
        case kRowsFp8: return K % MOE_QUANT_GROUP == 0 && K <= kMaxCols;
        default: return K % 16 == 0 && K <= MOE_MAX_INT8_K;
    }
}

}  // namespace

extern "C" {

MOE_API int moe_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int32_t rows,
                        int32_t cols, int32_t quant, void* residual_out, void* y, uint8_t* codes, void* scales,
                        hipStream_t stream) {
    const int group = quant_group(quant);
    if (rows < 0 || cols <= 0 || group < 0 || !(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (cols % (group ? group : 8) != 0 || cols > MOE_MAX_NORM_COLS) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!x || !weight || !aligned(x, 16) || !aligned(weight, 16) || !aligned(residual, 16) ||
        !aligned(residual_out, 16) || !aligned(y, 16) || (residual_out && !residual) ||
        (!residual_out && !y && !codes))
        return MOE_ERR_INVALID_ARG;
    const int st = check_codes(codes, scales, group);
    if (st != MOE_OK) return st;
    const int64_t n = int64_t(rows) * cols;
    if (clash({{residual_out, 2 * n}, {y, 2 * n}, {codes, n}, {scales, scale_bytes(n, group)}},
              {{x, 2 * n}, {residual, 2 * n}, {weight, 2 * int64_t(cols)}}, 2))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.weight = static_cast<const uint16_t*>(weight);
    a.residual_out = static_cast<uint16_t*>(residual_out);
    a.y = static_cast<uint16_t*>(y);
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.inv_cols = 1.0 / cols;
    return hip_status(launch_norm(a, quant_kind(group), stream));
}

MOE_API int moe_silu_mul(const void* h, int32_t rows, int32_t cols, float clamp_limit, int32_t quant, void* y,
                         uint8_t* codes, void* scales, hipStream_t stream) {
    const int group = quant_group(quant);
    if (rows < 0 || cols <= 0 || group < 0 || !(clamp_limit >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (cols % (group ? group : 8) != 0 || cols > kMaxCols) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!h || !aligned(h, 16) || !aligned(y, 16) || (group == 0 && !y)) return MOE_ERR_INVALID_ARG;
    const int st = check_codes(codes, scales, group);
    if (st != MOE_OK) return st;
    const int64_t n = int64_t(rows) * cols;
    if (clash({{y, 2 * n}, {codes, n}, {scales, scale_bytes(n, group)}}, {{h, 4 * n}}, 0)) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_silu_mul(static_cast<const uint16_t*>(h), rows, cols, clamp_limit, quant_kind(group),
                                      static_cast<uint16_t*>(y), codes, scales, stream));
}

MOE_API int moe_gemm_plan(int32_t rows, int32_t E, int32_t N, int32_t K, int32_t wdtype, moe_gemm_plan_info* out) {
    if (rows < 1 || E < 0 || E > MOE_MAX_EXPERTS || N <= 0 || K <= 0 || !out) return MOE_ERR_INVALID_ARG;
    if (wdtype == MOE_WDTYPE_MXFP8) return MOE_ERR_UNSUPPORTED;
    RowsKind kind;
    if (!rows_kind(wdtype, kind)) return MOE_ERR_INVALID_ARG;
    if ((E == 0 && kind == kRowsBf16) || !fits_k(kind, K) || rows > kMaxRows || N > kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    static const int32_t there = 0;   // the plan looks at no offset
    RowsGemmArgs g{};
    g.offsets = E > 0 ? &there : nullptr;
    g.rows = rows;
    g.E = E > 0 ? E : 1;
    g.N = N;
    g.K = K;
    const RowsPlan p = plan_rows_gemm(g, kind);
    *out = moe_gemm_plan_info{p.split ? 1 : p.per_cu == 2 ? 2 : 0, p.bw, p.bt, p.one_pass};
    return MOE_OK;
}

MOE_API int moe_gemm_fp8(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int32_t M,
                         int32_t N, int32_t K, void* out, hipStream_t stream) {
    if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % MOE_QUANT_GROUP != 0 || M > kMaxRows || N > kMaxRows || K > kMaxCols) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    const int st = check_product(a, a_scale, w, w_scale, out, true);
    if (st != MOE_OK) return st;
    const int64_t mk = int64_t(M) * K, nk = int64_t(N) * K, kb = K / MOE_QUANT_GROUP;
    if (clash({{out, 2 * int64_t(M) * N}},
              {{a, mk}, {a_scale, 4 * kb * M}, {w, nk}, {w_scale, 4 * ((int64_t(N) + 127) / 128) * kb}}, 0))
        return MOE_ERR_INVALID_ARG;
    RowsGemmArgs g{};
    g.a = a;
    g.a_scale = a_scale;
    g.w = w;
    g.w_scale = w_scale;
    g.offsets = nullptr;
    g.out = static_cast<uint16_t*>(out);
    g.rows = M;
    g.E = 1;
    g.N = N;
    g.K = K;
    return hip_status(launch_rows_gemm(g, kRowsFp8, stream));
}

MOE_API int moe_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w, const float* w_scale, int32_t M,
                          int32_t N, int32_t K, void* out, hipStream_t stream) {
    if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (!fits_k(kRowsInt8, K) || M > kMaxRows || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    const int st = check_product(a, a_scale, w, w_scale, out, true);
    if (st != MOE_OK) return st;
    if (clash({{out, 2 * int64_t(M) * N}},
              {{a, int64_t(M) * K}, {a_scale, 4 * int64_t(M)}, {w, int64_t(N) * K}, {w_scale, 4 * int64_t(N)}}, 0))
        return MOE_ERR_INVALID_ARG;
    RowsGemmArgs g{};
    g.a = reinterpret_cast<const uint8_t*>(a);
    g.a_scale = a_scale;
    g.w = reinterpret_cast<const uint8_t*>(w);
    g.w_scale = w_scale;
    g.offsets = nullptr;
    g.out = static_cast<uint16_t*>(out);
    g.rows = M;
    g.E = 1;
    g.N = N;
    g.K = K;
    return hip_status(launch_rows_gemm(g, kRowsInt8, stream));
}

MOE_API int moe_grouped_gemm(const void* a, const float* a_scale, const void* w, const float* w_scale,
                             const int32_t* offsets, int32_t rows, int32_t E, int32_t N, int32_t K, int32_t wdtype,
                             void* out, hipStream_t stream) {
    if (rows < 0 || E < 1 || E > MOE_MAX_EXPERTS || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (wdtype == MOE_WDTYPE_MXFP8) return MOE_ERR_UNSUPPORTED;
    RowsKind kind;
    if (!rows_kind(wdtype, kind)) return MOE_ERR_INVALID_ARG;
    if (!fits_k(kind, K) || rows > kMaxRows || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    const int st = check_product(a, a_scale, w, w_scale, out, kind != kRowsBf16);
    if (st != MOE_OK) return st;
    if (!offsets || !aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
    const int64_t es = kind == kRowsBf16 ? 2 : 1;
    // scales of a row of a, and of an expert's weights
    const int64_t sa = kind == kRowsFp8 ? K / MOE_QUANT_GROUP : 1;
    const int64_t sw = kind == kRowsFp8 ? (int64_t(N) + 127) / 128 * (K / MOE_QUANT_GROUP) : N;
    if (clash({{out, 2 * int64_t(rows) * N}},
              {{a, es * rows * K}, {a_scale, 4 * sa * rows}, {w, es * E * N * K}, {w_scale, 4 * sw * E},
               {offsets, 4 * (int64_t(E) + 1)}}, 0))
        return MOE_ERR_INVALID_ARG;
    RowsGemmArgs g{};
    g.a = static_cast<const uint8_t*>(a);
    g.a_scale = a_scale;
    g.w = static_cast<const uint8_t*>(w);
    g.w_scale = w_scale;
    g.offsets = offsets;
    g.out = static_cast<uint16_t*>(out);
    g.rows = rows;
    g.E = E;
    g.N = N;
    g.K = K;
    return hip_status(launch_rows_gemm(g, kind, stream));
}

}  // extern "C"
