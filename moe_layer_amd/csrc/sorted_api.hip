// C ABI of the operators that sort a batch by expert and bring it back, and
// that quantise rows to int8: argument checks and launches of moe_sort_rows,
// moe_combine_rows, moe_combine_rows_bwd, moe_quant_act_int8 and
// moe_silu_mul_int8 (documented in include/moe.h).
#include "moe.h"

#include "api_checks.h"
#include "sorted.h"

using namespace moe;

namespace {

bool known(int32_t type) {
    return type == MOE_WDTYPE_BF16 || type == MOE_WDTYPE_FP8_E4M3 || type == MOE_WDTYPE_INT8;
}
// columns that a row of this type is a multiple of
int whole_cols(int32_t type) { return type == MOE_WDTYPE_BF16 ? 8 : type == MOE_WDTYPE_INT8 ? 16 : MOE_QUANT_GROUP; }
int64_t row_bytes(int32_t type, int32_t cols) { return type == MOE_WDTYPE_BF16 ? 2 * int64_t(cols) : cols; }
int row_scales_of(int32_t type, int32_t cols) {
    return type == MOE_WDTYPE_BF16 ? 0 : type == MOE_WDTYPE_INT8 ? 1 : cols / MOE_QUANT_GROUP;
}
bool bad_routing(int32_t T, int32_t topk) { return T < 0 || topk < 1 || topk > MOE_MAX_TOPK; }

int check_int8_rows(const void* x, int32_t rows, int32_t cols, int64_t x_cols, const int8_t* codes,
                    const float* scales) {
    if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t r = rows;
    return clash({{codes, r * cols}, {scales, 4 * r}}, {{x, 2 * r * x_cols}}, 0) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int quant_int8(const void* x, int32_t rows, int32_t cols, bool gated, float limit, int8_t* codes, float* scales,
               hipStream_t stream) {
    if (cols % 16 != 0 || cols > MOE_MAX_INT8_K) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    const int st = check_int8_rows(x, rows, cols, gated ? 2 * int64_t(cols) : cols, codes, scales);
    if (st != MOE_OK) return st;
    return hip_status(launch_quant_int8({static_cast<const uint16_t*>(x), codes, scales, rows, cols, limit}, gated,
                                        stream));
}

// sizes that both directions of the combine share
int check_combine(int32_t T, int32_t topk, int32_t cols, int32_t num_rows) {
    if (bad_routing(T, topk) || cols <= 0 || num_rows < 0) return MOE_ERR_INVALID_ARG;
    if (cols % 8 != 0 || cols > kMaxCols || int64_t(T) * topk > kMaxRows || num_rows > kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

MOE_API int moe_quant_act_int8(const void* x, int32_t rows, int32_t cols, int8_t* codes, float* scales,
                               hipStream_t stream) {
    if (rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    return quant_int8(x, rows, cols, false, 0.0f, codes, scales, stream);
}

MOE_API int moe_silu_mul_int8(const void* h, int32_t rows, int32_t cols, float clamp_limit, int8_t* codes,
                              float* scales, hipStream_t stream) {
    if (rows < 0 || cols <= 0 || !(clamp_limit >= 0.0f)) return MOE_ERR_INVALID_ARG;
    return quant_int8(h, rows, cols, true, clamp_limit, codes, scales, stream);
}

MOE_API int64_t moe_sort_scratch_bytes(int32_t T, int32_t topk, int32_t E) {
    if (bad_routing(T, topk) || E < 1 || E > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_ARG;
    const int64_t R = int64_t(T) * topk;
    if (R > kMaxRows) return MOE_ERR_UNSUPPORTED;
    return int64_t(plan_sort(R).blocks) * E * 4;
}

MOE_API int moe_sort_rows(const void* x, const float* x_scale, const int32_t* topk_ids, int32_t T, int32_t topk,
                          int32_t E, int32_t cols, int32_t xtype, int32_t rowtype, void* rows, float* row_scales,
                          int32_t* offsets, int32_t* inv, void* scratch, int64_t scratch_bytes, hipStream_t stream) {
    if (bad_routing(T, topk) || E < 1 || E > MOE_MAX_EXPERTS || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (xtype == MOE_WDTYPE_MXFP8 || rowtype == MOE_WDTYPE_MXFP8) return MOE_ERR_UNSUPPORTED;
    if (!known(xtype) || !known(rowtype) || (xtype != rowtype && xtype != MOE_WDTYPE_BF16)) return MOE_ERR_INVALID_ARG;
    const bool to_int8 = xtype != rowtype && rowtype == MOE_WDTYPE_INT8;
    const int64_t R = int64_t(T) * topk;
    if (cols % whole_cols(xtype) != 0 || cols % whole_cols(rowtype) != 0 || cols > kMaxCols ||
        (to_int8 && cols > MOE_MAX_INT8_K) || R > kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    if (!offsets || !aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
    const int xs = row_scales_of(xtype, cols), rs = row_scales_of(rowtype, cols);
    const int64_t xb = row_bytes(xtype, cols), rb = row_bytes(rowtype, cols);
    const int64_t need = moe_sort_scratch_bytes(T, topk, E);
    if (T > 0) {
        if (!x || !topk_ids || !rows || !inv || !aligned(x, 16) || !aligned(topk_ids, 4) || !aligned(rows, 16) ||
            !aligned(inv, 4) || (xs > 0) != (x_scale != nullptr) || (rs > 0) != (row_scales != nullptr) ||
            !aligned(x_scale, 4) || !aligned(row_scales, 4))
            return MOE_ERR_INVALID_ARG;
        if (need > 0 && (!scratch || !aligned(scratch, 4) || scratch_bytes < need)) return MOE_ERR_WORKSPACE;
        if (clash({{rows, R * rb}, {row_scales, 4 * R * rs}, {offsets, 4 * (int64_t(E) + 1)}, {inv, 4 * R},
                   {need > 0 ? scratch : nullptr, need}},
                  {{x, T * xb}, {x_scale, 4 * int64_t(T) * xs}, {topk_ids, 4 * R}}, 0))
            return MOE_ERR_INVALID_ARG;
    }
    SortArgs a{};
    a.x = static_cast<const uint8_t*>(x);
    a.x_scale = x_scale;
    a.ids = topk_ids;
    a.rows = static_cast<uint8_t*>(rows);
    a.row_scales = row_scales;
    a.offsets = offsets;
    a.inv = inv;
    a.counts = static_cast<int32_t*>(scratch);
    a.T = T;
    a.topk = topk;
    a.E = E;
    a.R = int(R);
    a.units = int(rb / 16);
    a.scales = rs;
    const SortMode mode = xtype == rowtype ? kSortCopy : to_int8 ? kSortInt8 : kSortFp8;
    return hip_status(launch_sort_rows(a, mode, stream));
}

MOE_API int moe_combine_rows(const void* rows, const int32_t* inv, const float* weights, int32_t T, int32_t topk,
                             int32_t cols, int32_t num_rows, void* out, hipStream_t stream) {
    const int st = check_combine(T, topk, cols, num_rows);
    if (st != MOE_OK || T == 0) return st;
    if ((!rows && num_rows > 0) || !inv || !out || !aligned(rows, 16) || !aligned(inv, 4) || !aligned(weights, 4) ||
        !aligned(out, 16))
        return MOE_ERR_INVALID_ARG;
    const int64_t R = int64_t(T) * topk;
    if (clash({{out, 2 * int64_t(T) * cols}}, {{rows, 2 * int64_t(num_rows) * cols}, {inv, 4 * R}, {weights, 4 * R}}, 0))
        return MOE_ERR_INVALID_ARG;
    CombineArgs a{};
    a.rows = static_cast<const uint16_t*>(rows);
    a.inv = inv;
    a.weights = weights;
    a.out = static_cast<uint16_t*>(out);
    a.T = T;
    a.topk = topk;
    a.cols = cols;
    a.num_rows = num_rows;
    return hip_status(launch_combine_rows(a, stream));
}

MOE_API int moe_combine_rows_bwd(const void* grad_out, const void* rows, const int32_t* inv, const float* weights,
                                 int32_t T, int32_t topk, int32_t cols, int32_t num_rows, void* grad_rows,
                                 float* grad_weights, hipStream_t stream) {
    const int st = check_combine(T, topk, cols, num_rows);
    if (st != MOE_OK || T == 0) return st;
    const bool dots = grad_weights != nullptr;
    if (!grad_out || !inv || (num_rows > 0 && (!grad_rows || (dots && !rows))) || !aligned(grad_out, 16) ||
        !aligned(rows, 16) || !aligned(inv, 4) || !aligned(weights, 4) || !aligned(grad_rows, 16) ||
        !aligned(grad_weights, 4) || (rows && !dots))
        return MOE_ERR_INVALID_ARG;
    const int64_t R = int64_t(T) * topk, rb = 2 * int64_t(num_rows) * cols;
    if (clash({{grad_rows, rb}, {grad_weights, 4 * R}},
              {{grad_out, 2 * int64_t(T) * cols}, {rows, rb}, {inv, 4 * R}, {weights, 4 * R}}, 0))
        return MOE_ERR_INVALID_ARG;
    CombineArgs a{};
    a.rows = static_cast<const uint16_t*>(rows);
    a.inv = inv;
    a.weights = weights;
    a.grad_out = static_cast<const uint16_t*>(grad_out);
    a.grad_rows = static_cast<uint16_t*>(grad_rows);
    a.grad_weights = grad_weights;
    a.T = T;
    a.topk = topk;
    a.cols = cols;
    a.num_rows = num_rows;
    return hip_status(launch_combine_rows_bwd(a, stream));
}

}  // extern "C"
