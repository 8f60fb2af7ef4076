// SiLU-gated multiply of a product's gate and up halves (+ fp8 quantisation):
// the fused kernel of P2 section 1.2 as an operator of its own, with the
// rounding points of the fused epilogue,
//   a = bf16(bf16(silu(g)) * u),  silu(g) = g / (1 + exp(-g)),
// the optional clamp of the bf16 gate and up values before it, and codes and
// scales by moe_quant_act's rule.
//
// g is a bf16 value, so bf16(silu(g)) is a function of 16 bits; silu_f32
// (dev_silu.h) gives its correct rounding for every finite g (a test compares all of them
// with 64-bit arithmetic), so the outputs are the definition's bit for bit.
//
// A thread makes 8 columns from 16 bytes of gate and 16 of up; a 128-column
// quantisation group is 16 neighbouring lanes.  HBM-bound (4 bytes read per
// output, 1 + 4/128 or 2 written) as long as the vector unit keeps up: with 254
// vector instructions for 8 outputs 20011 x 2048 to fp8 takes 38.4 us, 5.4 TB/s
// (a 1 GiB copy 5.15 TB/s); with 390, a 64-bit division for the row among them,
// it took 44.3.  Two or four vectors a thread, or loads and stores past the
// caches' replacement, were no faster.  16 x 2048 2.6 us, of which an empty
// kernel takes 2.2.
#include "moe.h"

#include <algorithm>

#include "dev_silu.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct ActArgs {
    const uint16_t* h;      // [rows, 2 cols]
    uint16_t* y;            // [rows, cols] or null
    uint8_t* codes;
    void* scales;
    uint32_t total;         // rows * cols / 8, below 2^31
    uint32_t per_row;       // cols / 8
    uint32_t magic, shift;  // i / per_row = i magic >> shift for i below 2^31
    float limit;
};

template <int kQuant, bool kClamp>
__global__ __launch_bounds__(kThreads) void silu_mul_kernel(ActArgs a) {
    const uint32_t mine = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
    const bool live = mine < a.total;                // a quantisation group is live as a whole
    const uint32_t i = min(mine, a.total - 1);
    const uint32_t row = uint32_t(uint64_t(i) * a.magic >> a.shift);
    const uint64_t at = uint64_t(i) * 8;             // first output column, over all rows
    const uint16_t* src = a.h + (uint64_t(row) * a.per_row + i) * 8;
    const uint32_t cols = a.per_row * 8;
    const i32x4 gw = *reinterpret_cast<const i32x4*>(src);
    const i32x4 uw = *reinterpret_cast<const i32x4*>(src + cols);
    const i32x4 o = silu_mul8<kClamp>(gw, uw, a.limit);
    if (live && a.y) *reinterpret_cast<i32x4*>(a.y + at) = o;
    if constexpr (kQuant != 0) {
        constexpr int kLanes = kQuant == 1 ? 16 : 4;
        uint32_t lo, hi;
        const float s = quant8<kLanes>(o, lo, hi);
        if (live) {
            *reinterpret_cast<uint2*>(a.codes + at) = uint2{lo, hi};
            if ((threadIdx.x & (kLanes - 1)) == 0) {
                const uint32_t group = i / kLanes;
                if constexpr (kQuant == 1) static_cast<float*>(a.scales)[group] = s;
                else static_cast<uint8_t*>(a.scales)[group] = uint8_t(__float_as_uint(s) >> 23);
            }
        }
    }
}

template <bool kClamp>
hipError_t launch(const ActArgs& a, int quant, hipStream_t s) {
    void (*kern)(ActArgs) = quant == 0   ? silu_mul_kernel<0, kClamp>
                            : quant == 1 ? silu_mul_kernel<1, kClamp> : silu_mul_kernel<2, kClamp>;
    return start(kern, dim3((a.total + kThreads - 1) / kThreads), kThreads, s, a);
}

}  // namespace

hipError_t launch_silu_mul(const uint16_t* h, int rows, int cols, float clamp_limit, int quant, uint16_t* y,
                           uint8_t* codes, void* scales, hipStream_t s) {
    ActArgs a{};
    a.per_row = uint32_t(cols) >> 3;
    a.limit = clamp_limit;
    // magic = floor(2^shift / d) + 1 with shift = 31 + ceil(log2 d): i magic / 2^shift
    // exceeds i / d by less than 1 / d for i < 2^31, so its whole part is that of i / d
    a.shift = 31;
    while (uint64_t(1) << (a.shift - 31) < a.per_row) ++a.shift;
    a.magic = uint32_t((uint64_t(1) << a.shift) / a.per_row + 1);
    // at most 2^31 - 1 threads' indices in a launch
    const int most = int(std::min<int64_t>(rows, INT32_MAX / int64_t(a.per_row)));
    for (int r0 = 0; r0 < rows; r0 += std::min(most, rows - r0)) {
        const int64_t at = int64_t(r0) * cols;
        a.h = h + 2 * at;
        a.y = y ? y + at : nullptr;
        a.codes = codes ? codes + at : nullptr;
        const int64_t unit = quant == 1 ? at / MOE_QUANT_GROUP * 4 : at / MOE_MX_BLOCK;
        a.scales = scales ? static_cast<uint8_t*>(scales) + unit : nullptr;
        a.total = uint32_t(std::min(most, rows - r0)) * a.per_row;
        const hipError_t e = clamp_limit > 0.0f ? launch<true>(a, quant, s) : launch<false>(a, quant, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
