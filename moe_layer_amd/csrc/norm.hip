// Residual add + RMSNorm (+ fp8 quantisation) of bf16 rows:
//   s = fl32(x + r);  r' = bf16(s);  y = bf16(s * w / sqrt(mean(s^2) + eps));
//   codes and scales of y by moe_quant_act's rule.
//
// The mean of squares and the two products behind y are computed in fp64 and
// rounded to fp32 and then bf16 once, so y (and with it the codes and scales,
// whose scale doubles at a border of the group's maximum) does not depend on
// the order of the sum: the result is the same for every launch shape.
//
// One workgroup per row, the row held in registers between the two passes, so
// it is read once and every load of a row precedes its first store (the
// outputs may replace the inputs).  A thread holds CH chunks of 8 columns
// (16 bytes); a 128-column quantisation group is 16 neighbouring lanes.
// HBM-bound: 2 bytes read (4 with a residual), 2 written for each of r' and y,
// 1 + 4/128 for the codes and scales.  8192 x 7168 with all of them 94.5 us,
// 5.6 TB/s (a 1 GiB copy 5.15 TB/s), 1537 x 4096 to MXFP8 6.8 us; 1 x 7168
// 2.7 us, of which an empty kernel takes 2.2.  Rows of more than 16384 columns
// (1024 threads of four chunks, 128 registers each) keep 100-108 bytes a lane of
// theirs in scratch: 4096 x 32768 303 us, 4.0 TB/s, 1024 x 20480 73 us, 2.6 TB/s.
#include "moe.h"

#include "dense.h"

namespace moe {

namespace {

// A wave's sum, the same bits in every lane: lane permutations inside the
// vector unit (through LDS, as shuffles go, a sum's six steps wait for it)
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, 0xf, 0xf, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b >> 32)), CTRL, 0xf, 0xf, false));
    return v + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_add<0xb1>(v);                                  // quad_perm [1,0,3,2]
    v = dpp_add<0x4e>(v);                                  // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);                                 // row_half_mirror
    v = dpp_add<0x140>(v);                                 // row_mirror
    auto half = [](double x, auto swap) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const auto lo = swap(uint32_t(b)), hi = swap(uint32_t(b >> 32));
        return __builtin_bit_cast(double, uint64_t(hi[0]) << 32 | lo[0]) +
               __builtin_bit_cast(double, uint64_t(hi[1]) << 32 | lo[1]);
    };
    v = half(v, [](uint32_t w) { return __builtin_amdgcn_permlane16_swap(w, w, false, false); });
    return half(v, [](uint32_t w) { return __builtin_amdgcn_permlane32_swap(w, w, false, false); });
}

// 1 / sqrt(x) to about 2^-51: the hardware's estimate (good to 2^-14 or better)
// and three Newton steps, each doubling its bits
__device__ __forceinline__ double rsqrt64(double x) {
    double y = __builtin_amdgcn_rsq(x);
#pragma unroll
    for (int i = 0; i < 3; ++i) y = __fma_rn(y * 0.5, __fma_rn(-x * y, y, 1.0), y);
    return y;
}

template <int NT, int CH, int kQuant>
__global__ __launch_bounds__(NT) void norm_kernel(NormArgs a) {
    __shared__ double s_part[NT / 64];
    const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    if (row >= a.rows) return;
    const int nvec = a.cols >> 3;
    const uint16_t* x = a.x + row * a.cols;
    const uint16_t* r = a.residual ? a.residual + row * a.cols : nullptr;

    float v[CH][8];
    i32x4 w[CH];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = threadIdx.x + c * NT;
        // without a residual r = -0, which leaves every x as it is
        constexpr int kNegZero = int(0x80008000u);
        i32x4 xv = {0, 0, 0, 0}, rv = {kNegZero, kNegZero, kNegZero, kNegZero};
        w[c] = i32x4{0, 0, 0, 0};
        if (i < nvec) {
            xv = *reinterpret_cast<const i32x4*>(x + i * 8);
            if (r) rv = *reinterpret_cast<const i32x4*>(r + i * 8);
            w[c] = *reinterpret_cast<const i32x4*>(a.weight + i * 8);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[c][2 * q] = __fadd_rn(bf16_lo(xv[q]), bf16_lo(rv[q]));
            v[c][2 * q + 1] = __fadd_rn(bf16_hi(xv[q]), bf16_hi(rv[q]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) sum = __fma_rn(double(v[c][q]), double(v[c][q]), sum);
    }
    sum = wave_sum(sum);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) sum += s_part[i];
    }
    const double inv = rsqrt64(__fma_rn(sum, a.inv_cols, double(a.eps)));

#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = threadIdx.x + c * NT;
        const bool live = i < nvec;
        const int64_t at = row * a.cols + i * 8;
        if (live && a.residual_out) {
            i32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = int(pack_bf16(v[c][2 * q], v[c][2 * q + 1]));
            *reinterpret_cast<i32x4*>(a.residual_out + at) = o;
        }
        i32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float y0 = float(double(v[c][2 * q]) * inv * double(bf16_lo(w[c][q])));
            const float y1 = float(double(v[c][2 * q + 1]) * inv * double(bf16_hi(w[c][q])));
            o[q] = int(pack_bf16(y0, y1));
        }
        if (live && a.y) *reinterpret_cast<i32x4*>(a.y + at) = o;
        if constexpr (kQuant != 0) {
            uint32_t lo, hi;
            constexpr int kLanes = kQuant == 1 ? 16 : 4;
            const float s = quant8<kLanes>(o, lo, hi);   // cols % group == 0: a group is live as a whole
            if (live) {
                *reinterpret_cast<uint2*>(a.codes + at) = uint2{lo, hi};
                if ((threadIdx.x & (kLanes - 1)) == 0) {
                    const int64_t g = at / (8 * kLanes);
                    if constexpr (kQuant == 1) static_cast<float*>(a.scales)[g] = s;
                    else static_cast<uint8_t*>(a.scales)[g] = uint8_t(__float_as_uint(s) >> 23);
                }
            }
        }
    }
}

template <int NT, int CH>
hipError_t launch(const NormArgs& a, int quant, hipStream_t s) {
    void (*kern)(NormArgs) = quant == 0 ? norm_kernel<NT, CH, 0>
                             : quant == 1 ? norm_kernel<NT, CH, 1> : norm_kernel<NT, CH, 2>;
    return start(kern, grid_of(a.rows), NT, s, a);
}

}  // namespace

// Threads and chunks: few chunks a thread without idle waves.  us, 256 / 512
// threads: 1537 x 4096 7.05 / 7.47, 1024 x 7168 13.0 / 12.4, 8192 x 7168 95.6 /
// 94.7, 3000 x 5120 26.1 / 25.0; 128 or 1024 threads are slower throughout.
hipError_t launch_norm(const NormArgs& a, int quant, hipStream_t s) {
    const int nvec = a.cols >> 3;
    if (nvec <= 64) return launch<64, 1>(a, quant, s);
    if (nvec <= 256) return launch<256, 1>(a, quant, s);
    if (nvec <= 512) return launch<256, 2>(a, quant, s);
    if (nvec <= 1024) return launch<512, 2>(a, quant, s);
    if (nvec <= 2048) return launch<512, 4>(a, quant, s);
    static_assert(MOE_MAX_NORM_COLS <= 1024 * 4 * 8, "a row in one workgroup's registers");
    return launch<1024, 4>(a, quant, s);
}

}  // namespace moe
