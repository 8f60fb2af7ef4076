// int8 quantisation of bf16 rows with one scale each, as they are or behind the
// SiLU-gated multiply of a product's gate and up halves:
//   m = max(|v|max, 1e-10), scale = fl32(m / 127), code = RNE(v fl32(127 / m)),
//   gated: v = bf16(bf16(silu(g)) * u) after the optional clamp (dev_silu.h).
//
// A row is held in the registers of L lanes, CH chunks of 8 columns each, so it is
// read once; the maximum of the row's bf16 bits is joined through lane permutations
// and, where several waves have a row, LDS.  Rows of up to 32 chunks share a wave (24265
// x 80 gated 4.6 us, a wave to a row 11.6).  Many rows are bound by their bytes
// (32771 x 1536 gated 46-47 us, 5.4 TB/s), few by the launch (3.6-4 us).
#include "moe.h"

#include "dev_silu.h"
#include "sorted.h"

namespace moe {

namespace {

// threads of a workgroup whose rows are L lanes' each
template <int L>
constexpr int kThreads = L <= 256 ? 256 : L;

template <int L, int CH, bool kGated, bool kClamp, bool kPast>
__global__ __launch_bounds__(kThreads<L>) void quant_int8_kernel(Int8Args a) {
    constexpr int NT = kThreads<L>;
    __shared__ uint32_t s_max[NT / 64];
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t mine = wg * (NT / L) + threadIdx.x / L;
    if (L == 64 && mine >= a.rows) return;
    const int64_t row = min(mine, int64_t(a.rows) - 1);
    const int tid = threadIdx.x % L, nvec = a.cols >> 3;
    const uint16_t* x = a.x + row * a.cols * (kGated ? 2 : 1);
    i32x4 v[CH], u[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = min(tid + c * L, nvec - 1);     // behind the row: its last chunk again
        v[c] = load16<kPast>(x + i * 8);
        if constexpr (kGated) u[c] = load16<kPast>(x + a.cols + i * 8);
    }
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (kGated) v[c] = silu_mul8<kClamp>(v[c], u[c], a.limit);
        most = pk_max_u16(most, abs_max8(v[c]));
    }
    uint32_t bits = lanes_max_u16<(L < 64 ? L : 64)>(most);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = bits;
        __syncthreads();
        const int first = threadIdx.x / L * (L / 64);
#pragma unroll
        for (int i = 0; i < L / 64; ++i) bits = max(bits, s_max[first + i]);
    }
    float inverse;
    const float scale = int8_scale(bits, inverse);
    if (mine >= a.rows) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = tid + c * L;
        if (i < nvec) *reinterpret_cast<uint2*>(a.codes + row * a.cols + i * 8) = int8_codes(v[c], inverse);
    }
    if (tid == 0) a.scales[row] = scale;
}

// Rows from which a wave takes a whole row, up to kWaveVecs chunks of 8 columns; below
// it four waves do, which need less time for a row.  us, one wave / four, outputs that
// stay in the caches: gated, 128 rows of 4096 5.0 / 3.7, 512 of 2560 4.4 / 3.9, 1536 of
// 2048 5.2 / 4.8, 2048 of 2560 6.9 / 8.4, 16384 of 1536 22.9 / 28.4, of 2560 39.3 / 47.1,
// of 4096, gate and up half in 64 registers each, 64.6 / 60.9; not gated, 16384 of 1536
// 12.0 / 12.6, of 4096 29.4 / 28.6, 4096 of 4096 8.0 / 9.1.
constexpr int kManyRows = 2048;
template <bool kGated>
constexpr int kWaveVecs = kGated ? 384 : 512;

template <bool kGated, bool kClamp>
hipError_t launch(const Int8Args& a, hipStream_t s) {
    auto go = [&](auto lanes, auto ch) {
        constexpr int L = decltype(lanes)::value, CH = decltype(ch)::value, kRows = kThreads<L> / L;
        const int64_t n = (int64_t(a.rows) + kRows - 1) / kRows;
        void (*kern)(Int8Args) = a.past ? quant_int8_kernel<L, CH, kGated, kClamp, true>
                                        : quant_int8_kernel<L, CH, kGated, kClamp, false>;
        return start(kern, grid_of(n), kThreads<L>, s, a);
    };
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    const integral_constant<int, 64> wave;
    const integral_constant<int, 256> waves4;
    const integral_constant<int, 1024> waves16;
    const int nvec = a.cols >> 3;
    if (nvec <= 8) return go(integral_constant<int, 8>(), one);
    if (nvec <= 16) return go(integral_constant<int, 16>(), one);
    if (nvec <= 32) return go(integral_constant<int, 32>(), one);
    if (nvec <= 64) return go(wave, one);
    if (a.rows >= kManyRows && nvec <= kWaveVecs<kGated>) {
        if (nvec <= 128) return go(wave, two);
        if (nvec <= 192) return go(wave, integral_constant<int, 3>());
        if (nvec <= 256) return go(wave, four);
        if (nvec <= 384) return go(wave, integral_constant<int, 6>());
        if constexpr (!kGated) return go(wave, integral_constant<int, 8>());
    }
    if (nvec <= 256) return go(waves4, one);
    if (nvec <= 512) return go(waves4, two);
    if (nvec <= 1024) return go(waves4, four);
    if (nvec <= 2048) return go(waves16, two);
    static_assert(MOE_MAX_INT8_K <= 1024 * 4 * 8, "a row in one workgroup's registers");
    return go(waves16, four);
}

}  // namespace

hipError_t launch_quant_int8(const Int8Args& all, bool gated, hipStream_t s) {
    // three quarters of the cache, whose rest the codes take (us as they are / past, gated,
    // and with a kernel that writes x in front: 96 MiB 22.7 / 23.4 (51 / 52), 192 MiB 39.8 /
    // 41.9 (118 / 112), 256 MiB 62.7 / 55.1 (171 / 150), 384 MiB 96 / 81 (250 / 232))
    Int8Args a = all;
    const int64_t row_bytes = int64_t(a.cols) * (gated ? 4 : 2);
    a.past = a.rows * row_bytes >= kLastCacheBytes / 4 * 3 && reads_past(a.x, row_bytes);
    if (!gated) return launch<false, false>(a, s);
    return a.limit > 0.0f ? launch<true, true>(a, s) : launch<true, false>(a, s);
}

}  // namespace moe
