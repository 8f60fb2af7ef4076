// Rows sorted by expert back at their tokens, weighted, and the gradient:
//   out[t] = bf16(sum_j w[t, j] rows[inv[t, j]])               (fp32, in slot order)
//   grad_rows[inv[t, j]] = bf16(w[t, j] grad_out[t])
//   grad_weights[t, j] = sum_h grad_out[t, h] rows[inv[t, j], h]   (fp32)
// A slot whose inv lies outside [0, num_rows) has no row: it adds nothing, and
// its weight's gradient is 0.
//
// Every row is read once and every output written once, so both are bound by bytes:
// the combine of 8192 x 7168 and 8 slots 193 us, 5.5 TB/s (a large copy 5.1), 179 where the
// last output is in the last-level cache yet; the gradient of 4096 x 4096 and 8 slots 113
// us, 5.05 TB/s.  A thread has one piece of 16
// bytes of a token, which fills the CUs from a few tokens on, with the loads of eight
// slots in flight; gathering by token needs no atomics and sums in slot order.
#include "sorted.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;   // slots whose loads are in flight together

// wave-wide sum, the same bits in every lane
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return __fadd_rn(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xb1>(v);                                  // quad_perm [1,0,3,2]
    v = dpp_add<0x4e>(v);                                  // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);                                 // row_half_mirror
    v = dpp_add<0x140>(v);                                 // row_mirror
    const uint32_t b = __float_as_uint(v);
    const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    v = __fadd_rn(__uint_as_float(x[0]), __uint_as_float(x[1]));
    const uint32_t c = __float_as_uint(v);
    const auto y = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return __fadd_rn(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

struct Columns {
    uint32_t total;         // T * cols / 8 of this launch, below 2^31
    uint32_t per_row;       // cols / 8
    uint32_t magic, shift;  // i / per_row = i magic >> shift for i below 2^31
};

// A thread makes 8 columns of a token.  kUniform: a wave's 512 columns are one
// token's, whose positions and weights are then scalar loads.
template <bool kUniform, bool kWeights, bool kPast>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(CombineArgs a, Columns n) {
    const uint32_t mine = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
    if (mine >= n.total) return;
    uint32_t t = uint32_t(uint64_t(mine) * n.magic >> n.shift);
    const uint32_t h = (mine - t * n.per_row) * 8;
    if constexpr (kUniform) t = __builtin_amdgcn_readfirstlane(t);
    const int32_t* inv = a.inv + int64_t(t) * a.topk;
    const float* weights = a.weights + int64_t(t) * a.topk;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.topk; j0 += kSlots) {
        i32x4 v[kSlots];
        float w[kSlots];
        bool there[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            const int j = min(j0 + u, a.topk - 1);
            const int r = inv[j];
            there[u] = j0 + u < a.topk && uint32_t(r) < uint32_t(a.num_rows);
            w[u] = kWeights ? weights[j] : 1.0f;
            v[u] = i32x4{0, 0, 0, 0};
            if (there[u]) v[u] = load16<kPast>(a.rows + int64_t(r) * a.cols + h);
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            if (!there[u]) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (kWeights) {
                    acc[2 * q] = __builtin_fmaf(w[u], bf16_lo(v[u][q]), acc[2 * q]);
                    acc[2 * q + 1] = __builtin_fmaf(w[u], bf16_hi(v[u][q]), acc[2 * q + 1]);
                } else {
                    acc[2 * q] = __fadd_rn(acc[2 * q], bf16_lo(v[u][q]));
                    acc[2 * q + 1] = __fadd_rn(acc[2 * q + 1], bf16_hi(v[u][q]));
                }
            }
        }
    }
    i32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = int(pack_bf16(acc[2 * q], acc[2 * q + 1]));
    *reinterpret_cast<i32x4*>(a.out + int64_t(t) * a.cols + h) = o;
}

// A token by W waves, which go over its columns in turn; a lane's part of every
// slot's dot product stays in registers until the end.
template <int W, bool kDots, bool kWeights, bool kPast>
__global__ __launch_bounds__(W <= 4 ? 256 : 64 * W) void combine_rows_bwd_kernel(CombineArgs a) {
    constexpr int NT = W <= 4 ? 256 : 64 * W, kTokens = NT / 64 / W;
    __shared__ float s_dot[NT / 64][kSlots];
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t mine = wg * kTokens + threadIdx.x / (64 * W);
    if (W == 1 && mine >= a.T) return;
    const int t = __builtin_amdgcn_readfirstlane(int(min(mine, int64_t(a.T) - 1)));
    const int tid = threadIdx.x % (64 * W), nvec = a.cols >> 3;
    const int32_t* inv = a.inv + int64_t(t) * a.topk;
    const uint16_t* grad = a.grad_out + int64_t(t) * a.cols;
    for (int j0 = 0; j0 < a.topk; j0 += kSlots) {
        int r[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            const int j = min(j0 + u, a.topk - 1);
            r[u] = j0 + u < a.topk && mine < a.T ? inv[j] : -1;
            w[u] = kWeights ? a.weights[int64_t(t) * a.topk + j] : 1.0f;
            if (uint32_t(r[u]) >= uint32_t(a.num_rows)) r[u] = -1;
            r[u] = __builtin_amdgcn_readfirstlane(r[u]);
            dot[u] = 0.0f;
        }
        for (int i = tid; i < nvec; i += 64 * W) {
            const i32x4 g = load16<kPast>(grad + i * 8);
            i32x4 v[kSlots];
            if constexpr (kDots) {
#pragma unroll
                for (int u = 0; u < kSlots; ++u)
                    if (r[u] >= 0) v[u] = load16<kPast>(a.rows + int64_t(r[u]) * a.cols + i * 8);
            }
#pragma unroll
            for (int u = 0; u < kSlots; ++u) {
                if (r[u] < 0) continue;
                i32x4 o = g;
                if constexpr (kWeights) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = int(pack_bf16(__fmul_rn(w[u], bf16_lo(g[q])), __fmul_rn(w[u], bf16_hi(g[q]))));
                }
                store16<kPast>(a.grad_rows + int64_t(r[u]) * a.cols + i * 8, o);
                if constexpr (kDots) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        dot[u] = __builtin_fmaf(bf16_lo(g[q]), bf16_lo(v[u][q]), dot[u]);
                        dot[u] = __builtin_fmaf(bf16_hi(g[q]), bf16_hi(v[u][q]), dot[u]);
                    }
                }
            }
        }
        if constexpr (kDots) {
            float sum = 0.0f;                              // lane u keeps slot j0 + u's
#pragma unroll
            for (int u = 0; u < kSlots; ++u) {
                const float whole = wave_sum(dot[u]);
                if ((threadIdx.x & 63) == u) sum = whole;
            }
            if constexpr (W > 1) {
                __syncthreads();                           // the group before has been read
                if ((threadIdx.x & 63) < kSlots) s_dot[threadIdx.x >> 6][threadIdx.x & 63] = sum;
                __syncthreads();
                if (tid < kSlots) {
                    const int first = threadIdx.x / (64 * W) * W;
                    sum = s_dot[first][tid];
#pragma unroll
                    for (int i = 1; i < W; ++i) sum = __fadd_rn(sum, s_dot[first + i][tid]);
                }
            }
            if (tid < kSlots && j0 + tid < a.topk && mine < a.T)
                a.grad_weights[int64_t(t) * a.topk + j0 + tid] = sum;
        }
    }
}

template <int W, bool kDots, bool kWeights>
hipError_t launch_bwd(const CombineArgs& a, hipStream_t s) {
    constexpr int NT = W <= 4 ? 256 : 64 * W, kTokens = NT / 64 / W;
    const int64_t n = (int64_t(a.T) + kTokens - 1) / kTokens;
    void (*kern)(CombineArgs) = a.past ? combine_rows_bwd_kernel<W, kDots, kWeights, true>
                                       : combine_rows_bwd_kernel<W, kDots, kWeights, false>;
    return start(kern, grid_of(n), NT, s, a);
}

// Columns up to which a wave takes a token (us, one wave / four: 2048 tokens of 256
// and 8 slots 5.7 / 9.1, of 512 7.1 / 10.0, of 1024 14.3 / 14.3, of 4096 48 / 47), and
// tokens up to which sixteen waves do (four / sixteen: 64 x 7168 7.7 / 7.1, 200 x 7168
// 10.7 / 9.6, 400 x 7168 17.6 / 18.7, 600 x 4096 15.3 / 19.1).
constexpr int kWaveCols = 512, kFewTokens = 256;

template <bool kDots, bool kWeights>
hipError_t launch_bwd(const CombineArgs& a, hipStream_t s) {
    if (a.cols <= kWaveCols) return launch_bwd<1, kDots, kWeights>(a, s);
    if (a.T <= kFewTokens && a.cols > 2048) return launch_bwd<16, kDots, kWeights>(a, s);
    return launch_bwd<4, kDots, kWeights>(a, s);
}

// Whether there are more rows than stay in the last-level cache (us as they are / past
// it: the combine of 224 MiB 39.4 / 46.5, 448 MiB 104 / 93, 896 MiB 206 / 178 (an
// output whose last lines are in the cache yet; 206 / 193 otherwise); its
// gradient, rows read and written, of 224 MiB 105 / 102, 256 MiB 118 / 113, 896 MiB 405 /
// 395.  The combine's output is left to the caches: 179 / 183)
bool streamed(const CombineArgs& a) {
    return std::min<int64_t>(int64_t(a.T) * a.topk, a.num_rows) * a.cols * 2 >= kLastCacheBytes;
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& all, hipStream_t s) {
    CombineArgs a = all;
    Columns n{};
    n.per_row = uint32_t(a.cols) >> 3;
    // as in act.hip: i magic >> shift is i / per_row for i below 2^31
    n.shift = 31;
    while (uint64_t(1) << (n.shift - 31) < n.per_row) ++n.shift;
    n.magic = uint32_t((uint64_t(1) << n.shift) / n.per_row + 1);
    const int most = int(std::min<int64_t>(a.T, INT32_MAX / int64_t(n.per_row)));
    const bool uniform = n.per_row % 64 == 0;
    a.past = streamed(a) && reads_past(a.rows, int64_t(a.cols) * 2);
    void (*const kern)(CombineArgs, Columns) =
        pick(uniform, [&](auto u) {
            return pick(a.weights != nullptr, [&](auto w) {
                return pick(a.past, [&](auto p) -> void (*)(CombineArgs, Columns) {
                    return combine_rows_kernel<u.value, w.value, p.value>;
                });
            });
        });
    for (int t0 = 0; t0 < all.T; t0 += std::min(most, all.T - t0)) {
        a.inv = all.inv + int64_t(t0) * a.topk;
        a.weights = all.weights ? all.weights + int64_t(t0) * a.topk : nullptr;
        a.out = all.out + int64_t(t0) * a.cols;
        n.total = uint32_t(std::min(most, all.T - t0)) * n.per_row;
        const hipError_t e = start(kern, dim3((n.total + kThreads - 1) / kThreads), kThreads, s, a, n);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_combine_rows_bwd(const CombineArgs& all, hipStream_t s) {
    CombineArgs a = all;
    a.past = streamed(a) && whole_lines(a.grad_rows, int64_t(a.cols) * 2);
    if (a.grad_weights) return a.weights ? launch_bwd<true, true>(a, s) : launch_bwd<true, false>(a, s);
    return a.weights ? launch_bwd<false, true>(a, s) : launch_bwd<false, false>(a, s);
}

}  // namespace moe
