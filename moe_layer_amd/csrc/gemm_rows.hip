// Dense and grouped products of rows with K-contiguous weights:
//   out[r, n] = bf16(sum_k a[r, k] w[e, n, k]),  offsets[e] <= r < offsets[e + 1]
// (dense: one group of all rows), for bf16 operands or e4m3 ones with an fp32
// scale per row and 128 K (a) and per 128 x 128 block (w).
//
// The weight rows are the MFMA M side and the token rows the N side, so a lane
// holds one token and four neighbouring outputs of it.  A workgroup owns 16
// weight rows and a block of 16 NT rows of one group; its waves take the
// 128-byte K steps in turn and their sums are added through LDS in wave order.
// Both operands go straight to registers: lane l takes bytes 16 (l / 16) and
// 64 + 16 (l / 16) of row l % 16's 128-byte step (any order of K inside a step
// is the same product, as both operands take it).
#include <algorithm>

#include "dense.h"

namespace moe {

namespace {

// The group and first row of row block `slot` when every group is cut into
// blocks of BM rows: groups in order, each with ceil(rows / BM) blocks.  Every
// lane of the wave returns the same; false when there are fewer blocks.
// Offsets are held to [0, rows] and the block to its group's rows, so a bad
// table reads and writes in bounds.
template <int BM>
__device__ __forceinline__ bool find_block(const RowsGemmArgs& g, int slot, int& e, int& row0, int& row1) {
    if (!g.offsets) {
        e = 0;
        row0 = slot * BM;
        row1 = g.rows;
        return row0 < g.rows;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;                                  // blocks of the groups below e0
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        const int i = e0 + lane;
        int lo = 0, hi = 0;
        if (i < g.E) {
            lo = min(max(g.offsets[i], 0), g.rows);
            hi = min(max(g.offsets[i + 1], lo), g.rows);
        }
        const int n = (hi - lo + BM - 1) / BM;
        int sum = n;                                 // blocks of groups e0 .. i
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int up = __shfl_up(sum, m);
            if (lane >= m) sum += up;
        }
        const int total = __shfl(sum, 63);
        if (slot < before + total) {
            const int at = slot - before;            // the first lane whose sum passes it
            const uint64_t past = __ballot(sum > at);
            const int src = max(__ffsll((unsigned long long)past) - 1, 0);
            const int first = __builtin_amdgcn_readfirstlane(__shfl(lo, src));
            e = __builtin_amdgcn_readfirstlane(e0 + src);
            row0 = __builtin_amdgcn_readfirstlane(first + (at - (__shfl(sum, src) - __shfl(n, src))) * BM);
            row1 = __builtin_amdgcn_readfirstlane(__shfl(hi, src));
            return row0 >= first && row0 < row1;
        }
        before += total;
    }
    return false;
}

// outputs n .. n+3 of row r
__device__ __forceinline__ void store4(const RowsGemmArgs& g, int64_t r, int n, const f32x4& v) {
    uint16_t* p = g.out + r * g.N + n;
    const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
    if ((g.N & 3) == 0) {                            // 8-byte aligned rows, and n + 3 < N with n
        if (n < g.N) *reinterpret_cast<uint2*>(p) = uint2{lo, hi};
        return;
    }
    if (n < g.N) p[0] = uint16_t(lo);
    if (n + 1 < g.N) p[1] = uint16_t(lo >> 16);
    if (n + 2 < g.N) p[2] = uint16_t(hi);
    if (n + 3 < g.N) p[3] = uint16_t(hi >> 16);
}

template <bool FP8>
__device__ __forceinline__ f32x4 mma_step(i32x4 a0, i32x4 a1, i32x4 b0, i32x4 b1, f32x4 c) {
    if constexpr (FP8) {
        const i32x8 av = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
        const i32x8 bv = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 0, 0, 0, 0, 0, 0);
    } else {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a0), __builtin_bit_cast(bf16x8, b0),
                                                    c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a1),
                                                       __builtin_bit_cast(bf16x8, b1), c, 0, 0, 0);
    }
}

template <bool FP8, int NT, int W>
__global__ __launch_bounds__(64 * W) void rows_stream_kernel(RowsGemmArgs g, int ntiles, int slots) {
    constexpr int BM = 16 * NT;
    __shared__ f32x4 s_part[W][NT][64];
    const int64_t item = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int slot = int(item / ntiles), tile = int(item - int64_t(slot) * ntiles);
    int e, row0, row1;
    if (slot >= slots || !find_block<BM>(g, slot, e, row0, row1)) return;   // the whole workgroup alike

    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t kbytes = int64_t(g.K) * (FP8 ? 1 : 2);
    const int steps = int(kbytes >> 7);
    const uint8_t* wp = g.w + (int64_t(e) * g.N + min(tile * 16 + lr, g.N - 1)) * kbytes + 16 * lk;
    const float* ws = FP8 ? g.w_scale + (int64_t(e) * ((g.N + 127) >> 7) + (tile >> 3)) * steps : nullptr;
    const uint8_t* ap[NT];
    const float* as[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t r = min(row0 + 16 * t + lr, row1 - 1);
        ap[t] = g.a + r * kbytes + 16 * lk;
        as[t] = FP8 ? g.a_scale + r * steps : nullptr;
    }
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    for (int s = wv; s < steps; s += W) {
        const int64_t o = int64_t(s) << 7;
        const i32x4 w0 = *reinterpret_cast<const i32x4*>(wp + o), w1 = *reinterpret_cast<const i32x4*>(wp + o + 64);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const i32x4 a0 = *reinterpret_cast<const i32x4*>(ap[t] + o);
            const i32x4 a1 = *reinterpret_cast<const i32x4*>(ap[t] + o + 64);
            if constexpr (FP8) {
                const f32x4 p = mma_step<true>(w0, w1, a0, a1, f32x4{0, 0, 0, 0});
                const float sc = __fmul_rn(as[t][s], ws[s]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(sc, p[i], acc[t][i]);
            } else {
                acc[t] = mma_step<false>(w0, w1, a0, a1, acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) s_part[wv][t][lane] = acc[t];
    __syncthreads();
    for (int t = wv; t < NT; t += W) {
        f32x4 v = s_part[0][t][lane];
#pragma unroll
        for (int i = 1; i < W; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = __fadd_rn(v[q], s_part[i][t][lane][q]);
        const int64_t r = int64_t(row0) + 16 * t + lr;
        if (r < row1) store4(g, r, tile * 16 + 4 * lk, v);
    }
}

// Row blocks of BM rows there can be: every group with rows ends in at most
// one part block.
int64_t block_slots(const RowsGemmArgs& g, int bm) {
    if (!g.offsets) return (int64_t(g.rows) + bm - 1) / bm;
    const int64_t most = int64_t(g.rows) / bm + std::min(g.E, g.rows);
    return std::min<int64_t>(most, g.rows);
}

template <bool FP8, int NT, int W>
hipError_t launch_stream(const RowsGemmArgs& g, hipStream_t s) {
    const int ntiles = (g.N + 15) / 16;
    const int64_t slots = block_slots(g, 16 * NT);
    void (*kern)(RowsGemmArgs, int, int) = rows_stream_kernel<FP8, NT, W>;
    hipLaunchKernelGGL(kern, grid_of(slots * ntiles), dim3(64 * W), 0, s, g, ntiles, int(slots));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_gemm(const RowsGemmArgs& g, bool fp8, hipStream_t s) {
    return fp8 ? launch_stream<true, 4, 8>(g, s) : launch_stream<false, 4, 8>(g, s);
}

}  // namespace moe
