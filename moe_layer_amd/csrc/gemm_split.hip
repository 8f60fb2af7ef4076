// Dense and grouped products of few rows, or of few tiles:
//   out[r, n] = bf16(sum_k a[r, k] w[e, n, k]),  offsets[e] <= r < offsets[e + 1]
// (dense: one group of all rows), for bf16 operands or e4m3 ones with an fp32
// scale per row and 128 K (a) and per 128 x 128 block (w).  gemm_tile.hip has
// the form for many tiles.
//
// The weight rows are the MFMA M side and the token rows the N side, so a lane
// holds one token and four neighbouring outputs of it.  A workgroup owns BW
// weight rows and a block of BT rows of one group; its waves take the 128-byte
// K steps in turn, each with the whole tile and a ring of its own, so no wave
// waits for another before their sums are added through LDS in wave order.
//
// Both operands move global -> LDS with direct-to-LDS loads of 8 whole
// 128-byte row pieces: the same bytes fetched in the shape of the MFMA operand
// (16 rows x 64 bytes per load) come at 9.8 TB/s from L2 over the card, whole
// row pieces at 25-33 TB/s.
//
// Bound by the weights' bytes and the loads' latency at few rows (1 x 4096 x
// 7168 fp8, 29 MB: 7.1 us, 4.1 TB/s; 64 x 7168 x 2048, 16 MB: 6.2 us), beyond
// by the bytes a CU gets into its LDS (gemm_pick.hip).
#include "dev_rows.h"

namespace moe {

namespace {

template <bool FP8, int BW, int BT, int W, int D, bool NTW>
__global__ __launch_bounds__(64 * W) void rows_split_kernel(RowsGemmArgs g, int ntiles, int slots) {
    constexpr int SA = BW / 16, SB = BT / 16;
    // the step's scales behind its rows: BT of the tokens, then the weights' one
    constexpr int kScaleLoads = FP8 ? BT / 64 + 1 : 0;
    constexpr int kSlot = (BW + BT) * 128 + 256 * kScaleLoads;
    constexpr int NL = (BW + BT) / 8 + kScaleLoads;
    constexpr int kSum = W * SA * SB * 1024;                     // the waves' sums
    constexpr int kOut = BT * kOutRow<BW>;                       // the finished tile
    constexpr int kLds = std::max(W * D * kSlot, std::max(kSum, kOut));
    static_assert(kLds <= 160 * 1024, "LDS");
    // one LDS object: with several, the compiler waits for every direct-to-LDS
    // load before each LDS read
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int64_t item = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int slot = int(item / ntiles), tile = int(item - int64_t(slot) * ntiles);
    int e, row0, row1;
    if (slot >= slots || !find_block<BT>(g, slot, e, row0, row1)) return;   // the whole workgroup alike

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t kbytes = int64_t(g.K) * (FP8 ? 1 : 2);
    const int steps = int(kbytes >> 7);
    const int n0 = tile * BW;
    lds_t* const ring = (lds_t*)lds + wv * D * kSlot;

    const uint8_t* wbase = g.w + (int64_t(e) * g.N + n0) * kbytes;
    const uint8_t* abase = g.a + int64_t(row0) * kbytes;
    const int last_w = g.N - 1 - n0, last_a = row1 - 1 - row0;
    // piece j: rows 8 j + lane / 8, chunk (lane % 8) ^ (row % 8) at position lane % 8
    const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) << 4;
    uint32_t off[(BW + BT) / 8];
#pragma unroll
    for (int j = 0; j < (BW + BT) / 8; ++j) {
        const int r = 8 * j + (lane >> 3);
        off[j] = uint32_t(8 * j < BW ? min(r, last_w) : min(r - BW, last_a)) * uint32_t(kbytes) + chunk;
    }
    const float* sp[kScaleLoads + 1];                            // this lane's scale rows
#pragma unroll
    for (int j = 0; j < kScaleLoads; ++j) {
        const int r = 64 * j + lane;
        sp[j] = r < BT ? g.a_scale + (int64_t(row0) + min(r, last_a)) * steps
                       : g.w_scale + (int64_t(e) * ((g.N + 127) >> 7) + (n0 >> 7)) * steps;
    }
    auto issue = [&](int i) {                                    // this wave's i-th step
        const int s = wv + W * i;
        lds_t* to = ring + (i % D) * kSlot;
#pragma unroll
        for (int j = 0; j < kScaleLoads; ++j)
            __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(sp[j] + s), to + (BW + BT) * 128 + 256 * j,
                                             4, 0, 0);
#pragma unroll
        for (int j = 0; j < (BW + BT) / 8; ++j) {
            const uint8_t* base = (8 * j < BW ? wbase : abase) + (int64_t(s) << 7);
            load_piece<NTW>(base + off[j], to + j * 1024, 8 * j < BW);
        }
    };
    const uint32_t c0 = uint32_t(lr * 128) + (uint32_t(lk ^ (lr & 7)) << 4), c1 = c0 ^ 64;

    f32x4 acc[SA][SB];
#pragma unroll
    for (int i = 0; i < SA; ++i)
#pragma unroll
        for (int t = 0; t < SB; ++t) acc[i][t] = f32x4{0, 0, 0, 0};

    const int mine = steps > wv ? (steps - wv + W - 1) / W : 0;  // this wave's steps
    for (int i = 0; i < D && i < mine; ++i) issue(i);
    for (int i = 0; i < mine; ++i) {
        wait_stages<NL, D - 1>(min(i + D - 1, mine - 1) - i);
        __builtin_amdgcn_sched_barrier(0);
        const lds_t* from = ring + (i % D) * kSlot;
        i32x4 a0[SA], a1[SA], b0[SB], b1[SB];
        float sc[SB];
        const lds_t* scales = from + (BW + BT) * 128;
        const float sw = FP8 ? *reinterpret_cast<lds_f*>(scales + 4 * BT) : 0.0f;
#pragma unroll
        for (int t = 0; t < SB; ++t) {
            b0[t] = *reinterpret_cast<lds_v4*>(from + (BW + 16 * t) * 128 + c0);
            b1[t] = *reinterpret_cast<lds_v4*>(from + (BW + 16 * t) * 128 + c1);
            if constexpr (FP8)
                sc[t] = __fmul_rn(*reinterpret_cast<lds_f*>(scales + (16 * t + lr) * 4), sw);
        }
#pragma unroll
        for (int m = 0; m < SA; ++m) {
            a0[m] = *reinterpret_cast<lds_v4*>(from + 16 * m * 128 + c0);
            a1[m] = *reinterpret_cast<lds_v4*>(from + 16 * m * 128 + c1);
        }
        wait_lgkm0();                                            // the slot is in registers: it takes step i + D
        __builtin_amdgcn_sched_barrier(0);
        if (i + D < mine) issue(i + D);
        using Op = Operand<FP8>;
        Op bv[SB];
#pragma unroll
        for (int t = 0; t < SB; ++t) bv[t] = Op(b0[t], b1[t]);
#pragma unroll
        for (int m = 0; m < SA; ++m) {
            const Op av(a0[m], a1[m]);
            f32x4 p[SB];                                         // fp8: the step's own sums, to be scaled
#pragma unroll
            for (int k = 0; k < Op::kParts; ++k)
#pragma unroll
                for (int t = 0; t < SB; ++t) {
                    if constexpr (FP8) p[t] = mma(av.part[k], bv[t].part[k], k == 0 ? f32x4{0, 0, 0, 0} : p[t]);
                    else acc[m][t] = mma(av.part[k], bv[t].part[k], acc[m][t]);
                }
            if constexpr (FP8) {
#pragma unroll
                for (int t = 0; t < SB; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[m][t][q] = __builtin_fmaf(sc[t], p[t][q], acc[m][t][q]);
            }
        }
    }
    __syncthreads();                                             // the rings are idle: the sums take their place
    f32x4* part = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int m = 0; m < SA; ++m)
#pragma unroll
        for (int t = 0; t < SB; ++t) part[(wv * SA * SB + m * SB + t) * 64 + lane] = acc[m][t];
    __syncthreads();
    constexpr int kMine = (SA * SB + W - 1) / W;
    f32x4 v[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int j = min(wv + W * q, SA * SB - 1);
        v[q] = part[j * 64 + lane];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const f32x4 o = part[(i * SA * SB + j) * 64 + lane];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[q][k] = __fadd_rn(v[q][k], o[k]);
        }
    }
    if ((g.N & 3) == 0) {                                        // whole 8-byte pieces of a row
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int j = wv + W * q, r = row0 + 16 * (j % SB) + lr, n = n0 + 16 * (j / SB) + 4 * lk;
            if (j < SA * SB && r < row1 && n < g.N)
                *reinterpret_cast<uint2*>(g.out + int64_t(r) * g.N + n) =
                    uint2{pack_bf16(v[q][0], v[q][1]), pack_bf16(v[q][2], v[q][3])};
        }
        return;
    }
    __syncthreads();                                             // the finished tile takes the sums' place
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int j = wv + W * q;
        if (j < SA * SB) stage4<BW>((lds_t*)lds, 16 * (j % SB) + lr, 16 * (j / SB) + 4 * lk, v[q]);
    }
    __syncthreads();
    store_tile<BW, BT, 64 * W, false>(g, (lds_t*)lds, row0, row1, n0);
}

template <bool FP8, int BW, int BT, int W, int D>
hipError_t launch_split(const RowsGemmArgs& g, bool one_pass, hipStream_t s) {
    const int ntiles = (g.N + BW - 1) / BW;
    const int64_t slots = block_slots(g, BT);
    void (*kern)(RowsGemmArgs, int, int) =
        one_pass ? rows_split_kernel<FP8, BW, BT, W, D, true> : rows_split_kernel<FP8, BW, BT, W, D, false>;
    return start(kern, grid_of(slots * ntiles), 64 * W, s, g, ntiles, int(slots));
}

template <bool FP8>
hipError_t launch(const RowsGemmArgs& g, int shape, bool one_pass, hipStream_t s) {
    switch (shape) {
        case 0: return launch_split<FP8, 16, 16, 8, 4>(g, one_pass, s);
        case 1: return launch_split<FP8, 32, 16, 8, 3>(g, one_pass, s);
        case 2: return launch_split<FP8, 32, 32, 8, 2>(g, one_pass, s);
        case 3: return launch_split<FP8, 64, 32, 8, 1>(g, one_pass, s);
        case 4: return launch_split<FP8, 64, 48, 8, 1>(g, one_pass, s);
        case 5: return launch_split<FP8, 64, 64, 8, 1>(g, one_pass, s);
        default: break;
    }
    // of converted e4m3 operands these would not fit the registers
    if constexpr (!FP8) {
        if (shape == 6) return launch_split<false, 64, 80, 8, 1>(g, one_pass, s);
        if (shape == 7) return launch_split<false, 128, 48, 6, 1>(g, one_pass, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows_split(const RowsGemmArgs& g, bool fp8, int shape, bool one_pass, hipStream_t s) {
    return fp8 ? launch<true>(g, shape, one_pass, s) : launch<false>(g, shape, one_pass, s);
}

}  // namespace moe
