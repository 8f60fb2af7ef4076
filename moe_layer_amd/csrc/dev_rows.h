// Device code shared by the dense and grouped products (gemm_split.hip,
// gemm_tile.hip): finding a row block in the ragged groups, the matrix step
// and the output store.
#pragma once

#include <algorithm>
#include <type_traits>

#include "dense.h"

namespace moe {

namespace {

typedef __attribute__((address_space(3))) uint8_t lds_t;
typedef const __attribute__((address_space(3))) i32x4 lds_v4;
typedef const __attribute__((address_space(3))) float lds_f;

template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}
// wait until at most `ahead` stages of NL loads each are in flight
template <int NL, int MAXA>
__device__ __forceinline__ void wait_stages(int ahead) {
    if constexpr (MAXA <= 0) {
        wait_vm<0>();
    } else {
        if (ahead >= MAXA) wait_vm<MAXA * NL>();
        else wait_stages<NL, MAXA - 1>(ahead);
    }
}

// 16 bytes per lane global -> LDS (lane i's at to + 16 i).  NTW: weights that
// one row block alone reads go past the caches' replacement (131 rows on 73 of
// 128 experts of 4096 x 1536 bf16, 0.92 GB: 159 -> 141 us, 6.5 TB/s; weights
// that several row blocks read must not: 256-row blocks of the same experts,
// 32768 rows 518 -> 545 us).
template <bool NTW>
__device__ __forceinline__ void load_piece(const uint8_t* from, lds_t* to, bool weights) {
    if (NTW && weights)
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from), to, 16, 0, 2);
    else
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from), to, 16, 0, 0);
}

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

// The row blocks of BM rows the groups are cut into (find_block's slots).
template <int BM>
__device__ __forceinline__ int count_blocks(const RowsGemmArgs& g) {
    if (!g.offsets) return (g.rows + BM - 1) / BM;
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int i = lane; i < g.E; i += 64) {
        const int lo = min(max(g.offsets[i], 0), g.rows);
        n += (min(max(g.offsets[i + 1], lo), g.rows) - lo + BM - 1) / BM;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
    return __builtin_amdgcn_readfirstlane(n);
}

// count_blocks and find_block for the same BM with one look at the offsets: up to
// kHeldGroups groups stay in the wave's registers, four a lane.  Every workgroup starts
// with this and loads nothing before (188 rows in 256 int8 groups of 440 x 368 10.2 ->
// 7.0 us, 131 in 128 of 4096 x 1536 76 -> 70, 32768 in 128 300 -> 292).  Of more groups
// the offsets are read for each; kTotal false: only to find a block (1 row in 1024 fp8
// groups of 496 x 1280 7.9 us, with the count in front 10.1; 10 in 512 bf16 ones of 352 x
// 1792 6.8, 8.1).
template <int BM, bool kTotal>
struct RowBlocks {
    static constexpr int kPer = 4, kHeldGroups = 64 * kPer;
    int lo[kPer], hi[kPer];
    int own, sum;            // the lane's blocks, and with those of the lanes before
    int total;               // (kTotal)
    bool held;

    __device__ __forceinline__ explicit RowBlocks(const RowsGemmArgs& g) : held(g.offsets && g.E <= kHeldGroups) {
        if (!held) {
            if constexpr (kTotal) total = count_blocks<BM>(g);
            return;
        }
        const int lane = threadIdx.x & 63;
        int at[kPer + 1];
#pragma unroll
        for (int k = 0; k <= kPer; ++k) at[k] = g.offsets[min(kPer * lane + k, g.E)];
        own = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {                 // behind the last group twice the same offset
            lo[k] = min(max(at[k], 0), g.rows);
            hi[k] = kPer * lane + k < g.E ? min(max(at[k + 1], lo[k]), g.rows) : lo[k];
            own += (hi[k] - lo[k] + BM - 1) / BM;
        }
        sum = wave_scan(own);
        total = __builtin_amdgcn_readlane(sum, 63);
    }

    __device__ __forceinline__ bool find(const RowsGemmArgs& g, int slot, int& e, int& row0, int& row1) const {
        if (!held) return find_block<BM>(g, slot, e, row0, row1);
        if (slot >= total) return false;
        const int src = max(__ffsll((unsigned long long)__ballot(sum > slot)) - 1, 0);
        int in = slot - (__builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(own, src));
        e = kPer * src;
        bool found = false;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int first = __builtin_amdgcn_readlane(lo[k], src), last = __builtin_amdgcn_readlane(hi[k], src);
            const int n = (last - first + BM - 1) / BM;
            if (!found && in < n) {
                found = in >= 0;
                e += k;
                row0 = first + in * BM;
                row1 = last;
            }
            in -= n;
        }
        return found && row0 < row1;
    }
};

// Workgroup -> item of `total`.  The hardware deals workgroups to the 8 XCDs in
// turn; every XCD gets one contiguous range of the items, so that neighbours
// share its L2.  False past the range.
__device__ __forceinline__ bool xcd_item(int64_t total, int64_t& item) {
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t xcd = wg & 7;
    item = xcd * total / 8 + (wg >> 3);
    return item < (xcd + 1) * total / 8;
}

// A finished tile on its way out: BT rows of BW bf16 outputs in LDS, rows 16
// bytes apart beyond their length, so that whole 16-byte pieces of a row leave
// by one lane each (a lane's four outputs straight from the accumulator are 8
// bytes of a row; where N is odd they would be four stores of 2 bytes).
template <int BW>
constexpr int kOutRow = 2 * BW + 16;

// outputs 4 j .. 4 j + 3 of tile row t
template <int BW>
__device__ __forceinline__ void stage4(lds_t* tile, int t, int n, const f32x4& v) {
    typedef __attribute__((address_space(3))) i32x2 lds_v2;
    *reinterpret_cast<lds_v2*>(tile + t * kOutRow<BW> + 2 * n) =
        i32x2{int(pack_bf16(v[0], v[1])), int(pack_bf16(v[2], v[3]))};
}

// Eight outputs per lane by THREADS neighbouring lanes, 16 bytes a store wherever a
// row starts (global stores take any alignment; 6565 x 5413 x 496 int8 54.7 -> 45.2 us
// against 2 bytes a store where N is odd), the last N % 8 of a row one by one.  kPast:
// past the caches' replacement, of rows that are whole lines.
template <int BW, int BT, int THREADS, bool kPast>
__device__ __forceinline__ void store_rows(const RowsGemmArgs& g, const lds_t* tile, int row0, int row1, int n0) {
    typedef __attribute__((ext_vector_type(4), aligned(2))) int anywhere_v4;
    typedef const __attribute__((address_space(3))) uint16_t lds_u16;
    constexpr int kPer = BW / 8, kTurns = (BT * kPer + THREADS - 1) / THREADS;
    const int live = min(BT, row1 - row0);
    // several pieces read ahead of their stores
#pragma unroll(kTurns < 8 ? kTurns : 4)
    for (int q = 0; q < kTurns; ++q) {
        const int i = threadIdx.x % THREADS + q * THREADS;
        const int r = i / kPer, c = (i % kPer) * 8;
        if (r >= live || n0 + c >= g.N) continue;
        const lds_t* const from = tile + r * kOutRow<BW> + 2 * c;
        uint16_t* const to = g.out + int64_t(row0 + r) * g.N + n0 + c;
        if constexpr (kPast) {
            __builtin_nontemporal_store(*reinterpret_cast<lds_v4*>(from), reinterpret_cast<i32x4*>(to));
        } else if (n0 + c + 8 <= g.N) {
            *reinterpret_cast<anywhere_v4*>(to) = *reinterpret_cast<lds_v4*>(from);
        } else {
            for (int k = 0; n0 + c + k < g.N; ++k) to[k] = *reinterpret_cast<lds_u16*>(from + 2 * k);
        }
    }
}
// NT: tiles of 256 weight rows.  Outputs whose rows are whole lines go past the caches'
// replacement; of others the two halves of a line that tiles share should meet in L2.
// The choice stands around the loops: of two stores in one the compiler makes a plain
// one.  us past it / not, and with moe_silu_mul reading the result; whole lines:
// bf16 3000 x 2048 x 512 12.0 / 12.9 (20.3 / 21.1), 8000 rows in 32 groups of 5120 x 640
// 70 / 81 (103 / 102), 8192 x 8192 x 1024 123 / 121 (152 / 150); fp8 6000 in 16 of 1024 x
// 1024 19.1 / 20.4 (25.1 / 25.8), 8192 x 8192 x 1024 136 / 138 (169 / 168); int8 the two
// 12.9 / 14.3 (18.7 / 20.0), 77.8 / 78.3 (108 / 108), 32768 in 128 of 4096 x 1536 288 /
// 293 (344 / 350).  Not: bf16 16384 x 2064 x 512 59 / 54 (74 / 70), 8192 x 8192 x 1024
// 16 bytes off a line 134 / 123 (160 / 152), 8000 in 32 of 5136 x 640 77 / 83 (106 / 104);
// fp8 16384 x 2064 x 512 60 / 54 (77 / 71); int8 35.7 / 33.5 (52 / 50), 8192 x 8192 x 1024
// off a line 89 / 79 (115 / 109), 4000 x 2080 x 2048 24.6 / 26.2 (30.8 / 32.2).
template <int BW, int BT, int THREADS, bool NT>
__device__ __forceinline__ void store_tile(const RowsGemmArgs& g, const lds_t* tile, int row0, int row1, int n0) {
    if constexpr (NT) {
        if (((reinterpret_cast<uintptr_t>(g.out) | 2 * uintptr_t(g.N)) & 127) == 0)
            return store_rows<BW, BT, THREADS, true>(g, tile, row0, row1, n0);
    }
    store_rows<BW, BT, THREADS, false>(g, tile, row0, row1, n0);
}

// One operand of a 16-row subtile for a 128-byte step of K, from this lane's two
// 16-byte chunks of its row: bf16 as it is, e4m3 codes as the bf16 values they
// stand for (exact: 4 significant bits).  The fp8 matrix instructions take the
// codes themselves and twice as many a cycle, but drop the bits of a product
// below about 2^-14 of the largest of eight (256 - 256 + 126 times 2^-6 gives 0),
// and these outputs decide roundings, a gated multiply's codes among them; bf16
// products are summed in fp32.  int8 codes go to the matrix cores as they are and
// are summed in 32-bit integers, exactly.  Which K a lane's chunks hold does not
// matter as long as both operands agree.
template <RowsKind KIND>
struct Operand {
    static constexpr int kParts = KIND == kRowsFp8 ? 4 : 2;
    using Part = std::conditional_t<KIND == kRowsInt8, i32x4, bf16x8>;
    Part part[kParts];
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ Operand(i32x4 c0, i32x4 c1) {
        if constexpr (KIND == kRowsFp8) {
            part[0] = e4m3x8_to_bf16(c0[0], c0[1], 1.0f);
            part[1] = e4m3x8_to_bf16(c0[2], c0[3], 1.0f);
            part[2] = e4m3x8_to_bf16(c1[0], c1[1], 1.0f);
            part[3] = e4m3x8_to_bf16(c1[2], c1[3], 1.0f);
        } else {
            part[0] = __builtin_bit_cast(Part, c0);
            part[1] = __builtin_bit_cast(Part, c1);
        }
    }
};
__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mma(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}
// a lane's four sums of a 16 x 16 subtile
template <RowsKind KIND>
using Sums = std::conditional_t<KIND == kRowsInt8, i32x4, f32x4>;

// int8: rows of K bytes, any multiple of 16, so the last step of 128 may be a part
// of one.  Lanes whose 16-byte chunk lies behind a row's end fetch zeros there.
__device__ const __attribute__((aligned(16))) uint8_t kNoChunk[16] = {};

// The outputs of four int8 sums: fl32(fl32(sum) a_scale) w_scale, each rounded
__device__ __forceinline__ f32x4 scaled(i32x4 sum, float sa, f32x4 sw) {
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __fmul_rn(__fmul_rn(float(sum[q]), sa), sw[q]);
    return v;
}

// A grid of at least n workgroups, a multiple of 8 of them (xcd_item)
inline dim3 xcd_grid(int64_t n) { return grid_of((n + 7) / 8 * 8); }

// Row blocks of BM rows there can be: every group with rows ends in at most
// one part block.
inline int64_t block_slots(const RowsGemmArgs& g, int bm) {
    if (!g.offsets) return (int64_t(g.rows) + bm - 1) / bm;
    const int64_t most = int64_t(g.rows) / bm + std::min(g.E, g.rows);
    return std::min<int64_t>(most, g.rows);
}

}  // namespace

}  // namespace moe
