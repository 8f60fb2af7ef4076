// Device code shared by the dense and grouped products (gemm_split.hip,
// gemm_tile.hip): finding a row block in the ragged groups, the matrix step
// and the output store.
#pragma once

#include <algorithm>

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

// V outputs per lane, V * 2 bytes aligned in every row (N % V == 0), by THREADS
// neighbouring lanes.  NT: past the caches' replacement (tile_product).
template <int BW, int BT, int THREADS, bool NT, int V, typename T>
__device__ __forceinline__ void store_rows(const RowsGemmArgs& g, const lds_t* tile, int row0, int row1, int n0) {
    typedef const __attribute__((address_space(3))) T lds_T;
    constexpr int kPer = BW / V, kTurns = (BT * kPer + THREADS - 1) / THREADS;
    const int live = min(BT, row1 - row0);
    // several pieces read ahead of their stores
#pragma unroll(kTurns < 8 ? kTurns : 4)
    for (int q = 0; q < kTurns; ++q) {
        const int i = threadIdx.x % THREADS + q * THREADS;
        const int r = i / kPer, c = (i % kPer) * V;
        if (r < live && n0 + c < g.N) {
            const T v = *reinterpret_cast<lds_T*>(tile + r * kOutRow<BW> + 2 * c);
            T* const to = reinterpret_cast<T*>(g.out + int64_t(row0 + r) * g.N + n0 + c);
            if constexpr (NT) __builtin_nontemporal_store(v, to);
            else *to = v;
        }
    }
}
template <int BW, int BT, int THREADS, bool NT>
__device__ __forceinline__ void store_tile(const RowsGemmArgs& g, const lds_t* tile, int row0, int row1, int n0) {
    if ((g.N & 7) == 0) store_rows<BW, BT, THREADS, NT, 8, i32x4>(g, tile, row0, row1, n0);
    else if ((g.N & 1) == 0) store_rows<BW, BT, THREADS, NT, 2, uint32_t>(g, tile, row0, row1, n0);
    else store_rows<BW, BT, THREADS, NT, 1, uint16_t>(g, tile, row0, row1, n0);
}

// One operand of a 16-row subtile for a 128-byte step of K, from this lane's two
// 16-byte chunks of its row: bf16 as it is, e4m3 codes as the bf16 values they
// stand for (exact: 4 significant bits).  The fp8 matrix instructions take the
// codes themselves and twice as many a cycle, but drop the bits of a product
// below about 2^-14 of the largest of eight (256 - 256 + 126 times 2^-6 gives 0),
// and these outputs decide roundings, a gated multiply's codes among them; bf16
// products are summed in fp32.  Which K a lane's chunks hold does not matter as
// long as both operands agree.
template <bool FP8>
struct Operand {
    static constexpr int kParts = FP8 ? 4 : 2;
    bf16x8 part[kParts];
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ Operand(i32x4 c0, i32x4 c1) {
        if constexpr (FP8) {
            part[0] = e4m3x8_to_bf16(c0[0], c0[1], 1.0f);
            part[1] = e4m3x8_to_bf16(c0[2], c0[3], 1.0f);
            part[2] = e4m3x8_to_bf16(c1[0], c1[1], 1.0f);
            part[3] = e4m3x8_to_bf16(c1[2], c1[3], 1.0f);
        } else {
            part[0] = __builtin_bit_cast(bf16x8, c0);
            part[1] = __builtin_bit_cast(bf16x8, c1);
        }
    }
};
__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
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
