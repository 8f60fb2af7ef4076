// Tokens' rows sorted by the expert they go to, quantised on the way where
// asked for:
//   offsets[e] = #{f : id_f < e},  inv[f] = offsets[id_f] + #{f' < f : id_f' = id_f},
//   rows[inv[f]] = x[t] for the routed slots f = t topk + j, inv[f] = -1 for the others.
// The position of a slot is the number of routed slots before it in the order
// (expert, slot), so it is the same whichever form finds it:
//   few slots   in the launch that moves the rows: every workgroup counts the
//               slots before its token's own over all ids;
//   many slots  blocks of slots are counted by expert (sort_count_kernel), every
//               block adds the counts before its own and ranks its slots with a
//               ballot multisplit (sort_place_kernel), then the rows are moved.
// A row is read once and stored topk times.
#include "dev_align.h"
#include "moe.h"
#include "sorted.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kOneLaunchSlots = 2048;
constexpr int kMostBlocks = 256;

template <int CTRL>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ int wave_sum(int v) {
    v = dpp_add<0xb1>(v);                                  // quad_perm [1,0,3,2]
    v = dpp_add<0x4e>(v);                                  // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);                                 // row_half_mirror
    v = dpp_add<0x140>(v);                                 // row_mirror
    const auto a = __builtin_amdgcn_permlane16_swap(uint32_t(v), uint32_t(v), false, false);
    v = int(a[0] + a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(uint32_t(v), uint32_t(v), false, false);
    return int(b[0] + b[1]);
}

// Exclusive scan over the workgroup's threads of v[0 .. PER) in thread order;
// s: one int per wave.  Returns this thread's start.
template <int PER>
__device__ __forceinline__ int scan_start(const int (&v)[PER], int* s) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += v[i];
    int sum = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int up = __shfl_up(sum, m);
        if (lane >= m) sum += up;
    }
    if (lane == 63) s[w] = sum;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < w; ++i) before += s[i];
    return before + sum - mine;
}

// offsets of all experts by one workgroup of NT threads
template <int NT>
__device__ __forceinline__ void write_offsets(const SortArgs& a) {
    constexpr int kPer = kMaxE / NT;
    __shared__ int count[kMaxE];
    __shared__ int s_scan[NT / 64];
    for (int e = threadIdx.x; e < kMaxE; e += NT) count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.R; i += NT) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < uint32_t(a.E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    int n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = count[threadIdx.x * kPer + i];
    int at = scan_start(n, s_scan);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e <= a.E) a.offsets[e] = at;
        at += n[i];
    }
    if (a.E == kMaxE && threadIdx.x == NT - 1) a.offsets[kMaxE] = at;
}

// positions of token t's slots into pos[topk], by all waves of the workgroup
template <int NT>
__device__ __forceinline__ void find_positions(const SortArgs& a, int t, int* pos) {
    constexpr int kNW = NT / 64, kAt = 4;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int j0 = wv; j0 < a.topk; j0 += kAt * kNW) {
        uint32_t e[kAt];
        int f[kAt], n[kAt];
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            f[q] = t * a.topk + min(j0 + q * kNW, a.topk - 1);
            e[q] = uint32_t(a.ids[f[q]]);
            n[q] = 0;
        }
#pragma unroll 4
        for (int i = lane; i < a.R; i += 64) {
            const uint32_t id = uint32_t(a.ids[i]);         // an unrouted one is past every expert
#pragma unroll
            for (int q = 0; q < kAt; ++q) n[q] += id < e[q] + (i < f[q] ? 1u : 0u) ? 1 : 0;
        }
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            const int sum = wave_sum(n[q]);
            if (lane == 0 && j0 + q * kNW < a.topk) pos[j0 + q * kNW] = e[q] < uint32_t(a.E) ? sum : -1;
        }
    }
}

// counts[b * E + e] = slots of expert e among block b's
__global__ __launch_bounds__(kThreads) void sort_count_kernel(SortArgs a, int slots) {
    __shared__ int count[kMaxE];
    for (int e = threadIdx.x; e < a.E; e += kThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * slots;
    const int last = int(min(int64_t(a.R), first + slots));
#pragma unroll 4
    for (int i = int(first) + threadIdx.x; i < last; i += kThreads) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < uint32_t(a.E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.counts[int64_t(blockIdx.x) * a.E + e] = count[e];
}

// inv of block b's slots; block 0 writes the offsets
__global__ __launch_bounds__(kThreads) void sort_place_kernel(SortArgs a, int slots, int blocks) {
    constexpr int kPer = kMaxE / kThreads;
    __shared__ int run[kWaves * kMaxE];     // a wave's next position in each expert
    __shared__ int before[kMaxE], total[kMaxE];
    __shared__ int s_scan[kWaves];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const uint64_t lower = (uint64_t(1) << lane) - 1;
    const int bits = a.E > 1 ? 32 - __clz(a.E - 1) : 0;
    for (int i = threadIdx.x; i < kWaves * a.E; i += kThreads) run[i] = 0;
    for (int e = threadIdx.x; e < kMaxE; e += kThreads) before[e] = total[e] = 0;
    __syncthreads();
    // a wave's slots: a contiguous quarter of the block's, a multiple of 64
    const int64_t base = int64_t(blockIdx.x) * slots + wv * (slots / kWaves);
    const int first = int(min(int64_t(a.R), base)), last = int(min(int64_t(a.R), base + slots / kWaves));
    int* const mine = run + wv * a.E;
    for (int i = first; i < last; i += 64) {
        const int e = i + lane < last ? a.ids[i + lane] : -1;
        if (uint32_t(e) < uint32_t(a.E)) atomicAdd(&mine[e], 1);
    }
    // the blocks' counts: threads of `step` experts side by side, the rest over the blocks
    int step = 64;
    while (step < a.E && step < kThreads) step <<= 1;
    for (int e = threadIdx.x % step; e < a.E; e += step) {
        int b = 0, n = 0;
#pragma unroll 8
        for (int q = threadIdx.x / step; q < blocks; q += kThreads / step) {
            const int c = a.counts[int64_t(q) * a.E + e];
            n += c;
            b += q < int(blockIdx.x) ? c : 0;
        }
        atomicAdd(&total[e], n);
        atomicAdd(&before[e], b);
    }
    __syncthreads();
    int n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = total[threadIdx.x * kPer + i];
    int at = scan_start(n, s_scan);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (blockIdx.x == 0 && e <= a.E) a.offsets[e] = at;
        if (e < a.E) {
            int to = at + before[e];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int c = run[w * a.E + e];
                run[w * a.E + e] = to;
                to += c;
            }
        }
        at += n[i];
    }
    if (blockIdx.x == 0 && a.E == kMaxE && threadIdx.x == kThreads - 1) a.offsets[kMaxE] = at;
    __syncthreads();
    for (int i = first; i < last; i += 64) {
        const int f = i + lane;
        const int e = f < last ? a.ids[f] : -1;
        const bool routed = uint32_t(e) < uint32_t(a.E);
        const uint64_t same = peers(e, routed, bits);
        if (routed) {
            const int to = mine[e];
            a.inv[f] = to + __popcll(same & lower);
            // every lane's read of mine[e] precedes the first one's update (one wave, in order)
            if ((same & lower) == 0) mine[e] = to + __popcll(same);
        } else if (f < last) {
            a.inv[f] = -1;
        }
    }
}

// A token's row (kSortInt8) or a part of it to the positions of its slots.
// kOne: the positions are found here, and one more workgroup writes the offsets.
template <SortMode kMode, int NT, int CH, bool kOne>
__global__ __launch_bounds__(NT) void sort_move_kernel(SortArgs a, int parts, int span) {
    __shared__ int pos[MOE_MAX_TOPK];
    __shared__ uint32_t s_max[NT / 64];
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t token = wg / parts;
    if (token >= a.T) {                                    // the whole workgroup alike
        if (kOne && wg == int64_t(a.T) * parts) write_offsets<NT>(a);
        return;
    }
    const int t = int(token), part = int(wg - token * parts);
    const int u0 = part * span + threadIdx.x, u1 = min(a.units, (part + 1) * span);
    i32x4 v[CH];
    const uint8_t* src = a.x + token * a.units * 16;
#pragma unroll
    for (int c = 0; c < CH; ++c) {                         // behind the part: its last piece again
        const int u = min(u0 + c * NT, u1 - 1);
        v[c] = *reinterpret_cast<const i32x4*>(src + int64_t(u) * 16);
    }
    if constexpr (kOne) {
        find_positions<NT>(a, t, pos);
    } else {
        if (threadIdx.x < unsigned(a.topk)) pos[threadIdx.x] = a.inv[token * a.topk + threadIdx.x];
    }
    uint32_t bits = 0;
    if constexpr (kMode == kSortInt8) {
#pragma unroll
        for (int c = 0; c < CH; ++c) bits = pk_max_u16(bits, abs_max8(v[c]));
        bits = wave_max_u16(bits);
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = bits;
    }
    __syncthreads();
    if (kOne && part == 0 && threadIdx.x < unsigned(a.topk)) a.inv[token * a.topk + threadIdx.x] = pos[threadIdx.x];
    if constexpr (kMode == kSortCopy) {
        for (int j = 0; j < a.topk; ++j) {
            const int p = __builtin_amdgcn_readfirstlane(pos[j]);
            if (p < 0) continue;
            uint8_t* to = a.rows + int64_t(p) * a.units * 16;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int u = u0 + c * NT;
                if (u < u1) *reinterpret_cast<i32x4*>(to + int64_t(u) * 16) = v[c];
            }
        }
        if (part == 0)
            for (int i = threadIdx.x; i < a.scales; i += NT) {
                const float s = a.x_scale[token * a.scales + i];
                for (int j = 0; j < a.topk; ++j)
                    if (pos[j] >= 0) a.row_scales[int64_t(pos[j]) * a.scales + i] = s;
            }
    } else {
        uint2 q[CH];
        float s[CH];
        if constexpr (kMode == kSortInt8) {
#pragma unroll
            for (int i = 0; i < NT / 64; ++i) bits = max(bits, s_max[i]);
            float inverse;
            s[0] = int8_scale(bits, inverse);
#pragma unroll
            for (int c = 0; c < CH; ++c) q[c] = int8_codes(v[c], inverse);
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) s[c] = quant8<16>(v[c], q[c].x, q[c].y);   // parts are whole groups
        }
        for (int j = 0; j < a.topk; ++j) {
            const int p = __builtin_amdgcn_readfirstlane(pos[j]);
            if (p < 0) continue;
            uint8_t* to = a.rows + int64_t(p) * a.cols;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int u = u0 + c * NT;
                if (u < u1) {
                    *reinterpret_cast<uint2*>(to + int64_t(u) * 8) = q[c];
                    if (kMode == kSortFp8 && (threadIdx.x & 15) == 0)
                        a.row_scales[int64_t(p) * a.scales + (u >> 4)] = s[c];
                }
            }
            if (kMode == kSortInt8 && threadIdx.x == 0) a.row_scales[p] = s[0];
        }
    }
}

template <SortMode kMode, int NT, int CH>
hipError_t launch_move(const SortArgs& a, bool one, hipStream_t s) {
    // parts of at most NT * CH pieces, of equal length but for the rounding to whole groups
    const int parts = kMode == kSortInt8 ? 1 : (a.units + NT * CH - 1) / (NT * CH);
    const int span = kMode == kSortInt8 ? a.units : ((a.units + parts - 1) / parts + 15) / 16 * 16;
    const int64_t n = int64_t(a.T) * parts + (one ? 1 : 0);
    void (*kern)(SortArgs, int, int) =
        one ? sort_move_kernel<kMode, NT, CH, true> : sort_move_kernel<kMode, NT, CH, false>;
    return start(kern, grid_of(n), NT, s, a, parts, span);
}

hipError_t launch_move(const SortArgs& a, SortMode mode, bool one, hipStream_t s) {
    if (mode == kSortCopy) return launch_move<kSortCopy, 256, 1>(a, one, s);
    if (mode == kSortFp8) return launch_move<kSortFp8, 256, 1>(a, one, s);
    if (a.units <= 256) return launch_move<kSortInt8, 256, 1>(a, one, s);
    if (a.units <= 512) return launch_move<kSortInt8, 256, 2>(a, one, s);
    if (a.units <= 1024) return launch_move<kSortInt8, 256, 4>(a, one, s);
    if (a.units <= 2048) return launch_move<kSortInt8, 1024, 2>(a, one, s);
    static_assert(MOE_MAX_INT8_K <= 1024 * 4 * 8, "a row in one workgroup's registers");
    return launch_move<kSortInt8, 1024, 4>(a, one, s);
}

}  // namespace

SortPlan plan_sort(int64_t R, int E) {
    (void)E;
    if (R <= kOneLaunchSlots) return {0, 0};
    // 1024 slots a block, more where there would be over kMostBlocks of them (a
    // block reads the counts of all)
    const int64_t slots = std::max<int64_t>(1024, (R + kMostBlocks - 1) / kMostBlocks + 255) / 256 * 256;
    return {int(slots), int((R + slots - 1) / slots)};
}

hipError_t launch_sort_rows(const SortArgs& a, SortMode mode, hipStream_t s) {
    const SortPlan p = plan_sort(a.R, a.E);
    if (p.blocks == 0) return launch_move(a, mode, true, s);
    hipError_t e = start(sort_count_kernel, dim3(p.blocks), kThreads, s, a, p.slots);
    if (e == hipSuccess) e = start(sort_place_kernel, dim3(p.blocks), kThreads, s, a, p.slots, p.blocks);
    return e == hipSuccess ? launch_move(a, mode, false, s) : e;
}

}  // namespace moe
