// Tokens' rows sorted by the expert they go to, quantised on the way where
// asked for:
//   offsets[e] = #{f : id_f < e},  inv[f] = offsets[id_f] + #{f' < f : id_f' = id_f},
//   rows[inv[f]] = x[t] for the routed slots f = t topk + j, inv[f] = -1 for the others.
// The position of a slot is the number of routed slots before it in the order
// (expert, slot), so it is the same whichever form finds it:
//   few ids     every workgroup that moves a row compares its token's slots with
//               all ids (sort_move_kernel<.., true>);
//   batch       every workgroup counts all ids by expert in LDS, for several
//               tokens at a time (sort_batch_kernel);
//   counted     blocks of slots are counted by expert (sort_count_kernel), every
//               block adds the counts before its own and ranks its slots
//               (sort_place_kernel), then the rows are moved: three launches, for
//               more ids than every workgroup should read.
// A row is read once and stored topk times: large batches are bound by those bytes
// (8192 x 7168 bf16 to 8 of 256 experts 216 us with x from HBM, 4.9 TB/s, 187 with x from
// the last-level cache; 10 of them to find the positions), single tokens by the launch
// (kernel 2.7 us), batches in between by the look at all ids in front (1031 x 4096 to
// int8 11.4 us, 8.3 of them bytes).  8 of 256 experts, in a graph, us (bytes at 5.07 TB/s):
// to fp8 64 x 4096 4.5 (0.5), 1031 x 4096 12.3 (8.6), 8192 x 7168 105 (119); fp8 codes with
// their scales 4.7 (0.5), 12.0 (7.7), 105 (108); int8 codes 1031 x 4096 12.2 (7.5), 8192 x
// 7168 106 (104).
#include "dev_align.h"
#include "moe.h"
#include "sorted.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kPlaceThreads = 1024;
// Slots up to which every workgroup of the batch form counts all ids.  us, batch /
// counted, 8 of 256 experts: 4000 tokens of 4096 to int8 30.3 / 33.2, bf16 50.2 / 54.2, of
// 1024 18.2 / 20.4; 6000 (48000 slots) 44.9 / 45.4, 95.2 / 98.2, 26.3 / 27.2; 8000 71.7 /
// 69.7, 127.8 / 126.7, 34.3 / 33.2.
constexpr int kBatchMostSlots = 49152;
constexpr int kMostBlocks = 256;
constexpr int kBatchThreads = 512;
constexpr int kBatchSpan = 1024;                           // pieces of a part of a row that is not int8's
// slots of a workgroup of the batch form, at most kBatchMostSlots / 512 of T / 512 tokens and those of 4 more
constexpr int kBatchSlots = kBatchMostSlots / 512 + 4 * MOE_MAX_TOPK;

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

// Exclusive scan over the workgroup's W waves' threads of v[0 .. PER) in thread order;
// s: one int per wave.  Returns this thread's start.
template <int W, int PER>
__device__ __forceinline__ int scan_start(const int (&v)[PER], int* s) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += v[i];
    const int sum = wave_scan(mine);
    if (lane == 63) s[w] = sum;
    __syncthreads();
    int before = sum - mine;
#pragma unroll
    for (int i = 0; i < W; ++i) before += i < w ? s[i] : 0;
    return before;
}

// f(i, ids[i]) for every i below R, by NT threads: 16-byte loads, kFlight of them in
// flight, and single ones in front of the first 16-byte border and behind the last.
// load_first() may precede each() by other work.
template <int NT, int kFlight>
struct EachId {
    const int32_t* ids;
    const i32x4* four;
    int R, head, quads;
    i32x4 v[kFlight];

    __device__ __forceinline__ EachId(const int32_t* p, int n) : ids(p), R(n) {
        head = min(R, int(-(reinterpret_cast<uintptr_t>(ids) >> 2) & 3));
        quads = (R - head) >> 2;
        four = reinterpret_cast<const i32x4*>(ids + head);
    }
    __device__ __forceinline__ void load(int q0) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) v[u] = four[min(q0 + u * NT + int(threadIdx.x), quads - 1)];
    }
    __device__ __forceinline__ void load_first() {
        if (quads > 0) load(0);
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        for (int q0 = 0; q0 < quads; q0 += NT * kFlight) {
            if (q0 > 0) load(q0);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int q = q0 + u * NT + threadIdx.x;
                if (q < quads) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) f(head + 4 * q + w, v[u][w]);
                }
            }
        }
        const int rest = R - 4 * quads;                    // in front and behind, 6 at most
        if (int(threadIdx.x) < rest) {
            const int i = int(threadIdx.x) < head ? int(threadIdx.x) : int(threadIdx.x) + 4 * quads;
            f(i, ids[i]);
        }
    }
};
template <int NT, int kFlight, typename F>
__device__ __forceinline__ void each_id(const int32_t* p, int n, F f) {
    EachId<NT, kFlight> ids(p, n);
    ids.load_first();
    ids.each(f);
}

// Workgroups that write the offsets beside those that move rows
constexpr int offset_groups(int R, int E) { return R <= kHeldIds ? E / 16 + 1 : 1; }

// workgroup x of them
template <int NT>
__device__ __forceinline__ void write_offsets(const SortArgs& a, int x) {
    constexpr int kPer = kMaxE / NT;
    __shared__ __attribute__((aligned(16))) int count[kMaxE];
    __shared__ int s_scan[NT / 64];
    if (a.R <= kHeldIds) {
        // 16 experts, one a lane, and NT / 16 parts of the ids
        static_assert(kHeldIds <= kMaxE, "ids in count");
        const int e = 16 * x + (threadIdx.x & 15), part = threadIdx.x >> 4;
        const int quads = (a.R + 3) >> 2;
        for (int i = threadIdx.x; i < 4 * quads; i += NT) count[i] = i < a.R ? a.ids[i] : -1;
        __syncthreads();
        int n = 0;
        for (int q = part; q < quads; q += NT / 16) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(count + 4 * q);
#pragma unroll
            for (int w = 0; w < 4; ++w) n += uint32_t(v[w]) < uint32_t(e) ? 1 : 0;
        }
        n += __shfl_xor(n, 16);
        n += __shfl_xor(n, 32);
        __syncthreads();
        const int lane = threadIdx.x & 63;
        if (lane < 16) count[(threadIdx.x >> 6) * 16 + lane] = n;
        __syncthreads();
        if (threadIdx.x >= 16) return;
        for (int w = 1; w < NT / 64; ++w) n += count[16 * w + lane];
        if (e <= a.E) a.offsets[e] = n;
        return;
    }
    for (int e = threadIdx.x; e < kMaxE; e += NT) count[e] = 0;
    __syncthreads();
    each_id<NT, 2>(a.ids, a.R, [&](int, int id) {
        if (uint32_t(id) < uint32_t(a.E)) atomicAdd(&count[id], 1);
    });
    __syncthreads();
    int n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = count[threadIdx.x * kPer + i];
    int at = scan_start<NT / 64>(n, s_scan);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e <= a.E) a.offsets[e] = at;
        at += n[i];
    }
    if (a.E == kMaxE && threadIdx.x == NT - 1) a.offsets[kMaxE] = at;
}

// positions of token t's slots into pos[topk], a slot a wave, which holds all ids, Q a
// lane (16 a lane for any number of ids: 16 x 4096 4.1 us, not 3.6)
template <int NT, int Q>
__device__ __forceinline__ void compare_held(const SortArgs& a, int t, int* pos) {
    const int lane = threadIdx.x & 63, own = t * a.topk;
    const int mine = lane < a.topk ? a.ids[own + lane] : -1;
    int id[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) id[q] = 64 * q + lane < a.R ? a.ids[64 * q + lane] : -1;
    for (int j = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); j < a.topk; j += NT / 64) {
        const uint32_t e = uint32_t(__builtin_amdgcn_readlane(mine, j));
        int n = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            n += __popcll(__ballot(uint32_t(id[q]) < e + (64 * q + lane < own + j ? 1u : 0u)));
        if (lane == 0) pos[j] = e < uint32_t(a.E) ? n : -1;
    }
}

// positions of token t's slots into pos[topk] (set to 0 before, with a barrier); of
// many ids eight slots at a time, every wave counting over its share of the ids
template <int NT>
__device__ __forceinline__ void find_positions(const SortArgs& a, int t, int* pos) {
    constexpr int kAt = kSlotsAtOnce;
    const int lane = threadIdx.x & 63, own = t * a.topk;
    if (a.R <= 64) return compare_held<NT, 1>(a, t, pos);
    if (a.R <= 256) return compare_held<NT, 4>(a, t, pos);
    if (a.R <= 512) return compare_held<NT, 8>(a, t, pos);
    if (a.R <= kHeldIds) return compare_held<NT, kHeldIds / 64>(a, t, pos);
    for (int j0 = 0; j0 < a.topk; j0 += kAt) {
        uint32_t e[kAt];
        int n[kAt];
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            e[q] = uint32_t(a.ids[own + min(j0 + q, a.topk - 1)]);
            n[q] = 0;
        }
        // a slot before counts where its expert is not above, one from the slot on
        // where it is below; an unrouted id is above every expert
        each_id<NT, 2>(a.ids, a.R, [&](int i, int id) {
#pragma unroll
            for (int q = 0; q < kAt; ++q) n[q] += uint32_t(id) < e[q] + (i < own + j0 + q ? 1u : 0u) ? 1 : 0;
        });
        int mine = 0;                                      // lane q: slot j0 + q
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            const int sum = e[q] < uint32_t(a.E) ? wave_sum(n[q]) : -1;
            if (lane == q) mine = sum;
        }
        if (lane < kAt && j0 + lane < a.topk) atomicAdd(&pos[j0 + lane], mine);
    }
}

// inv of slots first .. last - 1 by one wave, given each expert's next position and
// the ids of the first 64 slots; also into pos[0 ..] where that is not null
__device__ __forceinline__ void place_slots(const SortArgs& a, int first, int last, int e, int* next, int* pos) {
    const int lane = threadIdx.x & 63;
    const uint64_t lower = (uint64_t(1) << lane) - 1;
    const int bits = a.E > 1 ? 32 - __clz(a.E - 1) : 0;
    for (int i = first; i < last; i += 64) {
        const int f = i + lane;
        if (i > first) e = f < last ? a.ids[f] : -1;
        const bool routed = uint32_t(e) < uint32_t(a.E);
        const uint64_t same = peers(e, routed, bits);
        int at = -1;
        if (routed) {
            const int to = next[e];
            at = to + __popcll(same & lower);
            // every lane's read of next[e] precedes the first one's update (one wave, in order)
            if ((same & lower) == 0) next[e] = to + __popcll(same);
        }
        if (f < last) {
            a.inv[f] = at;
            if (pos) pos[f - first] = at;
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
__global__ __launch_bounds__(kPlaceThreads) void sort_place_kernel(SortArgs a, int slots, int blocks) {
    constexpr int kPer = kMaxE / kPlaceThreads, kWaves = kPlaceThreads / 64;
    __shared__ int run[kWaves * kMaxE];     // a wave's next position in each expert
    __shared__ int before[kMaxE], total[kMaxE];
    __shared__ int s_scan[kWaves];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kWaves * a.E; i += kPlaceThreads) run[i] = 0;
    for (int e = threadIdx.x; e < kMaxE; e += kPlaceThreads) before[e] = total[e] = 0;
    __syncthreads();
    // a wave's slots: a contiguous part of the block's, a multiple of 64
    const int64_t base = int64_t(blockIdx.x) * slots + wv * (slots / kWaves);
    const int first = int(min(int64_t(a.R), base)), last = int(min(int64_t(a.R), base + slots / kWaves));
    int* const mine = run + wv * a.E;
    for (int i = first; i < last; i += 64) {
        const int e = i + lane < last ? a.ids[i + lane] : -1;
        if (uint32_t(e) < uint32_t(a.E)) atomicAdd(&mine[e], 1);
    }
    // the blocks' counts: threads of `step` experts side by side, the rest over the blocks
    int step = 64;
    while (step < a.E && step < kPlaceThreads) step <<= 1;
    for (int e = threadIdx.x % step; e < a.E; e += step) {
        int b = 0, n = 0;
#pragma unroll 8
        for (int q = threadIdx.x / step; q < blocks; q += kPlaceThreads / step) {
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
    int at = scan_start<kWaves>(n, s_scan);
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
    if (blockIdx.x == 0 && a.E == kMaxE && threadIdx.x == kPlaceThreads - 1) a.offsets[kMaxE] = at;
    __syncthreads();
    place_slots(a, first, last, first + lane < last ? a.ids[first + lane] : -1, mine, nullptr);
}

// ---------------------------------------------------------------------------
// rows on their way: pieces of 16 bytes (copied) or of 16 columns (quantised),
// which leave as 16 bytes either way
// ---------------------------------------------------------------------------
template <SortMode kMode>
struct Piece {
    static constexpr int kLoads = kMode == kSortCopy ? 1 : 2;
    i32x4 v[kLoads];
    __device__ __forceinline__ void load(const uint8_t* row, int u) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = *reinterpret_cast<const i32x4*>(row + int64_t(u * kLoads + i) * 16);
    }
};

// the row's pieces u0, u0 + stride, .. below u1 (CH of them in p) to the
// positions of the token's slots.  kSortInt8: bits is the row's largest magnitude;
// kSortFp8: a lane's piece and its neighbours' make whole groups.  kWaves: a wave's
// lanes have one token.
template <SortMode kMode, int CH, bool kWaves, bool kPast>
__device__ __forceinline__ void store_pieces(const SortArgs& a, const Piece<kMode> (&p)[CH], const int* pos, int u0,
                                             int u1, int stride, uint32_t bits) {
    i32x4 out[CH];
    float s[CH], inverse = 0.0f;
    if constexpr (kMode == kSortInt8) s[0] = int8_scale(bits, inverse);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (kMode == kSortCopy) {
            out[c] = p[c].v[0];
        } else if constexpr (kMode == kSortInt8) {
            const uint2 lo = int8_codes(p[c].v[0], inverse), hi = int8_codes(p[c].v[1], inverse);
            out[c] = i32x4{int(lo.x), int(lo.y), int(hi.x), int(hi.y)};
        } else {
            s[c] = quant16(p[c].v[0], p[c].v[1], out[c]);
        }
    }
    for (int j = 0; j < a.topk; ++j) {
        const int at = kWaves ? __builtin_amdgcn_readfirstlane(pos[j]) : pos[j];
        if (at < 0) continue;
        uint8_t* to = a.rows + int64_t(at) * a.units * 16;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = u0 + c * stride;
            if (u < u1) {
                store16<kPast>(to + int64_t(u) * 16, out[c]);
                if (kMode == kSortFp8 && (u & 7) == 0) a.row_scales[int64_t(at) * a.scales + (u >> 3)] = s[c];
            }
        }
        if (kMode == kSortInt8 && u0 == 0) a.row_scales[at] = s[0];
    }
}

// the scales of a token's codes by `lanes` lanes, whose first ones were read ahead
__device__ __forceinline__ float first_scale(const SortArgs& a, int64_t token, int lane) {
    return lane < a.scales ? a.x_scale[token * a.scales + lane] : 0.0f;
}
__device__ __forceinline__ void copy_scales(const SortArgs& a, int64_t token, const int* pos, int lane, int lanes,
                                            float first) {
    for (int i = lane; i < a.scales; i += lanes) {
        const float s = i == lane ? first : a.x_scale[token * a.scales + i];
        for (int j = 0; j < a.topk; ++j)
            if (pos[j] >= 0) a.row_scales[int64_t(pos[j]) * a.scales + i] = s;
    }
}

// A token's row (kSortInt8) or a part of it by a workgroup.  kOne: the positions
// are found here, and further workgroups write the offsets.
template <SortMode kMode, int NT, int CH, bool kOne, bool kPast>
__global__ __launch_bounds__(NT) void sort_move_kernel(SortArgs a, int parts, int span) {
    __shared__ int pos[MOE_MAX_TOPK];
    __shared__ uint32_t s_max[NT / 64];
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t token = wg / parts;
    if (token >= a.T) {                                    // the whole workgroup alike
        const int64_t x = wg - int64_t(a.T) * parts;
        if (kOne && x < offset_groups(a.R, a.E)) write_offsets<NT>(a, int(x));
        return;
    }
    const int t = int(token), part = int(wg - token * parts);
    const int u0 = part * span + threadIdx.x, u1 = min(a.units, (part + 1) * span);
    Piece<kMode> p[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c)                           // behind the part: its last piece again
        p[c].load(a.x + token * a.units * (16 * Piece<kMode>::kLoads), min(u0 + c * NT, u1 - 1));
    const float scale = kMode == kSortCopy && part == 0 ? first_scale(a, token, threadIdx.x) : 0.0f;
    if constexpr (kOne) {
        if (threadIdx.x < unsigned(a.topk)) pos[threadIdx.x] = 0;
        __syncthreads();
        find_positions<NT>(a, t, pos);
    } else {
        if (threadIdx.x < unsigned(a.topk)) pos[threadIdx.x] = a.inv[token * a.topk + threadIdx.x];
    }
    uint32_t bits = 0;
    if constexpr (kMode == kSortInt8) {
#pragma unroll
        for (int c = 0; c < CH; ++c) bits = pk_max_u16(bits, pk_max_u16(abs_max8(p[c].v[0]), abs_max8(p[c].v[1])));
        bits = lanes_max_u16<64>(bits);
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = bits;
    }
    __syncthreads();
    if (kOne && part == 0 && threadIdx.x < unsigned(a.topk))
        a.inv[token * a.topk + threadIdx.x] = max(pos[threadIdx.x], -1);
    if constexpr (kMode == kSortInt8) {
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) bits = max(bits, s_max[i]);
    }
    store_pieces<kMode, CH, true, kPast>(a, p, pos, u0, u1, NT, bits);
    if (kMode == kSortCopy && part == 0) copy_scales(a, token, pos, threadIdx.x, NT, scale);
}

// The counted form's rows of L pieces or fewer, L lanes to a token
template <SortMode kMode, int L, bool kPast>
__global__ __launch_bounds__(kThreads) void sort_narrow_kernel(SortArgs a) {
    const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t mine = wg * (kThreads / L) + threadIdx.x / L, token = min(mine, int64_t(a.T) - 1);
    const int u = threadIdx.x % L;
    Piece<kMode> p[1];
    p[0].load(a.x + token * a.units * (16 * Piece<kMode>::kLoads), min(u, a.units - 1));
    const float scale = kMode == kSortCopy ? first_scale(a, token, u) : 0.0f;
    uint32_t bits = 0;
    if constexpr (kMode == kSortInt8)
        bits = lanes_max_u16<L>(pk_max_u16(abs_max8(p[0].v[0]), abs_max8(p[0].v[1])));
    if (mine >= a.T) return;
    const int* const pos = a.inv + token * a.topk;
    store_pieces<kMode, 1, false, kPast>(a, p, pos, u, a.units, L, bits);
    if (kMode == kSortCopy) copy_scales(a, token, pos, u, L, scale);
}

// Tokens first .. first + per - 1 by a workgroup, L lanes to a token's row (up to 64
// for one of as many pieces or fewer) or, of long rows that are not int8's, a part of
// `span` pieces of it.  The workgroup counts all ids by expert, those before its own
// slots apart, in `1 << rep` copies (lanes of one expert add to different ones), and
// ranks its own slots; its first rows are on their way meanwhile.  Two waves to a long
// row: 1031 x 4096 to int8 12.7 us, one 14.5, four 12.8; 4000 tokens 32.7 / 36.8 / 31.9
// (11.3 and 30.3 since the ids are on their way before the counters are cleared).
template <SortMode kMode, int CH, int L, bool kPast>
__global__ __launch_bounds__(kBatchThreads) void sort_batch_kernel(SortArgs a, int per, int rep, int span) {
    constexpr int NT = kBatchThreads, kPer = kMaxE / NT, kTeams = NT / L, kWaves = L / 64;
    static_assert(L <= 64 ? CH == 1 : L % 64 == 0, "lanes");
    // [before, from][E][1 << rep], then a slot's next position in each expert
    __shared__ __attribute__((aligned(16))) int count[2 * kMaxE];
    __shared__ int pos[kBatchSlots];
    __shared__ int s_scan[NT / 64];
    __shared__ uint32_t s_max[2][NT / 64];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int team = L >= 64 ? wv / kWaves : int(threadIdx.x) / L, at_row = threadIdx.x % L;
    const int first = blockIdx.x * per, last = min(a.T, first + per);
    const int64_t row_bytes = int64_t(a.units) * (16 * Piece<kMode>::kLoads);
    const int u0 = int(blockIdx.y) * span, u1 = min(a.units, u0 + span);
    Piece<kMode> p[CH];
    float scale = 0.0f;
    auto load = [&](int t, int u) {                        // behind the part: its last piece again
#pragma unroll
        for (int c = 0; c < CH; ++c) p[c].load(a.x + t * row_bytes, min(u + at_row + L * c, u1 - 1));
        if (kMode == kSortCopy && u == 0) scale = first_scale(a, t, at_row);
    };
    EachId<NT, 8> ids(a.ids, a.R);
    ids.load_first();
    const int own = first * a.topk, copy = lane & ((1 << rep) - 1);
    const int own_id = own + lane < last * a.topk ? a.ids[own + lane] : -1;
    load(min(first + team, a.T - 1), u0);

    for (int i = threadIdx.x; i < 2 * kMaxE; i += NT) count[i] = 0;
    __syncthreads();
    ids.each([&](int i, int id) {
        if (uint32_t(id) < uint32_t(a.E)) atomicAdd(&count[((i >= own ? a.E : 0) + id << rep) + copy], 1);
    });
    __syncthreads();
    int before[kPer], n[kPer];
    auto add_copies = [&](auto copies) {
        constexpr int C = decltype(copies)::value;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            before[i] = n[i] = 0;
            if (e < a.E) {
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    before[i] += count[e * C + r];
                    n[i] += count[(a.E + e) * C + r];
                }
                n[i] += before[i];
            }
        }
    };
    if (rep == 0) add_copies(std::integral_constant<int, 1>());
    else if (rep == 1) add_copies(std::integral_constant<int, 2>());
    else if (rep == 2) add_copies(std::integral_constant<int, 4>());
    else add_copies(std::integral_constant<int, 8>());
    int at = scan_start<NT / 64>(n, s_scan);               // (a barrier behind every read of count)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (blockIdx.x == 0 && e <= a.E) a.offsets[e] = at;
        if (e < a.E) count[e] = at + before[i];
        at += n[i];
    }
    if (blockIdx.x == 0 && a.E == kMaxE && threadIdx.x == NT - 1) a.offsets[kMaxE] = at;
    __syncthreads();
    if (wv == 0) place_slots(a, own, last * a.topk, own_id, count, pos);
    __syncthreads();
    const bool whole = u1 - u0 <= L * CH;                  // the part in the team's registers
    for (int k = 0; k * kTeams < per; ++k) {               // every wave as often: there is a barrier in it
        const int t = first + team + k * kTeams;
        bool loaded = k == 0;
        uint32_t bits = 0;
        if constexpr (kMode == kSortInt8) {
            for (int u = u0; u < u1 && t < last; u += L * CH) {
                if (!loaded) load(t, u);
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    bits = pk_max_u16(bits, pk_max_u16(abs_max8(p[c].v[0]), abs_max8(p[c].v[1])));
                loaded = whole;
            }
            bits = lanes_max_u16<(L < 64 ? L : 64)>(bits);
            if constexpr (L > 64) {
                if (lane == 0) s_max[k & 1][wv] = bits;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWaves; ++i) bits = max(bits, s_max[k & 1][team * kWaves + i]);
            }
        }
        if (t >= last) continue;
        const int* mine = pos + (t - first) * a.topk;
        for (int u = u0; u < u1; u += L * CH) {
            if (!loaded) load(t, u);
            store_pieces<kMode, CH, L >= 64, kPast>(a, p, mine, u + at_row, u1, L, bits);
            loaded = false;
        }
        if (kMode == kSortCopy && u0 == 0) copy_scales(a, t, mine, at_row, L, scale);
    }
}

template <SortMode kMode, bool kPast>
hipError_t launch_batch(const SortArgs& a, hipStream_t s) {
    const int per = batch_tokens(a.T);
    const int span = kMode == kSortInt8 ? a.units : kBatchSpan;
    int rep = 0;
    while (rep < 3 && (2 * a.E << (rep + 1)) <= 2 * kMaxE) ++rep;
    const int most = std::min(a.units, span);
    void (*kern)(SortArgs, int, int, int) = most <= 8     ? sort_batch_kernel<kMode, 1, 8, kPast>
                                            : most <= 16  ? sort_batch_kernel<kMode, 1, 16, kPast>
                                            : most <= 32  ? sort_batch_kernel<kMode, 1, 32, kPast>
                                            : most <= 64  ? sort_batch_kernel<kMode, 1, 64, kPast>
                                            : most <= 128 ? sort_batch_kernel<kMode, 1, 128, kPast>
                                            : most <= 256 ? sort_batch_kernel<kMode, 2, 128, kPast>
                                            : most <= 512 ? sort_batch_kernel<kMode, 4, 128, kPast>
                                                          : sort_batch_kernel<kMode, 8, 128, kPast>;
    const dim3 grid((a.T + per - 1) / per, (a.units + span - 1) / span);
    return start(kern, grid, kBatchThreads, s, a, per, rep, span);
}

template <SortMode kMode, bool kPast>
hipError_t launch_narrow(const SortArgs& a, hipStream_t s) {
    const int lanes = a.units <= 8 ? 8 : a.units <= 16 ? 16 : a.units <= 32 ? 32 : 64;
    void (*kern)(SortArgs) = lanes == 8    ? sort_narrow_kernel<kMode, 8, kPast>
                             : lanes == 16 ? sort_narrow_kernel<kMode, 16, kPast>
                             : lanes == 32 ? sort_narrow_kernel<kMode, 32, kPast>
                                           : sort_narrow_kernel<kMode, 64, kPast>;
    return start(kern, grid_of((int64_t(a.T) * lanes + kThreads - 1) / kThreads), kThreads, s, a);
}

template <SortMode kMode, int NT, int CH>
hipError_t launch_move(const SortArgs& a, bool counted, hipStream_t s) {
    // parts of at most NT * CH pieces, of equal length but for the rounding to whole groups
    const int parts = kMode == kSortInt8 ? 1 : (a.units + NT * CH - 1) / (NT * CH);
    const int span = kMode == kSortInt8 ? a.units : ((a.units + parts - 1) / parts + 7) / 8 * 8;
    const int batch_parts = kMode == kSortInt8 ? 1 : (a.units + kBatchSpan - 1) / kBatchSpan;
    if (!counted && !few_ids(a.T, a.topk, parts, batch_parts, a.units))
        return a.past ? launch_batch<kMode, true>(a, s) : launch_batch<kMode, false>(a, s);
    if (counted && a.units <= 64)
        return a.past ? launch_narrow<kMode, true>(a, s) : launch_narrow<kMode, false>(a, s);
    const int64_t n = int64_t(a.T) * parts + (counted ? 0 : offset_groups(a.R, a.E));
    void (*kern)(SortArgs, int, int) = !counted ? sort_move_kernel<kMode, NT, CH, true, false>
                                       : a.past ? sort_move_kernel<kMode, NT, CH, false, true>
                                                : sort_move_kernel<kMode, NT, CH, false, false>;
    return start(kern, grid_of(n), NT, s, a, parts, span);
}

hipError_t launch_move(const SortArgs& a, SortMode mode, bool counted, hipStream_t s) {
    if (mode == kSortCopy) return launch_move<kSortCopy, 256, 1>(a, counted, s);
    if (mode == kSortFp8) return launch_move<kSortFp8, 256, 1>(a, counted, s);
    if (a.units <= 256) return launch_move<kSortInt8, 256, 1>(a, counted, s);
    if (a.units <= 512) return launch_move<kSortInt8, 256, 2>(a, counted, s);
    if (a.units <= 1024) return launch_move<kSortInt8, 256, 4>(a, counted, s);
    static_assert(MOE_MAX_INT8_K <= 1024 * 2 * 16, "a row in one workgroup's registers");
    return launch_move<kSortInt8, 1024, 2>(a, counted, s);
}

}  // namespace

SortPlan plan_sort(int64_t R) {
    if (R <= kBatchMostSlots) return {0, 0};
    // 1024 slots a block, more where there would be over kMostBlocks of them (a
    // block reads the counts of all)
    const int64_t slots = (R / kMostBlocks + kPlaceThreads) / kPlaceThreads * kPlaceThreads;
    return {int(slots), int((R + slots - 1) / slots)};
}

hipError_t launch_sort_rows(const SortArgs& all, SortMode mode, hipStream_t s) {
    // us as they are / past (8 slots, bf16 rows, and with moe_combine_rows behind): 224 MiB
    // 39.6 / 51.5 (82 / 97), 448 MiB 106 / 99 (229 / 193), 896 MiB 213 / 187 (432 / 368): x,
    // an eighth of it, stays in the cache for all its reads.  Where x is not there to begin
    // with, 213 / 216.
    SortArgs a = all;
    a.past = int64_t(a.R) * a.units * 16 >= kLastCacheBytes && whole_lines(a.rows, int64_t(a.units) * 16);
    const SortPlan p = plan_sort(a.R);
    if (p.blocks == 0) return launch_move(a, mode, false, s);
    hipError_t e = start(sort_count_kernel, dim3(p.blocks), kThreads, s, a, p.slots);
    if (e == hipSuccess) e = start(sort_place_kernel, dim3(p.blocks), kPlaceThreads, s, a, p.slots, p.blocks);
    return e == hipSuccess ? launch_move(a, mode, true, s) : e;
}

}  // namespace moe
