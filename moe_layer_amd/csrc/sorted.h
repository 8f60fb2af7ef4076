// Launchers and shared device code of the operators that sort a batch by
// expert and bring it back (sort_rows.hip, combine_rows.hip) and that quantise
// rows to int8 (quant_int8.hip).
#pragma once

#include <algorithm>
#include <type_traits>

#include "dense.h"

namespace moe {

// What moe_sort_rows does with a row on its way
enum SortMode { kSortCopy, kSortInt8, kSortFp8 };

struct SortArgs {
    const uint8_t* x;          // [T, row_bytes]
    const float* x_scale;      // [T, scales] (codes) or null
    const int32_t* ids;        // [T, topk]
    uint8_t* rows;             // [T * topk] rows of row_bytes (copy) or cols codes
    float* row_scales;         // [T * topk, scales] or null
    int32_t* offsets;          // [E + 1]
    int32_t* inv;              // [T, topk]
    int32_t* counts;           // scratch [blocks, E]
    int T, topk, E, R;         // R = T * topk
    int units;                 // 16-byte pieces of a row of `rows`
    int scales;                // scales of a row that is copied or made
    bool past;                 // rows are stored past the caches' replacement (but in the few-ids form)
};
// slots per block of the counted form, and its blocks; 0 blocks where the
// positions are found without counts
struct SortPlan {
    int slots, blocks;
};
SortPlan plan_sort(int64_t R);

// Ids up to which a wave holds them all, for the positions of a token's slots, and
// workgroups of 16 experts each compare them, for the offsets; more are counted in LDS
// (us in a graph, 8 of 256 experts, to int8, held / counted: 16 x 4096 3.6 / 4.9, 64 x
// 4096 3.9 / 5.2, 128 x 4096 4.4 / 4.9).
constexpr int kHeldIds = 1024;
// slots of a token whose positions are found with one look at all of more ids
constexpr int kSlotsAtOnce = 8;
// tokens of a workgroup of the batch form: about 512 workgroups
constexpr int batch_tokens(int T) { return std::max((T + 2047) / 2048, 1) * 4; }

// Whether the workgroups that move `parts` parts of every token's row of `units` pieces
// compare its slots with all ids themselves, or, in the batch form, `batch_parts` parts
// to a workgroup's tokens, count the ids for several tokens at once.  Comparing reads
// all ids again for every kSlotsAtOnce slots.  That many reads in all are made in the
// time of the batch form's start where it has workgroups enough; fewer than 96 of them
// take longer, for their tokens have all slots' rows to store.  And one workgroup's
// reads, one after the other, take the time of its row.
// us, comparing / batch, with the reads in all, of 256 experts: 8 slots: 256 x 7168 (2.1 M)
// 9.7 / 11.3, 320 x 7168 (3.3) 11.9 / 12.2, 400 (5.1) 15.0 / 13.3, 512 x 4096 to int8 (2.1)
// 9.0 / 9.1, 700 (3.9) 12.7 / 10.0; 16 slots: 128 x 7168 (2.1) 10.9 / 14.4, 256 x 7168 (8.4)
// 19.0 / 15.8; 64 slots: 32 x 7168 (2.1) 23.7 / 35.1, 32 x 2048 (0.5) 22.2 / 15.2, 64 x 16384
// (17) 44 / 41, 256 x 2048 (34) 81 / 20, 256 x 7168 (134) 153 / 42.  Over 1082 shapes from
// 1 to 1000 tokens of 512 to 65536 columns 0.7 % slower than the faster form in the
// geometric mean, 32 % at worst.
constexpr bool few_ids(int T, int topk, int parts, int batch_parts, int units) {
    const int64_t R = int64_t(T) * topk;
    const int64_t reads = R * (R > kHeldIds ? (topk + kSlotsAtOnce - 1) / kSlotsAtOnce : 1);
    const int64_t batch = int64_t((T + batch_tokens(T) - 1) / batch_tokens(T)) * batch_parts;
    return reads <= 6144 * int64_t((units + 255) / 256) &&
           T * reads * parts * std::min<int64_t>(batch, 96) <= (int64_t(5) << 19) * 96;
}

hipError_t launch_sort_rows(const SortArgs& a, SortMode mode, hipStream_t s);

struct CombineArgs {
    const uint16_t* rows;      // bf16 [num_rows, cols]
    const int32_t* inv;        // [T, topk]
    const float* weights;      // [T, topk] or null
    uint16_t* out;             // bf16 [T, cols]
    const uint16_t* grad_out;  // bf16 [T, cols]
    uint16_t* grad_rows;       // bf16 [num_rows, cols]
    float* grad_weights;       // [T, topk] or null
    int T, topk, cols, num_rows;
    bool past;                 // rows (and grad_rows) go past the caches' replacement
};
hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s);
hipError_t launch_combine_rows_bwd(const CombineArgs& a, hipStream_t s);

struct Int8Args {
    const uint16_t* x;         // bf16 [rows, cols], gated: [rows, 2 cols]
    int8_t* codes;             // [rows, cols]
    float* scales;             // [rows]
    int rows, cols;
    float limit;
    bool past;                 // x is read past the caches' replacement
};
hipError_t launch_quant_int8(const Int8Args& a, bool gated, hipStream_t s);

// The last-level (Infinity) cache.  Rows that are streamed once and are as many bytes
// go past the replacement of the caches: a stream that cannot stay there reads at up to
// 6.5 TB/s and is written at up to 6, instead of 5.1, and evicts nothing; smaller ones
// stay for the kernel that comes next.
// Written so only where rows are whole lines, and read so where they are that or long:
// lines that two rows share should meet in a cache (us as they are / past, called on the
// same rows again, so that x or the output is in the last-level cache: 8192 tokens of 8
// slots, sort 7168 columns 208 / 184, 7176 246 / 249, 5000 166 / 176, 65536 of 1000
// 277 / 295; combine 204 / 177, 203 / 185, 142 / 130, 226 / 215, 200000 of 328 226 / 234).
constexpr int64_t kLastCacheBytes = int64_t(256) << 20;
inline bool whole_lines(const void* rows, int64_t row_bytes) {
    return (reinterpret_cast<uintptr_t>(rows) | uintptr_t(row_bytes)) % 128 == 0;
}
inline bool reads_past(const void* rows, int64_t row_bytes) {
    return whole_lines(rows, row_bytes) || row_bytes >= 1536;
}

namespace {

// (kPast is no argument: of two accesses that differ in their caching alone the
// compiler makes a plain one)
template <bool kPast>
__device__ __forceinline__ i32x4 load16(const void* from) {
    const i32x4* p = static_cast<const i32x4*>(from);
    if constexpr (kPast) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool kPast>
__device__ __forceinline__ void store16(void* to, const i32x4& v) {
    i32x4* p = static_cast<i32x4*>(to);
    if constexpr (kPast) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// f(std::bool_constant<b>())
template <typename F>
auto pick(bool b, F f) {
    return b ? f(std::true_type()) : f(std::false_type());
}

// ---------------------------------------------------------------------------
// int8 rows: m = max(|v|max, 1e-10), scale = fl32(m / 127), and the code of v
// the whole number nearest to v fl32(127 / m) (ties to even; at most 127)
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t abs_max8(const i32x4& w) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return pk_max_u16(pk_max_u16(uint32_t(w[0]) & kAbs, uint32_t(w[1]) & kAbs),
                      pk_max_u16(uint32_t(w[2]) & kAbs, uint32_t(w[3]) & kAbs));
}
// the largest half of L neighbouring lanes' words, in each of them; the bits of a
// bf16 without their sign order as the magnitudes do
template <int L>
__device__ __forceinline__ uint32_t lanes_max_u16(uint32_t m) {
    static_assert(L == 8 || L == 16 || L == 32 || L == 64, "lanes");
    m = dpp_max_u16<0xb1>(m);                              // quad_perm [1,0,3,2]
    m = dpp_max_u16<0x4e>(m);                              // quad_perm [2,3,0,1]
    m = dpp_max_u16<0x141>(m);                             // row_half_mirror
    if constexpr (L > 8) m = dpp_max_u16<0x140>(m);        // row_mirror
    if constexpr (L > 16) {
        const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
        m = pk_max_u16(a[0], a[1]);
    }
    if constexpr (L > 32) {
        const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        m = pk_max_u16(b[0], b[1]);
    }
    return max(m & 0xffffu, m >> 16);
}
// scale and inverse from the row's largest magnitude (its bf16 bits); a row with
// an infinity or a NaN gets the scale NaN, so what is made of it is NaN
__device__ __forceinline__ float int8_scale(uint32_t bits, float& inverse) {
    const float m = fmaxf(__uint_as_float(bits << 16), 1e-10f);
    inverse = __fdiv_rn(127.0f, m);
    return bits >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(m, 127.0f);
}
// codes of 8 packed bf16 values.  v inverse + 1.5 2^23 is rounded once, to a whole
// number (ties to even), whose low byte is the code.
__device__ __forceinline__ uint2 int8_codes(const i32x4& w, float inverse) {
    constexpr float kWhole = 12582912.0f;
    uint32_t pair[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        pair[q] = __builtin_amdgcn_perm(__float_as_uint(__builtin_fmaf(bf16_hi(w[q]), inverse, kWhole)),
                                        __float_as_uint(__builtin_fmaf(bf16_lo(w[q]), inverse, kWhole)), 0x0c0c0400u);
    return uint2{pair[0] | pair[1] << 16, pair[2] | pair[3] << 16};
}

// fp8 codes and scale, moe_quant_act's bit for bit, of 16 columns by each of 8
// neighbouring lanes, which hold a 128-column group; returns the scale.  Its maximum
// passes over a NaN, whose code is -448's, and an infinity makes the scale infinite and
// its inverse 0.
__device__ __forceinline__ float quant16(const i32x4& a, const i32x4& b, i32x4& codes) {
    uint32_t m = pk_max_u16(abs_max8(a), abs_max8(b));
    m = dpp_max_u16<0xb1>(m);                              // quad_perm [1,0,3,2]
    m = dpp_max_u16<0x4e>(m);                              // quad_perm [2,3,0,1]
    m = dpp_max_u16<0x141>(m);                             // row_half_mirror
    m = max(m & 0xffffu, m >> 16);
    if (m > 0x7f80u) {                                     // a NaN, above every number's bits (the 8 lanes alike)
        auto number = [](uint32_t h) { return h > 0x7f80u ? 0u : h; };
        m = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            m = max(max(m, number(uint32_t(a[q]) & 0x7fffu)), number(uint32_t(a[q]) >> 16 & 0x7fffu));
            m = max(max(m, number(uint32_t(b[q]) & 0x7fffu)), number(uint32_t(b[q]) >> 16 & 0x7fffu));
        }
        m = dpp_max_u16<0x141>(dpp_max_u16<0x4e>(dpp_max_u16<0xb1>(m)));
    }
    const float s = fp8_group_scale(__uint_as_float(m << 16));
    // 1 / s, as in quant8; an infinity's mirrored exponent is below 0
    const float inv = __int_as_float(max(int(254u << 23) - __float_as_int(s), 0));
    // the clamp is for what no number is: the middle of three takes a NaN for the lowest
    auto code = [&](float v) { return __builtin_amdgcn_fmed3f(__fmul_rn(v, inv), -448.0f, 448.0f); };
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t w0 = uint32_t(q < 2 ? a[2 * q] : b[2 * q - 4]), w1 = uint32_t(q < 2 ? a[2 * q + 1] : b[2 * q - 3]);
        codes[q] = int(pack_e4m3(code(bf16_lo(w0)), code(bf16_hi(w0)), code(bf16_lo(w1)), code(bf16_hi(w1))));
    }
    return s;
}

}  // namespace

}  // namespace moe
