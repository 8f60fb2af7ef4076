// LDS-tiled dense and grouped products (see gemm_split.hip for the products and
// the operand sides).
//
// A workgroup owns BW weight rows x BT token rows of one group.  A stage is
// 128 bytes of K of every row (128 e4m3 or 64 bf16 elements, one fp8 scale
// block), moved global -> LDS with direct-to-LDS loads of 8 whole 128-byte row
// pieces into an S-slot ring, S - 1 stages ahead; each wave waits for its own
// loads, then one barrier per stage publishes the slot and frees the one read
// before.  LDS rows are 128 bytes with chunk c of row r at position
// c ^ (r & 7), so the 8 lanes that read 8 rows at one chunk hit all banks.
//
// fp8: the codes are converted to bf16 on their way from LDS to the matrix cores
// (Operand); a stage's products p, four MFMAs per 16 x 16 tile, are folded with
// acc += (a_scale w_scale) p.  The scales of 8 stages at a time sit in a two-slot
// LDS table that is filled along with the ring.
//
// What bounds it: at 8192 x 4096 x 7168 fp8 (410 us, 1.17 PFLOP/s; a library
// product of bf16 operands of that size 363 us, this file's bf16 form 373) the
// bf16 matrix cores are busy for 48 % of the cycles (counted in a profiled run)
// and the vector unit, two conversions and a fold a matrix instruction, for most
// of the rest:
// without the conversions it took 350 of 422 us, without the folds 386, without
// the loads 383.  Tiles of 256 x 256, which convert a quarter less, spill (620 us).
// Reading a stage's first operands in the stage before, 32 x 32 subtiles and loads
// spread between the products together gave 0-5 % and were not kept.  Large
// groups (32768 x 4096 x 1536 bf16 in 128: 515 us, 0.8 PFLOP/s) are bound by the
// bytes that leave the Infinity Cache and HBM, 2.2 GB read of 1.7 GB operands and
// 0.27 written at 4.8 TB/s, with 4-5 us a tile in which a workgroup stores its
// outputs and computes nothing.
#include "dev_rows.h"

namespace moe {

namespace {

// Weight tiles that an XCD's workgroups of one time share with some row blocks
// (256 x 256 tiles, 2 / 4 / 8 / 16: 32768 x 4096 x 1536 in 128 bf16 groups
// 542 / 530 / 530 / 542 us).
constexpr int kBand = 4;

// Bytes of LDS: the ring and the scale table's two slots
template <bool FP8, int BW, int BT, int S>
constexpr int tile_lds() {
    const int rows = FP8 ? (BT + (BW + 127) / 128 + 7) / 8 * 8 : 0;
    return S * (BW + BT) * 128 + 2 * rows * 32;
}

// One tile: weight rows n0 .. n0 + BW - 1 against rows row0 .. min(row0 + BT, row1) - 1 of group e
template <bool FP8, int BW, int BT, int WW, int WT, int S, bool NTW>
__device__ __forceinline__ void tile_product(const RowsGemmArgs& g, lds_t* ring, int e, int row0, int row1, int n0) {
    constexpr int W = WW * WT;
    constexpr int SA = BW / WW / 16, SB = BT / WT / 16;      // 16-row subtiles per wave
    constexpr int kPieces = (BW + BT) / 8;                   // 1 KB loads per stage
    constexpr int NL = (kPieces + W - 1) / W;                // loads per wave per stage
    constexpr int kSlot = (BW + BT) * 128;
    // A ring of two, bf16: every wave has the tokens in registers by the first
    // subtile row and half of its weight rows half-way through the stage, so a
    // second barrier there lets three quarters of the stage after next start
    // (32768 x 4096 x 1536, 128 groups 589 -> 575 us).
    constexpr bool kEarly = !FP8 && S == 2;
    constexpr int kHalf0 = NL - BW / 16 / W;                 // its loads of half 0
    static_assert(!kEarly || 2 * 8 * W == BW / WW, "halves of a wave's weight rows");
    constexpr int kScaleRows = FP8 ? (BT + (BW + 127) / 128 + 7) / 8 * 8 : 0;
    constexpr int kTab = kScaleRows * 32;                    // 8 stages of fp32 scales per row
    constexpr int kParts = (kScaleRows / 8 + W - 1) / W;     // table loads per wave per 8 stages
    static_assert((BW / 8) % W == 0 && S >= 2 && S - 1 + kParts <= 8, "tile shape");
    static_assert(W * 16 * kOutRow<BW / WW> <= S * kSlot, "outputs in the ring's place");
    lds_t* const tab = ring + S * kSlot;

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wv % WW, wt = wv / WW;
    const int lr = lane & 15, lk = lane >> 4;
    const int64_t kbytes = int64_t(g.K) * (FP8 ? 1 : 2);
    const int steps = int(kbytes >> 7);

    const uint8_t* wbase = g.w + (int64_t(e) * g.N + n0) * kbytes;
    const uint8_t* abase = g.a + int64_t(row0) * kbytes;
    uint32_t off[NL];                                        // this lane's bytes of each piece
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const int r = 8 * min(wv + W * j, kPieces - 1) + (lane >> 3);
        const int src = j < BW / 8 / W ? min(r, g.N - 1 - n0) : min(r - BW, row1 - 1 - row0);
        off[j] = uint32_t(src) * uint32_t(kbytes) + (((lane & 7) ^ (lane >> 3)) << 4);
    }
    auto load = [&](int st, int j) {
        const uint8_t* base = (j < BW / 8 / W ? wbase : abase) + (int64_t(st) << 7);
        load_piece<NTW>(base + off[j], ring + (st % S) * kSlot + min(wv + W * j, kPieces - 1) * 1024, j < BW / 8 / W);
    };
    // pieces of half 0: the tokens and the first half of each wave's weight rows; of half 1: the rest
    auto half_of = [](int j) { return j < BW / 8 / W ? j & 1 : 0; };
    auto issue = [&](int st, int half) {
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (half < 0 || half == half_of(j)) load(st, j);
    };
    // held in scalars: a lane's choice between two kernel arguments would be a
    // load of its own, and its wait one for every load in flight
    const float *a_scale = g.a_scale, *w_scale = g.w_scale;
    asm("" : "+s"(a_scale), "+s"(w_scale));
    // part p of the scales of stages 8 c .. 8 c + 7: one load of 8 table rows
    auto issue_scales = [&](int c, int p) {
        if constexpr (FP8) {
            const int piece = min(wv + W * p, kScaleRows / 8 - 1);
            const int r = 8 * piece + (lane >> 3);
            const int nb = (g.N + 127) >> 7;
            const int64_t row = r < BT ? min(row0 + r, row1 - 1)
                                       : int64_t(e) * nb + min((n0 >> 7) + r - BT, nb - 1);
            const float* src = (r < BT ? a_scale : w_scale) + row * steps + min(8 * c + (lane & 7), steps - 1);
            __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(src), tab + (c & 1) * kTab + piece * 256, 4,
                                             0, 0);
        }
    };
    // the loads of stage st; its chunk of 8 stages starts the next one's scales
    // once the chunk before is out of use (S - 1 stages in)
    auto issue_stage = [&](int st, int half) {
        if constexpr (FP8) {
            const int p = (st & 7) - (S - 1);
            if (half != 0 && p >= 0 && p < kParts && (st >> 3) * 8 + 8 < steps) issue_scales((st >> 3) + 1, p);
        }
        issue(st, half);
    };
    // stage s has landed; fewer loads than are in flight at most: the table's
    // come before a stage's own
    auto wait_stage = [&](int s) {
        if constexpr (!kEarly) wait_stages<NL, S - 2>(min(s + S - 2, steps - 1) - s);
        else if (s + 1 < steps) wait_vm<kHalf0>();
        else wait_vm<0>();
    };
    auto issue_at_start = [&](int s) {
        if (s + S - 1 < steps) issue_stage(s + S - 1, kEarly ? 1 : -1);
    };
    // half-way through stage s every wave has read the tokens and half 0 of the weights
    auto issue_half_way = [&](int s) {
        barrier();
        issue_stage(s + S, 0);
    };

    // fragment addresses
    const uint32_t arow = uint32_t(wm * (BW / WW) + lr) * 128;
    const uint32_t brow = uint32_t(BW + wt * (BT / WT) + lr) * 128;
    const uint32_t c0 = uint32_t(lk ^ (lr & 7)) << 4, c1 = c0 ^ 64;

    f32x4 acc[SA][SB];
#pragma unroll
    for (int i = 0; i < SA; ++i)
#pragma unroll
        for (int t = 0; t < SB; ++t) acc[i][t] = f32x4{0, 0, 0, 0};

    f32x4 prev[SB];                                          // fp8: the last subtile row's sums over a stage
    float sc[SB];                                            // and their scales
#pragma unroll
    for (int t = 0; t < SB; ++t) {
        prev[t] = f32x4{0, 0, 0, 0};
        sc[t] = 0.0f;
    }

    if constexpr (FP8) {
#pragma unroll
        for (int p = 0; p < kParts; ++p) issue_scales(0, p);
    }
    for (int st = 0; st < S - 1 && st < steps; ++st) issue_stage(st, -1);
    if (kEarly && S - 1 < steps) issue_stage(S - 1, 0);
    // a wave whose tokens or weight rows all lie past the end only loads
    const bool idle = wt * (BT / WT) >= row1 - row0 || n0 + wm * (BW / WW) >= g.N;
    for (int s = 0; idle && s < steps; ++s) {
        wait_stage(s);
        barrier();
        issue_at_start(s);
        if (kEarly && s + S < steps) issue_half_way(s);
    }
    using Op = Operand<FP8>;
    // a bf16 stage
    auto stage = [&](int s, auto half_way) {
        wait_stage(s);
        barrier();
        // the stages, short in K, need their loads as early as can be (grouped 32768
        // x 4096 x 1536 600 against 616 us behind the first reads)
        issue_at_start(s);
        const lds_t* from = ring + (s % S) * kSlot;
        // The first product needs one subtile of each operand: those are read
        // first.  Subtile row i is multiplied while row i + 1 is read, behind the
        // row's first product (in front of it the compiler waits for them as well).
        i32x4 a0 = *reinterpret_cast<lds_v4*>(from + arow + c0), a1 = *reinterpret_cast<lds_v4*>(from + arow + c1);
        i32x4 b0[SB], b1[SB];
#pragma unroll
        for (int t = 0; t < SB; ++t) {
            b0[t] = *reinterpret_cast<lds_v4*>(from + brow + t * 2048 + c0);
            b1[t] = *reinterpret_cast<lds_v4*>(from + brow + t * 2048 + c1);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < SA; ++i) {
            i32x4 n0, n1;
#pragma unroll
            for (int t = 0; t < SB; ++t) {
                const Op av(a0, a1), bv(b0[t], b1[t]);
                acc[i][t] = mma(av.part[1], bv.part[1], mma(av.part[0], bv.part[0], acc[i][t]));
                __builtin_amdgcn_sched_barrier(0);
                if (t == 0 && i + 1 < SA) {
                    n0 = *reinterpret_cast<lds_v4*>(from + arow + (i + 1) * 2048 + c0);
                    n1 = *reinterpret_cast<lds_v4*>(from + arow + (i + 1) * 2048 + c1);
                }
                if (half_way.value && t == 0 && i == SA / 2) {
                    issue_half_way(s);
                    __builtin_amdgcn_sched_barrier(0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            a0 = n0;
            a1 = n1;
        }
    };
    // An fp8 stage: subtile row i is multiplied while row i + 1 is read and
    // converted and row i - 1 (for i = 0 the last of the stage before) is folded.
    auto stage8 = [&](int s) {
        wait_stage(s);
        barrier();
        const lds_t* from = ring + (s % S) * kSlot;
        i32x4 a0 = *reinterpret_cast<lds_v4*>(from + arow + c0), a1 = *reinterpret_cast<lds_v4*>(from + arow + c1);
        i32x4 b0[SB], b1[SB];
#pragma unroll
        for (int t = 0; t < SB; ++t) {
            b0[t] = *reinterpret_cast<lds_v4*>(from + brow + t * 2048 + c0);
            b1[t] = *reinterpret_cast<lds_v4*>(from + brow + t * 2048 + c1);
        }
        const lds_t* row = tab + ((s >> 3) & 1) * kTab + (s & 7) * 4;
        const float sw = *reinterpret_cast<lds_f*>(row + (BT + wm * (BW / WW) / 128) * 32);
        float sb[SB];
#pragma unroll
        for (int t = 0; t < SB; ++t) sb[t] = *reinterpret_cast<lds_f*>(row + (wt * (BT / WT) + 16 * t + lr) * 32);
        __builtin_amdgcn_sched_barrier(0);
        issue_at_start(s);                                   // behind the first reads
        __builtin_amdgcn_sched_barrier(0);
        Op av(a0, a1), bv[SB];
#pragma unroll
        for (int t = 0; t < SB; ++t) bv[t] = Op(b0[t], b1[t]);
#pragma unroll
        for (int i = 0; i < SA; ++i) {
            Op next;
            f32x4 p[SB];
            if (i + 1 < SA) {
                a0 = *reinterpret_cast<lds_v4*>(from + arow + (i + 1) * 2048 + c0);
                a1 = *reinterpret_cast<lds_v4*>(from + arow + (i + 1) * 2048 + c1);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int t = 0; t < SB; ++t) {
                    p[t] = mma(av.part[k], bv[t].part[k], k == 0 ? f32x4{0, 0, 0, 0} : p[t]);
                    f32x4& to = acc[(i + SA - 1) % SA][t];
                    to[k] = __builtin_fmaf(sc[t], prev[t][k], to[k]);
                }
                if (k >= 2 && i + 1 < SA) {                  // the next row's reads have had two parts' time
                    const i32x4 c = k == 2 ? a0 : a1;
                    next.part[2 * k - 4] = e4m3x8_to_bf16(c[0], c[1], 1.0f);
                    next.part[2 * k - 3] = e4m3x8_to_bf16(c[2], c[3], 1.0f);
                }
                if (i > 0) __builtin_amdgcn_sched_barrier(0);
            }
            av = next;
#pragma unroll
            for (int t = 0; t < SB; ++t) {
                prev[t] = p[t];
                if (i == 0) sc[t] = __fmul_rn(sb[t], sw);
            }
        }
    };
    const int mine = idle ? 0 : steps;
    int s = 0;
    if constexpr (FP8) {
        for (; s < mine; ++s) stage8(s);
#pragma unroll
        for (int t = 0; t < SB; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[SA - 1][t][q] = __builtin_fmaf(sc[t], prev[t][q], acc[SA - 1][t][q]);
    } else {
        // the last two stages, which start no third, are their own loop
        for (; kEarly && s + S < mine; ++s) stage(s, std::bool_constant<kEarly>());
        for (; s < mine; ++s) stage(s, std::false_type());
    }
    // The ring is idle: each wave's outputs pass through 16 rows of its own, as
    // it needs no other wave.  The stores of 256 weight rows, long streams for
    // the most part, are past the caches' replacement: 32768 x 4096 x 1536 in 128
    // bf16 groups 574 -> 550 us, and 635 -> 623 us with moe_silu_mul reading the
    // result.
    __syncthreads();
    constexpr int kCols = BW / WW;
    lds_t* const rows16 = ring + wv * (16 * kOutRow<kCols>);
#pragma unroll
    for (int t = 0; t < SB; ++t) {
#pragma unroll
        for (int i = 0; i < SA; ++i) stage4<kCols>(rows16, lr, 16 * i + 4 * lk, acc[i][t]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        store_tile<kCols, 16, 64, BW == 256>(g, rows16, row0 + wt * (BT / WT) + 16 * t, row1, n0 + wm * kCols);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <bool FP8, int BW, int BT, int WW, int WT, int S, bool NTW>
__global__ __launch_bounds__(64 * WW * WT) void rows_tile_kernel(RowsGemmArgs g, int ntiles, int band) {
    // The last block of a group, of half the rows or fewer: the room of the
    // missing ones goes into a third slot and all waves share the rest (20000
    // rows in 64 bf16 groups of 2000 x 1024 120 -> 115 us).
    constexpr bool kPart64 = BW == 256, kPart128 = BW == 256 && BT == 256;
    constexpr int kLds = std::max({tile_lds<FP8, BW, BT, S>(), kPart64 ? tile_lds<FP8, BW, 64, 3>() : 0,
                                   kPart128 ? tile_lds<FP8, BW, 128, 3>() : 0});
    // one LDS object: with several, the compiler waits for every direct-to-LDS
    // load before each LDS read
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    static_assert(kLds <= 160 * 1024, "LDS");
    lds_t* const ring = (lds_t*)lds;

    // item -> (band of weight tiles, row block, tile in the band): the items an
    // XCD works on at a time share `band` weight tiles and some row blocks
    const int slots = count_blocks<BT>(g);
    int64_t item;
    if (!xcd_item(int64_t(slots) * ntiles, item)) return;    // the whole workgroup alike
    const int64_t per_band = int64_t(band) * slots;
    const int b = int(item / per_band);
    const int64_t in = item - b * per_band;
    const int wide = min(band, ntiles - b * band);
    const int slot = int(in / wide), n0 = (b * band + int(in % wide)) * BW;
    int e, row0, row1;
    if (!find_block<BT>(g, slot, e, row0, row1)) return;

    if constexpr (kPart64) {
        if (row1 - row0 <= 64) return tile_product<FP8, BW, 64, 4, 2, 3, NTW>(g, ring, e, row0, row1, n0);
    }
    if constexpr (kPart128) {
        if (row1 - row0 <= 128) return tile_product<FP8, BW, 128, 4, 2, 3, NTW>(g, ring, e, row0, row1, n0);
    }
    tile_product<FP8, BW, BT, WW, WT, S, NTW>(g, ring, e, row0, row1, n0);
}

template <bool FP8, int BW, int BT, int WW, int WT, int S>
hipError_t launch_tile(const RowsGemmArgs& g, bool one_pass, hipStream_t s) {
    const int ntiles = (g.N + BW - 1) / BW;
    const int64_t slots = block_slots(g, BT);
    void (*kern)(RowsGemmArgs, int, int) =
        one_pass ? rows_tile_kernel<FP8, BW, BT, WW, WT, S, true> : rows_tile_kernel<FP8, BW, BT, WW, WT, S, false>;
    return start(kern, xcd_grid(slots * ntiles), 64 * WW * WT, s, g, ntiles, std::min(kBand, ntiles));
}

template <bool FP8>
hipError_t launch(const RowsGemmArgs& g, int shape, bool one_pass, hipStream_t s) {
    switch (shape) {
        case 0: return launch_tile<FP8, 64, 32, 2, 2, 4>(g, one_pass, s);
        case 1: return launch_tile<FP8, 128, 64, 4, 1, 3>(g, one_pass, s);
        case 2: return launch_tile<FP8, 128, 128, 2, 4, 4>(g, one_pass, s);
        case 3: return launch_tile<FP8, 256, 128, 4, 2, 3>(g, one_pass, s);
        default: break;
    }
    if constexpr (!FP8) {                                    // of converted e4m3 operands: out of registers
        if (shape == 4) return launch_tile<false, 256, 256, 2, 4, 2>(g, one_pass, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows_tile(const RowsGemmArgs& g, bool fp8, int shape, bool one_pass, hipStream_t s) {
    return fp8 ? launch<true>(g, shape, one_pass, s) : launch<false>(g, shape, one_pass, s);
}

}  // namespace moe
