// The tile a dense or grouped product runs in.
//
// Both forms (gemm_split.hip, gemm_tile.hip) are bound by the bytes a CU gets
// from L2 into its LDS, 50-80 GB/s by tile, for most sizes, fp8 tiles of many
// rows by the conversion of their operands and the bf16 matrix cores behind it: a
// workgroup of BW x BT outputs fetches (BW + BT) 128-byte rows per K step, so
// large tiles move fewer bytes and small ones fill the 256 CUs.  The time of a
// tile shape is modelled as
//   start + rounds (round + steps step),
// rounds = workgroups / 256, rounded up (above 4 half a round more than the
// quotient), steps = K steps of 128 bytes, and at least the bytes that have to
// come from HBM; the fastest shape is taken.  The constants are least-squares
// fits: for fp8 over 62 dense shapes from 1 x 512 x 512 to 8192 x 4096 x 7168,
// each timed in every tile (those of 256 weight rows where there are more than
// 128 token rows; residual 6-17 %).  Over those and 20 grouped ones the pick is
// 1.4 % slower than the best tile in the geometric mean, 15 % at worst (150 rows
// in 128 groups of 700 x 768).  The bf16 ones were
// fitted to products of as many bytes that go to the matrix cores as they are, not
// to bf16 itself: over 24 shapes the pick is 6 % slower than the best tile, 49 %
// at worst (4096 x 4096 x 4096 in one group).
#include <algorithm>
#include <cmath>

#include "dense.h"

namespace moe {

namespace {

struct Tile {
    bool split;        // gemm_split.hip, else gemm_tile.hip
    int shape;         // its number there
    int bw, bt;        // weight rows and token rows
    float start, round, step;   // us
    int per_cu = 1;    // workgroups that a CU works on at a time
};

constexpr Tile kTilesBf16[] = {
    {true, 0, 16, 16, 1.18f, 1.14f, 0.0561f},    {true, 1, 32, 16, 1.10f, 1.27f, 0.0830f},
    {true, 2, 32, 32, 0.95f, 1.49f, 0.1069f},    {true, 3, 64, 32, 0.83f, 1.91f, 0.1562f},
    {true, 4, 64, 48, 0.68f, 2.53f, 0.1813f},    {true, 5, 64, 64, 0.59f, 2.97f, 0.2185f},
    {true, 6, 64, 80, 0.49f, 3.54f, 0.2398f},    {true, 7, 128, 48, 0.68f, 3.77f, 0.2805f},
    {false, 0, 64, 32, 2.57f, 0.29f, 0.1760f},   {false, 1, 128, 64, 2.66f, 0.79f, 0.4171f},
    {false, 2, 128, 128, 0.20f, 3.07f, 0.4869f}, {false, 3, 256, 128, 0.48f, 4.37f, 0.8250f},
    {false, 4, 256, 256, -1.06f, 7.37f, 1.3169f},
};
// int8: from the bf16 constants (as many bytes that go to the matrix cores as they
// are) by a search for the ones whose picks are the fastest over 347 shapes, dense
// and grouped, each timed in every tile; fitted to half of them 2.8 % above the best tile
// over the other half.  The kernels have changed since then (few rows' K out of step,
// stores): timed again, the picks are 2.3 % above the best tile in the geometric mean (155
// dense shapes 1.4 %, 192 grouped 3.0 %), 44 % at worst (1568 rows in 100 groups of 360 x
// 128, 6.6 us; dense 15 %, 1 x 104 x 512).  When fitted, the best tile without the two
// workgroups a CU of the last one was 48 % slower at worst (7189 rows in 256 groups of
// 504 x 256).
constexpr Tile kTilesInt8[] = {
    {true, 0, 16, 16, 1.18f, 1.14f, 0.0561f},    {true, 1, 32, 16, 1.20f, 1.52f, 0.0748f},
    {true, 2, 32, 32, 1.03f, 1.24f, 0.1195f},    {true, 3, 64, 32, 0.79f, 2.11f, 0.1240f},
    {true, 4, 64, 48, 0.77f, 2.92f, 0.2077f},    {true, 5, 64, 64, 0.49f, 3.40f, 0.2386f},
    {true, 6, 64, 80, 0.60f, 4.14f, 0.2479f},    {true, 7, 128, 48, 0.66f, 4.27f, 0.2781f},
    {false, 0, 64, 32, 2.57f, 0.29f, 0.1660f},   {false, 1, 128, 64, 3.13f, 0.73f, 0.4171f},
    {false, 2, 128, 128, 0.19f, 3.34f, 0.5316f}, {false, 3, 256, 128, 0.64f, 4.37f, 0.9328f},
    {false, 4, 256, 256, -1.09f, 5.56f, 1.1392f}, {false, 5, 256, 128, 1.42f, 0.54f, 1.9746f, 2},
};
constexpr Tile kTilesFp8[] = {
    {true, 0, 16, 16, 1.18f, 1.19f, 0.0662f},     {true, 1, 32, 16, 1.14f, 1.34f, 0.0960f},
    {true, 2, 32, 32, 1.02f, 1.59f, 0.1218f},     {true, 3, 64, 32, 0.92f, 2.06f, 0.1785f},
    {true, 4, 64, 48, 0.76f, 2.73f, 0.2215f},     {true, 5, 64, 64, 0.68f, 3.18f, 0.2750f},
    {false, 0, 64, 32, 2.81f, 0.26f, 0.2599f},    {false, 1, 128, 64, 2.83f, 0.72f, 0.6596f},
    {false, 2, 128, 128, -0.20f, 3.46f, 0.9265f}, {false, 3, 256, 128, 0.62f, 4.31f, 1.6690f},
};

constexpr double kHbmBytesPerUs = 5.8e6;   // streaming reads and writes (6 TB/s reads alone)

double time_us(const Tile& t, const RowsGemmArgs& g, RowsKind kind) {
    const double es = kind == kRowsBf16 ? 2 : 1, steps = std::ceil(g.K * es / 128);
    const int64_t groups = g.offsets ? std::min(g.E, g.rows) : 1;
    // row blocks: of a group's rows, known on the device only, the last one is
    // half full on average
    const double blocks = g.offsets ? std::max(double(groups), double(g.rows) / t.bt + 0.5 * groups)
                                    : std::ceil(double(g.rows) / t.bt);
    const double fill = blocks * ((g.N + t.bw - 1) / t.bw) / (256 * t.per_cu);
    const double rounds = fill <= 4 ? std::ceil(fill) : fill + 0.5;
    const double us = t.start + rounds * (t.round + steps * t.step);
    const double bytes = (double(groups) * g.N + g.rows) * g.K * es + 2.0 * g.rows * g.N;
    const double hbm = bytes / kHbmBytesPerUs;
    // long streams overlap with the rest in part only
    return hbm < 20 ? us : std::max(us, hbm) + (t.split ? 0.3 : 0.2) * std::min(us, hbm);
}

// Whether the weights pass once and are too many to stay in the 256 MB Infinity
// Cache for the next call: one row block (for groups, whose sizes are known on
// the device only, half a one on average) and 128 MiB of weights or more
// (load_piece).  us without / with them: dense 16 x 2112 x 7168
// (15 MB) 6.3 / 7.2, 8 x 20000 x 7168 (143 MB) 31.0 / 27.6; 131 fp8 rows in 32
// groups of 4096 x 2048 (268 MB) 49.4 / 44.1; 8192 in 256 groups of 512 x 4096,
// half-full 64-row blocks 142 / 136; 32768 bf16 rows in 128 groups of 4096 x 1536,
// as many as fill a 256-row block each 518 / 545.  Not where K (int8) is no whole
// number of lines: two steps have a part of each line, and the second would fetch it
// again (6059 rows in 128 groups of 2568 x 3056 254 / 345; 1 x 20000 x 7184 25.8 /
// 37.5; 300 in 128 of 2048 x 2064 78 / 88).
bool one_pass(const RowsGemmArgs& g, int bm, RowsKind kind) {
    const int64_t groups = g.offsets ? std::min(g.E, g.rows) : 1;
    const int64_t rows = g.offsets ? 2 * int64_t(g.rows) : g.rows;
    const int64_t row_bytes = g.K * (kind == kRowsBf16 ? 2 : 1);
    return rows <= bm * groups && groups * g.N * row_bytes >= int64_t(128) << 20 && row_bytes % 128 == 0;
}

template <int N>
const Tile& fastest(const Tile (&tiles)[N], const RowsGemmArgs& g, RowsKind kind) {
    const Tile* best = tiles;
    double least = time_us(tiles[0], g, kind);
    for (const Tile& t : tiles) {
        const double us = time_us(t, g, kind);
        if (us < least) {
            best = &t;
            least = us;
        }
    }
    return *best;
}

}  // namespace

RowsPlan plan_rows_gemm(const RowsGemmArgs& g, RowsKind kind) {
    const Tile& t = kind == kRowsFp8    ? fastest(kTilesFp8, g, kind)
                    : kind == kRowsInt8 ? fastest(kTilesInt8, g, kind) : fastest(kTilesBf16, g, kind);
    return {t.split, t.shape, t.bw, t.bt, t.per_cu, one_pass(g, t.bt, kind)};
}

hipError_t launch_rows_gemm(const RowsGemmArgs& g, RowsKind kind, hipStream_t s) {
    const RowsPlan p = plan_rows_gemm(g, kind);
    return p.split ? launch_rows_split(g, kind, p.shape, p.one_pass, s)
                   : launch_rows_tile(g, kind, p.shape, p.one_pass, s);
}

}  // namespace moe
