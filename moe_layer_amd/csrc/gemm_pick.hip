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
constexpr Tile kTilesFp8[] = {
    {true, 0, 16, 16, 1.18f, 1.19f, 0.0662f},     {true, 1, 32, 16, 1.14f, 1.34f, 0.0960f},
    {true, 2, 32, 32, 1.02f, 1.59f, 0.1218f},     {true, 3, 64, 32, 0.92f, 2.06f, 0.1785f},
    {true, 4, 64, 48, 0.76f, 2.73f, 0.2215f},     {true, 5, 64, 64, 0.68f, 3.18f, 0.2750f},
    {false, 0, 64, 32, 2.81f, 0.26f, 0.2599f},    {false, 1, 128, 64, 2.83f, 0.72f, 0.6596f},
    {false, 2, 128, 128, -0.20f, 3.46f, 0.9265f}, {false, 3, 256, 128, 0.62f, 4.31f, 1.6690f},
};

constexpr double kHbmBytesPerUs = 5.8e6;   // streaming reads and writes (6 TB/s reads alone)

double time_us(const Tile& t, const RowsGemmArgs& g, bool fp8) {
    const double es = fp8 ? 1 : 2, steps = g.K * es / 128;
    const int64_t groups = g.offsets ? std::min(g.E, g.rows) : 1;
    // row blocks: of a group's rows, known on the device only, the last one is
    // half full on average
    const double blocks = g.offsets ? std::max(double(groups), double(g.rows) / t.bt + 0.5 * groups)
                                    : std::ceil(double(g.rows) / t.bt);
    const double fill = blocks * ((g.N + t.bw - 1) / t.bw) / 256;
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
// as many as fill a 256-row block each 518 / 545.
bool one_pass(const RowsGemmArgs& g, int bm, bool fp8) {
    const int64_t groups = g.offsets ? std::min(g.E, g.rows) : 1;
    const int64_t rows = g.offsets ? 2 * int64_t(g.rows) : g.rows;
    return rows <= bm * groups && groups * g.N * g.K * (fp8 ? 1 : 2) >= int64_t(128) << 20;
}

template <int N>
const Tile& fastest(const Tile (&tiles)[N], const RowsGemmArgs& g, bool fp8) {
    const Tile* best = tiles;
    double least = time_us(tiles[0], g, fp8);
    for (const Tile& t : tiles) {
        const double us = time_us(t, g, fp8);
        if (us < least) {
            best = &t;
            least = us;
        }
    }
    return *best;
}

}  // namespace

RowsPlan plan_rows_gemm(const RowsGemmArgs& g, bool fp8) {
    const Tile& t = fp8 ? fastest(kTilesFp8, g, true) : fastest(kTilesBf16, g, false);
    return {t.split, t.shape, t.bw, t.bt, one_pass(g, t.bt, fp8)};
}

hipError_t launch_rows_gemm(const RowsGemmArgs& g, bool fp8, hipStream_t s) {
    const RowsPlan p = plan_rows_gemm(g, fp8);
    return p.split ? launch_rows_split(g, fp8, p.shape, p.one_pass, s) : launch_rows_tile(g, fp8, p.shape, p.one_pass, s);
}

}  // namespace moe
