// Host rules of the ragged grouped products: tile height and K segments, from
// the sizes that the host knows (rows in all, groups, widths).
#include <algorithm>

#include "kernels.hpp"

namespace bsg {

static int elt(int dtype) { return dtype == kE4m3 ? 1 : dtype == kBf16 ? 2 : 4; }

// Tiles to expect of a launch with tiles of `rows` rows: every group of its
// mean size (the sizes themselves are on the device).
static int64_t tiles_expected(int64_t M, int E, int N, int epi, int rows) {
    const int64_t ne = E < M ? E : M, mean = (M + ne - 1) / ne;
    const int w = epi == kEpiSiluMul ? 128 : 256;
    return ne * ((mean + rows - 1) / rows) * ((N + w - 1) / w);
}

// Tile rows: 128 where a tile is over before one workgroup's loads and stores
// can hide behind its products (at most 2 KB of K a row), where groups have
// too few rows for 256, and where tiles of 256 rows would be fewer than the
// compute units and the groups long enough to be cut in two; otherwise 256,
// whose operands each cross LDS half as often.  Measured, 128 / 256: bf16 64
// experts of 256 rows, K 512, 67 / 85 us; skewed 131072 rows, K 1024, 1243 /
// 1344 us and K 4096, 1282 / 1113 us; 8 experts of 128 rows, K 4096, 499 / 441
// us; e4m3 8 experts of 2048 rows, K 4096, 2070 / 1852 us.
static int tile_rows(int64_t M, int E, int K, int N, int epi, int dtype, int ncu) {
    if ((int64_t)K * elt(dtype) <= 2048 || M / E <= 96) return 128;
    return M / E > 256 && tiles_expected(M, E, N, epi, 256) < ncu ? 128 : 256;
}

// Weight gradients: the reduction is a group's rows.  Short ones run two
// workgroups a compute unit; narrower tiles where wide ones are few.
// Measured, 128 / 256 rows a tile: 64 experts of 256 rows 53 / 62 us, of 2048
// rows 1099 / 1071 us.
//
// Segments of a group's rows where even narrow tiles are fewer than a third of
// what two workgroups a unit take, of 256 rows or more, while the segments'
// sums (fp32, written and read once) stay below half the operands' bytes.
GroupedPlan grouped_wgrad_plan(int64_t M, int K, int N, int E, int dtype, int ncu,
                               int64_t max_segments) {
    const int64_t tn = (N + 255) / 256, few = dtype == kF32 ? 2 * (int64_t)ncu : ncu;
    const int64_t narrow = E * (((int64_t)K + 127) / 128) * ((N + 127) / 128);
    if (3 * narrow <= 2 * (int64_t)ncu) {
        const int64_t operands = M * ((int64_t)K + N) * elt(dtype);
        const int64_t share = (int64_t)E * K * N * 8;
        const int64_t n = std::min({2 * (int64_t)ncu / narrow, M / E / 256, operands / (2 * share),
                                    max_segments, (int64_t)kMaxSegments});
        if (n >= 2) return {128, 128, (int)n};
    }
    if (N <= 128 || E * (((int64_t)K + 127) / 128) * tn < few) return {128, 128, 1};
    return {M / E <= 512 || E * (((int64_t)K + 255) / 256) * tn < few ? 128 : 256, 256, 1};
}

// K segments: a launch that would leave more than a third of the compute
// units without a tile cuts its sums until there are about two workgroups for
// each of them, if a segment keeps kMinSegment K-tiles (64 bytes of K a row
// each) or more and the segments' sums, written and read once in fp32, stay
// below a quarter of the operands' bytes.  Measured, split / not: bf16, K
// 14336, N 4096, 8 experts of 128 rows 220 / 293 us, one row of two experts 41
// / 178 us; but K 4096, N 14336 (SILU_MUL), one row of two experts, in two
// segments 98 / 85 us: 224 workgroups fill the memory's queues already.  Nor
// are groups of few rows split whose narrow tiles fill the units: K 14336, N
// 4096, 8 experts of 12 rows, four segments / 128 columns, bf16 165 / 145 us,
// e4m3 93 / 88 us.
//
// Columns: 128 (under 128 rows, unsplit, one product) where the wider tile
// would be more than half empty or leave compute units idle: fewer tiles than
// units, of 256 rows fewer than half as many, of fp32, whose products take
// sixteen times as long, fewer than two a unit.  Measured, 128 x 128 / wider:
// fp32 24 experts of 96 rows, K 672, N 728, 45 / 157 us; bf16 64 experts of 256
// rows, K 2048, N 512 (128 tiles of 256 x 256), 50 / 47 us.
GroupedPlan grouped_plan(int64_t M, int K, int N, int E, int epi, int dtype, int ncu,
                         int64_t max_segments) {
    constexpr int kMinSegment = 16;
    const bool dual = epi == kEpiSiluMul;
    const int mats = dual ? 2 : 1;
    const int64_t ne = E < M ? E : M;
    GroupedPlan p{tile_rows(M, E, K, N, epi, dtype, ncu), 256, 1};
    const int64_t tiles = tiles_expected(M, E, N, epi, p.rows);
    const bool narrow_fills = M / E <= 96 && 2 * tiles >= ncu;
    int64_t n = 2 * (int64_t)ncu / tiles;
    if (n >= 3 && (dual || !narrow_fills)) {
        const int64_t operands = (M * (int64_t)K + ne * (int64_t)K * N * mats) * elt(dtype);
        const int64_t share = M * (int64_t)N * mats * 8;
        n = std::min(n, ((int64_t)K * elt(dtype) / 64) / kMinSegment);
        n = std::min({n, operands / (4 * share), max_segments, (int64_t)kMaxSegments});
        if (n >= 2) {
            p.segments = (int)n;
            return p;
        }
    }
    if (!dual) {
        const int64_t few = dtype == kF32 ? 2 * (int64_t)ncu : p.rows == 256 ? ncu / 2 : ncu;
        if (N <= 128 || ((M / E > 64 || narrow_fills) && tiles < few)) p.rows = p.cols = 128;
    }
    return p;
}

}  // namespace bsg
