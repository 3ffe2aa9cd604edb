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
int grouped_tile_rows(int64_t M, int E, int K, int N, int epi, int dtype, int ncu) {
    if ((int64_t)K * elt(dtype) <= 2048 || M / E <= 96) return 128;
    return M / E > 256 && tiles_expected(M, E, N, epi, 256) < ncu ? 128 : 256;
}

// K segments: a launch that would leave more than a third of the compute
// units without a tile cuts its sums until there are about two workgroups for
// each of them, if a segment keeps kMinSegment K-tiles (64 bytes of K a row
// each) or more and the segments' sums, written and read once in fp32, stay
// below a quarter of the operands' bytes.  Measured, split / not: bf16, K
// 14336, N 4096, 8 experts of 12 rows 165 / 212 us, of 128 rows 220 / 293 us,
// one row of two experts 41 / 178 us; e4m3, 12 rows, 93 / 138 us; but K 4096,
// N 14336 (SILU_MUL), one row of two experts, in two segments 98 / 85 us: 224
// workgroups fill the memory's queues already.
int grouped_segments(int64_t M, int K, int N, int E, int epi, int dtype, int ncu) {
    constexpr int kMinSegment = 16;
    const int mats = epi == kEpiSiluMul ? 2 : 1;
    const int64_t ne = E < M ? E : M;
    const int64_t tiles =
        tiles_expected(M, E, N, epi, grouped_tile_rows(M, E, K, N, epi, dtype, ncu));
    const int64_t operands = (M * (int64_t)K + ne * (int64_t)K * N * mats) * elt(dtype);
    const int64_t share = M * (int64_t)N * mats * 8;
    int64_t n = 2 * (int64_t)ncu / tiles;
    if (n < 3) return 1;
    n = std::min(n, ((int64_t)K * elt(dtype) / 64) / kMinSegment);
    n = std::min(n, operands / (4 * share));
    n = std::min<int64_t>(n, kMaxSegments);
    return n < 2 ? 1 : (int)n;
}

}  // namespace bsg
