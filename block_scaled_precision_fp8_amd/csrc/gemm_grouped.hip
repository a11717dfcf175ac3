// gemm_grouped.hip -- which form a grouped block-of-128 FP8 product runs on (gfx950).
//
// The groups' sizes are on the device, so the choice goes by their number and the rows in all: as if
// the rows were spread evenly, half a tile of each group empty.  Times are microseconds on MI355X, of calls
// in a captured graph.
#include "gemm_grouped.h"

#include <algorithm>

namespace bsfp8 {

namespace {

enum Form { FEW, T64x128, T128, T256 };

// Rows by expert.  A tiled form runs `stage` per 128 K and tile on each CU, and `tile` besides; the
// form for few rows moves 32 bytes per K and 16 x 16 tile at 10 TB/s.  The weights of the groups that have rows
// are read at 5 TB/s (6 by the form for few rows), which hides behind the tiled products by some 70%.
// 64 groups, N 2048, K 4096, 16-bit output (few rows, 64 x 128, 128 x 128, 256 x 256): 128 rows 84, 110, 113,
// 116; 512 rows 106, 123, 127, 129; 1024 rows 164, 124, 127, 130; 4096 rows 520, 136, 131, 135; 8192
// rows 991, 168, 151, 143; 16384 rows 1941, 256, 205, 188.  16384 rows of 8 groups, N 14336: -,
// 1440, 1039, 763; 8 rows of 16 groups, N 1024: 8.7, 15.5, 16.9, 37.0.
// With few columns the form for few rows has few workgroups, each of which walks its group's 16-row tiles one after
// another, at 0.25 us and 1 us per 1024 K each (K 512: 0.75 to 0.9, K 4096: 4.3): the largest group, taken as
// twice the mean, sets the time, the first tile being in the 4 us of every form.  N 16, K 4096 (few rows,
// 64 x 128): 2 groups of 64 rows 21, 12.2; 8 of 16 rows 8.9, 12.3; 8 of 64 rows 21.5, 12.4; 64 of 8 rows 5.8, 12.3; 64 of
// 32 rows 15.6, 14.8; 8 of 2048 rows 557, 19.3; K 512: 8 of 16 rows 2.9, 4.4; 8 of 64 rows 5.3, 4.4; 2 of 1024 rows 50, 4.5.
Form choose_rows(const GroupedArgs& t) {
    const bool wide = t.out == BSFP8_OUT_F32;
    const double M = static_cast<double>(t.M), N = static_cast<double>(t.N), K = static_cast<double>(t.K);
    const double groups = static_cast<double>(std::min<int64_t>(t.M, t.groups)), stages = std::max(1.0, K / 128.0);
    const double weights = groups * N * K / 5.0e6;
    auto row_tiles = [&](double rows) { return std::max(groups, M / rows + groups / 2); };
    auto total = [&](double products) { return 4.0 + std::max(weights, products) + 0.3 * std::min(weights, products); };
    Form form = FEW;
    // (a workgroup of up to 1024 threads per 16 columns and group; threads are counted in 32 bits)
    const double walk = std::max(0.0, 2.0 * M / groups / 16.0 - 1.0) * (0.25 + K / 1024.0);
    double best = 4.0 + std::max({groups * N * K / 6.0e6, row_tiles(16) * (N / 16.0) * K * 32.0 / 10.0e6, walk});
    if ((t.N + 15) / 16 * t.groups >= int64_t(1) << 22) best = 1e300;
    struct Cost { Form form; int rows, columns; double stage, stage_f32, tile; };
    static constexpr Cost kCost[3] = {{T64x128, 64, 128, 0.37, 0.51, 0.0}, {T128, 128, 128, 0.56, 0.88, 0.0}, {T256, 256, 256, 1.35, 1e9, 8.0}};
    for (const Cost& c : kCost) {
        if (c.form == T256 && (wide || !t.fast_ok())) continue;
        const double tiles = row_tiles(c.rows) * std::max(1.0, N / c.columns) / 256.0;
        const double rounds = c.form == T256 ? static_cast<double>(static_cast<int64_t>(tiles + 1.0)) : std::max(1.0, tiles);
        const double time = total(rounds * (stages * (wide ? c.stage_f32 : c.stage) + c.tile));
        if (time < best) {
            best = time;
            form = c.form;
        }
    }
    return form;
}

// K values by expert.  Narrow: 32 x 32 tiles, three workgroups per CU, K over four waves.
// 8192 rows of 4 groups, 256 x 256 (narrow, 128 x 128, 256 x 256): 7.4, 12.4, 24.9; 300 rows of 8 groups, 256 x 256:
// 4.4, 5.1, 9.6; 64 rows of 64 groups, 512 x 512: 71, 17, 21; 2222 rows of 32 groups, 1000 x 2000: 287,
// 69, 60 (1000 x 2001: 294, 72, 64); 16384 rows of 8 groups, 4096 x 4096: -, 344, 245, and FP32 -, 521, 445 (with
// C -, 590, 535).  Over 120 sizes (128 to 8192 rows of 1 to 32 groups, 256 x 256 to 4096 x 1024) the choice is within 13% of
// the best form, but for one long group: 8192 rows, 1000 x 2000, FP32 runs narrow, 83 where 128 x 128 takes 53.
Form choose_columns(const GroupedKArgs& t) {
    const bool wide = t.out == BSFP8_OUT_F32;
    // (columns: the rows in all and up to 127 more per group)
    const double blocks = std::max(1.0, static_cast<double>(t.columns) / 128.0 / t.groups);
    auto tiles = [&](int64_t side) { return static_cast<double>((t.M + side - 1) / side * ((t.N + side - 1) / side) * t.groups); };
    const double few = tiles(32);
    double best = 4.0 + (few <= 768 ? 0.22 * blocks + 1.5 : few / 768 * (0.22 * blocks + 3.7));
    if (few >= (1 << 24)) best = 1e300;              // threads are counted in 32 bits
    Form form = FEW;
    const double t128 = 4.0 + std::max(1.0, tiles(128) / 256) * (blocks * (wide ? 0.88 : 0.56) + 2.5);
    if (t128 < best) best = t128, form = T128;
    const double t256 = 4.0 + static_cast<double>(static_cast<int64_t>((tiles(256) + 255) / 256)) * (blocks * (wide ? 3.05 : 1.35) + 9.0);
    if (t.fast_ok() && t256 < best) form = T256;
    return form;
}

}  // namespace

hipError_t launch_gemm_grouped(const GroupedArgs& t) {
    if (t.K == 0) return launch_gemm_grouped_rows(t);
    switch (choose_rows(t)) {
    case T64x128: return launch_gemm_grouped_1x2(t);
    case T128: return launch_gemm_grouped_2x2(t);
    case T256: return launch_gemm_grouped_4x4(t);
    default: return launch_gemm_grouped_rows(t);
    }
}

int gemm_grouped_form(int64_t M, int64_t N, int64_t K, int groups, int out, int64_t ldd, int64_t ldc, float beta) {
    GroupedArgs t{};
    t.M = M, t.N = N, t.K = K, t.groups = groups, t.out = out, t.ldd = ldd, t.ep.ldc = ldc, t.ep.beta = beta;
    return K == 0 ? FEW : choose_rows(t);
}

int gemm_wgrad_form(int64_t M, int64_t N, int64_t columns, int groups, int out, int64_t ldd, int64_t ldc, float beta) {
    GroupedKArgs t{};
    t.M = M, t.N = N, t.columns = columns, t.groups = groups, t.out = out, t.ldd = ldd, t.ep.ldc = ldc, t.ep.beta = beta;
    return choose_columns(t);
}

hipError_t launch_gemm_grouped_wgrad(const GroupedKArgs& t) {
    switch (choose_columns(t)) {
    case T128: return launch_gemm_wgrad_2x2(t);
    case T256: return t.out == BSFP8_OUT_F32 ? launch_gemm_wgrad_4x4_f32(t) : launch_gemm_wgrad_4x4(t);
    default: return launch_gemm_wgrad_narrow(t);
    }
}

}  // namespace bsfp8
