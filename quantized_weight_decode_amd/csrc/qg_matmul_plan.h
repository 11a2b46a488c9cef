// qg_matmul_plan.h -- which kernel a product of two 8-bit operands takes, in which
// tiles and parts of K: rules on sizes and the number of CUs (host only, no GPU).
#pragma once

#include <initializer_list>

namespace qg {

// Rows of y, experts (0: dense), columns of x, rows of W.
struct MatmulSizes {
    int R, E, I, O;
    bool bf16, gated;                    // results
    int outputs() const { return gated ? O / 2 : O; }
    int steps() const { return (I + 127) / 128; }
};

// The tile kernel's kinds of tiles (matmul_tile.h).
struct TileKind {
    int bt, bw, waves;                   // rows of x, rows of W, waves
    double step, fixed;                  // us per K step and per tile
};
constexpr TileKind TILE_KINDS[] = {{256, 256, 8, 1.5, 14.0},
                                   {192, 256, 8, 1.27, 13.0},
                                   {128, 256, 8, 0.97, 12.0},
                                   {64, 256, 8, 0.64, 10.0},
                                   {128, 128, 4, 1.0, 10.0}};
constexpr int SQUARE = 4;                // the only one for f32, or rows that are not on 16 bytes
constexpr int SCALE_STEPS = 4;           // K steps whose scales are fetched together

// How the tile kernel takes a product: tiles of `kind`, K in `parts` (dense); the
// first `head` columns of y, if any, by a launch of their own, of `head_kind`.
struct TilePlan {
    int kind, parts, head, head_kind;
    double us;                           // estimated (dense)
};

// K steps of one of `parts` parts: whole groups of scales.
inline int steps_per_part(int steps, int parts)
{
    return ((steps + parts - 1) / parts + SCALE_STEPS - 1) / SCALE_STEPS * SCALE_STEPS;
}

// Tiles of a kind for n columns of y.
inline long long tiles_of(const MatmulSizes &p, int kind, int n)
{
    const TileKind &k = TILE_KINDS[kind];
    const int cols = k.bw / (p.gated ? 2 : 1);
    return (long long)((p.R + k.bt - 1) / k.bt) * ((n + cols - 1) / cols);
}

// The plan of n columns in one launch: the kind, and the parts of K where tiles leave
// CUs without work, for which the busiest CU ends first (1501 x 16384 x 7168: 224 tiles
// of 192 rows 196 us, 168 of 256 rows 219, those in three parts 236).  One workgroup (of
// the square kind two) per CU at a time; joining parts costs a launch and their sums'
// way to memory and back.
inline TilePlan plan_columns(const MatmulSizes &p, bool any, int n, long long ncu)
{
    const int steps = p.steps();
    TilePlan best{};
    best.us = -1.0;
    for (int i = any ? 0 : SQUARE; i <= SQUARE; i++) {
        const TileKind &k = TILE_KINDS[i];
        const long long tiles = tiles_of(p, i, n), slots = i == SQUARE ? 2 * ncu : ncu;
        const double c = p.bf16 ? k.step : 2 * k.step;
        for (const int f : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (f > 1 && (tiles * f > slots || p.R > 4096)) break;
            const int per = steps_per_part(steps, f);
            if ((steps + per - 1) / per != f) continue;
            double us = (double)((tiles * f + slots - 1) / slots) *
                        ((f > 1 ? per : steps) * c + k.fixed);
            if (f > 1) us += 5.0 + 8e-6 * f * p.R * (double)p.O / 5.0;
            if (best.us < 0.0 || us < best.us) best = TilePlan{i, f, 0, 0, us};
        }
    }
    return best;
}

// The tile kernel's plan; direct: rows of both operands on 16 bytes.
// Dense: the faster of one launch and of two, the first with as many columns as give
// every CU the same number of one kind's tiles, the second with the rest, by what suits
// that.  us: 2048 x 6144 x 12288, 384 tiles of 256 x 256 at once 177 (gated 179); 256 of
// them, then the rest in 512 of 128 x 128 159 (161), in 256 of 128 x 256, whose estimate
// is 0.6 higher, 157 (159); 2040 x 6144 x 12290 at once 206 (211), the rest in tiles of
// 192 rows 197 (201).
// Grouped by expert 128 x 256, whose three stages suit experts of few rows, bound by
// their weights' bytes, up to 512 rows per expert on average.  us, 128 and 256 rows per
// tile, unevenly routed: 64 experts of 7168 x 2048 with 128 rows each 275 and 294, 256
// rows 428 and 387, 512 rows 704 and 590, 1024 rows 1223 and 1023; 8 experts with 128
// rows 66 and 88, 384 rows 79 and 106, 512 rows 130 and 105.  (Between 256 and 512 rows
// many experts would gain from 256, few would lose.)
inline TilePlan plan_tiles(const MatmulSizes &p, bool direct, long long ncu)
{
    const bool any = p.bf16 && direct;
    if (p.E) return TilePlan{!any ? SQUARE : p.R / p.E < 512 ? 2 : 0, 1, 0, 0, 0.0};
    const int oc = p.outputs();
    TilePlan best = plan_columns(p, any, oc, ncu);
    for (int i = 0; any && i < SQUARE; i++) {
        const TileKind &k = TILE_KINDS[i];
        const int cols = k.bw / (p.gated ? 2 : 1);
        const long long ntm = (p.R + k.bt - 1) / k.bt, rounds = tiles_of(p, i, oc) / ncu;
        const long long head = rounds * ncu / ntm * cols;
        if (rounds < 1 || head < cols || head >= oc) continue;
        const double us = rounds * (p.steps() * k.step + k.fixed) + 7.0;
        if (us >= best.us) continue;
        TilePlan rest = plan_columns(p, any, oc - (int)head, ncu);
        rest.us += us;
        rest.head = (int)head;
        rest.head_kind = i;
        if (rest.us < best.us) best = rest;
    }
    return best;
}

// The kernel of a product and the rows of its row tiles.
struct MatmulPlan {
    bool tile;
    TilePlan plan;
    int bm;
};

// The tile kernel, or up to 64 rows the stream kernel where it is estimated to be
// faster: 7 us and its weights at 5 TB/s, 1, 1.8 or 3.2 times for tiles of 16, 32 or
// 64 rows (whose products take the longer part).  us of a call by stream and tile, bf16
// results (f32): 5 x 16384 x 7168 34 and 31 (34 and 40), 16 rows 43 and 32 (43 and 41),
// 5 x 4096 x 4096 15 and 19 (15 and 19), 64 x 6144 x 12288 66 and 30 (65 and 35).  (Up
// to 16 rows of weights below 64 MB always, without estimating: 16 x 4096 x 4096.)
// Grouped by expert the tile kernel from 17 rows on: of 256 experts, 7168 x 2048, 16
// rows 62 and 65 (61 and 67), 32 rows 107 and 94 (107 and 95), 128 rows 261 and 235 (262
// and 248).  Where experts are few that is too early: of 8, 32 rows 33 and 51 (33 and
// 55), 64 rows 42 and 53 (42 and 56).
// fits: the tile kernel's offsets are within 32 bits.
inline MatmulPlan plan_matmul(const MatmulSizes &p, bool fits, bool direct, long long ncu)
{
    MatmulPlan c{};
    const int rows = p.E ? (p.R + p.E - 1) / p.E : p.R;
    const double bytes = p.O * (double)p.I;
    c.bm = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    if (fits && (p.E ? p.R > 16 : rows > 16 || bytes > 64e6)) {
        c.plan = plan_tiles(p, direct, ncu);
        const double w = c.bm == 16 ? 1.0 : c.bm == 32 ? 1.8 : 3.2;
        c.tile = p.E || rows > 64 || c.plan.us < 7.0 + w * bytes / 5e6;
    }
    if (c.tile) c.bm = TILE_KINDS[c.plan.kind].bt;
    else c.plan.parts = 1;
    return c;
}

}  // namespace qg
