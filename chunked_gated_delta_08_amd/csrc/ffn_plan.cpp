// ffn_plan.cpp -- which tile and how many splits a product of the feed-forward block takes.
#include "ffn_plan.hpp"

#include <algorithm>

namespace ffn {

namespace {
// Of each tile: its sizes, how many workgroups a CU holds, and in us the time of a step where one of them has
// the CU, where as many as it holds share it (all of them), and of the rest of a tile, for 16-bit types and fp32
// (0: not used, the smaller tiles are as fast; an fp32 step is bound by the matrix unit whatever the tile).
// Fitted to 9036 (16-bit) and 8696 (fp32) timings of the products, 62 and 47 sizes from 100 to 16384 tokens,
// every tile and number of splits.  What the estimate picks, measured on 350 and 134 other sizes of 65 to 16384 tokens: a
// forward takes 1.0 % longer than with the fastest tile and splits of gate and up, or of down, on average and 22 % at
// worst, a backward 1.0 % and 23 % for dh.
struct Tile {
    int bm, bn, held;
    float one[2], all[2], rest[2];
};
constexpr Tile TILE[] = {
    {256, 256, 1, {1.38f, 0.f}, {1.38f, 0.f}, {2.0f, 0.f}},
    {256, 128, 1, {0.78f, 0.f}, {0.78f, 0.f}, {1.8f, 0.f}},
    {128, 128, 2, {0.585f, 1.88f}, {0.836f, 3.56f}, {0.1f, 1.4f}},
    {128, 128, 1, {0.47f, 0.f}, {0.47f, 0.f}, {1.1f, 0.f}},
    {64, 128, 2, {0.327f, 1.01f}, {0.57f, 1.9f}, {0.65f, 1.0f}},
    {64, 64, 2, {0.194f, 0.534f}, {0.369f, 1.0f}, {0.41f, 1.2f}},
};
constexpr float JOIN = 3.f, JOIN_SUM = 1.1e-6f;   // the launch that joins splits, and for each sum of a split
// The same for up to 64 rows of a product with weights stored [n][k] (GATE_UP, DOWN), with the time that the join takes
// for each split. From 2600 and 2700 timings of the products, 192 sizes each with 1 to 64 tokens; measured on 1927 and 962 other
// sizes: a forward takes 1.0 to 1.7 % longer than with the fastest choice for either product, at worst 16 % (splits wherever
// CUs were free took 6 %: whole forwards in a graph, us,
// 25 x 512 x 1408 bf16 11.6 and now 9.7, 64 x 1024 x 2816 17.3 and 14.1, 64 x 4096 x 5632 fp32 112 and 94).
constexpr Tile FEW[] = {
    {32, 64, 2, {0.135f, 0.327f}, {0.241f, 0.62f}, {1.7f, 1.1f}},
    {64, 128, 2, {0.305f, 1.04f}, {0.744f, 1.99f}, {2.0f, 2.4f}},
    {64, 64, 2, {0.186f, 0.578f}, {0.459f, 1.05f}, {1.9f, 1.0f}},
};
constexpr int FEW_CONFIG[] = {THIN, LOW, SMALL};
constexpr float FEW_JOIN[] = {1.2f, 1.3f}, FEW_SPLIT[] = {0.25f, 0.3f}, FEW_SUM[] = {1.9e-6f, 1.1e-6f};
constexpr int CUS = 256;

Shape shape(Kind kind, int c, int bm, int bn, int M, int N, int all, int want) {
    const int bt = kind == GATE_UP ? bn / 2 : bn;
    Shape s{c, 1, 0, (M + bm - 1) / bm, (N + bt - 1) / bt};
    s.steps = (all + want - 1) / want;
    if (s.steps) s.splits = (all + s.steps - 1) / s.steps;
    return s;
}
}  // namespace

// The tile and the splits of least estimated time: each CU takes its share of the workgroups, as
// many at once as it holds; splits add the sums' way through memory.
Shape shape_of(Kind kind, int M, int N, int K, int esize) {
    const int ke = 128 / esize, all = (K + ke - 1) / ke, wide = esize == 4, pair = kind == GATE_UP ? 2 : 1;
    const bool few = M <= 64 && (kind == GATE_UP || kind == DOWN);
    Shape best{};
    float least = 0.f;
    auto consider = [&](const Tile& t, int c) {
        for (int want = 1; want <= (few ? 32 : 16); want++) {
            const Shape s = shape(kind, c, t.bm, t.bn, M, N, all, want);
            const int64_t tiles = (int64_t)s.tilesM * s.tilesN;
            if (want > 1 && (all < (few ? 2 : 4) * want || tiles * (want - 1) >= (few ? 4 : 2) * CUS)) break;
            if (want > 1 && s.splits != want) continue;
            const int64_t each = (tiles * s.splits + CUS - 1) / CUS, full = each / t.held, odd = each % t.held;
            float us = full * (s.steps * t.all[wide] + t.rest[wide]) + odd * (s.steps * t.one[wide] + t.rest[wide]);
            if (s.splits > 1) {
                us += few ? FEW_JOIN[wide] + FEW_SPLIT[wide] * s.splits : JOIN;
                us += (few ? FEW_SUM[wide] : JOIN_SUM) * s.splits * M * N * pair;
            }
            if (best.tilesM == 0 || us < least) least = us, best = s;
        }
    };
    if (few) {
        for (int i = 0; i < 3; i++)
            if ((M <= 32) == (FEW_CONFIG[i] == THIN)) consider(FEW[i], FEW_CONFIG[i]);
    } else {
        for (int c = 0; c < THIN; c++)
            if (TILE[c].one[wide] != 0.f) consider(TILE[c], c);
    }
    return best;
}

size_t part_floats(Kind kind, int M, int N, int K, int esize) {
    const Shape s = shape_of(kind, M, N, K, esize);
    return s.splits > 1 ? (size_t)s.splits * M * N * (kind == GATE_UP ? 2 : 1) : 0;
}

namespace {
// When the workgroups of the gradients' products are through, in us: they start in their order wherever a place is free,
// those of a product take the same time.  The constants, as TILE's, from 17 sizes with each tile and number of splits; on the 350
// and 134 sizes named there a backward takes 2.5 % (fp32 3.4 %) longer than with the fastest tile and splits, at worst 19 %.
float makespan(const Shape (&s)[3], const Tile& t, int wide) {
    struct { float at; int64_t places; } level[8];
    int64_t total = 0;
    for (const Shape& x : s) total += (int64_t)x.tilesM * x.tilesN * x.splits;
    const bool alone = total <= CUS;
    const int64_t places = alone ? CUS : (int64_t)CUS * t.held;
    int n = 1;
    level[0] = {0.f, places};
    float end = 0.f;
    for (const Shape& x : s) {
        int64_t left = (int64_t)x.tilesM * x.tilesN * x.splits;
        const float d = x.steps * (alone ? t.one : t.all)[wide] + t.rest[wide];
        const int64_t rounds = left / places;   // every place gets as many
        for (int i = 0; i < n; i++) level[i].at += rounds * d, end = std::max(end, level[i].at);
        left -= rounds * places;
        while (left > 0) {   // the earliest places
            int e = 0;
            for (int i = 1; i < n; i++)
                if (level[i].at < level[e].at) e = i;
            const int64_t m = std::min(left, level[e].places);
            const float at = level[e].at + d;
            end = std::max(end, at);
            left -= m;
            if (m == level[e].places || n == 8) level[e].at = at;
            else level[e].places -= m, level[n++] = {at, m};
        }
    }
    return end;
}
constexpr Tile GRAD_TILE[] = {
    {256, 256, 1, {1.55f, 0.f}, {1.55f, 0.f}, {6.4f, 0.f}},
    {256, 128, 1, {0.89f, 0.f}, {0.89f, 0.f}, {4.2f, 0.f}},
    {128, 128, 2, {0.71f, 1.88f}, {0.96f, 3.56f}, {1.3f, 1.4f}},
    {64, 64, 2, {0.f, 0.534f}, {0.f, 1.0f}, {0.f, 1.2f}},
};
constexpr int GRAD_CONFIG[] = {BIG, WIDE, MIDDLE, SMALL};
// The weights' gradients sum over the tokens, up to 2^24 of them.  Steps that a split adds up at most, for 16-bit types and
// fp32, 4096 matrix instructions of 32 and of 4 products: an fp32 sum of equal signs loses a unit in the last place
// with each (2^24 equal tokens in fp32, in four splits of a million instructions: 5 % off; 131072 and 16384 tokens a split now).
constexpr int LONGEST[] = {2048, 512};
// The join's time for each split, where they are more than the four that JOIN counts.  Backward, us, with 4, 8, 16, 32, 64 and 128
// splits of these sums, bf16: 16384 x 64 x 64 47.0, 27.6, 20.4, 17.9, 18.8, 25.6; 16384 x 128 x 256 57.9, 38.4, 31.1, 32.3,
// 35.0, 46.0; 65536 x 256 x 512 331, 229, 201, 206, 243, 279; 65536 x 1024 x 2816 2328, 2351, 2423, 2555, 2904, 3658.
constexpr float JOIN_SPLIT = 0.25f;
}  // namespace

GradPlan grad_plan(int T, int D, int F, int esize) {
    const int ke = 128 / esize, wide = esize == 4;
    const int M[3] = {T, 2 * F, D}, N[3] = {D, D, F}, K[3] = {2 * F, T, T};
    static const int by_dx[3] = {0, 1, 2}, by_dw[3] = {1, 2, 0}, dx_splits[] = {1, 2, 3, 4, 6, 8};
    int first = 1;   // splits of the sums over the tokens: powers of two from here on
    while ((T + ke - 1) / ke > first * LONGEST[wide]) first *= 2;
    const int* order = 2 * F >= T ? by_dx : by_dw;   // the longest sums first
    GradPlan best{};
    float least = -1.f;
    for (int c = 0; c < 4; c++) {
        const Tile& t = GRAD_TILE[c];
        if (t.one[wide] == 0.f) continue;
        auto fits = [&](int j, int want) {   // splits while there is work for them and room
            const Shape x = shape(DX, c, t.bm, t.bn, M[j], N[j], (K[j] + ke - 1) / ke, want);
            return (K[j] + ke - 1) / ke >= 4 * want && (int64_t)x.tilesM * x.tilesN * (want - 1) < 2 * CUS;
        };
        for (int sx : dx_splits) {
            if (sx > 1 && !fits(0, sx)) break;
            for (int sw = first; sw == first || (fits(1, sw) && fits(2, sw)); sw *= 2) {
                GradPlan p{GRAD_CONFIG[c], {}, {order[0], order[1], order[2]}};
                float us = sw > 4 ? JOIN_SPLIT * sw : 0.f;
                bool joined = false;
                for (int i = 0; i < 3; i++) {
                    const int j = order[i];
                    const Shape x = shape(DX, c, t.bm, t.bn, M[j], N[j], (K[j] + ke - 1) / ke, j == 0 ? sx : sw);
                    if (x.splits > 1) joined = true, us += JOIN_SUM * x.splits * M[j] * N[j];
                    p.s[i] = x;
                }
                us += makespan(p.s, t, wide) + (joined ? JOIN : 0.f);
                if (least < 0.f || us < least) least = us, best = p;
            }
        }
    }
    return best;
}

size_t grad_floats(const GradPlan& p, int T, int D, int F) {
    const size_t size[3] = {(size_t)T * D, 2 * (size_t)F * D, (size_t)D * F};
    size_t n = 0;
    for (int i = 0; i < 3; i++)
        if (p.s[i].splits > 1) n += p.s[i].splits * size[p.order[i]];
    return n;
}

}  // namespace ffn
