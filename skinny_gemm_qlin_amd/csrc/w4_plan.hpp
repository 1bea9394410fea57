// w4_plan.hpp -- how a forward call of the 4-bit weight operators is laid out:
// which kernel takes it, with how many rows, waves, passes and stages.  Sizes
// in, numbers out: plain C++ for the host (its layout functions serve the
// kernels, too).
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace qlin {

constexpr uint32_t kW4LdsBytes = 160 * 1024;  // of a compute unit

// ---------------------------------------------------------------- up to 16 tokens (w4_few.hpp)
// floats that an output's wave sums take: whole 16 bytes, not 16 of them so that rows start in different banks
constexpr int w4_few_red(int nw) { return nw > 12 ? 20 : (nw + 3) / 4 * 4; }

constexpr int kW4FewLoad = 512 + 8;  // elements that a 1 KB load of token rows takes: the next starts 16 bytes of banks on

// Dynamic LDS: each wave's lines of the token rows, X of its fold units, scales and zero points as they are in
// memory (from the 16-byte line their block starts in), the waves' sums.
struct W4FewLds { uint32_t xsum, s, z, red, total; };

constexpr W4FewLds w4_few_lds(int M, int U, int PL, int cols, int wrows, int groups, int nw) {
    auto up = [](uint32_t b) { return (b + 15u) / 16u * 16u; };
    W4FewLds o{};
    o.xsum = (uint32_t)(nw * ((PL * M + 1) / 2)) * kW4FewLoad * 2;
    o.s = o.xsum + (uint32_t)nw * (PL * (128 / U)) * (M > 8 ? 128 : 64);
    o.z = o.s + up((uint32_t)(wrows * groups * 2)) + 64;  // gated: two blocks, each with its own start and end
    o.red = o.z + up((uint32_t)(wrows * groups)) + 64;
    o.total = o.red + (uint32_t)(M * cols * w4_few_red(nw)) * 4;
    return o;
}

constexpr int kW4FewMaxM = 16;

// How a call is laid out; false if its token rows and the scales of one tile
// of rows do not fit LDS.  They do up to 5300 groups a row for 1 to 8 tokens
// and 2600 for 9 to 16 (the worst of all sizes; tiles of 16 rows), gated 2600
// and 1290 (two tiles): the rows for which qlin.h promises unrounded weights.
struct W4FewPlan { int pl, nw, passes, rows, depth; uint32_t lds; };

inline bool w4_few_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4FewPlan& o) {
    if (M > kW4FewMaxM) return false;
    const int U = group % 128 == 0 ? 128 : (group % 64 == 0 ? 64 : 32);
    const int64_t lines = (K + 255) / 256, groups = K / group;
    // one line a wave on short rows: more waves to hide latency (1024 x 1024: 3.3 us, two lines 3.4)
    // 9 to 16 tokens: one, or the two halves' operands would not fit the registers
    const bool full = M > 8;
    o.pl = lines <= 8 || full ? 1 : 2;
    const int TR = full ? 16 : 8;
    // One workgroup a compute unit, several (that LDS holds together) where a workgroup has few waves, at least
    // 8 columns each.  Where LDS does not hold a share, K is first walked in up to four times as many passes, then
    // the shares get smaller and the rounds of workgroups more.
    const int64_t least = (lines + 16 * o.pl - 1) / (16 * o.pl);
    const int64_t fewest = (lines + 4 * least * o.pl - 1) / (4 * least * o.pl), tile = TR * (glu ? 2 : 1);
    if (tile * groups >= kW4LdsBytes ||
        w4_few_lds((int)M, U, o.pl, glu ? 16 : 8, (int)tile, (int)groups, (int)fewest).total > kW4LdsBytes)
        return false;
    for (int64_t rounds = 1;; ++rounds) {  // ends at the latest with 8 columns and the fewest waves
        for (int64_t passes = least; passes <= 4 * least; ++passes) {
            o.nw = (int)((lines + passes * o.pl - 1) / (passes * o.pl));
            o.passes = (int)((lines + o.nw * o.pl - 1) / (o.nw * o.pl));
            for (int64_t per_cu = o.nw >= 12 ? 1 : 12 / o.nw; per_cu >= 1; --per_cu) {
                const int64_t wgs = 256 * per_cu * rounds;
                int64_t rows = (C + wgs - 1) / wgs;
                if (rows < 8) rows = 8;
                const int64_t wrows = (rows + TR - 1) / TR * TR * (glu ? 2 : 1);
                if (wrows >= 4096 || wrows * groups >= kW4LdsBytes) continue;
                o.rows = (int)rows;
                o.lds = w4_few_lds((int)M, U, o.pl, (int)rows * (glu ? 2 : 1), (int)wrows, (int)groups, o.nw).total;
                if (o.lds * per_cu > kW4LdsBytes && !(rows == 8 && o.lds <= kW4LdsBytes)) continue;
                // about 20 to 32 KB a compute unit in flight (17408 x 5120, 10 waves of two lines: one tile ahead
                // 11.5 us, two 11.4; 28672 x 4096 gated, 8 waves: 15.4 and 14.0).  Two tiles of 16 rows ahead do
                // not fit the registers with folds of 32 (16 tokens, 4096 x 4096, groups of 32: 8.9 and 11.9 us;
                // 9 tokens 8.0 and 10.1)
                o.depth = o.nw * o.pl * (full ? 2 : 1) > 16 || (full && U == 32) ? 1 : 2;
                return true;
            }
        }
    }
}

// ---------------------------------------------------------------- 17 to 64 tokens, small matrices (w4_mid.hpp)
constexpr int kW4MidStep = 256;

constexpr int w4_mid_stage(int XR, int NTL) { return (XR * 2 + NTL * 16) * kW4MidStep; }
// tokens whose sums are added at a time: the waves' sums take the first stage's LDS
constexpr int w4_mid_parts(int NTL) { return NTL > 1 ? 8 : 16; }

// scales and zero points of the workgroup's rows, as in memory from the 16-byte line each block starts in
constexpr uint32_t w4_mid_scales(int rows, int groups) {
    return ((uint32_t)(rows * groups * 2) + 15u) / 16u * 16u + ((uint32_t)(rows * groups) + 15u) / 16u * 16u + 128u;
}

constexpr uint32_t w4_mid_fixed_lds(int xr, int ntl, int stages) { return stages * w4_mid_stage(xr, ntl) + 256; }

// Stages: as many as leave 16 KB for scales, or one less where the scales take more.  A step's loads come back
// later than a step takes (48 tokens, 4096 x 7168, one row tile: two stages 28.8 us, three 22.4), so two, which
// one row tile goes down to, are for rows of more scales than fit next to three (64 tokens, 8192 rows, groups of 32:
// K = 17600, three stages, 55 us; K = 17632, two, 71 us, in the GEMM 302; K = 28672 107 us, in the GEMM 464).
constexpr int w4_mid_most_stages(int xr, int ntl) { return 4 * w4_mid_stage(xr, ntl) <= 144 * 1024 ? 4 : 3; }

struct W4MidPlan { int ntl, stages; uint32_t scales; float us; };  // row tiles, LDS of the scales, estimated time

// false if the scales of 32 rows do not fit LDS next to two stages.
// Row tiles of a workgroup.  A step of 256 K takes about 0.27 us and 0.29 us a tile with 32 tokens, 0.25 us and
// 0.4 us a tile with 64, and a call 6 us besides (17408 x 5120, 20 steps: 64 tokens, one tile in three rounds of
// workgroups 48 us, three tiles in one 35 us; 32 tokens 38 and 29 us), so the rounds decide.
inline bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o) {
    const int64_t groups = K / group, rows = glu ? 2 * C : C;
    if (groups > kW4LdsBytes / 64) return false;
    const int xr = M <= 32 ? 32 : (M <= 48 ? 48 : 64);
    o.ntl = 0;
    for (int ntl = 1; ntl <= 4; ++ntl) {
        const uint32_t scales = w4_mid_scales(32 * ntl, (int)groups);
        int stages = w4_mid_most_stages(xr, ntl);
        const int least = ntl == 1 ? 2 : stages - 1;
        while (stages > least && w4_mid_fixed_lds(xr, ntl, stages) + scales > kW4LdsBytes) --stages;
        if (w4_mid_fixed_lds(xr, ntl, stages) + scales > kW4LdsBytes) break;
        const int64_t wgs = ((rows + 32 * ntl - 1) / (32 * ntl)) * ((M + 63) / 64);
        const float step = (M <= 32 ? 0.27f + 0.29f * ntl : 0.25f + 0.4f * ntl) * (ntl == 1 && stages == 2 ? 1.3f : 1.f);
        const float us = 6.f + (float)((wgs + 255) / 256 * ((K + 255) / 256)) * step;
        if (o.ntl > 0 && us >= o.us) continue;
        o.us = us;
        o.ntl = ntl;
        o.stages = stages;
        o.scales = scales;
    }
    return o.ntl > 0;
}

// ---------------------------------------------------------------- more (w4_gemm.hpp)
// Estimated time of the GEMM with square tiles.  A 64-deep step of a 256 x 256 tile takes 1.95 us (one workgroup a
// compute unit), of a 128 x 128 tile 1.05 us alone on its unit and 1.2 to 1.4 us where two share one (2048 tokens,
// 17408 x 5120, 80 steps: 544 large tiles 478 us, 2176 small ones 489 us; 509 tokens, 4096 x 7168, 112 steps: 32
// large ones 203 us, 128 small ones 120 us; 256 tokens, 17408 x 5120, 272 small ones 120 us).
inline float w4_large_us(int64_t tiles, int64_t steps) { return (float)((tiles + 255) / 256 * steps) * 1.95f; }

inline float w4_small_us(int64_t tiles, int64_t steps) {
    const int64_t full = tiles / 512, rest = tiles - full * 512;
    return (float)steps * ((float)full * 1.22f + (rest == 0 ? 0.f : (rest <= 256 ? 1.05f : 1.4f)));
}

// Forward: `large` tile columns of 256 in large tiles, the rest in small ones.  Large tiles that would leave the
// last of several rounds of workgroups part empty give their last columns to small tiles (2048 tokens: 17408 x 5120,
// 2.1 rounds, 475 us in large tiles, 429 us so; 28672 x 4096 gated, 3.5 rounds, 532 and 521 us).
struct W4GemmPlan { int64_t large; float us; };

inline W4GemmPlan w4_gemm_plan(int64_t M, int64_t cols, int64_t R) {
    const int64_t steps = (R + 63) / 64, tm = (M + 255) / 256, tc = (cols + 255) / 256, tm2 = (M + 127) / 128;
    W4GemmPlan o{0, 10.f + w4_small_us(tm2 * ((cols + 127) / 128), steps)};
    const float all = 10.f + w4_large_us(tm * tc, steps);
    if (all <= o.us) o = {tc, all};
    const int64_t part = (tm * tc - 1) / 256 * 256 / tm;  // tile columns of all rounds but the last
    if (part > 0) {
        const float both = 15.f + w4_large_us(tm * part, steps) + w4_small_us(tm2 * ((cols - part * 256 + 127) / 128), steps);
        if (both < o.us) o = {part, both};
    }
    return o;
}

// The kernel for 17 to 64 tokens also takes longer batches, in blocks of 64, where the GEMM's tiles would leave
// compute units idle (128 tokens, 4096 x 7168: 22 us against 102), and matrices of fewer than four scales, which
// the GEMM loads four at a time.
inline bool w4_use_mid(int64_t M, int64_t N, int64_t K, int64_t group, const W4MidPlan& pl) {
    return N * (K / group) < 4 || pl.us < w4_gemm_plan(M, N, K).us;
}

}  // namespace qlin
