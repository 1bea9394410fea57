// i8ffn_plan.hpp -- which kernel the INT8 feed-forward operators take, by sizes
// alone: plain C++, so that a host test can ask too.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace qlin {

// ---------------------------------------------------------------- up to 16 tokens: i8ffn_few.hpp
constexpr int kFewPairs = 256;   // 16 tokens, 16 slots
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;  // one workgroup a compute unit: 16 waves, or two workgroups, are slower
constexpr int kFewTokens = 16;   // tokens of a chunk at most: four column sets
constexpr int kFewUnitsPerWave = 6, kFewUnits = kFewUnitsPerWave * kFewWaves;  // x 512 elements that a workgroup quantises
constexpr int kFewLds = 146 * 1024;  // dynamic LDS next to the lists, of 160 KB
constexpr int kFewSums = 16 * 1024;  // of which the down projection's sums
constexpr int kFewGrid = 256;        // compute units
static_assert(kFewSums / (16 * kFewPairs) >= 1, "LDS holds the sums of a row group");

// A turn: steps of 256 K that a wave's loads are ahead of its products.  An item's K is a whole number of turns, so
// three where that saves steps (K = 768: 3 instead of 4; 2064: 9 instead of 12).
constexpr int few_turn(int64_t K) {
    const int64_t steps = (K + 255) / 256;
    return (steps + 2) / 3 * 3 < (steps + 3) / 4 * 4 ? 3 : 4;
}
// LDS pitch of a code row: whole turns, and the four tokens of a column set 64 bytes (16 banks) apart
constexpr int few_pitch(int64_t K, int turn) { return (int)((K + 256 * turn - 1) / (256 * turn)) * (256 * turn) + 64; }
constexpr int few_pitch(int64_t K) { return few_pitch(K, few_turn(K)); }
static_assert(few_pitch(131072) <= kFewLds - kFewSums && few_pitch(131072 - 16) <= kFewLds - kFewSums, "LDS holds the longest row");

// All tokens' codes are in LDS at once.  (9 to 16 rows longer than that go to the GEMM.)
constexpr bool few_fits(int64_t M, int64_t K) { return M <= kFewTokens && M * few_pitch(K) <= kFewLds; }

// Each workgroup quantises the rows for itself, or copies the codes that a kernel ahead wrote.
constexpr bool few_quantise(int64_t rows, int64_t K) { return rows * ((K + 511) / 512) <= kFewUnits; }

// Column sets (of 4 tokens) a chunk has: all tokens where they are few, else a multiple of what an expert has on
// average, as four sets take four times the products and code reads of one (an expert that has more is taken in two
// chunks).  E = 0: dense.
constexpr int few_sets(int64_t M, int64_t topk, int64_t E) {
    const int64_t often = E > 0 ? 4 * M * topk / E + 3 : M, most = often < M ? often : M;
    return most <= 4 ? 1 : (most <= 8 ? 2 : 4);
}

// Pairs' code rows that LDS holds in the down projection, and the pairs of a chunk.
constexpr int64_t few_down_rows(int64_t P, int64_t I) {
    const int64_t n = (kFewLds - kFewSums) / few_pitch(I);
    return P < n ? P : n;
}
constexpr int64_t few_chunk(int64_t M, int64_t topk, int64_t E, int64_t I) {
    const int64_t n = few_down_rows(M * topk, I), s = 4 * few_sets(M, topk, E);
    return s < n ? s : n;
}

// Workgroups of the down projection, and the 4-row groups of the output whose sums one of them holds in LDS at once: a
// workgroup whose share has more takes them in blocks of that many.
constexpr int few_down_grid(int64_t H) { return H / 4 < kFewGrid ? (int)(H / 4) : kFewGrid; }
constexpr int few_down_most(int64_t H) { return (int)((H / 4 + few_down_grid(H) - 1) / few_down_grid(H)); }
constexpr int few_down_block(int64_t P, int64_t H) {
    const int n = (int)(kFewSums / (16 * P));  // at least 4: P <= kFewPairs
    return few_down_most(H) < n ? few_down_most(H) : n;
}

// ---------------------------------------------------------------- more: i8ffn_gemm.hpp
// Code rows of an expert's tile, by what experts have on average.  64 experts, top 6, 7168 x 2048, calls: 17 tokens 368
// us with 32 rows, 463 with 64; 150 tokens 527 and 536.  Front and down with 28 pairs each: 345 + 216 us with 64 rows,
// 372 + 258 with 128; with 94 pairs each 509 + 349 and 409 + 303.
constexpr int i8_tile_rows(int64_t P, int64_t E) { return P <= 16 * E ? 32 : (P <= 56 * E ? 64 : 128); }

// Tile (code rows x weight rows) of a dense front: smaller ones where the larger leave half of the compute units idle.
// 2 x 4096 x 7168: 64 tokens 29 us with 64 x 64, 36 with 64 x 128; 128 tokens 30, 36 and 44 with 128 x 128.
// 2 x 14336 x 4096, 64 tokens: 36 us with 64 x 64, 34 with 64 x 128.  The rings of 128 x 128 are four deep, one workgroup
// a compute unit; two deep where that lets all of them run at once (2 x 14336 x 4096: 200 tokens, 448 workgroups, 50 us
// with two, 55 with four; 300 tokens, 672 workgroups, 82 and 76).
enum I8DenseTile { kI8Tile64x64 = 0, kI8Tile64x128 = 1, kI8Tile128x128 = 2, kI8TwoOf128x128 = 3 };
constexpr I8DenseTile i8_dense_tile(int64_t M, int64_t I) {
    const int64_t columns = (I + 63) / 64;  // gated: 128 weight rows give 64 columns
    const int64_t large = (M + 127) / 128 * columns;
    if ((M + 63) / 64 * columns <= 128) return kI8Tile64x64;
    if (M <= 64 || large <= 128) return kI8Tile64x128;
    return large <= 256 || large > 512 ? kI8Tile128x128 : kI8TwoOf128x128;
}

// Output columns of a dense front that 256 x 256 tiles (128 columns) compute in whole rounds of 256.
constexpr int64_t i8_large_columns(int64_t M, int64_t I) {
    if (M < 1024) return 0;
    const int64_t mt = (M + 255) / 256, all = mt * (I / 128), rounds = all / 256;
    return rounds * 256 / mt * 128;
}

}  // namespace qlin
