// i8ffn_plan.hpp -- which kernel the INT8 feed-forward operators take, by sizes
// alone: plain C++, so that a host test can ask too.
//
// Times beside the rules are microseconds of a whole call without its host part
// (captured, cold weights), the smallest of four to seven rounds, both sides in turn.  A
// front's sizes are tokens x (2 x outputs) x K, a layer's tokens, experts top slots,
// H x I.
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
// three where that saves steps (K = 768: 3 instead of 4; 2064: 9 instead of 12), four where it does not.  One token, 2 x
// 14336 outputs, turns of three and four: K = 768 8.4 and 8.7, 2064 15.2 and 15.9, 4096 24.4 and 22.4; 2 x 28672 x 1024
// 17.1 and 13.8; layer of 16 tokens, 128 top 8, 2048 x 768: 4 in the front and 3 down 85.3, all three 92.4, all four 88.6.
constexpr int few_turn(int64_t K) {
    const int64_t steps = (K + 255) / 256;
    return (steps + 2) / 3 * 3 < (steps + 3) / 4 * 4 ? 3 : 4;
}
// LDS pitch of a code row: whole turns, and the four tokens of a column set 64 bytes (16 banks) apart
constexpr int few_pitch(int64_t K, int turn) { return (int)((K + 256 * turn - 1) / (256 * turn)) * (256 * turn) + 64; }
constexpr int few_pitch(int64_t K) { return few_pitch(K, few_turn(K)); }
static_assert(few_pitch(131072) <= kFewLds - kFewSums && few_pitch(131072 - 16) <= kFewLds - kFewSums, "LDS holds the longest row");

// All tokens' codes are in LDS at once: M x few_pitch(K) <= 146 KB.  16 tokens fit up to K = 9216, 8 up to 18432, 2 up to
// 74496, one always.  Longer rows go to the GEMM, which takes 1.4 to 3 times as long there: 2 x 2051 outputs, 16 tokens
// 16.2 at K = 9216 and 34.1 at 9232, 11 tokens 19.0 at 13312 and 44.9 at 13328, 2 tokens 69 at 73728 and 219 at 74512;
// 16 x (2 x 14336): 50 at 9216 and 68 at 9232.
constexpr bool few_fits(int64_t M, int64_t K) { return M <= kFewTokens && M * few_pitch(K) <= kFewLds; }

// Each workgroup quantises the rows for itself, or copies the codes that a kernel ahead wrote (a launch more).  The first
// and the second way: 1 x (2 x 2048) x 4096 (8 units) 7.3 and 9.8, 1 x (2 x 14336) x 4096 22.0 and 24.1, 4 x the same (32)
// 23.8 and 24.1, 2 x (2 x 4096) x 12288 (48) 24.3 and 25.0; layer of one token, 64 top 6, 7168 x 2048 (14 and 24) 51.1 and
// 53.1.  Between 33 and 48 units of more than two rows the second is 0.6 to 1.9 us faster: 6 x (2 x 14336) x 4096 25.7 and
// 24.4, 16 x (2 x 4096) x 1536 10.8 and 8.9.  Beyond 48 the first needs 12 loads a lane: 8 x (2 x 14336) x 4096 (64) 27.7
// and 24.7, 12 x (2 x 4096) x 4096 (96) 18.1 and 13.1, 2 x (2 x 4096) x 16384 (64) 34.8 and 35.9.
constexpr bool few_quantise(int64_t rows, int64_t K) { return rows * ((K + 511) / 512) <= kFewUnits; }

// Column sets (of 4 tokens) a chunk has: all tokens where they are few, else a multiple of what an expert has on
// average, as four sets take four times the products and code reads of one (an expert that has more is taken in several
// chunks).  E = 0: dense.  With one, two and four sets: layers of 16 tokens, 64 top 6, 7168 x 2048 (rule: 4) 352, 329 and
// 336; 128 top 8, 2048 x 768 (2) 86, 89 and 95; 8 top 2, 4096 x 3584 (4) 82, 74 and 74; 8 tokens of 64 top 6 (2) 225, 225
// and 229; a front of 1 x (2 x 14336) x 4096 21.5, 21.6 and 22.5.  An expert with far more pairs than the average is read
// several times, at little cost: 16 tokens all to one of 128 experts, 2048 x 768 (1) 16.5, 16.2 and 16.9; half of the
// pairs of 64 top 6 to one (4) 393, 367 and 356.
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
// 372 + 258 with 128; with 94 pairs each 509 + 349 and 409 + 303.  With 256 pairs and more a layer of 128-row tiles is bound
// by the matrix cores: 8 top 2, 4096 x 14336, 1024 tokens 729 (64 rows: 805), 4096 tokens 2080 (2573).  The average is all
// that is known on the host: with half of the pairs to one expert 64 tokens of 64 top 6 (rule: 32) take 513, 518 with 64
// rows; 1000 tokens (128) 858, 855 with 64 and 1142 with 32; spread evenly 718, 859 and 980.
constexpr int i8_tile_rows(int64_t P, int64_t E) { return P <= 16 * E ? 32 : (P <= 56 * E ? 64 : 128); }

// Tile (code rows x weight rows) of a dense front: smaller ones where the larger leave half of the compute units idle.
// 2 x 4096 x 7168: 64 tokens 29 us with 64 x 64, 36 with 64 x 128; 128 tokens 30, 36 and 44 with 128 x 128.
// 2 x 14336 x 4096, 64 tokens: 36 us with 64 x 64, 34 with 64 x 128.  The rings of 128 x 128 are four deep, one workgroup
// a compute unit; two deep where that lets all of them run at once.  K = 4096, by workgroups, four deep and two deep: 256
// 32.0 and 42.0, 384 54.0 and 49.1, 448 53.4 and 51.5, 512 56.3 and 52.5, 516 69.2 and 71.8, 576 72.5 and 81.4, 672 74.2 and
// 82.0, 768 79.2 and 84.3, but 896 103.2 and 95.0.  K = 7168: 448 81.9 and 80.2, 672 110.9 and 131.5.  K = 1024 is faster two
// deep past 512 too: 672 32.3 and 28.0.
enum I8DenseTile { kI8Tile64x64 = 0, kI8Tile64x128 = 1, kI8Tile128x128 = 2, kI8TwoOf128x128 = 3 };
constexpr I8DenseTile i8_dense_tile(int64_t M, int64_t I) {
    const int64_t columns = (I + 63) / 64;  // gated: 128 weight rows give 64 columns
    const int64_t large = (M + 127) / 128 * columns;
    if ((M + 63) / 64 * columns <= 128) return kI8Tile64x64;
    if (M <= 64 || large <= 128) return kI8Tile64x128;
    return large <= 256 || large > 512 ? kI8Tile128x128 : kI8TwoOf128x128;
}

// Output columns of a dense front that 256 x 256 tiles (128 columns) compute in whole rounds of 256, from 1024 tokens on.
// With and without: 2 x 14336 x 4096, 1024 tokens 152.8 and 175.0, 1200 tokens 172.8 and 213.4; 2 x 8192 x 7168, 1024 tokens
// 123.5 and 161.7; 2 x 4096 x 7168, 2048 tokens 124.2 and 156.8.  Fewer tokens that fill a round would gain as well: 2 x
// 14336 x 4096, 768 tokens 122.5 with and 142.4 without; so would a round that is nearly full (512 tokens, 224 tiles: 78.4
// and 103.4) and not one that has just begun (600 tokens, all columns in large tiles: 135.4 and 122.8).
constexpr int64_t i8_large_columns(int64_t M, int64_t I) {
    if (M < 1024) return 0;
    const int64_t mt = (M + 255) / 256, all = mt * (I / 128), rounds = all / 256;
    return rounds * 256 / mt * 128;
}

}  // namespace qlin
