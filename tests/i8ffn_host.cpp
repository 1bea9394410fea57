// Host checks of the INT8 feed-forward operators' arithmetic and of the rules by which sizes choose a kernel.
//   quotients        every mantissa of a 16-bit x against every scale that a largest magnitude can give
//   plan ...         what i8ffn_plan.hpp answers
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "../skinny_gemm_qlin_amd/csrc/i8ffn_plan.hpp"

// codes by the kernels' way and by the division, for all x of `bits` mantissa bits up to the largest, 2^top .. 2^(top - down)
static long differ(int bits, int top, int down) {
    long bad = 0;
    const int one = 1 << bits;
    for (int ma = one; ma < 2 * one; ++ma) {
        const float amax = std::ldexp((float)ma, top - bits);
        const float s = amax / 127.0f;
        if (!(s >= 0x1p-100f)) continue;
        const float r = 1.0f / s;
        for (int e = 0; e <= down; ++e)
            for (int mx = one; mx < 2 * one; ++mx) {
                const float x = std::ldexp((float)mx, top - e - bits);
                if (x > amax) break;
                const float t = x * r;
                const float got = std::rint(std::fma(std::fma(-t, s, x), r, t));
                float want = std::rint(x / s);
                if (want > 127.0f) want = 127.0f;
                if (got != want) ++bad;
            }
    }
    return bad;
}

int main(int argc, char** argv) {
    using namespace qlin;
    if (argc > 1 && !std::strcmp(argv[1], "quotients")) {
        long bad = 0;
        for (int top : {0, 15, 127, -60, -93}) bad += differ(7, top, 24);
        for (int top : {0, 15, -14}) bad += differ(10, top, 10);
        std::printf("%ld\n", bad);
        return 0;
    }
    if (argc == 7 && !std::strcmp(argv[1], "plan")) {
        const int64_t M = std::atoll(argv[2]), K = std::atoll(argv[3]), I = std::atoll(argv[4]), topk = std::atoll(argv[5]),
                      E = std::atoll(argv[6]);
        std::printf("%d %d %d %d %lld %lld %lld %lld %lld\n", few_fits(M, K), few_quantise(M, K), few_turn(K),
                    few_sets(M, topk, E), (long long)few_down_rows(M * topk, I), (long long)few_chunk(M, topk, E, I),
                    (long long)(E > 0 ? i8_tile_rows(M * topk, E) : 0), (long long)i8_dense_tile(M, I),
                    (long long)i8_large_columns(M, I));
        return 0;
    }
    return 2;
}
