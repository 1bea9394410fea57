// What i8ffn_plan.hpp says of the down projection for up to 16 tokens: M H I topk E ->
//   fits, own codes, pairs, row groups a workgroup has at most, row groups a block, code rows in LDS, pairs a chunk
#include <cstdio>
#include <cstdlib>

#include "../skinny_gemm_qlin_amd/csrc/i8ffn_plan.hpp"

int main(int argc, char** argv) {
    using namespace qlin;
    if (argc != 6) return 2;
    const int64_t M = std::atoll(argv[1]), H = std::atoll(argv[2]), I = std::atoll(argv[3]), topk = std::atoll(argv[4]),
                  E = std::atoll(argv[5]), P = M * topk;
    std::printf("%d %d %lld %d %d %lld %lld\n", few_fits(M, H), few_quantise(P, I), (long long)P, few_down_most(H),
                few_down_block(P, H), (long long)few_down_rows(P, I), (long long)few_chunk(M, topk, E, I));
    return 0;
}
