// w4_dec_bf16_32.hip -- few-token 4-bit kernels, bf16, fold unit 32 (groups of other multiples of 32).
#include "w4_dec_launch.hpp"

namespace qlin {

hipError_t w4_dec_bf16_32(const W4DecParams& p, bool glu, hipStream_t st) { return w4_dec<kBf16, 32>(p, glu, st); }

}  // namespace qlin
