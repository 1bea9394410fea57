// w4_dec_fp16_128.hip -- few-token 4-bit kernels, fp16, fold unit 128 (groups that are multiples of 128).
#include "w4_dec_launch.hpp"

namespace qlin {

hipError_t w4_dec_fp16_128(const W4DecParams& p, bool glu, hipStream_t st) { return w4_dec<kFp16, 128>(p, glu, st); }

}  // namespace qlin
