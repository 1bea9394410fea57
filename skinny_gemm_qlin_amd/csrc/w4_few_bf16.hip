// w4_few_bf16.hip -- decode 4-bit kernels, bf16.
#include "w4_few_launch.hpp"

namespace qlin {

hipError_t w4_few_bf16(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    if (p.w.group % 128 == 0) return w4_few_u<kBf16, 128>(p, pl, st);
    if (p.w.group % 64 == 0) return w4_few_u<kBf16, 64>(p, pl, st);
    return w4_few_u<kBf16, 32>(p, pl, st);
}

}  // namespace qlin
