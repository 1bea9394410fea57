// w4_mid_launch.hpp -- launcher of the kernels for 17 to 64
// tokens and for small matrices.
#pragma once
#include "w4_mid.hpp"

namespace qlin {

hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st);

}  // namespace qlin
