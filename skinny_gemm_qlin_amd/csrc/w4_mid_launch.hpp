// w4_mid_launch.hpp -- plan and launcher of the kernels for 17 to 64
// tokens and for small matrices.
#pragma once
#include "w4_mid.hpp"

namespace qlin {

struct W4MidPlan { int ntl, stages; uint32_t scales; float us; };  // row tiles, LDS of the scales, estimated time

// false if the scales of 32 rows do not fit LDS next to two stages
bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o);
hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st);

}  // namespace qlin
