// w4_mid_launch.hpp -- plan and launcher of the kernels for 9 to 64 tokens.
#pragma once
#include "w4_mid.hpp"

namespace qlin {

constexpr int kW4MidMaxM = 64;

struct W4MidPlan { int ntl; uint32_t scales; };

// false if the scales of 32 rows do not fit LDS next to two stages
bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o);
hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st);

}  // namespace qlin
