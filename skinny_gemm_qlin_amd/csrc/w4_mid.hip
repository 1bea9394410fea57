// w4_mid.hip -- launchers of the kernels for 9 to 64 tokens (w4_mid.hpp).
#include "w4_mid_launch.hpp"
#include <stdlib.h>

namespace qlin {

namespace {

constexpr uint32_t kLdsBytes = 160 * 1024;

template <int T, int MT, int NTL, int STAGES>
hipError_t run(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int BM = 32 * MT, BN = 32 * NTL;
    const int CT = p.I > 0 ? BN / 2 : BN;
    const uint32_t ring = STAGES * w4_mid_stage<BM, BN>() + pl.scales, sums = 8 * BM * BN * 4;
    hipLaunchKernelGGL((w4_mid_kernel<T, MT, NTL, STAGES>), dim3((unsigned)((p.C + CT - 1) / CT)), dim3(512),
                       ring > sums ? ring : sums, st, p);
    return hipGetLastError();
}

template <int T>
hipError_t tokens(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    if (p.M <= 32) return pl.ntl == 2 ? run<T, 1, 2, 3>(p, pl, st) : run<T, 1, 1, 3>(p, pl, st);
    return pl.ntl == 2 ? run<T, 2, 2, 2>(p, pl, st) : run<T, 2, 1, 2>(p, pl, st);
}

}  // namespace

bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o) {
    if (M > kW4MidMaxM) return false;
    const int64_t groups = K / group;
    if (groups > kLdsBytes / 64) return false;
    const uint32_t ring1 = M <= 32 ? 3 * w4_mid_stage<32, 32>() : 2 * w4_mid_stage<64, 32>();
    const uint32_t ring2 = M <= 32 ? 3 * w4_mid_stage<32, 64>() : 2 * w4_mid_stage<64, 64>();
    o.scales = w4_mid_scales(32, (int)groups);
    if (ring1 + o.scales > kLdsBytes) return false;
    const uint32_t s2 = w4_mid_scales(64, (int)groups);
    static int f = getenv("W4_NTL") ? atoi(getenv("W4_NTL")) : 0;
    o.ntl = (glu ? 2 * C : C) > 256 * 32 && ring2 + s2 <= kLdsBytes ? 2 : 1;
    if (f) o.ntl = f;
    if (o.ntl == 2) o.scales = s2;
    return true;
}

hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    return dtype == kFp16 ? tokens<kFp16>(p, pl, st) : tokens<kBf16>(p, pl, st);
}

}  // namespace qlin
