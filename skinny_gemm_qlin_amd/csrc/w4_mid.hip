// w4_mid.hip -- launchers of the kernels for 17 to 64 tokens and small matrices (w4_mid.hpp).
#include "w4_mid_launch.hpp"

namespace qlin {

namespace {

constexpr uint32_t kLdsBytes = 160 * 1024;

template <int T, int XR, int NTL, int STAGES>
hipError_t run(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int BM = (XR + 31) / 32 * 32, BN = 32 * NTL;
    static_assert(STAGES >= 2 && STAGES <= 4, "stages");
    const int CT = p.I > 0 ? BN / 2 : BN;
    hipLaunchKernelGGL((w4_mid_kernel<T, XR, NTL, STAGES>),
                       dim3((unsigned)((p.C + CT - 1) / CT), (unsigned)((p.M + BM - 1) / BM)), dim3(512), pl.scales, st, p);
    return hipGetLastError();
}

constexpr uint32_t fixed_lds(int xr, int ntl, int stages) { return stages * w4_mid_stage(xr, ntl) + 256; }

// Stages: as many as leave 16 KB for scales, or one less where the scales take more.  A step's loads come back
// later than a step takes (48 tokens, 4096 x 7168, one row tile: two stages 28.8 us, three 22.4).
constexpr int most_stages(int xr, int ntl) { return 4 * w4_mid_stage(xr, ntl) <= 144 * 1024 ? 4 : 3; }

template <int T, int XR, int NTL>
hipError_t stages(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int most = most_stages(XR, NTL);
    return pl.stages == most ? run<T, XR, NTL, most>(p, pl, st) : run<T, XR, NTL, most - 1>(p, pl, st);
}

template <int T, int XR>
hipError_t tiles(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    switch (pl.ntl) {
        case 1: return stages<T, XR, 1>(p, pl, st);
        case 2: return stages<T, XR, 2>(p, pl, st);
        case 3: return stages<T, XR, 3>(p, pl, st);
        default: return stages<T, XR, 4>(p, pl, st);
    }
}

template <int T>
hipError_t tokens(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    if (p.M <= 32) return tiles<T, 32>(p, pl, st);
    return p.M <= 48 ? tiles<T, 48>(p, pl, st) : tiles<T, 64>(p, pl, st);
}

}  // namespace

// Row tiles of a workgroup.  A step of 256 K takes about 0.27 us and 0.29 us a tile with 32 tokens, 0.25 us and
// 0.4 us a tile with 64, and a call 6 us besides (17408 x 5120, 20 steps: 64 tokens, one tile in three rounds of
// workgroups 48 us, three tiles in one 35 us; 32 tokens 38 and 29 us), so the rounds decide.
bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o) {
    const int64_t groups = K / group, rows = glu ? 2 * C : C;
    if (groups > kLdsBytes / 64) return false;
    const int xr = M <= 32 ? 32 : (M <= 48 ? 48 : 64);
    o.ntl = 0;
    for (int ntl = 1; ntl <= 4; ++ntl) {
        const uint32_t scales = w4_mid_scales(32 * ntl, (int)groups);
        int stages = most_stages(xr, ntl);
        if (fixed_lds(xr, ntl, stages) + scales > kLdsBytes) --stages;
        if (fixed_lds(xr, ntl, stages) + scales > kLdsBytes) break;
        const int64_t wgs = ((rows + 32 * ntl - 1) / (32 * ntl)) * ((M + 63) / 64);
        const float us = 6.f + (float)((wgs + 255) / 256 * ((K + 255) / 256)) * (M <= 32 ? 0.27f + 0.29f * ntl : 0.25f + 0.4f * ntl);
        if (o.ntl > 0 && us >= o.us) continue;
        o.us = us;
        o.ntl = ntl;
        o.stages = stages;
        o.scales = scales;
    }
    return o.ntl > 0;
}

hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    return dtype == kFp16 ? tokens<kFp16>(p, pl, st) : tokens<kBf16>(p, pl, st);
}

}  // namespace qlin
