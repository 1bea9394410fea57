// w4_mid.hip -- launchers of the kernels for 17 to 64 tokens and small matrices (w4_mid.hpp).
#include "w4_mid_launch.hpp"

namespace qlin {

namespace {

constexpr uint32_t kLdsBytes = 160 * 1024;

template <int MT, int NTL, int STAGES>
constexpr uint32_t fixed_lds() { return STAGES * w4_mid_stage<32 * MT, 32 * NTL>() + 8 * (NTL > 2 ? 8 : 16) * 32 * NTL * 4 + 256; }

template <int T, int MT, int NTL, int STAGES>
hipError_t run(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int BM = 32 * MT, BN = 32 * NTL;
    const int CT = p.I > 0 ? BN / 2 : BN;
    hipLaunchKernelGGL((w4_mid_kernel<T, MT, NTL, STAGES>),
                       dim3((unsigned)((p.C + CT - 1) / CT), (unsigned)((p.M + BM - 1) / BM)), dim3(512), pl.scales, st, p);
    return hipGetLastError();
}

// stages by tokens (32, 64) and row tiles: as many as leave room for the scales of common sizes
constexpr int kStages[2][4] = {{4, 4, 3, 3}, {3, 2, 2, 2}};

template <int T, int MT>
hipError_t tiles(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    switch (pl.ntl) {
        case 1: return run<T, MT, 1, kStages[MT - 1][0]>(p, pl, st);
        case 2: return run<T, MT, 2, kStages[MT - 1][1]>(p, pl, st);
        case 3: return run<T, MT, 3, kStages[MT - 1][2]>(p, pl, st);
        default: return run<T, MT, 4, kStages[MT - 1][3]>(p, pl, st);
    }
}

template <int MT>
uint32_t fixed(int ntl) {
    switch (ntl) {
        case 1: return fixed_lds<MT, 1, kStages[MT - 1][0]>();
        case 2: return fixed_lds<MT, 2, kStages[MT - 1][1]>();
        case 3: return fixed_lds<MT, 3, kStages[MT - 1][2]>();
        default: return fixed_lds<MT, 4, kStages[MT - 1][3]>();
    }
}

}  // namespace

// Row tiles of a workgroup.  A step of 256 K takes about 0.27 us and 0.29 us a tile with 32 tokens, 0.25 us and
// 0.4 us a tile with 64, and a call 6 us besides (17408 x 5120, 20 steps: 64 tokens, one tile in three rounds of
// workgroups 48 us, three tiles in one 35 us; 32 tokens 38 and 29 us), so the rounds decide.
bool w4_mid_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4MidPlan& o) {
    const int64_t groups = K / group, rows = glu ? 2 * C : C;
    if (groups > kLdsBytes / 64) return false;
    o.ntl = 0;
    for (int ntl = 1; ntl <= 4; ++ntl) {
        const uint32_t scales = w4_mid_scales(32 * ntl, (int)groups);
        if ((M <= 32 ? fixed<1>(ntl) : fixed<2>(ntl)) + scales > kLdsBytes) break;
        const int64_t wgs = ((rows + 32 * ntl - 1) / (32 * ntl)) * ((M + 63) / 64);
        const float us = 6.f + (float)((wgs + 255) / 256 * ((K + 255) / 256)) * (M <= 32 ? 0.27f + 0.29f * ntl : 0.25f + 0.4f * ntl);
        if (o.ntl > 0 && us >= o.us) continue;
        o.us = us;
        o.ntl = ntl;
        o.scales = scales;
    }
    return o.ntl > 0;
}

hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    if (p.M <= 32) return dtype == kFp16 ? tiles<kFp16, 1>(p, pl, st) : tiles<kBf16, 1>(p, pl, st);
    return dtype == kFp16 ? tiles<kFp16, 2>(p, pl, st) : tiles<kBf16, 2>(p, pl, st);
}

}  // namespace qlin
