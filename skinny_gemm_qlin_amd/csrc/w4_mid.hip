// w4_mid.hip -- launchers of the kernels for 17 to 64 tokens and small matrices (w4_mid.hpp).
#include "w4_mid_launch.hpp"

namespace qlin {

namespace {

template <int T, int XR, int NTL, int STAGES>
hipError_t run(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int BM = (XR + 31) / 32 * 32, BN = 32 * NTL;
    static_assert(STAGES >= 2 && STAGES <= 4, "stages");
    const int CT = p.I > 0 ? BN / 2 : BN;
    hipLaunchKernelGGL((w4_mid_kernel<T, XR, NTL, STAGES>),
                       dim3((unsigned)((p.C + CT - 1) / CT), (unsigned)((p.M + BM - 1) / BM)), dim3(512), pl.scales, st, p);
    return hipGetLastError();
}

template <int T, int XR, int NTL>
hipError_t stages(const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    constexpr int most = w4_mid_most_stages(XR, NTL);
    if constexpr (NTL == 1) {
        if (pl.stages == 2) return run<T, XR, NTL, 2>(p, pl, st);
    }
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

hipError_t w4_mid(int dtype, const W4MidParams& p, const W4MidPlan& pl, hipStream_t st) {
    return dtype == kFp16 ? tokens<kFp16>(p, pl, st) : tokens<kBf16>(p, pl, st);
}

}  // namespace qlin
