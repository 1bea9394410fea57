// w4_few_launch.hpp -- launcher of the decode kernels (w4_few.hpp); one
// translation unit per dtype instantiates it.
#pragma once
#include "w4_few.hpp"

namespace qlin {

template <int T, int U, int RM, int PL, int D, bool FULL>
hipError_t w4_few_run(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    hipLaunchKernelGGL((w4_few_kernel<T, U, RM, PL, D, FULL>), dim3((unsigned)((p.C + p.rows - 1) / p.rows)),
                       dim3(64 * pl.nw), pl.lds, st, p);
    return hipGetLastError();
}

template <int T, int U, int RM, int PL, bool FULL>
hipError_t w4_few_d(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    if constexpr (FULL && U == 32) {
        return w4_few_run<T, U, RM, PL, 1, FULL>(p, pl, st);
    } else {
        return pl.depth == 1 ? w4_few_run<T, U, RM, PL, 1, FULL>(p, pl, st)
                             : w4_few_run<T, U, RM, PL, 2, FULL>(p, pl, st);
    }
}

template <int T, int U, int RM>
hipError_t w4_few_rm(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    return pl.pl == 1 ? w4_few_d<T, U, RM, 1, false>(p, pl, st) : w4_few_d<T, U, RM, 2, false>(p, pl, st);
}

template <int T, int U>
hipError_t w4_few_u(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    if (p.M <= 2) return w4_few_rm<T, U, 1>(p, pl, st);
    if (p.M <= 4) return w4_few_rm<T, U, 2>(p, pl, st);
    if (p.M <= 6) return w4_few_rm<T, U, 3>(p, pl, st);
    if (p.M <= 8) return w4_few_rm<T, U, 4>(p, pl, st);
    if (p.M <= 12) return w4_few_d<T, U, 3, 1, true>(p, pl, st);
    return w4_few_d<T, U, 4, 1, true>(p, pl, st);
}

hipError_t w4_few_bf16(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st);
hipError_t w4_few_fp16(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st);

}  // namespace qlin
