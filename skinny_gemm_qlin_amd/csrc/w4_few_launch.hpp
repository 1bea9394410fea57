// w4_few_launch.hpp -- launcher of the decode kernels (w4_few.hpp); one
// translation unit per dtype instantiates it.
#pragma once
#include "w4_few.hpp"

namespace qlin {

constexpr int kW4FewMaxM = 16;
constexpr uint32_t kW4LdsBytes = 160 * 1024;  // of a compute unit

// How a call is laid out; false if its token rows and scales do not fit LDS
// even one tile of rows at a time.
struct W4FewPlan { int pl, nw, passes, rows, depth; uint32_t lds; };

inline bool w4_few_plan(int64_t M, int64_t K, int64_t group, int64_t C, bool glu, W4FewPlan& o) {
    if (M > kW4FewMaxM) return false;
    const int U = group % 128 == 0 ? 128 : (group % 64 == 0 ? 64 : 32);
    const int64_t lines = (K + 255) / 256, groups = K / group;
    if (groups > kW4LdsBytes / 16) return false;
    // one line a wave on short rows: more waves to hide latency (1024 x 1024: 3.3 us, two lines 3.4)
    // 9 to 16 tokens: one, or the two halves' operands would not fit the registers
    const bool full = M > 8;
    o.pl = lines <= 8 || full ? 1 : 2;
    const int TR = full ? 16 : 8;
    // One workgroup a compute unit, several (that LDS holds together) where a workgroup has few waves, at least
    // 8 columns each.  Where LDS does not hold a share, K is first walked in up to four times as many passes, then
    // the shares get smaller and the rounds of workgroups more.
    const int64_t least = (lines + 16 * o.pl - 1) / (16 * o.pl);
    for (int64_t rounds = 1;; ++rounds) {
        bool smallest = true;
        for (int64_t passes = least; passes <= 4 * least; ++passes) {
            o.nw = (int)((lines + passes * o.pl - 1) / (passes * o.pl));
            o.passes = (int)((lines + o.nw * o.pl - 1) / (o.nw * o.pl));
            for (int64_t per_cu = o.nw >= 12 ? 1 : 12 / o.nw; per_cu >= 1; --per_cu) {
                const int64_t wgs = 256 * per_cu * rounds;
                int64_t rows = (C + wgs - 1) / wgs;
                if (rows < 8) rows = 8;
                smallest = smallest && rows == 8;
                const int64_t wrows = (rows + TR - 1) / TR * TR * (glu ? 2 : 1);
                if (wrows >= 4096 || wrows * groups >= kW4LdsBytes) continue;
                o.rows = (int)rows;
                o.lds = w4_few_lds((int)M, U, o.pl, (int)rows * (glu ? 2 : 1), (int)wrows, (int)groups, o.nw).total;
                if (o.lds * per_cu > kW4LdsBytes && !(rows == 8 && o.lds <= kW4LdsBytes)) continue;
                // about 20 to 32 KB a compute unit in flight (17408 x 5120, 10 waves: one tile ahead 11.2 us,
                // two 11.8; 28672 x 4096 gated, 8 waves: 14.9 and 13.1)
                o.depth = o.nw * o.pl * (full ? 2 : 1) > 16 ? 1 : 2;
                return true;
            }
        }
        if (smallest) return false;
    }
}

template <int T, int U, int RM, int PL, int D, bool FULL>
hipError_t w4_few_run(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    hipLaunchKernelGGL((w4_few_kernel<T, U, RM, PL, D, FULL>), dim3((unsigned)((p.C + p.rows - 1) / p.rows)),
                       dim3(64 * pl.nw), pl.lds, st, p);
    return hipGetLastError();
}

template <int T, int U, int RM, int PL, bool FULL>
hipError_t w4_few_d(const W4FewParams& p, const W4FewPlan& pl, hipStream_t st) {
    return pl.depth == 1 ? w4_few_run<T, U, RM, PL, 1, FULL>(p, pl, st) : w4_few_run<T, U, RM, PL, 2, FULL>(p, pl, st);
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
