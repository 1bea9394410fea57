// w4_gemm.hip -- launchers of the 4-bit weight GEMM (w4_gemm.hpp).
#include <algorithm>

#include "w4_few_launch.hpp"
#include "w4_mid_launch.hpp"
#include "w4_bwd.hpp"
#include "w4_gemm.hpp"

namespace qlin {

namespace {

// fold units (of 128, 64 or 32 elements) per group r: unit / r by multiplication, exact for
// unit * r < 2^32 (both at most 2^15); 0: r = 1
uint32_t ratio_magic(int64_t group, int unit) {
    const uint64_t r = (uint64_t)(group / unit);
    return r == 1 ? 0 : (uint32_t)(((1ull << 32) + r - 1) / r);
}

template <int T, bool BWD, int EPI, int BM, int BN, int WGM, int WGN>
hipError_t run(W4GemmParams p, int64_t c_first, int64_t c_count, int64_t splits, hipStream_t st) {
    constexpr int CT = EPI == kW4Glu || EPI == kW4GluBwd ? BN / 2 : BN;
    const int64_t tiles = ((p.M + BM - 1) / BM) * ((c_count + CT - 1) / CT);
    p.c_first = c_first;
    p.c_count = c_count;
    const int64_t nsteps = (p.R + 63) / 64;
    p.steps = (nsteps + splits - 1) / splits;
    p.ratio_magic = ratio_magic(p.w.group, 32);
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)((nsteps + p.steps - 1) / p.steps));
    hipLaunchKernelGGL((w4_gemm_kernel<T, BWD, EPI, BM, BN, WGM, WGN>), grid, dim3(64 * WGM * WGN), 0, st, p);
    return hipGetLastError();
}

template <int T, int EPI>
hipError_t forward(const W4GemmParams& p, hipStream_t st) {
    constexpr int fold = EPI == kW4Store ? 1 : 2;  // rows of W a column of the output takes
    const int64_t large = w4_gemm_plan(p.M, fold * p.C, p.R).large * 256 / fold, first = large < p.C ? large : p.C;
    if (first > 0) {
        const hipError_t e = run<T, false, EPI, 256, 256, 2, 4>(p, 0, first, 1, st);
        if (e != hipSuccess) return e;
    }
    return first == p.C ? hipSuccess : run<T, false, EPI, 128, 128, 2, 2>(p, first, p.C - first, 1, st);
}

template <int EPI>
hipError_t gemm(int dtype, const W4GemmParams& p, hipStream_t st) {
    return dtype == kFp16 ? forward<kFp16, EPI>(p, st) : forward<kBf16, EPI>(p, st);
}

hipError_t run_few(int dtype, W4FewParams p, const W4FewPlan& pl, hipStream_t st) {
    p.rows = pl.rows;
    p.passes = pl.passes;
    p.groups = (int)(p.w.K / p.w.group);
    p.ratio_magic = ratio_magic(p.w.group, p.w.group % 128 == 0 ? 128 : (p.w.group % 64 == 0 ? 64 : 32));
    return dtype == kFp16 ? w4_few_fp16(p, pl, st) : w4_few_bf16(p, pl, st);
}

hipError_t run_mid(int dtype, W4MidParams p, const W4MidPlan& pl, hipStream_t st) {
    p.groups = (int)(p.w.K / p.w.group);
    p.ratio_magic = ratio_magic(p.w.group, 32);
    return w4_mid(dtype, p, pl, st);
}

}  // namespace

hipError_t launch_gemv_w4(const W4LinearArgs& a, hipStream_t st) {
    W4FewPlan pl;
    if (w4_few_plan(a.M, a.w.K, a.w.group, a.w.N, false, pl)) {
        W4FewParams d{};
        d.x = a.x; d.ldx = a.ldx; d.M = (int)a.M; d.w = a.w; d.C = a.w.N;
        d.bias = a.bias; d.y = a.y; d.ldy = a.ldy;
        return run_few(a.dtype, d, pl, st);
    }
    W4MidPlan mp;
    if (w4_mid_plan(a.M, a.w.K, a.w.group, a.w.N, false, mp) && w4_use_mid(a.M, a.w.N, a.w.K, a.w.group, mp)) {
        W4MidParams d{};
        d.x = a.x; d.ldx = a.ldx; d.M = (int)a.M; d.w = a.w; d.C = a.w.N;
        d.bias = a.bias; d.y = a.y; d.ldy = a.ldy;
        return run_mid(a.dtype, d, mp, st);
    }
    W4GemmParams p{};
    p.x = a.x; p.ldx = a.ldx; p.M = a.M; p.R = a.w.K; p.C = a.w.N; p.w = a.w;
    p.bias = a.bias; p.y = a.y; p.ldy = a.ldy;
    return gemm<kW4Store>(a.dtype, p, st);
}

hipError_t launch_glu_w4(const W4GluArgs& a, hipStream_t st) {
    W4FewPlan pl;
    if (w4_few_plan(a.M, a.w.K, a.w.group, a.I, true, pl)) {
        W4FewParams d{};
        d.x = a.x; d.ldx = a.ldx; d.M = (int)a.M; d.w = a.w; d.I = a.I; d.C = a.I;
        d.y = a.y; d.ldy = a.ldy; d.gu = a.gu; d.ldgu = a.ldgu; d.dy = a.dy; d.lddy = a.lddy; d.act = a.act;
        return run_few(a.dtype, d, pl, st);
    }
    W4MidPlan mp;
    if (w4_mid_plan(a.M, a.w.K, a.w.group, a.I, true, mp) && w4_use_mid(a.M, a.w.N, a.w.K, a.w.group, mp)) {
        W4MidParams d{};
        d.x = a.x; d.ldx = a.ldx; d.M = (int)a.M; d.w = a.w; d.I = a.I; d.C = a.I;
        d.y = a.y; d.ldy = a.ldy; d.gu = a.gu; d.ldgu = a.ldgu; d.dy = a.dy; d.lddy = a.lddy; d.act = a.act;
        return run_mid(a.dtype, d, mp, st);
    }
    W4GemmParams p{};
    p.x = a.x; p.ldx = a.ldx; p.M = a.M; p.R = a.w.K; p.C = a.I; p.w = a.w; p.I = a.I;
    p.y = a.y; p.ldy = a.ldy; p.gu = a.gu; p.ldgu = a.ldgu; p.dy = a.dy; p.lddy = a.lddy; p.act = a.act;
    return a.dy ? gemm<kW4GluBwd>(a.dtype, p, st) : gemm<kW4Glu>(a.dtype, p, st);
}

// How the input gradient is laid out: shares of the reduction over N, so that short batches and narrow outputs
// fill the chip too; the shares' partial sums go through the workspace.
namespace {

struct BwdPlan { int cw; int64_t shares, per; };  // cw: codes of a lane (up to 64 tokens), 0: the GEMM; per: blocks or steps

BwdPlan bwd_plan(int64_t M, int64_t N, int64_t K) {
    BwdPlan o{};
    if (M <= 64) {
        o.cw = M <= 32 ? 16 : 8;
        const int64_t cols = (K + 16 * o.cw - 1) / (16 * o.cw), blocks = (N + 31) / 32;
        // one workgroup of 4 waves a compute unit, at least one block a wave (33 tokens, 4096 x 7168: 20 us, two 22,
        // half of one 28; one token, 17408 x 5120: 25, 24.4 and 39)
        int64_t shares = 256 / cols;
        if (shares > (blocks + 3) / 4) shares = (blocks + 3) / 4;
        o.per = shares > 1 ? (blocks + shares - 1) / shares : blocks;
        o.shares = (blocks + o.per - 1) / o.per;
        return o;
    }
    const int64_t tile = M <= 512 ? 128 : 256, tiles = ((M + tile - 1) / tile) * ((K + tile - 1) / tile);
    const int64_t steps = (N + 63) / 64;
    float best = 0.f;
    for (int64_t s = 1; s <= 8 && (s == 1 || steps / s >= 4); ++s) {
        // a step of a 256 x 256 tile 1.8 us, of a 128 x 128 tile 1.1 us; partial sums at 4 TB/s, written and read
        const float us = (float)((tiles * s + 255) / 256 * ((steps + s - 1) / s)) * (tile == 256 ? 1.8f : 1.1f) +
                         (s > 1 ? 5.f + (float)(s * M * K) * 8e-6f / 4.f : 0.f);
        if (s > 1 && us >= best) continue;
        best = us;
        o.per = (steps + s - 1) / s;
        o.shares = (steps + o.per - 1) / o.per;
    }
    return o;
}

template <int T>
hipError_t run_bwd(const W4BwdArgs& a, const BwdPlan& pl, hipStream_t st) {
    W4BwdParams p{a.dy, a.lddy, (int)a.M, a.w, a.dx, a.lddx, pl.shares > 1 ? a.part : nullptr, (int)pl.per};
    const dim3 grid((unsigned)((a.w.K + 16 * pl.cw - 1) / (16 * pl.cw)), (unsigned)pl.shares);
    if (a.M <= 16) hipLaunchKernelGGL((w4_bwd_kernel<T, 16, 1>), grid, dim3(256), 0, st, p);
    else if (a.M <= 32) hipLaunchKernelGGL((w4_bwd_kernel<T, 16, 2>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((w4_bwd_kernel<T, 8, 4>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int T>
hipError_t run_bwd_gemm(const W4BwdArgs& a, const BwdPlan& pl, hipStream_t st) {
    W4GemmParams p{};
    p.x = a.dy; p.ldx = a.lddy; p.M = a.M; p.R = a.w.N; p.C = a.w.K; p.w = a.w;
    p.y = a.dx; p.ldy = a.lddx; p.part = a.part;
    if (a.M <= 512)
        return pl.shares > 1 ? run<T, true, kW4Part, 128, 128, 2, 2>(p, 0, p.C, pl.shares, st)
                             : run<T, true, kW4Store, 128, 128, 2, 2>(p, 0, p.C, 1, st);
    return pl.shares > 1 ? run<T, true, kW4Part, 256, 256, 2, 4>(p, 0, p.C, pl.shares, st)
                         : run<T, true, kW4Store, 256, 256, 2, 4>(p, 0, p.C, 1, st);
}

template <int T>
hipError_t bwd(const W4BwdArgs& a, hipStream_t st) {
    const BwdPlan pl = bwd_plan(a.M, a.w.N, a.w.K);
    const hipError_t e = pl.cw ? run_bwd<T>(a, pl, st) : run_bwd_gemm<T>(a, pl, st);
    if (e != hipSuccess || pl.shares == 1) return e;
    const int64_t outputs = a.M * a.w.K;
    if (outputs >= 4 * 256 * 512)
        hipLaunchKernelGGL((w4_reduce_kernel<T, 4>), dim3((unsigned)((outputs / 4 + 255) / 256)), dim3(256), 0, st,
                           a.part, a.M, a.w.K, (int)pl.shares, a.dx, a.lddx);
    else
        hipLaunchKernelGGL((w4_reduce_kernel<T, 1>), dim3((unsigned)((outputs + 255) / 256)), dim3(256), 0, st, a.part,
                           a.M, a.w.K, (int)pl.shares, a.dx, a.lddx);
    return hipGetLastError();
}

}  // namespace

size_t w4_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const BwdPlan pl = bwd_plan(M, N, K);
    return pl.shares > 1 ? (size_t)(pl.shares * M * K) * 4 : 0;
}

hipError_t launch_gemv_w4_bwd(const W4BwdArgs& a, hipStream_t st) {
    return a.dtype == kFp16 ? bwd<kFp16>(a, st) : bwd<kBf16>(a, st);
}

hipError_t launch_gate_bwd(const W4GateBwdArgs& a, hipStream_t st) {
    const bool vec = a.I % 8 == 0 && (((uintptr_t)a.dy | (uintptr_t)a.gu | (uintptr_t)a.dgu) & 15) == 0 &&
                     (a.lddy | a.ldgu | a.lddgu) % 8 == 0;
    const int64_t n = a.M * (vec ? a.I / 8 : a.I);
    const dim3 grid((unsigned)std::min((n + 255) / 256, kW4GateBlocks));
    if (a.dtype == kFp16) {
        if (vec) hipLaunchKernelGGL((w4_gate_bwd_kernel<kFp16, 8>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((w4_gate_bwd_kernel<kFp16, 1>), grid, dim3(256), 0, st, a);
    } else {
        if (vec) hipLaunchKernelGGL((w4_gate_bwd_kernel<kBf16, 8>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((w4_gate_bwd_kernel<kBf16, 1>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace qlin
