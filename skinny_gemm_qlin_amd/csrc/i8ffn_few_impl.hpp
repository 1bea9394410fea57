// i8ffn_few_impl.hpp -- launchers of the kernels for up to 16 tokens, for one
// 16-bit type; see i8ffn_few.hpp.
#pragma once
#include <algorithm>

#include "i8ffn_few.hpp"
#include "i8ffn_few_launch.hpp"

namespace qlin {

template <int T, int SRC, int NS, int D>
hipError_t run_front(const FewFrontParams& p, hipStream_t st) {
    const size_t lds = (size_t)p.M * few_pitch(p.K, D);
    const int64_t chunks = p.E > 0 ? std::min<int64_t>(p.E, p.M * p.topk) : 1, n = chunks * ((p.I + 1) / 2);
    const unsigned grid = (unsigned)std::min<int64_t>(n, kFewGrid);
    auto k = SRC == kFewStaged || p.E <= 128 ? few_front_kernel<T, SRC, NS, D, 2>
                                             : few_front_kernel<T, SRC, NS, D, SRC == kFewStaged ? 2 : 16>;
    hipLaunchKernelGGL(k, dim3(grid), dim3(kFewThreads), lds, st, p);
    return hipGetLastError();
}

template <int T, int SRC>
hipError_t run_front(const FewFrontParams& p, int sets, hipStream_t st) {
    if (few_turn(p.K) == 3) {
        if (sets == 1) return run_front<T, SRC, 1, 3>(p, st);
        return sets == 2 ? run_front<T, SRC, 2, 3>(p, st) : run_front<T, SRC, 4, 3>(p, st);
    }
    if (sets == 1) return run_front<T, SRC, 1, 4>(p, st);
    return sets == 2 ? run_front<T, SRC, 2, 4>(p, st) : run_front<T, SRC, 4, 4>(p, st);
}

template <int T>
hipError_t run_prep(const FewPrepParams& p, hipStream_t st) {
    auto k = p.E <= 128 ? few_prep_kernel<T, 2> : few_prep_kernel<T, 16>;
    hipLaunchKernelGGL(k, dim3((unsigned)(p.rows + (p.list ? 1 : 0))), dim3(kFewThreads), 0, st, p);
    return hipGetLastError();
}

template <int T>
hipError_t few_front(FewFrontParams& p, int8_t* xq, int64_t ldxq, float* xs, int sets, int cap, FewList* list,
                     hipStream_t st) {
    p.ldxq = ldxq;
    if (few_quantise(p.M, p.K)) {
        p.xq_out = p.E > 0 ? nullptr : xq;
        p.xs_out = xs;
        return run_front<T, kFewQuantise>(p, sets, st);
    }
    FewPrepParams q{};
    q.x = p.x; q.ldx = p.ldx; q.rows = p.M; q.K = p.K; q.xq = xq; q.ldxq = ldxq; q.xs = xs; q.logits = p.logits;
    q.ldl = p.ldl; q.M = p.M; q.E = p.E; q.topk = p.topk; q.route = p.route; q.cap = cap; q.ids = p.ids; q.gw = p.gw;
    q.list = list;
    const hipError_t e = run_prep<T>(q, st);
    if (e != hipSuccess) return e;
    p.xq = xq;
    p.xs = xs;
    p.list = list;
    return run_front<T, kFewStaged>(p, sets, st);
}

template <int T, int SRC, int NS, int D>
hipError_t run_down(FewDownParams& p, hipStream_t st) {
    const int P = p.M * p.topk;
    p.rows = (int)few_down_rows(P, p.I);
    p.block = few_down_block(P, p.H);
    hipLaunchKernelGGL((few_down_kernel<T, SRC, NS, D>), dim3((unsigned)few_down_grid(p.H)), dim3(kFewThreads),
                       (size_t)p.block * P * 16 + (size_t)p.rows * few_pitch(p.I, D), st, p);
    return hipGetLastError();
}

template <int T, int SRC>
hipError_t run_down(FewDownParams& p, int sets, hipStream_t st) {
    if (few_turn(p.I) == 3) {
        if (sets == 1) return run_down<T, SRC, 1, 3>(p, st);
        return sets == 2 ? run_down<T, SRC, 2, 3>(p, st) : run_down<T, SRC, 4, 3>(p, st);
    }
    if (sets == 1) return run_down<T, SRC, 1, 4>(p, st);
    return sets == 2 ? run_down<T, SRC, 2, 4>(p, st) : run_down<T, SRC, 4, 4>(p, st);
}

template <int T>
hipError_t few_moe(const I8MoeArgs& a, const I8FewRegions& r, hipStream_t st) {
    FewList* list = (FewList*)r.list;
    const int64_t P = a.M * a.topk;
    FewFrontParams f{};
    f.x = a.x; f.ldx = a.ldx; f.M = (int)a.M; f.K = (int)a.H; f.logits = a.logits; f.ldl = a.ldl; f.E = (int)a.E;
    f.topk = (int)a.topk; f.route = a.route; f.ids = a.ids; f.gw = a.gw; f.w = a.w13; f.ldw = a.ldw13; f.I = a.I;
    f.ws = a.s13; f.ws_step = 1; f.act = a.act; f.y = r.h; f.ldy = a.I;
    const int sets = few_sets(a.M, a.topk, a.E), cap = (int)few_chunk(a.M, a.topk, a.E, a.I);
    hipError_t e = few_front<T>(f, r.xq, a.H, r.xs, sets, cap, list, st);
    if (e != hipSuccess) return e;
    FewDownParams d{};
    d.h = r.h; d.M = (int)a.M; d.I = (int)a.I; d.ids = a.ids; d.gw = a.gw; d.E = (int)a.E;
    d.topk = (int)a.topk; d.w = a.w2; d.ldw = a.ldw2; d.H = a.H; d.ws = a.s2; d.y = a.y; d.ldy = a.ldy;
    if (few_quantise(P, a.I)) return run_down<T, kFewQuantise>(d, sets, st);
    FewPrepParams q{};
    q.x = r.h; q.ldx = a.I; q.rows = (int)P; q.K = (int)a.I; q.xq = r.hq; q.ldxq = a.I; q.xs = r.hs; q.pairs = true; q.M = (int)a.M;
    q.E = (int)a.E; q.topk = (int)a.topk; q.cap = cap; q.ids = a.ids; q.gw = a.gw;
    q.list = few_quantise(a.M, a.H) ? list : nullptr;  // the front made its list for itself
    e = run_prep<T>(q, st);
    if (e != hipSuccess) return e;
    d.hq = r.hq;
    d.hs = r.hs;
    d.list = list;
    return run_down<T, kFewStaged>(d, sets, st);
}

template <int T>
hipError_t few_glu(const I8GluArgs& a, hipStream_t st) {
    FewFrontParams f{};
    f.x = a.x; f.ldx = a.ldx; f.M = (int)a.M; f.K = (int)a.K; f.w = a.w13; f.ldw = a.ldw; f.I = a.I; f.ws = a.s13;
    f.ws_step = a.ws_step; f.act = a.act; f.y = a.y; f.ldy = a.ldy;
    return few_front<T>(f, a.xq, a.ldxq, a.xs, few_sets(a.M, 0, 0), 0, nullptr, st);
}

}  // namespace qlin
