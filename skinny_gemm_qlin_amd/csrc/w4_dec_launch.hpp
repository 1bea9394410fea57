// w4_dec_launch.hpp -- launcher template of the few-token kernels
// (w4_dec.hpp); one translation unit per dtype and fold unit instantiates it.
#pragma once
#include "w4_dec.hpp"

namespace qlin {

constexpr int kW4DecMaxM = 64;          // tokens of the few-token kernels
constexpr int kW4StageBytes = 65536;    // token rows staged in LDS up to this size

template <int T, int U, int TR, int MT, int RM, int PB, bool XL, bool LOOP, bool GLU, int NTMAX>
hipError_t w4_dec_run(W4DecParams p, hipStream_t st) {
    constexpr int CT = GLU ? TR * 8 : TR * 16;
    int nw = (p.pieces + PB - 1) / PB;
    if (nw > NTMAX / 64) nw = NTMAX / 64;
    p.per_wave = (p.pieces + nw - 1) / nw;
    nw = (p.pieces + p.per_wave - 1) / p.per_wave;
    const size_t xb = XL ? (size_t)p.M * (p.pieces * 128 + kW4XPad) * 2 : 0;
    const size_t rb = (size_t)nw * p.M * TR * 64;
    hipLaunchKernelGGL((w4_dec_kernel<T, U, TR, MT, RM, PB, XL, LOOP, GLU, NTMAX>),
                       dim3((unsigned)((p.C + CT - 1) / CT)), dim3(64 * nw), xb > rb ? xb : rb, st, p);
    return hipGetLastError();
}

template <int T, int U, int TR, bool GLU>
hipError_t w4_dec_tokens(const W4DecParams& p, hipStream_t st) {
    if (p.M <= 4 && (int64_t)p.M * (p.pieces * 128 + kW4XPad) * 2 <= kW4StageBytes) {
        if (p.pieces <= 64) return w4_dec_run<T, U, TR, 1, 1, 4, true, false, GLU, 1024>(p, st);
        return w4_dec_run<T, U, TR, 1, 1, 2, true, true, GLU, 1024>(p, st);
    }
    if (p.M <= 16) {
        const bool one = p.pieces <= 48;
        if (p.M <= 4)
            return one ? w4_dec_run<T, U, TR, 1, 1, 4, false, false, GLU, 768>(p, st)
                       : w4_dec_run<T, U, TR, 1, 1, 2, false, true, GLU, 768>(p, st);
        if (p.M <= 8)
            return one ? w4_dec_run<T, U, TR, 1, 2, 4, false, false, GLU, 768>(p, st)
                       : w4_dec_run<T, U, TR, 1, 2, 2, false, true, GLU, 768>(p, st);
        return one ? w4_dec_run<T, U, TR, 1, 4, 4, false, false, GLU, 768>(p, st)
                   : w4_dec_run<T, U, TR, 1, 4, 2, false, true, GLU, 768>(p, st);
    }
    if (p.M <= 32) return w4_dec_run<T, U, TR, 2, 4, 2, false, true, GLU, 512>(p, st);
    return w4_dec_run<T, U, TR, 4, 4, 1, false, true, GLU, 512>(p, st);
}

template <int T, int U>
hipError_t w4_dec(const W4DecParams& p, bool glu, hipStream_t st) {
    if (glu) return w4_dec_tokens<T, U, 2, true>(p, st);
    return w4_dec_tokens<T, U, 2, false>(p, st);
}

hipError_t w4_dec_bf16_128(const W4DecParams& p, bool glu, hipStream_t st);
hipError_t w4_dec_bf16_32(const W4DecParams& p, bool glu, hipStream_t st);
hipError_t w4_dec_fp16_128(const W4DecParams& p, bool glu, hipStream_t st);
hipError_t w4_dec_fp16_32(const W4DecParams& p, bool glu, hipStream_t st);

}  // namespace qlin
