// w4_gemm.hpp -- tiled matrix-core GEMM on 4-bit weights, in both directions:
//   forward   out[m,n] = sum_k x[m,k] W[n,k]      (reduction over K, columns n)
//   backward  out[m,k] = sum_n dy[m,n] W[n,k]     (reduction over N, columns k)
// and, forward, the gated pair of products with its epilogue.
//
// Bound: the matrix cores (2 M N K operations; the weights are 4 times smaller
// than the 16-bit matrix and re-read from L2).  A workgroup owns BM tokens x
// BN columns and walks the reduction 64 deep.  The activation tile goes from
// global memory straight into LDS (global_load_lds); the codes of the next
// tile are loaded to registers, dequantised there once per workgroup - every
// thread has one run of 32 codes of one row, so one scale and one zero - and
// written to LDS as 16-bit weights while the matrix cores work on the current
// tile.  Both tiles are double-buffered, one barrier per 64-deep step.
//
// Rounding: here a weight is rounded once to the 16-bit type before it is
// multiplied (at most 2^-8 of its value in bf16, 2^-11 in fp16; sums are
// fp32).  A fold of the scales after the sum, which the small-M kernels use,
// is not possible backward (the scale varies along the reduction) and costs
// a second set of accumulators forward.
//
// Forward and backward differ only in which index of the weight tile is the
// reduction: forward it is the contiguous one and a B fragment is one 16-byte
// LDS read; backward the tile is stored as it comes, [64 n][BN k], and
// ds_read_b64_tr_b16 hands each lane four n of its own k.
#pragma once
#include "w4_device.hpp"
#include "w4_launch.hpp"

namespace qlin {

enum W4Epi { kW4Store = 0, kW4Glu = 1, kW4GluBwd = 2, kW4Part = 3 };

struct W4GemmParams {
    const uint16_t* x; int64_t ldx; int64_t M;  // left operand [M][R]
    int64_t R, C;                               // reduction length, output columns
    W4Weight w; int64_t I;                      // gated: columns C = I, rows n and I + n
    const uint16_t* bias; uint16_t* y; int64_t ldy;
    uint16_t* gu; int64_t ldgu; const uint16_t* dy; int64_t lddy; int act;
    float* part; int64_t steps;                 // 64-deep steps per split (gridDim.y splits)
};

__device__ __forceinline__ void w4_stage_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x70);  // vmcnt(0) lgkmcnt(0): this wave's loads into LDS and LDS writes are done
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

constexpr int64_t kW4BandM = 8;  // token tiles per raster band

template <int T, bool BWD, int EPI, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN, 2) void w4_gemm_kernel(const W4GemmParams p) {
    constexpr int NW = WGM * WGN, NT = 64 * NW;
    constexpr bool kGlu = EPI == kW4Glu || EPI == kW4GluBwd;
    constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;  // 32 x 32 tiles per wave
    constexpr int BR = 64;                                 // reduction depth of a step
    constexpr int XT = BM * BR * 2, WT = BN * BR * 2, ST = XT + WT;
    constexpr int XI = BM / 8 / NW;  // 1 KB loads per wave and step
    static_assert(2 * BN == NT, "one run of 32 codes per thread");
    static_assert(TM >= 1 && TN >= 1 && XI >= 1 && (!kGlu || (TN == 2 && !BWD)), "tile");
    __shared__ __align__(16) uint8_t w4_lds[2 * ST];

    const int64_t M = p.M, R = p.R, C = p.C;
    constexpr int CT = kGlu ? BN / 2 : BN;  // output columns per workgroup
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_c = (C + CT - 1) / CT, tiles = tiles_m * tiles_c;
    const int64_t t = (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;  // an XCD takes adjacent tiles
    if (t >= tiles) return;  // workgroup-uniform
    const int64_t bsz = kW4BandM * tiles_c, band = t / bsz, rr = t - band * bsz;
    const int64_t gm = tiles_m - band * kW4BandM < kW4BandM ? tiles_m - band * kW4BandM : kW4BandM;
    const int64_t c0 = (rr / gm) * CT, m0 = (band * kW4BandM + rr % gm) * BM;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int64_t nsteps = (R + BR - 1) / BR;
    const int64_t s0 = (int64_t)blockIdx.y * p.steps, s1 = s0 + p.steps < nsteps ? s0 + p.steps : nsteps;

    // ---- activation tile: LDS row r, slot c holds 16-byte chunk c ^ (r & 7)
    const uint16_t* xsrc[XI];
    int xchunk[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int r = (wv * XI + i) * 8 + (lane >> 3);
        const int64_t m = m0 + r < M ? m0 + r : M - 1;  // rows past M: clamped, not stored
        xchunk[i] = ((lane & 7) ^ (r & 7)) * 8;
        xsrc[i] = p.x + m * p.ldx + xchunk[i];
    }
    auto issue_x = [&](int64_t s, int slot) {
        uint8_t* base = w4_lds + slot * ST;
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const uint16_t* src = s * BR + xchunk[i] < R ? xsrc[i] + s * BR : (const uint16_t*)&kW4Zero16;
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void_t*)(base + (wv * XI + i) * 1024), 16, 0, 0);
        }
    };

    // ---- this thread's run of 32 codes: one row, one group
    const int64_t ngroups = p.w.K / p.w.group;
    const uint8_t* wsrc;
    const uint16_t* ssrc;
    const uint8_t* zsrc;
    int wdst;            // LDS offset of the run's first 16-byte piece (pieces placed below)
    int run_r;           // its first reduction index inside a step
    bool run_ok = true;  // the run's row / columns exist
    int64_t grem = 0, gstep = 0;
    if constexpr (!BWD) {
        const int r = tid >> 1, h = tid & 1;
        int64_t n;
        if constexpr (kGlu) {
            const int64_t col = c0 + (r >> 6) * 32 + (r & 31);
            n = (col < C ? col : C - 1) + ((r >> 5) & 1) * p.I;
        } else {
            n = c0 + r < C ? c0 + r : C - 1;
        }
        run_r = h * 32;
        const int64_t k = s0 * BR + run_r, g = k / p.w.group;
        grem = k - g * p.w.group;
        wsrc = p.w.w + n * p.w.ldw;
        ssrc = p.w.ws + n * ngroups + g;
        zsrc = p.w.wz + (p.w.wz ? n * ngroups + g : 0);
        wdst = r * (BR * 2);
    } else {
        constexpr int RPR = BN / 32;  // runs per row
        const int r = tid / RPR, cc = tid % RPR;
        int64_t k = c0 + cc * 32;
        run_ok = k < C;
        k = run_ok ? k : 0;
        run_r = r;
        const int64_t g = k / p.w.group;
        wsrc = p.w.w + k / 2;
        ssrc = p.w.ws + g;
        zsrc = p.w.wz + (p.w.wz ? g : 0);
        wdst = r * (BN * 2) + (cc ^ (r & 3)) * 64;
        gstep = cc;
    }
    struct Codes { u32x4_t q; uint32_t s, z; };
    auto load_codes = [&](int64_t s) {  // steps in order: s0, s0 + 1, ...
        Codes c;
        const int64_t i = s * BR + run_r;
        const bool ok = run_ok && i < R;
        if constexpr (!BWD) {
            c.q = *(const u32x4_t*)(wsrc + (ok ? i / 2 : 0));
            c.s = ok ? *ssrc : 0;  // past the end of K: scale 0, weights 0
            c.z = p.w.wz && ok ? *zsrc : 8;
            grem += BR;
#pragma unroll
            for (int j = 0; j < 2; ++j)  // group >= 32: at most two groups a step
                if (grem >= p.w.group && i + BR < R) {
                    grem -= p.w.group;
                    ++ssrc;
                    zsrc += p.w.wz ? 1 : 0;
                }
        } else {
            const int64_t n = i < R ? i : R - 1;
            c.q = *(const u32x4_t*)(wsrc + n * p.w.ldw);
            c.s = ok ? ssrc[n * ngroups] : 0;
            c.z = p.w.wz ? zsrc[n * ngroups] : 8;
        }
        return c;
    };
    // piece i (8 weights) of the run
    auto put_piece = [&](uint8_t* wt, const W4Scale<T>& sc, const u32x4_t& q, int i) {
        int off;
        if constexpr (!BWD) off = wdst + (((run_r >> 3) + i) ^ ((tid >> 1) & 7)) * 16;
        else off = wdst + (i ^ (((int)gstep >> 1) & 3)) * 16;
        *(u32x4_t*)(wt + off) = sc.weights8(q[i]);
    };

    const int wn = wv % WGN, wm = wv / WGN, row = lane & 31, half = lane >> 5;
    auto frag_b = [&](const uint8_t* wt, int j, int ks) {
        if constexpr (!BWD) {
            const int r = wn * (BN / WGN) + j * 32 + row;
            return *(const u32x4_t*)(wt + r * (BR * 2) + (((2 * ks + half) ^ (r & 7)) * 16));
        } else {
            // lanes 4r..4r+3 of 16 lend their addresses to row r of a 4 x 16 block; lane i gets its column i
            typedef short s16x4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
            const int cc = wn * (BN / WGN / 32) + j, sub = lane & 15;
            const int piece = ((lane >> 4) & 1) * 2 + ((sub & 3) >> 1);
            const int col = (cc ^ (sub >> 2)) * 64 + ((piece ^ ((cc >> 1) & 3)) * 16) + (sub & 1) * 8;
            const int r = ks * 16 + half * 8 + (sub >> 2);
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(wt + r * (BN * 2) + col));
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(wt + (r + 4) * (BN * 2) + col));
            const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
            return u32x4_t{l.x, l.y, h.x, h.y};
        }
    };

    f32x16v_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x16v_t{};

    Codes cur = load_codes(s0);
    issue_x(s0, 0);
    {
        W4Scale<T> sc;
        sc.set(cur.s, cur.z);
#pragma unroll
        for (int i = 0; i < 4; ++i) put_piece(w4_lds + XT, sc, cur.q, i);
    }
    if (s0 + 1 < s1) cur = load_codes(s0 + 1);
    for (int64_t s = s0; s < s1; ++s) {
        const int slot = (int)((s - s0) & 1);
        w4_stage_barrier();  // tile s is complete for everyone, and everyone is done with tile s - 1
        asm volatile("" : "+v"(cur.q), "+v"(cur.s), "+v"(cur.z));
        const uint8_t* xt = w4_lds + slot * ST;
        const uint8_t* wt = xt + XT;
        if (s * BR + BR > R && (R & 7)) {  // backward, odd N: clear the last chunk's tail (whatever the row pitch holds)
            const int e0 = (int)(R - s * BR), e1 = (e0 + 7) & ~7;
            for (int r = tid; r < BM; r += NT)
                for (int e = e0; e < e1; ++e)
                    *(uint16_t*)(w4_lds + slot * ST + r * (BR * 2) + (((e >> 3) ^ (r & 7)) * 16) + (e & 7) * 2) = 0;
            w4_stage_barrier();
        }
        const bool more = s + 1 < s1;
        if (more) issue_x(s + 1, slot ^ 1);
        W4Scale<T> sc;
        sc.set(cur.s, cur.z);
        const u32x4_t q = cur.q;
        if (s + 2 < s1) cur = load_codes(s + 2);
        uint8_t* wnext = w4_lds + (slot ^ 1) * ST + XT;
#pragma unroll
        for (int ks = 0; ks < BR / 16; ++ks) {
            u32x4_t a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = wm * (BM / WGM) + i * 32 + row;
                a[i] = *(const u32x4_t*)(xt + r * (BR * 2) + (((2 * ks + half) ^ (r & 7)) * 16));
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) b[j] = frag_b(wt, j, ks);
            if (more) put_piece(wnext, sc, q, ks);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma32<T>(a[i], b[j], acc[i][j]);
        }
    }

    // ---- epilogue: register e of a 32 x 32 tile holds token 8(e/4) + 4*half + e%4, column lane%32
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int64_t m = m0 + wm * (BM / WGM) + i * 32 + 8 * (e >> 2) + 4 * half + (e & 3);
            if (m >= M) continue;
            if constexpr (kGlu) {
                const int64_t c = c0 + wn * 32 + row;
                if (c >= C) continue;
                const float g = acc[i][0][e], u = acc[i][1][e];
                float av, dav;
                gate_act(g, p.act, av, dav);
                if constexpr (EPI == kW4Glu) {
                    p.y[m * p.ldy + c] = f32_to_h<T>(av * u);
                    if (p.gu) {
                        p.gu[m * p.ldgu + c] = f32_to_h<T>(g);
                        p.gu[m * p.ldgu + p.I + c] = f32_to_h<T>(u);
                    }
                } else {
                    const float d = h_to_f32<T>(p.dy[m * p.lddy + c]);
                    p.gu[m * p.ldgu + c] = f32_to_h<T>(d * u * dav);
                    p.gu[m * p.ldgu + p.I + c] = f32_to_h<T>(d * av);
                }
            } else {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int64_t c = c0 + wn * (BN / WGN) + j * 32 + row;
                    if (c >= C) continue;
                    float v = acc[i][j][e];
                    if constexpr (EPI == kW4Part) {
                        p.part[((int64_t)blockIdx.y * M + m) * C + c] = v;
                    } else {
                        if constexpr (!BWD) {
                            if (p.bias) v += h_to_f32<T>(p.bias[c]);
                        }
                        p.y[m * p.ldy + c] = f32_to_h<T>(v);
                    }
                }
            }
        }
}

// out[m,c] = sum over splits of part[s][m][c], in split order
template <int T>
__global__ __launch_bounds__(256) void w4_reduce_kernel(const float* part, int64_t M, int64_t C, int splits,
                                                        uint16_t* y, int64_t ldy) {
    const int64_t c4 = C / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // C % 32 == 0
    if (i >= M * c4) return;
    const int64_t m = i / c4, c = (i - m * c4) * 4;
    const float* src = part + m * C + c;
    f32x4v_t v = *(const f32x4v_t*)src;
    for (int s = 1; s < splits; ++s) v += *(const f32x4v_t*)(src + (int64_t)s * M * C);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[m * ldy + c + e] = f32_to_h<T>(v[e]);
}

// dgu = [dy u act'(g), dy act(g)], V columns a thread
template <int T, int V>
__global__ __launch_bounds__(256) void w4_gate_bwd_kernel(const W4GateBwdArgs a) {
    const int64_t per = a.I / V, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.M * per) return;
    const int64_t m = i / per, c = (i - m * per) * V;
    typedef uint16_t vec_t __attribute__((ext_vector_type(V)));
    vec_t d, g, u, og, ou;
    if constexpr (V == 1) {
        d[0] = a.dy[m * a.lddy + c];
        g[0] = a.gu[m * a.ldgu + c];
        u[0] = a.gu[m * a.ldgu + a.I + c];
    } else {
        d = *(const vec_t*)(a.dy + m * a.lddy + c);
        g = *(const vec_t*)(a.gu + m * a.ldgu + c);
        u = *(const vec_t*)(a.gu + m * a.ldgu + a.I + c);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float av, dav;
        const float dv = h_to_f32<T>(d[e]);
        gate_act(h_to_f32<T>(g[e]), a.act, av, dav);
        og[e] = f32_to_h<T>(dv * h_to_f32<T>(u[e]) * dav);
        ou[e] = f32_to_h<T>(dv * av);
    }
    if constexpr (V == 1) {
        a.dgu[m * a.lddgu + c] = og[0];
        a.dgu[m * a.lddgu + a.I + c] = ou[0];
    } else {
        *(vec_t*)(a.dgu + m * a.lddgu + c) = og;
        *(vec_t*)(a.dgu + m * a.lddgu + a.I + c) = ou;
    }
}

}  // namespace qlin
