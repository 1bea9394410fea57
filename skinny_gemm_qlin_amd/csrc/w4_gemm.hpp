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
    int64_t c_first, c_count;                   // of which this launch computes c_count from c_first
    W4Weight w; int64_t I;                      // gated: columns C = I, rows n and I + n
    const uint16_t* bias; uint16_t* y; int64_t ldy;
    uint16_t* gu; int64_t ldgu; const uint16_t* dy; int64_t lddy; int act;
    float* part; int64_t steps;                 // 64-deep steps per split (gridDim.y splits)
    uint32_t ratio_magic;                       // forward: 32-K units per group r: unit / r = mulhi(unit, magic), 0: r = 1
};

__device__ __forceinline__ void w4_stage_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x70);  // vmcnt(0) lgkmcnt(0): this wave's loads into LDS and LDS writes are done
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Slot of 16-byte chunk c in LDS row r of 128 bytes: c ^ swz(r).  Two rows fill the 64 banks once, so pairs of
// rows share a swizzle and 16 adjacent rows' copies of one chunk lie in different banks.
__device__ __forceinline__ int w4_swz(int r) { return (r >> 1) & 7; }

constexpr int64_t kW4BandM = 8;  // token tiles per raster band

template <int T, bool BWD, int EPI, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN, 2) void w4_gemm_kernel(const W4GemmParams p) {
    constexpr int NW = WGM * WGN, NT = 64 * NW;
    constexpr bool kGlu = EPI == kW4Glu || EPI == kW4GluBwd;
    constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;  // 32 x 32 tiles per wave
    constexpr int BR = 64;                                 // reduction depth of a step
    constexpr int XT = BM * BR * 2, WT = BN * BR * 2;
    constexpr int XI = BM / 8 / NW;  // 1 KB loads per wave and step
    static_assert(2 * BN == NT, "one run of 32 codes per thread");
    static_assert(TM >= 1 && TN >= 1 && XI >= 1 && (!kGlu || (TN == 2 && !BWD)), "tile");
    // an object of its own for each tile: the compiler then knows that a load into one of them need not be
    // waited for before another is read
    __shared__ __align__(16) uint8_t x_even[XT], x_odd[XT], w_even[WT], w_odd[WT];

    const int64_t M = p.M, R = p.R, C = p.C;
    constexpr int CT = kGlu ? BN / 2 : BN;  // output columns per workgroup
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_c = (p.c_count + CT - 1) / CT, tiles = tiles_m * tiles_c;
    const int64_t t = (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;  // an XCD takes adjacent tiles
    if (t >= tiles) return;  // workgroup-uniform
    const int64_t bsz = kW4BandM * tiles_c, band = t / bsz, rr = t - band * bsz;
    const int64_t gm = tiles_m - band * kW4BandM < kW4BandM ? tiles_m - band * kW4BandM : kW4BandM;
    const int64_t c0 = p.c_first + (rr / gm) * CT, m0 = (band * kW4BandM + rr % gm) * BM;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int64_t nsteps = (R + BR - 1) / BR;
    const int64_t s0 = (int64_t)blockIdx.y * p.steps, s1 = s0 + p.steps < nsteps ? s0 + p.steps : nsteps;

    // ---- activation tile
    const uint16_t* xsrc[XI];
    int xchunk[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int r = (wv * XI + i) * 8 + (lane >> 3);
        const int64_t m = m0 + r < M ? m0 + r : M - 1;  // rows past M: clamped, not stored
        xchunk[i] = ((lane & 7) ^ w4_swz(r)) * 8;
        xsrc[i] = p.x + m * p.ldx + xchunk[i];
    }
    auto issue_x = [&](int64_t s, uint8_t* base) {
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const uint16_t* src = s * BR + xchunk[i] < R ? xsrc[i] + s * BR : (const uint16_t*)&kW4Zero16;
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void_t*)(base + (wv * XI + i) * 1024), 16, 0, 0);
        }
    };

    // ---- this thread's run of 32 codes of a step: one row, one group
    const int64_t ngroups = p.w.K / p.w.group;
    const bool has_z = p.w.wz != nullptr;
    int wdst;            // LDS offset of the run's row or 64-byte block (pieces placed below)
    int run_r;           // its first reduction index inside a step
    int run_c = 0;       // backward: its 32-column block
    int run_row = 0;     // forward: its LDS row
    // forward.  A row gives 32 bytes to a step; loaded so, every 128-byte line would come from L2 four times.
    // Four threads therefore load 64 bytes of a row, two steps' worth, of rows r and r' = BN / 2 + (r ^ 4), and
    // exchange: threads 0, 1 keep row r, threads 2, 3 row r', each with one run of either step.
    const uint8_t* wsrc[2];
    const int j4 = tid & 3;
    // forward: the scales of 4 groups at a time
    const uint16_t* srow = nullptr;
    const uint8_t* zrow = nullptr;
    int left = 0;  // scales from the row's first to the matrix's last
    // backward: the columns are fixed
    const uint16_t* ssrc = nullptr;
    const uint8_t* zsrc = nullptr;
    bool run_ok = true;
    if constexpr (!BWD) {
        auto matrix_row = [&](int r) -> int64_t {
            if constexpr (kGlu) {
                const int64_t col = c0 + (r >> 6) * 32 + (r & 31);
                return (col < C ? col : C - 1) + ((r >> 5) & 1) * p.I;
            } else {
                return c0 + r < C ? c0 + r : C - 1;
            }
        };
        const int ra = tid >> 2, rb = BN / 2 + ((tid >> 2) ^ 4);
        run_row = j4 < 2 ? ra : rb;
        run_r = (j4 & 1) * 32;
        wsrc[0] = p.w.w + matrix_row(ra) * p.w.ldw;
        wsrc[1] = p.w.w + matrix_row(rb) * p.w.ldw;
        srow = p.w.ws + matrix_row(run_row) * ngroups;
        const int64_t rest = (p.w.N - matrix_row(run_row)) * ngroups;
        left = rest < (1 << 30) ? (int)rest : 1 << 30;
        zrow = has_z ? p.w.wz + matrix_row(run_row) * ngroups : (const uint8_t*)srow;  // without zeros: not used
        wdst = run_row * (BR * 2);
    } else {
        constexpr int RPR = BN / 32;  // runs per row
        const int r = tid / RPR, cc = tid % RPR;
        int64_t k = c0 + cc * 32;
        run_ok = k < C;
        k = run_ok ? k : 0;
        run_r = r;
        run_c = cc;
        const int64_t g = k / p.w.group;
        wsrc[0] = p.w.w + k / 2;
        ssrc = p.w.ws + g;
        zsrc = has_z ? p.w.wz + g : (const uint8_t*)ssrc;
        wdst = r * (BN * 2) + (cc ^ (r & 3)) * 64;
    }
    struct Codes { u32x4_t q; uint32_t s, z; };
    auto load_codes = [&](int64_t s) {  // backward
        Codes c;
        const int64_t i = s * BR + run_r, n = i < R ? i : R - 1;
        c.q = *(const u32x4_t*)(wsrc[0] + n * p.w.ldw);
        c.s = ssrc[n * ngroups];  // looked at when they are used, or this would wait for them
        c.z = zsrc[n * ngroups];
        return c;
    };
    auto set_scale = [&](W4Scale<T>& sc, const Codes& c, int64_t s) {
        sc.set(run_ok && s * BR + run_r < R ? c.s : 0, has_z ? c.z : 8);  // past the end: scale 0, weights 0
    };
    auto load_pair = [&](int64_t s, u32x4_t (&raw)[2]) {  // forward: the 128 K of steps s and s + 1
        const int64_t k = s * BR + j4 * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) raw[i] = *(const u32x4_t*)(wsrc[i] + (k < R ? k / 2 : 0));
    };
    auto exchange = [&](const u32x4_t (&raw)[2], u32x4_t& first, u32x4_t& second) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t send = j4 < 2 ? raw[1][d] : raw[0][d];
            const uint32_t got = (uint32_t)dpp_mov<0x4E>((int)send);  // quad_perm 2 3 0 1
            first[d] = j4 < 2 ? raw[0][d] : got;
            second[d] = j4 < 2 ? got : raw[1][d];
        }
    };
    // forward: scales and zeros of groups 4v .. 4v + 3 of the run's row, as one load each.  The four may reach into
    // the next row; at the end of the matrix they are its last four (there are four: the launcher sees to it).
    struct Window { uint2 s; uint32_t z; };
    auto window_first = [&](int v) { return v * 4 < left - 4 ? v * 4 : left - 4; };
    auto load_window = [&](int v) {
        Window w;
        const int first = window_first(v);
        __builtin_memcpy(&w.s, srow + first, 8);
        __builtin_memcpy(&w.z, zrow + first, 4);
        return w;
    };
    auto group_of = [&](int64_t unit) {  // group of the 32 elements from 32 * unit; uniform
        return p.ratio_magic ? (int)__umulhi((uint32_t)unit, p.ratio_magic) : (int)unit;
    };
    auto scale_of = [&](const Window& w, int v, int64_t s) {  // of this thread's run of step s
        const int g0 = group_of(s * 2), g1 = group_of(s * 2 + 1), at = (run_r ? g1 : g0) - window_first(v);
        const uint32_t d = at & 2 ? w.s.y : w.s.x;
        W4Scale<T> sc;
        sc.set(s * BR + run_r < R ? (d >> (16 * (at & 1))) & 0xFFFFu : 0u,  // past K: scale 0, weights 0
               has_z ? (w.z >> (8 * (at & 3))) & 0xFFu : 8u);
        return sc;
    };
    // piece i (8 weights) of the run
    auto put_piece = [&](uint8_t* wt, const W4Scale<T>& sc, const u32x4_t& q, int i) {
        int off;
        if constexpr (!BWD) off = wdst + (((run_r >> 3) + i) ^ w4_swz(run_row)) * 16;
        else off = wdst + (i ^ ((run_c >> 1) & 3) ^ (run_r & 1)) * 16;
        *(u32x4_t*)(wt + off) = sc.weights8(q[i]);
    };

    const int wn = wv % WGN, wm = wv / WGN, row = lane & 31, half = lane >> 5;
    auto frag_b = [&](const uint8_t* wt, int j, int ks) {
        if constexpr (!BWD) {
            const int r = wn * (BN / WGN) + j * 32 + row;
            return *(const u32x4_t*)(wt + r * (BR * 2) + (((2 * ks + half) ^ w4_swz(r)) * 16));
        } else {
            // lanes 4r..4r+3 of 16 lend their addresses to row r of a 4 x 16 block; lane i gets its column i
            typedef short s16x4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
            const int cc = wn * (BN / WGN / 32) + j, sub = lane & 15;
            const int piece = ((lane >> 4) & 1) * 2 + ((sub & 3) >> 1);
            const int col = (cc ^ (sub >> 2)) * 64 + ((piece ^ ((cc >> 1) & 3) ^ ((sub >> 2) & 1)) * 16) + (sub & 1) * 8;
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

    u32x4_t fa[2][TM], fb[2][TN];  // operands of the current and the next 16-deep slice
    auto load_frags = [&](int set, const uint8_t* xt, const uint8_t* wt, int ks) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = wm * (BM / WGM) + i * 32 + row;
            fa[set][i] = *(const u32x4_t*)(xt + r * (BR * 2) + (((2 * ks + half) ^ w4_swz(r)) * 16));
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[set][j] = frag_b(wt, j, ks);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma32<T>(fa[set][i], fb[set][j], acc[i][j]);
    };
    // backward, odd N: the last chunk of dy's rows is cleared past N (whatever the row pitch holds)
    auto clear_tail = [&](int64_t s, uint8_t* xt) {
        if (BWD && s * BR + BR > R && (R & 7) && s < s1) {
            const int e0 = (int)(R - s * BR), e1 = (e0 + 7) & ~7;
            for (int r = tid; r < BM; r += NT)
                for (int e = e0; e < e1; ++e)
                    *(uint16_t*)(xt + r * (BR * 2) + (((e >> 3) ^ w4_swz(r)) * 16) + (e & 7) * 2) = 0;
            w4_stage_barrier();
        }
    };

    // what is held for the next two steps' weights: backward their codes, forward the second run of a pair
    // (while it is needed) and the next pair as loaded, and two windows of scales
    Codes c1, c2;
    u32x4_t q1, q2, raw[2];
    Window win, next_win;
    int v = 0;
    (void)c1; (void)c2; (void)q1; (void)q2; (void)raw; (void)win; (void)next_win; (void)v;
    W4Scale<T> sc;
    if constexpr (BWD) {
        const Codes c = load_codes(s0);
        issue_x(s0, x_even);
        c1 = load_codes(s0 + 1);
        c2 = load_codes(s0 + 2);
        set_scale(sc, c, s0);
#pragma unroll
        for (int i = 0; i < 4; ++i) put_piece(w_even, sc, c.q, i);
    } else {
        v = group_of(s0 * 2) >> 2;
        win = load_window(v);
        load_pair(s0, raw);
        issue_x(s0, x_even);
        u32x4_t q0;
        exchange(raw, q0, q1);
        sc = scale_of(win, v, s0);
#pragma unroll
        for (int i = 0; i < 4; ++i) put_piece(w_even, sc, q0, i);
        load_pair(s0 + 2, raw);
        next_win = load_window(v + 1);
    }
    // forward: the window of step s
    auto turn_window = [&](int64_t s) {
        const int want = group_of(s * 2) >> 2;
        if (want != v) {  // uniform; the next one, since a window is at least 128 K
            win = next_win;
            v = want;
            next_win = load_window(v + 1);
        }
    };
    if constexpr (!BWD) turn_window(s0 + 1);
    w4_stage_barrier();
    clear_tail(s0, x_even);
    load_frags(0, x_even, w_even, 0);
    issue_x(s0 + 1 < s1 ? s0 + 1 : s0, x_odd);
    // one step on tiles xt, wt; the next one's are xn, wn
    auto step = [&](int64_t s, const bool odd, uint8_t* xt, uint8_t* wt, uint8_t* xn, uint8_t* wnext) {
        // slices 0-2 of step s, with step s + 1's codes dequantised on the way; operands are read one slice ahead
        u32x4_t q;
        if constexpr (BWD) {
            set_scale(sc, c1, s + 1);
            q = c1.q;
        } else {
            sc = scale_of(win, v, s + 1);
            q = q1;
        }
#pragma unroll
        for (int ks = 0; ks < 3; ++ks) {
            load_frags((ks + 1) & 1, xt, wt, ks + 1);
            put_piece(wnext, sc, q, ks);
            if (ks == 0) put_piece(wnext, sc, q, 3);
            multiply(ks & 1);
        }
        // everyone's reads of step s and writes of step s + 1 are done, and its activation tile is there;
        // the last slice's products run while the next step's operands are read
        w4_stage_barrier();
        clear_tail(s + 1, xn);
        load_frags(0, xn, wnext, 0);
        if constexpr (BWD) {
            c1 = c2;
            c2 = load_codes(s + 3);
        } else {
            if (!odd) {  // s + 2 opens a pair
                exchange(raw, q1, q2);
                load_pair(s + 4, raw);
            } else {
                q1 = q2;
            }
            turn_window(s + 2);
        }
        issue_x(s + 2 < s1 ? s + 2 : s, xt);  // past the end: the idle tile, again
        multiply(1);
    };
    for (int64_t s = s0; s < s1; s += 2) {
        step(s, false, x_even, w_even, x_odd, w_odd);
        if (s + 1 < s1) step(s + 1, true, x_odd, w_odd, x_even, w_even);
    }
    w4_wait_vmcnt<0>();  // no load into LDS outlives the workgroup

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

// out[m,c] = sum over splits of part[s][m][c], in split order; V columns a thread (4, or 1 where that leaves too
// few threads), eight splits' loads in flight at once
template <int T, int V>
__global__ __launch_bounds__(256) void w4_reduce_kernel(const float* part, int64_t M, int64_t C, int splits,
                                                        uint16_t* y, int64_t ldy) {
    typedef float vec_t __attribute__((ext_vector_type(V)));
    const int64_t cv = C / V, i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // C % 32 == 0
    if (i >= M * cv) return;
    const int64_t m = i / cv, c = (i - m * cv) * V;
    const float* src = part + m * C + c;
    vec_t sum = {};
    for (int s = 0; s < splits; s += 8) {
        vec_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __builtin_nontemporal_load((const vec_t*)(src + (int64_t)(s + e < splits ? s + e : s) * M * C));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (s + e < splits) sum += v[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) y[m * ldy + c + e] = f32_to_h<T>(sum[e]);
}

// dgu = [dy u act'(g), dy act(g)], V columns a thread; a grid of at most kW4GateBlocks workgroups, which then take
// more than one turn (a launch holds fewer than 2^32 threads, M * I may be more)
constexpr int64_t kW4GateBlocks = 1 << 22;

template <int T, int V>
__global__ __launch_bounds__(256) void w4_gate_bwd_kernel(const W4GateBwdArgs a) {
    const int64_t per = a.I / V;
    typedef uint16_t vec_t __attribute__((ext_vector_type(V)));
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.M * per; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / per, c = (i - m * per) * V;
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
}

}  // namespace qlin
