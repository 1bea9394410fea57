// i8ffn_gemm.hpp -- tiled INT8 matrix-core GEMM of the feed-forward operators,
// grouped by expert or dense (one group):
//   gated   y[r][i] = r16(act(g) u), rows i and I + i of the group's W13
//   down    part[r][n] = (acc * xs[r]) * ws[n]            (fp32)
// over the code rows r of a group.  acc is the exact int32 sum.
//
// A workgroup owns BM code rows x BN weight rows and walks K 128 bytes at a
// time.  Both tiles travel global -> LDS directly (global_load_lds_dwordx4, 8
// rows x one whole 128-byte line an instruction) into a ring of D buffers; one
// barrier a step.  The fragments of a 32-deep slice are read one slice ahead of
// their products, and those of the next step's first slice right behind the
// barrier, so a buffer is free for the loads of D steps later while the last
// slice's products still run: a load has D - 1 steps to arrive.
//
// D = 4 where a compute unit has one workgroup, as in a dense front of up to
// some hundred tokens (2 x 4096 x 7168, cold: 509 tokens 63 -> 48 us, 256 61 ->
// 44; 64 tokens in tiles of 64 rows 57 -> 36).  D = 2 where several share it
// and hide each other's waits (1000 tokens, 64 experts top 6, 7168 x 2048: 729
// us, 751 with 4), and in the 256 x 256 tile, whose two buffers fill LDS.  The
// last D steps have nothing left to request and load their own slice again, which
// the epilogue waits for: with D = 2 and K = 768 that is a quarter of the requests.
#pragma once
#include "i8ffn_device.hpp"

namespace qlin {

enum I8Epi { kI8Gated = 0, kI8Part = 1 };

// The group (expert) that a row tile belongs to: its first row tile, first row and number of rows.
struct I8Tile { int group, tile, row, rows; };

struct I8GemmParams {
    const int8_t* x; int64_t ldx; const float* xs;  // codes [rows][ldx] and their scales
    int64_t R;                                      // dense: rows
    const I8Tile* tiles; const int32_t* ntiles;     // grouped: of each row tile its group; null: dense
    const int32_t* perm; int div;                   // grouped: row r of the groups is pair perm[r], code row perm[r] / div
    int64_t K; const int8_t* w; int64_t ldw; int64_t N;  // N weight rows a group (gated: 2 I)
    const float* ws; int ws_step;                   // [E][N]
    int64_t C;                                      // output columns: I or N
    int64_t c_first, c_count;                       // of which this launch computes c_count from c_first
    int act; uint16_t* y; float* part; int64_t ldy;
};

__device__ const u32x4_t kI8Zero16 = {0u, 0u, 0u, 0u};

typedef int i32x16v_t __attribute__((ext_vector_type(16)));
typedef int i32x4v_t __attribute__((ext_vector_type(4)));

// Slot of 16-byte chunk c in LDS row r of 128 bytes: c ^ swz(r); see w4_gemm.hpp.
__device__ __forceinline__ int i8_swz(int r) { return (r >> 1) & 7; }

// This wave's loads into LDS but the last LATER are done, its reads too; then everyone's.
template <int LATER>
__device__ __forceinline__ void i8_stage_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((LATER & 15) | ((LATER >> 4) << 14) | 0x70);  // vmcnt(LATER) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

constexpr int kI8BandM = 8;  // row tiles per raster band

template <int T, int EPI, int BN, int BM, int WGN, int WGM, int D>
__global__ __launch_bounds__(64 * WGM * WGN, WGM * WGN == 16 ? 4 : 2) void i8_gemm_kernel(const I8GemmParams p) {
    constexpr int NW = WGM * WGN;
    constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;  // 32 x 32 tiles per wave
    constexpr int BK = 128, XT = BM * BK, WT = BN * BK;
    constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;      // 1 KB loads per wave and step
    constexpr int CT = EPI == kI8Gated ? BN / 2 : BN;      // output columns a tile
    static_assert(TM >= 1 && TN >= 1 && XI >= 1 && WI >= 1 && (EPI != kI8Gated || TN % 2 == 0), "tile");
    static_assert(D == 2 || D == 4, "ring");
    // an object of its own for each tile: a load into one need not be waited for before another is read
    __shared__ __align__(16) uint8_t x_even[XT], x_odd[XT], w_even[WT], w_odd[WT];
    __shared__ __align__(16) uint8_t x_third[D > 2 ? XT : 16], x_fourth[D > 2 ? XT : 16];
    __shared__ __align__(16) uint8_t w_third[D > 2 ? WT : 16], w_fourth[D > 2 ? WT : 16];
    __shared__ int32_t rows[BM];  // the tile's output rows, their codes' scales: no load between the stores of the end
    __shared__ float scale[BM];

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int tiles_c = (int)((p.c_count + CT - 1) / CT);
    int64_t c0, m0, cnt;  // first column; first row and number of rows of the tile
    int e = 0;
    const int b = blockIdx.x;
    if (p.tiles) {
        // an XCD (workgroups are dealt to the 8 of them in turn) takes a run of the tiles that the routing made:
        // expert by expert, column tile by column tile, the row tiles that share it next to each other
        const int tiles = *p.ntiles * tiles_c, per = (tiles + 7) / 8, t = (b & 7) * per + (b >> 3);
        if ((b >> 3) >= per || t >= tiles) return;  // workgroup-uniform
        const I8Tile g = p.tiles[t / tiles_c];  // some row tile of the group
        e = g.group;
        const int mt = (g.rows + BM - 1) / BM, rr = t - g.tile * tiles_c, ct = rr / mt, rt = rr - ct * mt;
        c0 = p.c_first + (int64_t)ct * CT;
        m0 = g.row + rt * BM;
        cnt = g.rows - rt * BM;
    } else {
        const int tiles_m = (int)((p.R + BM - 1) / BM), tiles = tiles_m * tiles_c, per = (tiles + 7) / 8;
        const int t = (b & 7) * per + (b >> 3);
        if ((b >> 3) >= per || t >= tiles) return;  // workgroup-uniform
        const int bsz = kI8BandM * tiles_c, band = t / bsz, rr = t - band * bsz;
        const int gm = tiles_m - band * kI8BandM < kI8BandM ? tiles_m - band * kI8BandM : kI8BandM, ct = rr / gm;
        c0 = p.c_first + (int64_t)ct * CT;
        m0 = (int64_t)(band * kI8BandM + rr - ct * gm) * BM;
        cnt = p.R - m0;
    }
    const int rows_here = cnt < BM ? (int)cnt : BM;
    const int64_t K = p.K, C = p.C, nsteps = (K + BK - 1) / BK;
    const int8_t* w = p.w + (int64_t)e * p.N * p.ldw;
    const float* ws = p.ws + (int64_t)e * p.N * p.ws_step;

    const uint8_t* xsrc[XI];
    const uint8_t* wsrc[WI];
    int xcol[XI], wcol[WI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int r = (wv * XI + i) * 8 + (lane >> 3);
        const int rc = r < rows_here ? r : rows_here - 1;  // rows past the group: clamped, not stored
        int64_t src = m0 + rc;
        if (p.tiles) src = p.perm[src] / p.div;
        xcol[i] = ((lane & 7) ^ i8_swz(r)) * 16;
        xsrc[i] = (const uint8_t*)p.x + src * p.ldx + xcol[i];
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int r = (wv * WI + i) * 8 + (lane >> 3);
        int64_t n;
        if constexpr (EPI == kI8Gated) {  // 32 gate rows, then their 32 up rows
            const int64_t c = c0 + (r >> 6) * 32 + (r & 31);
            n = (c < C ? c : C - 1) + ((r >> 5) & 1) * C;
        } else {
            n = c0 + r < C ? c0 + r : C - 1;
        }
        wcol[i] = ((lane & 7) ^ i8_swz(r)) * 16;
        wsrc[i] = (const uint8_t*)w + n * p.ldw + wcol[i];
    }
    for (int i = tid; i < BM; i += 64 * NW) {
        const int64_t at = m0 + (i < rows_here ? i : rows_here - 1);
        const int pair = p.tiles ? p.perm[at] : (int)at;
        rows[i] = pair;
        scale[i] = p.xs[p.tiles ? pair / p.div : pair];
    }
    auto issue = [&](int64_t s, uint8_t* xt, uint8_t* wt) {  // chunks past K are zeros
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const uint8_t* src = s * BK + xcol[i] < K ? xsrc[i] + s * BK : (const uint8_t*)&kI8Zero16;
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void_t*)(xt + (wv * XI + i) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            const uint8_t* src = s * BK + wcol[i] < K ? wsrc[i] + s * BK : (const uint8_t*)&kI8Zero16;
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void_t*)(wt + (wv * WI + i) * 1024), 16, 0, 0);
        }
    };

    const int wn = wv % WGN, wm = wv / WGN, row = lane & 31, half = lane >> 5;
    i32x16v_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x16v_t{};
    u32x4_t fa[2][TM], fb[2][TN];  // operands of the current and the next 32-deep slice
    auto load_frags = [&](int set, const uint8_t* xt, const uint8_t* wt, int ks) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = wm * (BM / WGM) + i * 32 + row;
            fa[set][i] = *(const u32x4_t*)(xt + r * BK + (((2 * ks + half) ^ i8_swz(r)) * 16));
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int r = wn * (BN / WGN) + j * 32 + row;
            fb[set][j] = *(const u32x4_t*)(wt + r * BK + (((2 * ks + half) ^ i8_swz(r)) * 16));
        }
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v_t, fa[set][i]),
                                                                  __builtin_bit_cast(i32x4v_t, fb[set][j]),
                                                                  acc[i][j], 0, 0, 0);
    };

    auto step = [&](int64_t s, uint8_t* xt, uint8_t* wt, uint8_t* xn, uint8_t* wnext) {
#pragma unroll
        for (int ks = 0; ks < 3; ++ks) {
            load_frags((ks + 1) & 1, xt, wt, ks + 1);
            multiply(ks & 1);
        }
        i8_stage_barrier<(D - 2) * (XI + WI)>();  // everyone's reads of step s are done, and the tiles of step s + 1 are there
        load_frags(0, xn, wnext, 0);
        issue(s + D < nsteps ? s + D : s, xt, wt);  // past the end: the idle tile, again
        multiply(1);
    };
    issue(0, x_even, w_even);
    issue(nsteps > 1 ? 1 : 0, x_odd, w_odd);
    if constexpr (D > 2) {
        issue(nsteps > 2 ? 2 : 0, x_third, w_third);
        issue(nsteps > 3 ? 3 : 0, x_fourth, w_fourth);
    }
    i8_stage_barrier<(D - 1) * (XI + WI)>();
    load_frags(0, x_even, w_even, 0);
    int64_t s = 0;
    if constexpr (D == 2) {
        for (; s < nsteps; s += 2) {
            step(s, x_even, w_even, x_odd, w_odd);
            if (s + 1 < nsteps) step(s + 1, x_odd, w_odd, x_even, w_even);
        }
    } else {
        for (; s + 4 <= nsteps; s += 4) {  // no branch inside: the compiler would wait for every load where two ways meet
            step(s, x_even, w_even, x_odd, w_odd);
            step(s + 1, x_odd, w_odd, x_third, w_third);
            step(s + 2, x_third, w_third, x_fourth, w_fourth);
            step(s + 3, x_fourth, w_fourth, x_even, w_even);
        }
        if (s < nsteps) step(s, x_even, w_even, x_odd, w_odd);
        if (s + 1 < nsteps) step(s + 1, x_odd, w_odd, x_third, w_third);
        if (s + 2 < nsteps) step(s + 2, x_third, w_third, x_fourth, w_fourth);
    }
    w4_wait_vmcnt<0>();  // no load into LDS outlives the workgroup

    // register v of a 32 x 32 tile holds code row 8(v/4) + 4*half + v%4, weight row lane%32
    constexpr int NC = EPI == kI8Gated ? TN / 2 : TN;  // output columns of a lane
    constexpr int CW = EPI == kI8Gated ? BN / WGN / 2 : BN / WGN;
    const int64_t cl = c0 + wn * CW + row;
    float sc[NC], su[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t c = cl + j * 32 < C ? cl + j * 32 : C - 1;
        sc[j] = ws[c * p.ws_step];
        su[j] = EPI == kI8Gated ? ws[(C + c) * p.ws_step] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int r = wm * (BM / WGM) + i * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
            if (r >= rows_here) continue;
            const int64_t at = (int64_t)rows[r] * p.ldy + cl;
            const float xs = scale[r];
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if (cl + j * 32 >= C) continue;
                if constexpr (EPI == kI8Gated)
                    p.y[at + j * 32] = f32_to_h<T>(gated(acc[i][2 * j][v], acc[i][2 * j + 1][v], xs, sc[j], su[j], p.act));
                else
                    p.part[at + j * 32] = ((float)acc[i][j][v] * xs) * sc[j];
            }
        }
}

}  // namespace qlin
