// w4_few.hpp -- 4-bit weight products for up to 16 tokens (decode): the linear
// layer and the gated feed-forward front.
//
// Bound: the weights are streamed once from HBM (K/2 bytes a row); everything
// else is small.  What that takes here:
//
// * Loads of whole 128-byte lines.  One load instruction brings 8 rows x 256 K:
//   lanes n and n + 8 (n = lane % 16, q = lane / 16) hold the two 128-K halves
//   of row n % 8, 32 codes each, chunk q of the half.  (Loads alone, 17408 x
//   5120: 8.2 us so, 10.2 us with 64 bytes of 16 rows an instruction.)
//
// * No transpose.  The 32 codes are a B operand of v_mfma_f32_16x16x32 four
//   times over (dword j for instruction j).  Columns n < 8 want the tokens'
//   first half and columns n >= 8 the second, so the A operand holds the (at
//   most 8) tokens twice: rows 0-7 with the first half of x, rows 8-15 with
//   the second.  Of D only the two blocks with matching halves are used, and
//   they are added at the end.  Row i of a half is token i/4 + 2 (i%4): a
//   lane's register r is token q%2 + 2r, so M tokens fold ceil(M / 2) registers.
//   9 to 16 tokens (FULL) need all 16 rows of A: tiles of 16 weight rows, and
//   the two loads of a line (rows 0-7, 8-15) exchange their 8-lane halves, one
//   DPP move per register; row i of A is token i/4 + 4 (i%4).
//
// * 7 instructions per 8 codes: two masks, a shift and four converts, for any
//   number of tokens (the vector unit is the second bound: about 5 us of its
//   time for 17408 x 5120, 7 to 8 us with the exchange of 9 to 16 tokens).
//   Scales stay out of the products: with D = sum code * x and X = sum x over a
//   group, y = sum s * D - sum (s * zero) * X, exact in code * x, fp32 sums, no
//   rounding of weights.  The second sum is a
//   product of its own, four groups at a time on v_mfma_f32_16x16x4_f32; X is
//   what the tokens' products with a B operand of ones give, found while the
//   weights are still in flight.  Groups that are no multiple of 128 (fold unit
//   U = 64 or 32) exchange dwords between the lane groups (v_permlane32_swap,
//   v_permlane16_swap) so that no instruction spans two groups.
//
// * One round of workgroups, evenly loaded.  A workgroup owns `rows` adjacent
//   rows (tiles of 8; rows past its share repeat the last row's addresses), N /
//   256 of them where that fits, and each of its waves PL lines of 256 K, all
//   rows of which it walks with D tiles requested ahead.  D is small on
//   purpose: about 20-32 KB a compute unit in flight.  With all loads requested
//   at once (17408 x 5120: 9 tiles) the first waves are served first and the
//   last one unpacks its whole share alone at the end (2 us more than D = 1);
//   two or more uneven rounds of workgroups cost 2 to 5 us.
//
// * Token rows, scales and zero points go to LDS ahead of the weights
//   (global_load_lds, no registers): the scales by the whole workgroup, one
//   barrier, which leaves the weight loads outstanding; its own lines of the
//   token rows by each wave, without a barrier, so that waves walk a long row
//   independently (with a barrier a pass and all tokens' slice shared: 14336 x
//   4099, 5 tokens 19.6 us, now 16.3).  The waves' sums are added in wave order
//   through LDS (deterministic, no workspace).  Rows longer than 16 waves'
//   lines (K > 8192 or 4096), or too long for LDS, are walked in passes.
//
// Nothing may be in private memory here: its loads return in order behind the
// weights' and would be waited for with them (the offsets of the scales in an
// array of private memory cost a call 1 to 2 us).
//
// Measured (bf16, zero points, groups of 128, weights cold): 17408 x 5120, one
// token 11.5 us (4.1 TB/s of codes and scales), 8 tokens 13.5, 16 tokens 16.1;
// 28672 x 4096 gated, one token 13.9 us (4.4 TB/s), 16 tokens 19.0; 1024 x 1024
// 3.6 us.
#pragma once
#include "w4_device.hpp"
#include "w4_launch.hpp"
#include "w4_plan.hpp"

namespace qlin {

struct W4FewParams {
    const uint16_t* x; int64_t ldx; int M;
    W4Weight w; int64_t I;            // I > 0: gated, rows n and I + n, columns C = I
    int64_t C;
    const uint16_t* bias; uint16_t* y; int64_t ldy;
    uint16_t* gu; int64_t ldgu; const uint16_t* dy; int64_t lddy; int act;
    int rows;                         // columns of a workgroup
    int passes;                       // K is walked in this many slices of (waves * PL) lines
    int groups;                       // K / group
    uint32_t ratio_magic;             // fold units per group r: unit / r = mulhi(unit, magic), 0: r = 1
};

template <int T, int U, int RM, int PL, int D, bool FULL>
__global__ __launch_bounds__(1024) void w4_few_kernel(const W4FewParams p) {
    static_assert(U == 128 || U == 64 || U == 32, "fold unit");
    constexpr int TR = FULL ? 16 : 8;  // rows of a tile
    constexpr int LH = FULL ? 2 : 1;   // halves of a line that a lane's row takes part in, loads of a line
    constexpr int UPH = 128 / U;       // fold units per half line
    constexpr int NU = PL * LH * UPH;  // of a wave, for each of its rows
    constexpr int NC = (NU + 3) / 4;   // fp32 matrix instructions that take out their zero points
    extern __shared__ __align__(16) uint8_t w4f_lds[];

    const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 63, wv = tid >> 6, NW = NT >> 6;
    const int n = lane & 15, q = lane >> 4, half = n >> 3, M = p.M;
    const int K = (int)p.w.K;
    const int64_t c0 = (int64_t)blockIdx.x * p.rows;
    const int CT = p.C - c0 < p.rows ? (int)(p.C - c0) : p.rows;  // columns of this workgroup, at least 1
    const int KP = NW * PL * 256, G = p.groups;  // KP: K of a pass
    const bool glu = p.I > 0;
    const int parts = glu ? 2 : 1, GT = (CT + TR - 1) / TR, TT = parts * GT;  // tiles; gated: gate and up alternate
    const W4FewLds at = w4_few_lds(M, U, PL, parts * CT, TT * TR, G, NW);
    const int xloads = (PL * M + 1) / 2;                    // of 1 KB: two token lines each
    uint16_t* xw = (uint16_t*)w4f_lds + wv * xloads * kW4FewLoad;  // this wave's [token][line][256], zero past K
    float* xsum = (float*)(w4f_lds + at.xsum);        // [wave][NU][16]
    float* red = (float*)(w4f_lds + at.red);          // [token][gate and up][CT][RS]: the waves' sums
    const int RS = w4_few_red(NW);

    // ---- staging, ahead of the weights (loads return in order) and straight into LDS: 16 bytes a thread
    auto stage = [&](const void* src, void* dst, uint32_t bytes) {  // both 16-byte aligned, bytes a multiple of 16
        for (uint32_t o = 0; o < bytes; o += NT * 16)
            if (o + tid * 16 < bytes)
                __builtin_amdgcn_global_load_lds((const void*)((const uint8_t*)src + o + tid * 16),
                                                 (lds_void_t*)((uint8_t*)dst + o + wv * 1024), 16, 0, 0);
    };
    // Each wave stages its own lines and so needs no barrier for them.  A load takes 512 bytes twice: a token's two
    // lines, or two tokens' one.  The 16-byte chunks of a line are permuted so that the A operands' reads (the same
    // chunk of 16 tokens, or of the two halves of 8) fall into different banks.
    auto place = [&](int chunk, int sub) {  // its own inverse
        return chunk ^ (PL > 1 ? (chunk >> 4) * 8 : sub * 8 ^ (chunk >> 4) * 4);
    };
    auto stage_x = [&](int k0) {
        const int sub = lane >> 5, k = k0 + (PL > 1 ? sub * 256 : 0) + place(lane & 31, sub) * 8;
        const bool in = k < K;
        const int64_t step = in ? (PL > 1 ? p.ldx : 2 * p.ldx) : 0;
        const uint16_t* src = in ? p.x + (PL > 1 ? 0 : sub * p.ldx) + k : (const uint16_t*)&kW4Zero16;
        for (int i = 0; i < xloads; ++i, src += step) {
            if (PL == 1 && 2 * i + 1 == M && in) src -= sub * p.ldx;  // no token M: the last one again
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void_t*)(xw + i * kW4FewLoad), 16, 0, 0);
        }
    };
    stage_x(wv * PL * 256);
    // The scales of adjacent rows are one contiguous block, which may start anywhere: the 16-byte lines that
    // hold it are copied (at most 15 bytes more at each end, of the same line), and read at its offset.
    const bool has_z = p.w.wz != nullptr;
    uint32_t sat[2], zat[2];  // LDS offsets of the gate and the up block (plain: the first)
    {
        uint32_t so = at.s, zo = at.z;
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // a trip count known here keeps the offsets in registers
            if (part == 1 && !glu) break;
            const int64_t first = (c0 + (part ? p.I : 0)) * G;
            const uint32_t count = (uint32_t)CT * G;
            const uintptr_t sa = (uintptr_t)(p.w.ws + first), za = (uintptr_t)(p.w.wz + (has_z ? first : 0));
            const uint32_t sm = (uint32_t)(sa & 15), zm = (uint32_t)(za & 15);
            const uint32_t sbytes = (sm + count * 2 + 15) / 16 * 16, zbytes = (zm + count + 15) / 16 * 16;
            stage((const void*)(sa - sm), w4f_lds + so, sbytes);
            sat[part] = so + sm;
            so += sbytes;
            if (has_z) stage((const void*)(za - zm), w4f_lds + zo, zbytes);
            zat[part] = zo + zm;
            zo += zbytes;
        }
    }

    // ---- the weights: D tiles of this wave in flight
    const uint8_t* base = p.w.w + c0 * p.w.ldw;
    const uint8_t* ubase = base + p.I * p.w.ldw;
    uint32_t koff[PL];
    u32x4_t w[D][PL][LH];
    auto load_tile = [&](int slot, int t) {
        const int first = (glu ? t >> 1 : t) * TR + (n & 7);
        const uint8_t* b = glu && (t & 1) ? ubase : base;
#pragma unroll
        for (int v = 0; v < LH; ++v) {  // 8 rows each; rows past the share repeat its last
            const int r = first + v * 8;
            const uint32_t roff = (uint32_t)(r < CT ? r : CT - 1) * (uint32_t)p.w.ldw;
#pragma unroll
            for (int l = 0; l < PL; ++l) w[slot][l][v] = ld_stream(b + (roff + koff[l]));
        }
    };

    // row n of A: half n / 8, token (n % 8) / 4 + 2 (n % 4); FULL: token n / 4 + 4 (n % 4).  Tokens past M
    // repeat the last (not stored).
    int tok = FULL ? (n >> 2) + 4 * (n & 3) : ((n & 7) >> 2) + 2 * (n & 3);
    tok = tok < M ? tok : M - 1;
    auto lane_k = [&](int j) {  // first of the 8 elements of instruction j, within the half line
        if constexpr (U == 128) return q * 32 + j * 8;
        else if constexpr (U == 64) return ((j >> 1) * 2 + (q & 1)) * 32 + ((j & 1) * 2 + (q >> 1)) * 8;
        else return j * 32 + ((q & 1) << 1 | (q >> 1)) * 8;
    };
    const uint32_t one = T == kBf16 ? 0x3F803F80u : 0x3C003C00u;
    const u32x4_t ones = {one, one, one, one};
    const f32x4v_t zero4 = {0.f, 0.f, 0.f, 0.f};
    u32x4_t a[PL][LH][4];
    // unit e of the lane's row: lane group q looks after unit 4c + q (two units: q % 2, one: all the same)
    auto unit_of = [&](int c) { return NU >= 4 ? c * 4 + q : (NU == 2 ? q & 1 : 0); };
    float nx[NC];  // -X of row n of A and that unit
    int gi[NC];    // index of the unit's scale in this lane's row of a tile

    // where this lane's sums go: token token0 + 4r (FULL) or + 2r of register r, column n of a tile
    const int token0 = FULL ? q : q & 1, red_step = (FULL ? 4 : 2) * parts * CT * RS;
    float* red_lane = red + (token0 * parts * CT + n) * RS + wv;

    // A tile is waited for, and then the load that follows it into flight is issued before the work on it begins;
    // left to itself the compiler issues that load before the wait or after the work.
    u32x4_t now[PL][LH];
    auto take = [&](int slot) {
#pragma unroll
        for (int l = 0; l < PL; ++l)
#pragma unroll
            for (int v = 0; v < LH; ++v) {
                now[l][v] = w[slot][l][v];
                asm volatile("" : "+v"(now[l][v]));
            }
    };

    // ---- products, tile by tile as the weights arrive
    auto tile = [&](int t, bool add) {
        const int up = glu ? t & 1 : 0, g0 = (glu ? t >> 1 : t) * TR * G;
        const uint16_t* ss = (const uint16_t*)(w4f_lds + (up ? sat[1] : sat[0])) + g0;
        const uint8_t* zs = w4f_lds + (up ? zat[1] : zat[0]) + g0;
        f32x4v_t acc = zero4;
        uint32_t sf[NC][4];  // scale of unit 4c + i, in every lane group
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float s = h_to_f32<T>(ss[gi[c]]);
            const uint32_t zb = zs[gi[c]];
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(nx[c], s * (has_z ? (float)zb : 8.0f), acc, 0, 0, 0);
            const uint32_t sb = __float_as_uint(s);
            if constexpr (NU >= 4) {
                spread4(sb, sf[c]);
            } else {
                sf[c][0] = sb;
                sf[c][1] = sb;
                if constexpr (NU == 2) swap16(sf[c][0], sf[c][1]);
            }
        }
#pragma unroll
        for (int l = 0; l < PL; ++l)
#pragma unroll
            for (int v = 0; v < LH; ++v) {  // FULL: half v of the line
                uint32_t d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d[j] = now[l][v][j];
                    if constexpr (FULL) {  // half 0: lanes n >= 8 fetch rows 8-15's first half, half 1: n < 8 rows 0-7's second
                        const int keep = (int)d[j], other = (int)now[l][v ^ (LH - 1)][j];
                        d[j] = (uint32_t)(v == 0 ? __builtin_amdgcn_update_dpp(keep, other, 0x128, 0xF, 0xC, false)
                                                 : __builtin_amdgcn_update_dpp(keep, other, 0x128, 0xF, 0x3, false));
                    }
                }
                // dword d of lane group c is chunk c, dword d.  U = 64: registers 0, 2 take chunks 0 and 1,
                // registers 1, 3 chunks 2 and 3.  U = 32: register 0, 2, 1, 3 takes chunk 0, 1, 2, 3
                if constexpr (U != 128) {
                    swap32(d[0], d[1]);
                    swap32(d[2], d[3]);
                }
                if constexpr (U == 32) {
                    swap16(d[0], d[2]);
                    swap16(d[1], d[3]);
                }
#pragma unroll
                for (int h = 0; h < UPH; ++h) {
                    f32x4v_t P = zero4;
#pragma unroll
                    for (int j = h * (U / 32); j < (h + 1) * (U / 32); ++j)
                        P = mfma16<T>(a[l][v][j], unpack8<T>(d[U == 128 ? j : ((j & 1) << 1 | (j >> 1))]), P);
                    const int e = (l * LH + v) * UPH + h;
                    const float s = __uint_as_float(sf[e / 4][e % 4]);
#pragma unroll
                    for (int r = 0; r < RM; ++r) acc[r] = fmaf(s, P[r], acc[r]);
                }
            }
        const int j0 = (glu ? t >> 1 : t) * TR;  // the tile's first column
        float* out = red_lane + (up * CT + j0) * RS;
        const bool mine = (FULL || (n < 8 && q < 2)) && n < CT - j0;
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            float sum = acc[r];
            if constexpr (!FULL) {  // add the two halves: lanes (n, q) and (n ^ 8, q ^ 2) hold the same rows and tokens
                uint32_t x = __float_as_uint(sum), y = x;
                swap32(x, y);  // x: lanes 0-31 twice, y: lanes 32-63 twice
                sum = __uint_as_float(x) + __int_as_float(dpp_mov<0x128>((int)y));
            }
            float* at = out + r * red_step;
            if (mine && token0 + r * (FULL ? 4 : 2) < M) *at = add ? *at + sum : sum;
        }
    };
    for (int pass = 0; pass < p.passes; ++pass) {
        const int k0 = pass * KP + wv * PL * 256;  // this wave's first element
#pragma unroll
        for (int l = 0; l < PL; ++l) {
            const int k = k0 + l * 256 + half * 128 + q * 32;
            koff[l] = k < K ? k / 2 : 0;  // past K: any codes, x is zero there
        }
        if (pass > 0) stage_x(k0);  // this wave has read the last pass's
#pragma unroll
        for (int t = 0; t < D; ++t) load_tile(t, t < TT ? t : TT - 1);
        __builtin_amdgcn_sched_barrier(0);
        w4_wait_vmcnt<D * PL * LH>();  // what was staged has arrived; the weights are on their way
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (pass == 0) w4_lds_barrier();  // the scales and zero points of the others, too

        // A operands and X of this wave's lines
#pragma unroll
        for (int l = 0; l < PL; ++l) {
            #pragma unroll
            for (int v = 0; v < LH; ++v) {
                const int sub = PL > 1 ? l : tok & 1;
                const uint16_t* row = xw + (PL > 1 ? tok : tok >> 1) * kW4FewLoad + sub * 256;
                const int first = (FULL ? v : half) * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[l][v][j] = even_odd(*(const u32x4_t*)(row + place(first + lane_k(j) / 8, sub) * 8));
#pragma unroll
                for (int h = 0; h < UPH; ++h) {  // D is the same in every column; one writes it
                    f32x4v_t s = zero4;
#pragma unroll
                    for (int j = h * (U / 32); j < (h + 1) * (U / 32); ++j) s = mfma16<T>(a[l][v][j], ones, s);
                    if (n == 0) *(f32x4v_t*)(xsum + (wv * NU + (l * LH + v) * UPH + h) * 16 + q * 4) = s;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = unit_of(c);
            const float x = xsum[(wv * NU + e) * 16 + n];  // this wave's own: LDS operations of a wave are in order
            nx[c] = NU >= 4 || q < NU ? -x : 0.f;
            const uint32_t line = (uint32_t)((pass * NW + wv) * PL + e / (LH * UPH));
            uint32_t u = line * 2 * UPH + (FULL ? e % (2 * UPH) : half * UPH + e % UPH);
            if (p.ratio_magic) u = __umulhi(u, p.ratio_magic);
            gi[c] = (FULL ? n : n & 7) * G + ((int)u < G ? (int)u : G - 1);
        }

        // no load under a branch in the main loop: the compiler's load counters stay exact
        int t = 0;
        for (; t + 2 * D <= TT; t += D) {
#pragma unroll
            for (int i = 0; i < D; ++i) {
                take(i);
                load_tile(i, t + i + D);
                tile(t + i, pass > 0);
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * D - 1; ++i) {
            if (t + i >= TT) break;
            take(i % D);
            if (t + i + D < TT) load_tile(i % D, t + i + D);
            tile(t + i, pass > 0);
        }
    }
    w4_lds_barrier();

    // ---- sums of the waves, in order: a wave to each token, or all to the only one
    const bool single = M == 1;
    for (int m = single ? 0 : wv; m < M; m += NW)
    for (int j = single ? tid : lane; j < CT; j += single ? NT : 64) {
        const int64_t c = c0 + j;
        const float* src = red + (m * parts * CT + j) * RS;
        auto total = [&](const float* f) {
            f32x4v_t part[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) part[k] = *(const f32x4v_t*)(f + (k * 4 < NW ? k * 4 : 0));
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) v += k < NW ? part[k >> 2][k & 3] : 0.f;
            return v;
        };
        float v = total(src);
        if (glu) {
            const float v2 = total(src + CT * RS);
            float av, dav;
            gate_act(v, p.act, av, dav);
            if (!p.dy) {
                p.y[m * p.ldy + c] = f32_to_h<T>(av * v2);
                if (p.gu) {
                    p.gu[m * p.ldgu + c] = f32_to_h<T>(v);
                    p.gu[m * p.ldgu + p.I + c] = f32_to_h<T>(v2);
                }
            } else {
                const float d = h_to_f32<T>(p.dy[m * p.lddy + c]);
                p.gu[m * p.ldgu + c] = f32_to_h<T>(d * v2 * dav);
                p.gu[m * p.ldgu + p.I + c] = f32_to_h<T>(d * av);
            }
        } else {
            if (p.bias) v += h_to_f32<T>(p.bias[c]);
            p.y[m * p.ldy + c] = f32_to_h<T>(v);
        }
    }
}

}  // namespace qlin
