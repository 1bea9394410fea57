// w4_bwd.hpp -- input gradient dx = dy W of the 4-bit layer for up to 64
// tokens (the GEMM takes more).
//
// Bound: the latency of the weights' stream (K/2 bytes a row): four waves a
// compute unit, each a block ahead.  Behind it the vector unit: the scale
// varies along the reduction, so a weight is dequantised before it is
// multiplied, (code - zero) * s in fp32 rounded once to the 16-bit type, 2.8
// instructions a code (5120 x 5120, 7 tokens: busy for 4 of 9.4 us).
//
// A B operand of v_mfma_f32_16x16x32 wants 8 successive n of one column k in a
// lane.  Lane (c = lane % 16, q = lane / 16) loads CW codes of row 8q + j for j
// = 0..7 (CW = 16: whole 128-byte lines of 4 rows an instruction) and takes
// for matrix instruction i code i of each of its 8 rows: the columns of
// instruction i are CW c + i, so no transpose is needed anywhere.  All codes of
// a lane in a row lie in one scale group (CW <= 32).
//
// A workgroup owns 16 CW columns and a share of the rows (gridDim.y shares, in
// whole blocks of 32), its 4 waves take those blocks in turn and add their sums
// in wave order through LDS, 16 tokens at a time; the shares' sums go through
// the workspace and are added in order by w4_reduce_kernel.
#pragma once
#include "w4_device.hpp"
#include "w4_launch.hpp"

namespace qlin {

struct W4BwdParams {
    const uint16_t* dy; int64_t lddy; int M;
    W4Weight w;
    uint16_t* dx; int64_t lddx;
    float* part;            // [share][M][K], or null: one share, stored to dx
    int share;              // blocks of 32 rows a share
};

template <int T, int CW, int MT>
__global__ __launch_bounds__(256, 2) void w4_bwd_kernel(const W4BwdParams p) {
    constexpr int COLS = 16 * CW, NW = 4, DW = CW / 8;  // dwords of a lane in a row
    __shared__ float red[NW * 16 * COLS];               // [wave][token % 16][column]
    typedef uint32_t codes_t __attribute__((ext_vector_type(DW)));

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, c = lane & 15, q = lane >> 4, M = p.M;
    const int64_t N = p.w.N, K = p.w.K, k0 = (int64_t)blockIdx.x * COLS, k = k0 + c * CW;
    const int64_t ngroups = K / p.w.group, kc = k < K ? k : 0;  // columns past K: not stored
    const bool has_z = p.w.wz != nullptr;
    const uint8_t* wcol = p.w.w + kc / 2;
    const uint16_t* scol = p.w.ws + kc / p.w.group;
    const uint8_t* zcol = has_z ? p.w.wz + kc / p.w.group : (const uint8_t*)scol;  // without zeros: not used
    const int64_t blocks = (N + 31) / 32, b0 = (int64_t)blockIdx.y * p.share;
    const int64_t b1 = b0 + p.share < blocks ? b0 + p.share : blocks;

    struct Block { codes_t d[8]; uint16_t s[8]; uint8_t z[8]; u32x4_t a[MT]; };
    auto load = [&](Block& b, int64_t blk) {
        const int64_t n0 = blk * 32 + q * 8;
#pragma unroll
        for (int m = 0; m < MT; ++m) {  // row c of A: token 16 m + c; past M repeats the last (not stored)
            const int t = m * 16 + c;
            b.a[m] = *(const u32x4_t*)(p.dy + (t < M ? t : M - 1) * p.lddy + (n0 < N ? n0 : 0));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + j < N ? n0 + j : N - 1;
            b.d[j] = __builtin_nontemporal_load((const codes_t*)(wcol + n * p.w.ldw));
            b.s[j] = scol[n * ngroups];
            b.z[j] = zcol[n * ngroups];
        }
    };
    f32x4v_t acc[MT][CW];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < CW; ++i) acc[m][i] = f32x4v_t{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](Block& b, int64_t blk) {
        const int64_t left = N - (blk * 32 + q * 8);  // rows past the end: scale 0 and dy 0, whatever the pitch holds
        float s[8], o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = j < left ? h_to_f32<T>(b.s[j]) : 0.f;
            o[j] = -(has_z ? (float)b.z[j] : 8.0f) * s[j];
        }
        if (left < 8) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b.a[m][j] &= (2 * j < left ? 0xFFFFu : 0u) | (2 * j + 1 < left ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < DW; ++w) {
            uint32_t e[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = b.d[j][w] & 0x0F0F0F0Fu;
                h[j] = (b.d[j][w] >> 4) & 0x0F0F0F0Fu;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = fmaf((float)(((i & 1 ? h[j] : e[j]) >> (8 * (i >> 1))) & 0xFFu), s[j], o[j]);
                u32x4_t bw;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2v_t pr = {v[2 * j], v[2 * j + 1]};
                    if constexpr (T == kBf16) bw[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2_t));
                    else bw[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, f16x2_t));
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m][w * 8 + i] = mfma16<T>(b.a[m], bw, acc[m][w * 8 + i]);
            }
        }
    };
    // the next block is on its way while one is dequantised
    Block cur;
    int64_t blk = b0 + wv;
    if (blk < b1) {
        load(cur, blk);
        for (; blk + NW < b1; blk += NW) {
            Block nxt;
            load(nxt, blk + NW);
            compute(cur, blk);
            cur = nxt;
        }
        compute(cur, blk);
    }

    // ---- sums of the waves, in order: register r of instruction i is token 4q + r, column CW c + i
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m * 16 >= M) break;  // workgroup-uniform
        if (m > 0) w4_lds_barrier();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < CW; i += 4)
                *(f32x4v_t*)(red + (wv * 16 + 4 * q + r) * COLS + c * CW + i) =
                    f32x4v_t{acc[m][i][r], acc[m][i + 1][r], acc[m][i + 2][r], acc[m][i + 3][r]};
        w4_lds_barrier();
        const int tokens = M - m * 16 < 16 ? M - m * 16 : 16;
        for (int e = tid; e < tokens * (COLS / 4); e += 256) {
            const int t = e / (COLS / 4), j = (e - t * (COLS / 4)) * 4;
            if (k0 + j >= K) continue;  // K is a multiple of 32: four columns at once
            f32x4v_t v = *(const f32x4v_t*)(red + t * COLS + j);
#pragma unroll
            for (int w = 1; w < NW; ++w) v += *(const f32x4v_t*)(red + (w * 16 + t) * COLS + j);
            const int64_t tok = m * 16 + t;
            if (p.part) {
                *(f32x4v_t*)(p.part + ((int64_t)blockIdx.y * M + tok) * K + k0 + j) = v;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) p.dx[tok * p.lddx + k0 + j + x] = f32_to_h<T>(v[x]);
            }
        }
    }
}

}  // namespace qlin
