// w4_dec.hpp -- 4-bit weight products for few tokens (M <= 64): the linear
// layer and the gated feed-forward front.
//
// Bound: the weights are streamed once from HBM (K/2 bytes a row); nothing is
// written but the M outputs.  A workgroup owns TR tiles of 16 weight rows and
// all of K; its waves split K in runs of 128-K pieces (64 bytes a row) and add
// their sums in wave order through LDS (deterministic, no workspace).
//
// One load instruction brings one piece of 16 rows: lane (n = lane % 16,
// q = lane / 16) holds the 32 codes 32q..32q+31 of row n - already a B operand
// of v_mfma_f32_16x16x32 four times over, dword j for matrix instruction j, if
// the A operand (tokens) takes the same 8 elements 32q + 8j.. of x.  No
// transpose, no LDS for the weights, and the unpacking is 7 instructions per 8
// codes (two masks, a shift, four converts) for any number of tokens, which is
// why even one token runs on the matrix cores.
//
// Scales stay out of the products.  With D = sum code * x and X = sum x over
// one group, the group adds s * (D - zero * X): exact in code * x, fp32 sums,
// no rounding of weights.  X comes from one more matrix instruction whose B
// operand is all ones.  A group must not share a matrix instruction with
// another: for groups that are no multiple of 128 the dwords of the four lane
// groups are exchanged (v_permlane32_swap, v_permlane16_swap) so that
// instruction j covers the 32 codes of chunk j.
//
// D row i holds token (i / 4) + 4 (i % 4): a lane's register r is token
// lane/16 + 4r, so M tokens need ceil(M / 4) of the four registers folded.
#pragma once
#include "w4_device.hpp"
#include "w4_launch.hpp"

namespace qlin {

struct W4DecParams {
    const uint16_t* x; int64_t ldx; int M;
    W4Weight w; int64_t I;            // gated: rows n and I + n, columns C = I
    int64_t C;
    const uint16_t* bias; uint16_t* y; int64_t ldy;
    uint16_t* gu; int64_t ldgu; const uint16_t* dy; int64_t lddy; int act;
    int pieces, per_wave;             // K / 128 rounded up; pieces of a wave
    uint32_t ratio_magic;             // units per group r: unit / r = mulhi(unit, magic), magic 0: r = 1
};

__device__ __forceinline__ u32x4_t even_odd(const u32x4_t& v) {  // elements 0 2 4 6 1 3 5 7, the order codes unpack in
    return u32x4_t{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                   __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
}

template <int T>
__device__ __forceinline__ u32x4_t unpack8(uint32_t d) {
    const uint32_t e = d & 0x0F0F0F0Fu, o = (d >> 4) & 0x0F0F0F0Fu;
    return u32x4_t{codes2<T, false>(e), codes2<T, true>(e), codes2<T, false>(o), codes2<T, true>(o)};
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {  // a's lanes 32.. <-> b's lanes ..31
    typedef unsigned u2_t __attribute__((ext_vector_type(2)));
    const u2_t r = __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(a, b, false, false));
    a = r[0];
    b = r[1];
}

__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {  // a's odd rows of 16 lanes <-> b's even rows
    typedef unsigned u2_t __attribute__((ext_vector_type(2)));
    const u2_t r = __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane16_swap(a, b, false, false));
    a = r[0];
    b = r[1];
}

// v of lane group 0..3 in every lane: out[i] = v of lanes 16i..16i+15
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&out)[4]) {
    uint32_t a = v, b = v;
    swap32(a, b);
    out[0] = a;
    out[1] = a;
    out[2] = b;
    out[3] = b;
    swap16(out[0], out[1]);
    swap16(out[2], out[3]);
}

constexpr int kW4XPad = 8;  // elements between staged token rows: 16 bytes, so the rows start in different banks

template <int T, int U, int TR, int MT, int RM, int PB, bool XL, bool LOOP, bool GLU, int NTMAX>
__global__ __launch_bounds__(NTMAX) void w4_dec_kernel(const W4DecParams p) {
    static_assert(U == 128 || U == 32, "fold unit");
    static_assert(!GLU || TR % 2 == 0, "gate and up tiles come in pairs");
    constexpr int UPP = 128 / U;                // fold units per piece
    constexpr int SL = (PB * UPP + 3) / 4;      // scale loads per tile and batch: four units each
    constexpr int CT = GLU ? TR * 8 : TR * 16;  // output columns of a workgroup
    extern __shared__ __align__(16) uint8_t w4d_lds[];

    const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 63, wv = tid >> 6, NW = NT >> 6;
    const int n = lane & 15, q = lane >> 4, M = p.M;
    const int64_t K = p.w.K;
    const int64_t c0 = (int64_t)blockIdx.x * CT;
    const int p0 = wv * p.per_wave, p1 = p0 + p.per_wave < p.pieces ? p0 + p.per_wave : p.pieces;
    const int KP = p.pieces * 128, XP = KP + kW4XPad;  // staged token row, elements

    // ---- token rows to LDS, in unpacking order, zero past K
    uint16_t* xs = (uint16_t*)w4d_lds;
    const int per_row = KP / 8, total = M * per_row;
    auto x_chunk = [&](int c) {
        const int m = c / per_row, k = (c - m * per_row) * 8;
        return k < K ? *(const u32x4_t*)(p.x + m * p.ldx + k) : u32x4_t{0u, 0u, 0u, 0u};
    };
    auto x_put = [&](int c, const u32x4_t& v) {
        const int m = c / per_row, k = (c - m * per_row) * 8;
        *(u32x4_t*)(xs + m * XP + k) = even_odd(v);
    };
    constexpr int XC = 2;  // chunks a thread requests ahead of the weights
    u32x4_t xv[XC];
    if constexpr (XL) {
        for (int c = tid + XC * NT; c < total; c += NT) x_put(c, x_chunk(c));
#pragma unroll
        for (int i = 0; i < XC; ++i)
            if (tid + i * NT < total) xv[i] = x_chunk(tid + i * NT);
    }

    // ---- this lane's row of each tile
    const int64_t ngroups = K / p.w.group;
    const uint8_t* wrow[TR];
    const uint16_t* srow[TR];
    const uint8_t* zrow[TR];
#pragma unroll
    for (int t = 0; t < TR; ++t) {
        const int64_t col = GLU ? c0 + (t >> 1) * 16 + n : c0 + t * 16 + n;
        const int64_t r = (col < p.C ? col : p.C - 1) + (GLU && (t & 1) ? p.I : 0);  // rows past the end: not stored
        wrow[t] = p.w.w + r * p.w.ldw;
        srow[t] = p.w.ws + r * ngroups;
        zrow[t] = p.w.wz + (p.w.wz ? r * ngroups : 0);
    }

    // A operand row n is token n/4 + 4 (n%4) of each 16; tokens past M repeat the last (not stored)
    int tok[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = mt * 16 + (n >> 2) + 4 * (n & 3);
        tok[mt] = m < M ? m : M - 1;
    }
    // first of the 8 elements that this lane supplies to matrix instruction j of a piece
    auto lane_k = [&](int j) { return U == 32 ? j * 32 + ((q & 1) << 1 | (q >> 1)) * 8 : q * 32 + j * 8; };

    struct Batch { u32x4_t w[PB][TR]; uint32_t s[SL][TR], z[SL][TR]; u32x4_t a[XL ? 1 : PB][4][MT]; };
    const uint32_t units = (uint32_t)((K + U - 1) / U);
    auto load = [&](Batch& b, int pc) {
        if constexpr (!XL) {  // ahead of the weights: loads return in order, and the first product needs both
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int64_t k = (int64_t)(pc + i) * 128 + lane_k(j);
                        const bool ok = k < K && pc + i < p1;
                        const u32x4_t v = *(const u32x4_t*)(p.x + tok[mt] * p.ldx + (ok ? k : 0));
                        b.a[i][j][mt] = ok ? v : u32x4_t{0u, 0u, 0u, 0u};
                    }
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int64_t k = (int64_t)(pc + i) * 128 + q * 32;
            const int64_t off = k < K && pc + i < p1 ? k / 2 : 0;  // past the end: any codes, x is zero there
#pragma unroll
            for (int t = 0; t < TR; ++t) b.w[i][t] = ld_stream(wrow[t] + off);
        }
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            uint32_t u = (uint32_t)pc * UPP + i * 4 + q;
            u = u < units ? u : units - 1;
            const uint32_t g = p.ratio_magic ? __umulhi(u, p.ratio_magic) : u;
#pragma unroll
            for (int t = 0; t < TR; ++t) {
                b.s[i][t] = srow[t][g];
                b.z[i][t] = p.w.wz ? zrow[t][g] : 8;
            }
        }
    };

    f32x4v_t acc[TR][MT];
#pragma unroll
    for (int t = 0; t < TR; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = f32x4v_t{0.f, 0.f, 0.f, 0.f};

    const uint32_t one = T == kBf16 ? 0x3F803F80u : 0x3C003C00u;
    const u32x4_t ones = {one, one, one, one};

    auto compute = [&](const Batch& b, int pc) {
        uint32_t sz[SL][TR][4];
#pragma unroll
        for (int i = 0; i < SL; ++i)
#pragma unroll
            for (int t = 0; t < TR; ++t) spread4((b.s[i][t] << 16) | b.z[i][t], sz[i][t]);
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            if (pc + i >= p1) break;  // wave-uniform
            uint32_t d[TR][4];
#pragma unroll
            for (int t = 0; t < TR; ++t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[t][j] = b.w[i][t][j];
                if constexpr (U == 32) {
                    // dword d of lane group c is chunk c, dword d; afterwards register j holds chunk
                    // {0, 2, 1, 3}[j] and lane group q its dword {0, 2, 1, 3}[q]
                    swap32(d[t][0], d[t][1]);
                    swap32(d[t][2], d[t][3]);
                    swap16(d[t][0], d[t][2]);
                    swap16(d[t][1], d[t][3]);
                }
            }
            f32x4v_t D[TR][MT], X[MT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // after the swaps register 0, 2, 1, 3 is chunk 0, 1, 2, 3: walk the chunks in order
                const int reg = U == 32 ? ((j & 1) << 1 | (j >> 1)) : j;
                u32x4_t a[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (XL) a[mt] = *(const u32x4_t*)(xs + tok[mt] * XP + (pc + i) * 128 + lane_k(j));
                    else a[mt] = even_odd(b.a[i][j][mt]);
                }
                const bool first = U == 32 || j == 0;
                const f32x4v_t zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) X[mt] = mfma16<T>(a[mt], ones, first ? zero4 : X[mt]);
#pragma unroll
                for (int t = 0; t < TR; ++t) {
                    const u32x4_t bw = unpack8<T>(d[t][reg]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) D[t][mt] = mfma16<T>(a[mt], bw, first ? zero4 : D[t][mt]);
                }
                if (U == 32 || j == 3) {
                    const int u = U == 32 ? i * 4 + j : i;
#pragma unroll
                    for (int t = 0; t < TR; ++t) {
                        const uint32_t v = sz[u >> 2][t][u & 3];
                        const float s = T == kBf16 ? __uint_as_float(v & 0xFFFF0000u) : h_to_f32<kFp16>(v >> 16);
                        const float z = (float)(v & 0xFFu);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int r = 0; r < RM; ++r)
                                acc[t][mt][r] = fmaf(s, fmaf(-z, X[mt][r], D[t][mt][r]), acc[t][mt][r]);
                    }
                }
            }
        }
    };

    Batch cur;
    load(cur, p0 < p1 ? p0 : 0);
    if constexpr (XL) {
#pragma unroll
        for (int i = 0; i < XC; ++i)
            if (tid + i * NT < total) x_put(tid + i * NT, xv[i]);
        __syncthreads();
    }
    if constexpr (LOOP) {
        for (int pc = p0; pc < p1; pc += PB) {
            Batch nxt;
            const bool more = pc + PB < p1;
            if (more) load(nxt, pc + PB);
            compute(cur, pc);
            if (more) cur = nxt;
        }
    } else {
        compute(cur, p0);
    }

    // ---- sums of the waves, in wave order.  red[wave][token][tile][16]
    if constexpr (XL) __syncthreads();  // the token rows are no longer needed
    float* red = (float*)w4d_lds;
#pragma unroll
    for (int t = 0; t < TR; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                const int m = mt * 16 + q + 4 * r;
                if (m < M) red[((wv * M + m) * TR + t) * 16 + n] = acc[t][mt][r];
            }
    __syncthreads();
    for (int o = tid; o < M * CT; o += NT) {
        const int m = o / CT, j = o - m * CT, t0 = GLU ? (j >> 4) * 2 : j >> 4, jn = j & 15;
        const int64_t c = c0 + j;
        if (c >= p.C) continue;
        const float* src = red + (m * TR + t0) * 16 + jn;
        float v = 0.f, v2 = 0.f;
        for (int k = 0; k < NW; ++k) {
            v += src[k * M * TR * 16];
            if constexpr (GLU) v2 += src[k * M * TR * 16 + 16];
        }
        if constexpr (GLU) {
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
