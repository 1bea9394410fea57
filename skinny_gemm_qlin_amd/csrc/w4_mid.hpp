// w4_mid.hpp -- 4-bit weight products for 17 to 64 tokens, and for more where
// the matrix is too small for the GEMM's tiles (blocks of 64 tokens): the
// linear layer and the gated feed-forward front.
//
// Bound: the weights' stream from HBM, the activations' from L2 (every
// workgroup reads all of x, M K 2 bytes), and the vector unit's dequantisation
// come out within a factor of two of each other; so a workgroup owns 32 to 128
// weight rows (gated: half of them gate, half up) for all tokens, the x of a
// step is shared in LDS, and a weight is dequantised once for 64 tokens.
//
// A step is 256 K: codes of BN rows (one 128-byte line each) and x of BM tokens
// go straight to LDS (global_load_lds, XOR-swizzled slots), STAGES - 1 steps
// ahead.  The 8 waves split the step's K: wave w multiplies elements 32w..32w+31
// of all rows and tokens on v_mfma_f32_32x32x16 - its 32 codes of a row are
// 16 bytes, of which lane half h takes dwords 2h and 2h + 1, one for each of
// two matrix instructions, and x is read in the same order.  Codes are
// dequantised in registers on the way, rounded once to the 16-bit type.  The
// waves' sums are added in wave order through the first stage's LDS at the
// end, 16 or 8 tokens at a time.
//
// Measured (weights cold): 48 tokens, 4096 x 4096 14.0 us, 8192 x 8192 29.5,
// 2 x 2051 x 7168 gated 21.2; 64 tokens, 17408 x 5120 36.9 us (the vector unit
// busy for 14 of them, the matrix cores for 5); 509 tokens, 4096 x 7168 57 us.
// With few rows half the compute units are idle, and a step takes what its
// token rows take to arrive: 0.36 us with 32 of them, 0.5 with 48, 0.6 with 64.
#pragma once
#include "w4_device.hpp"
#include "w4_launch.hpp"
#include "w4_plan.hpp"

namespace qlin {

struct W4MidParams {
    const uint16_t* x; int64_t ldx; int M;
    W4Weight w; int64_t I;            // I > 0: gated, rows n and I + n, columns C = I
    int64_t C;
    const uint16_t* bias; uint16_t* y; int64_t ldy;
    uint16_t* gu; int64_t ldgu; const uint16_t* dy; int64_t lddy; int act;
    int groups;                       // K / group
    uint32_t ratio_magic;             // 32-K chunks per group r: chunk / r = mulhi(chunk, magic), 0: r = 1
};

template <int T, int XR, int NTL, int STAGES>  // XR: token rows staged, 32, 48 or 64; 2 <= STAGES <= 4
__global__ __launch_bounds__(512) void w4_mid_kernel(const W4MidParams p) {
    constexpr int MT = (XR + 31) / 32, BM = 32 * MT, BN = 32 * NTL, NW = 8, NT = 512, STEP = kW4MidStep;
    constexpr int XI = XR / 2 / NW;                   // x loads of a wave and step: 2 rows of 512 bytes each
    constexpr int WL = BN / 8;                        // code loads of a step: 8 rows of 128 bytes each
    constexpr int WI = (WL + NW - 1) / NW;            // of a wave; the last only of waves below WL % NW
    constexpr int ST = w4_mid_stage(XR, NTL);
    extern __shared__ __align__(16) uint8_t w4m_lds[];  // scales
    __shared__ __align__(16) uint8_t st0[ST], st1[ST], st2[STAGES > 2 ? ST : 16], st3[STAGES > 3 ? ST : 16];
    constexpr int RT = w4_mid_parts(NTL);
    static_assert(NW * RT * BN * 4 <= ST, "the sums fit a stage");
    float* red = (float*)st0;                           // after the last step: [wave][token % RT][row]

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, G = p.groups;
    const int64_t m0 = (int64_t)blockIdx.y * BM;
    const int M = p.M - m0 < BM ? (int)(p.M - m0) : BM;  // tokens of this workgroup
    const int K = (int)p.w.K, steps = (K + STEP - 1) / STEP;
    const bool glu = p.I > 0;
    const int CT = glu ? BN / 2 : BN;                 // columns of a workgroup
    const int64_t c0 = (int64_t)blockIdx.x * CT;
    const int CL = p.C - c0 < CT ? (int)(p.C - c0) : CT;
    // local row lr of the workgroup: column and matrix row (gated: gate rows, then up rows)
    auto row_of = [&](int lr) {
        const int c = glu && lr >= CT ? lr - CT : lr;
        return c0 + (c < CL ? c : CL - 1) + (glu && lr >= CT ? p.I : 0);  // rows past the end: not stored
    };

    // ---- scales: 16-byte lines that hold the rows' contiguous blocks (at most 15 bytes more at each end)
    const bool has_z = p.w.wz != nullptr;
    uint32_t sat[2], zat[2];  // LDS offsets of the gate and the up block (plain: the first)
    {
        auto stage = [&](const void* src, uint32_t at, uint32_t bytes) {
            for (uint32_t o = 0; o < bytes; o += NT * 16)
                if (o + tid * 16 < bytes)
                    __builtin_amdgcn_global_load_lds((const void*)((const uint8_t*)src + o + tid * 16),
                                                     (lds_void_t*)(w4m_lds + at + o + wv * 1024), 16, 0, 0);
        };
        uint32_t at = 0;
        const uint32_t count = (uint32_t)CL * G;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            if (part == 1 && !glu) break;
            const int64_t first = (c0 + (part ? p.I : 0)) * G;
            const uintptr_t sa = (uintptr_t)(p.w.ws + first);
            const uint32_t sm = (uint32_t)(sa & 15), sbytes = (sm + count * 2 + 15) / 16 * 16;
            stage((const void*)(sa - sm), at, sbytes);
            sat[part] = at + sm;
            at += sbytes;
            zat[part] = sat[part];
            if (has_z) {
                const uintptr_t za = (uintptr_t)(p.w.wz + first);
                const uint32_t zm = (uint32_t)(za & 15), zbytes = (zm + count + 15) / 16 * 16;
                stage((const void*)(za - zm), at, zbytes);
                zat[part] = at + zm;
                at += zbytes;
            }
        }
    }

    // ---- this lane's sources: slot s of an LDS row holds 16-byte chunk s ^ row (mod the row's chunks)
    const uint16_t* xsrc[XI];
    int xk[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int r = (wv * XI + i) * 2 + (lane >> 5);
        xk[i] = ((lane & 31) ^ (r & 31)) * 8;
        xsrc[i] = p.x + (m0 + (r < M ? r : M - 1)) * p.ldx + xk[i];
    }
    const uint8_t* wsrc[WI];
    int wk[WI];
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int r = (i * NW + wv) * 8 + (lane >> 3);
        wk[i] = ((lane & 7) ^ (r & 7)) * 32;
        wsrc[i] = p.w.w + row_of(r < BN ? r : 0) * p.w.ldw + wk[i] / 2;
    }
    const bool full = WL % NW == 0 || wv < WL % NW;  // this wave has WI code loads, not WI - 1
    auto issue = [&](int s, uint8_t* base) {
        const int k0 = s * STEP;
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const void* src = k0 + xk[i] < K ? (const void*)(xsrc[i] + k0) : (const void*)&kW4Zero16;
            __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(base + (wv * XI + i) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < WI; ++i) {  // past K: zero codes, and x is zero there
            const void* src = k0 + wk[i] < K ? (const void*)(wsrc[i] + k0 / 2) : (const void*)&kW4Zero16;
            uint8_t* dst = base + XR * STEP * 2 + (i * NW + wv) * 1024;
            if (i + 1 < WI || full) __builtin_amdgcn_global_load_lds(src, (lds_void_t*)dst, 16, 0, 0);
        }
    };

    const int row = lane & 31, half = lane >> 5;
    int lrow[NTL];
    uint32_t sbase[NTL], zbase[NTL];  // of this lane's row of each tile
#pragma unroll
    for (int t = 0; t < NTL; ++t) {
        const int lr = t * 32 + row, up = glu && lr >= CT, c = up ? lr - CT : lr;
        lrow[t] = lr;
        const int at = (c < CL ? c : CL - 1) * G;
        sbase[t] = (up ? sat[1] : sat[0]) + at * 2;
        zbase[t] = (up ? zat[1] : zat[0]) + at;
    }
    f32x16v_t acc[MT][NTL];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NTL; ++t) acc[m][t] = f32x16v_t{};

    struct Operands { u32x4_t a[MT][2]; uint2 q[NTL]; uint32_t s[NTL], z[NTL]; };
    Operands now;
    auto multiply = [&]() {
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
            W4Scale<T> sc;
            sc.set(now.s[t], has_z ? now.z[t] : 8u);
            const u32x4_t b0 = sc.weights8(now.q[t].x), b1 = sc.weights8(now.q[t].y);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                acc[m][t] = mfma32<T>(now.a[m][0], b0, acc[m][t]);
                acc[m][t] = mfma32<T>(now.a[m][1], b1, acc[m][t]);
            }
        }
    };

    // step s on stage `xt`: its operands are read while those of step s - 1 are multiplied, where registers hold both
    // (48 tokens, 8192 x 8192, two row tiles: 29.6 and 27.3 us), and the stage that step s - 1 used is filled again
    constexpr bool kAhead = NTL <= 2;
    auto step = [&](int s, const uint8_t* xt, uint8_t* refill) {
        // this wave's loads of step s have arrived once at most those of the next STAGES - 2 steps are left
        if (s + STAGES - 2 < steps) {
            if (full) w4_wait_vmcnt<(STAGES - 2) * (XI + WI)>();
            else w4_wait_vmcnt<(STAGES - 2) * (XI + WI - 1)>();
        } else {
            w4_wait_vmcnt<0>();
        }
        w4_lds_barrier();  // step s is complete for everyone, and everyone is done with step s - 1
        const uint8_t* wt = xt + XR * STEP * 2;
        uint32_t g = (uint32_t)(s * (STEP / 32) + wv);
        if (p.ratio_magic) g = __umulhi(g, p.ratio_magic);
        if ((int)g >= G) g = G - 1;  // past K
        Operands next;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const int r = m * 32 + row < XR ? m * 32 + row : XR - 1;  // past the staged rows: not stored
                next.a[m][ks] = *(const u32x4_t*)(xt + r * (STEP * 2) + (((wv * 4 + 2 * half + ks) ^ (r & 31)) * 16));
            }
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
            const int lr = lrow[t];
            next.q[t] = *(const uint2*)(wt + lr * (STEP / 2) + ((wv ^ (lr & 7)) * 16) + half * 8);
            next.s[t] = *(const uint16_t*)(w4m_lds + sbase[t] + g * 2);
            next.z[t] = w4m_lds[zbase[t] + g];
        }
        if (s + STAGES - 1 < steps) issue(s + STAGES - 1, refill);
        if (kAhead && s > 0) multiply();
        now = next;
        if (!kAhead) multiply();
    };
    uint8_t* const ring[4] = {st0, st1, st2, st3};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < steps) issue(s, ring[s]);
    for (int s = 0; s < steps; s += STAGES) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            if (s + i < steps) step(s + i, ring[i], ring[(i + STAGES - 1) % STAGES]);
    }

    // ---- sums of the waves, in order, RT tokens at a time: register e of a tile is token 8(e/4) + 4*half + e%4
    if (kAhead) multiply();
    w4_lds_barrier();  // everyone is done with the stages; no load into them is left
#pragma unroll
    for (int part = 0; part < BM / RT; ++part) {
        if (part * RT >= M) break;  // workgroup-uniform
        if (part > 0) w4_lds_barrier();
        constexpr int PT = 32 / RT;  // parts of a tile
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int e = 0; e < RT / 2; ++e) {
                const int tok = 8 * (e >> 2) + 4 * half + (e & 3);
                red[(wv * RT + tok) * BN + t * 32 + row] = acc[part / PT][t][(part % PT) * (RT / 2) + e];
            }
        w4_lds_barrier();
        auto total = [&](int m, int lr) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) v += red[(k * RT + m) * BN + lr];
            return v;
        };
        for (int o = tid; o < RT * CT; o += NT) {
            const int mm = glu ? o / (BN / 2) : o / BN, j = o - mm * CT;
            const int64_t m = m0 + part * RT + mm, c = c0 + j;
            if (j >= CL || part * RT + mm >= M) continue;
            float v = total(mm, j);
            if (glu) {
                const float v2 = total(mm, CT + j);
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
}

}  // namespace qlin
