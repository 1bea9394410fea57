// i8ffn.hip -- the INT8 feed-forward operators: row quantiser, routing, pair
// sort and combine kernels, and the launchers of the gated front
// (qlin_glu_i8) and the routed expert layer (qlin_moe_ffn_i8).
#include "i8ffn_few_launch.hpp"
#include "i8ffn_gemm.hpp"
#include "i8ffn_launch.hpp"
#include "i8ffn_plan.hpp"

namespace qlin {

namespace {

// One workgroup per row: largest magnitude, then codes (i8ffn_device.hpp).
// ids, if given: a row whose id is outside [0, E) is not read or written.
constexpr int kI8QuantThreads = 512;

template <int T>
__global__ __launch_bounds__(kI8QuantThreads) void i8_quant_kernel(const uint16_t* x, int64_t ldx, int64_t K, int8_t* xq,
                                                                   int64_t ldxq, float* xs, const int32_t* ids, int E) {
    const int64_t m = blockIdx.x;
    if (ids && (uint32_t)ids[m] >= (uint32_t)E) return;  // workgroup-uniform
    quantise_row_wg<T, kI8QuantThreads>(x + m * ldx, K, xq + m * ldxq, xs + m);
}

hipError_t quantise(int dtype, const uint16_t* x, int64_t ldx, int64_t rows, int64_t K, int8_t* xq, int64_t ldxq, float* xs,
                    const int32_t* ids, int64_t E, hipStream_t st) {
    auto k = dtype == kFp16 ? i8_quant_kernel<kFp16> : i8_quant_kernel<kBf16>;
    hipLaunchKernelGGL(k, dim3((unsigned)rows), dim3(kI8QuantThreads), 0, st, x, ldx, K, xq, ldxq, xs, ids, (int)E);
    return hipGetLastError();
}

// A workgroup a token: 8 waves quantise it, a ninth routes it (NR > 0).
struct I8TokenParams {
    const uint16_t* x; int64_t ldx; int64_t K; int8_t* xq; float* xs;
    const float* logits; int64_t ldl; int E, topk, route; int32_t* ids; float* gw;
};

template <int T, int NR>
__global__ __launch_bounds__(kI8QuantThreads + (NR > 0 ? 64 : 0)) void i8_token_kernel(const I8TokenParams p) {
    const int64_t m = blockIdx.x;
    if constexpr (NR > 0) {
        if (threadIdx.x >= kI8QuantThreads) {
            const int lane = threadIdx.x & 63;
            int id;
            float w;
            route_token<NR>(p.logits + m * p.ldl, p.E, p.topk, p.route, lane, id, w);
            if (lane < p.topk) {
                p.ids[m * p.topk + lane] = id;
                p.gw[m * p.topk + lane] = w;
            }
        }
    }
    quantise_row_wg<T, kI8QuantThreads>(p.x + m * p.ldx, p.K, p.xq + m * p.K, p.xs + m);
}

// Pairs by expert (perm), and the row tiles of bm pairs that they make, each
// with its expert.  One workgroup, LDS counters: the order of an
// expert's pairs is arbitrary, which no result depends on (every pair's row is
// computed on its own, the combine adds in slot order).  A thread's ids are
// loaded together, eight at a time, and kept where they are no more.
constexpr int kI8MaxE = 1024;

__global__ __launch_bounds__(1024) void i8_sort_kernel(const int32_t* ids, int P, int E, int bm, I8Tile* tiles,
                                                       int32_t* ntiles, int32_t* perm) {
    __shared__ int32_t cnt[kI8MaxE], cur[kI8MaxE], wsum[16], wtile[16];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int32_t id[8];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = base + i * 1024 + tid;
            const int32_t e = ids[p < P ? p : P - 1];
            id[i] = p < P && (uint32_t)e < (uint32_t)E ? e : -1;
        }
    };
    load(0);
    cnt[tid] = 0;
    __syncthreads();
    for (int base = 0;;) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (id[i] >= 0) atomicAdd(&cnt[id[i]], 1);
        base += 8192;
        if (base >= P) break;
        load(base);
    }
    __syncthreads();
    const int c = cnt[tid], t = (c + bm - 1) / bm;
    int ci = c, ti = t;  // inclusive sums
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const int a = __shfl_up(ci, s), b = __shfl_up(ti, s);
        if (lane >= s) {
            ci += a;
            ti += b;
        }
    }
    if (lane == 63) {
        wsum[wv] = ci;
        wtile[wv] = ti;
    }
    __syncthreads();
    for (int q = 0; q < wv; ++q) {
        ci += wsum[q];
        ti += wtile[q];
    }
    cur[tid] = ci - c;
    for (int k = 0; k < t; ++k) tiles[ti - t + k] = I8Tile{tid, ti - t, ci - c, c};
    if (tid == kI8MaxE - 1) *ntiles = ti;  // experts past E count nothing
    __syncthreads();
    for (int base = 0; base < P; base += 8192) {
        if (P > 8192) load(base);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (id[i] >= 0) perm[atomicAdd(&cur[id[i]], 1)] = base + i * 1024 + tid;
    }
}

// y[t,n] = r16(sum_j gw[t,j] part[t,j,n]) in slot order, four columns a thread.
template <int T>
__global__ __launch_bounds__(256) void i8_combine_kernel(const float* part, const int32_t* ids, const float* gw, int64_t M,
                                                         int topk, int E, int64_t N, uint16_t* y, int64_t ldy) {
    const int64_t nv = N / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // N % 16 == 0
    if (i >= M * nv) return;
    const int64_t t = i / nv, n = (i - t * nv) * 4;
    f32x4v_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < topk; ++j) {
        const int64_t p = t * topk + j;
        if ((uint32_t)ids[p] >= (uint32_t)E) continue;
        const f32x4v_t v = __builtin_nontemporal_load((const f32x4v_t*)(part + p * N + n));
        const float g = gw[p];
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] = fmaf(g, v[c], sum[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) y[t * ldy + n + c] = f32_to_h<T>(sum[c]);
}

// columns [first, first + count) of the product with row_tiles tiles of BM rows (at most, where they are grouped)
template <int T, int EPI, int BN, int BM, int WGN, int WGM, int D = 2>  // D: i8ffn_gemm.hpp
hipError_t run_gemm(I8GemmParams p, int64_t row_tiles, int64_t first, int64_t count, hipStream_t st) {
    constexpr int CT = EPI == kI8Gated ? BN / 2 : BN;
    p.c_first = first;
    p.c_count = count;
    const int64_t tiles = row_tiles * ((count + CT - 1) / CT);
    hipLaunchKernelGGL((i8_gemm_kernel<T, EPI, BN, BM, WGN, WGM, D>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(64 * WGN * WGM), 0, st, p);
    return hipGetLastError();
}

// row tiles that P pairs of E groups can make at most
int64_t most_tiles(int64_t P, int64_t E, int64_t bm) { return P / bm + (E < P ? E : P); }

struct MoeRegions { size_t xq, xs, h, hq, hs, part, tiles, ntiles, perm, list, total; };

MoeRegions regions(int64_t M, int64_t H, int64_t I, int64_t topk, int64_t E) {
    MoeRegions r{};
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += ((size_t)bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t P = M * topk;
    r.xq = take(M * H);
    r.xs = take(M * 4);
    r.h = take(P * I * 2);
    r.hq = take(P * I);
    r.hs = take(P * 4);
    r.part = take(P * H * 4);
    r.tiles = take(most_tiles(P, E, 32) * (int64_t)sizeof(I8Tile));
    r.ntiles = take(4);
    r.perm = take(P * 4);
    r.list = take((int64_t)few_list_bytes());
    r.total = at;
    return r;
}

template <int T>
hipError_t moe(const I8MoeArgs& a, hipStream_t st) {
    const MoeRegions r = regions(a.M, a.H, a.I, a.topk, a.E);
    const int64_t P = a.M * a.topk;
    uint8_t* ws = a.workspace;
    int8_t *xq = (int8_t*)(ws + r.xq), *hq = (int8_t*)(ws + r.hq);
    float *xs = (float*)(ws + r.xs), *hs = (float*)(ws + r.hs), *part = (float*)(ws + r.part);
    uint16_t* h = (uint16_t*)(ws + r.h);
    I8Tile* tiles = (I8Tile*)(ws + r.tiles);
    int32_t *ntiles = (int32_t*)(ws + r.ntiles), *perm = (int32_t*)(ws + r.perm);
    if (few_fits(a.M, a.H)) {
        const I8FewRegions f{xq, xs, h, hq, hs, ws + r.list};
        return T == kFp16 ? few_moe_fp16(a, f, st) : few_moe_bf16(a, f, st);
    }
    const int bm = (int)i8_tile_rows(P, a.E);
    const I8TokenParams q{a.x, a.ldx, a.H, xq, xs, a.logits, a.ldl, (int)a.E, (int)a.topk, a.route, a.ids, a.gw};
    auto token = !a.logits ? i8_token_kernel<T, 0>
                           : (a.E <= 64 ? i8_token_kernel<T, 1>
                                        : (a.E <= 128 ? i8_token_kernel<T, 2>
                                                      : (a.E <= 256 ? i8_token_kernel<T, 4> : i8_token_kernel<T, 16>)));
    hipLaunchKernelGGL(token, dim3((unsigned)a.M), dim3(kI8QuantThreads + (a.logits ? 64 : 0)), 0, st, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(i8_sort_kernel, dim3(1), dim3(1024), 0, st, a.ids, (int)P, (int)a.E, bm, tiles, ntiles, perm);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    I8GemmParams g{};
    g.x = xq; g.ldx = a.H; g.xs = xs; g.tiles = tiles; g.ntiles = ntiles; g.perm = perm; g.div = (int)a.topk;
    g.K = a.H; g.w = a.w13; g.ldw = a.ldw13; g.N = 2 * a.I; g.ws = a.s13; g.ws_step = 1; g.C = a.I; g.act = a.act;
    g.y = h; g.ldy = a.I;
    const int64_t most = most_tiles(P, a.E, bm);
    e = bm == 32   ? run_gemm<T, kI8Gated, 128, 32, 2, 1>(g, most, 0, a.I, st)
        : bm == 64 ? run_gemm<T, kI8Gated, 128, 64, 2, 2>(g, most, 0, a.I, st)
                   : run_gemm<T, kI8Gated, 128, 128, 2, 4>(g, most, 0, a.I, st);
    if (e != hipSuccess) return e;
    e = quantise(T, h, a.I, P, a.I, hq, a.I, hs, a.ids, a.E, st);
    if (e != hipSuccess) return e;
    g.x = hq; g.ldx = a.I; g.xs = hs; g.div = 1; g.K = a.I; g.w = a.w2; g.ldw = a.ldw2; g.N = a.H; g.ws = a.s2;
    g.C = a.H; g.y = nullptr; g.part = part; g.ldy = a.H;
    e = bm == 32   ? run_gemm<T, kI8Part, 128, 32, 4, 1>(g, most, 0, a.H, st)
        : bm == 64 ? run_gemm<T, kI8Part, 128, 64, 4, 2>(g, most, 0, a.H, st)
                   : run_gemm<T, kI8Part, 128, 128, 2, 4>(g, most, 0, a.H, st);
    if (e != hipSuccess) return e;
    const int64_t n = a.M * (a.H / 4);
    hipLaunchKernelGGL(i8_combine_kernel<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, part, a.ids, a.gw, a.M,
                       (int)a.topk, (int)a.E, a.H, a.y, a.ldy);
    return hipGetLastError();
}

template <int T>
hipError_t glu(const I8GluArgs& a, hipStream_t st) {
    if (few_fits(a.M, a.K)) return T == kFp16 ? few_glu_fp16(a, st) : few_glu_bf16(a, st);
    const hipError_t e = quantise(T, a.x, a.ldx, a.M, a.K, a.xq, a.ldxq, a.xs, nullptr, 0, st);
    if (e != hipSuccess) return e;
    I8GemmParams g{};
    g.x = a.xq; g.ldx = a.ldxq; g.xs = a.xs; g.R = a.M; g.div = 1;
    g.K = a.K; g.w = a.w13; g.ldw = a.ldw; g.N = 2 * a.I; g.ws = a.s13; g.ws_step = a.ws_step; g.C = a.I; g.act = a.act;
    g.y = a.y; g.ldy = a.ldy;
    const int64_t large = i8_large_columns(a.M, a.I), rest = a.I - large;
    if (large > 0) {
        const hipError_t l = run_gemm<T, kI8Gated, 256, 256, 4, 4>(g, (a.M + 255) / 256, 0, large, st);
        if (l != hipSuccess || rest == 0) return l;
    }
    switch (i8_dense_tile(a.M, rest)) {
        case kI8Tile64x64: return run_gemm<T, kI8Gated, 64, 64, 1, 2, 4>(g, (a.M + 63) / 64, large, rest, st);
        case kI8Tile64x128: return run_gemm<T, kI8Gated, 128, 64, 2, 2, 4>(g, (a.M + 63) / 64, large, rest, st);
        case kI8TwoOf128x128: return run_gemm<T, kI8Gated, 128, 128, 2, 4>(g, (a.M + 127) / 128, large, rest, st);
        default: return run_gemm<T, kI8Gated, 128, 128, 2, 4, 4>(g, (a.M + 127) / 128, large, rest, st);
    }
}

}  // namespace

size_t moe_ffn_i8_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk, int64_t E) {
    return regions(M, H, I, topk, E).total;
}

hipError_t launch_glu_i8(const I8GluArgs& a, hipStream_t st) {
    return a.dtype == kFp16 ? glu<kFp16>(a, st) : glu<kBf16>(a, st);
}

hipError_t launch_moe_ffn_i8(const I8MoeArgs& a, hipStream_t st) {
    return a.dtype == kFp16 ? moe<kFp16>(a, st) : moe<kBf16>(a, st);
}

}  // namespace qlin
