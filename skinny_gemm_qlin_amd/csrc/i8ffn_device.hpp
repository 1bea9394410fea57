// i8ffn_device.hpp -- quantisation rule, routing and epilogue arithmetic shared
// by the INT8 feed-forward kernels.
//
// Quantisation of a row (the INT8 rule of qlin_device.hpp, for either 16-bit
// type): s = amax / 127 and q = clamp(rne(x / s)), both quotients IEEE fp32;
// amax = 0 gives s = 0 and codes 0.  The maximum is taken over the magnitude
// bits as whole numbers, which order like the values and put infinities and
// NaNs above every finite one: a row that holds one gets s = NaN and codes 0,
// so all it feeds is NaN and no other row is touched.
#pragma once
#include "w4_device.hpp"

namespace qlin {

// largest 16-bit magnitude (sign cleared) of 8 values, as a whole number; two halves in one register
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    const u16x2_t r = __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b));
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t mag8(const u32x4_t& v, uint32_t m) {
    m = pk_max_u16(m, v.x & 0x7FFF7FFFu);
    m = pk_max_u16(m, v.y & 0x7FFF7FFFu);
    m = pk_max_u16(m, v.z & 0x7FFF7FFFu);
    return pk_max_u16(m, v.w & 0x7FFF7FFFu);
}

// the larger half of the packed maximum, over the whole wave
__device__ __forceinline__ uint32_t wave_mag(uint32_t m) {
    m = pk_max_u16(m, (uint32_t)dpp_mov<0x128>((int)m));
    m = pk_max_u16(m, (uint32_t)dpp_mov<0x124>((int)m));
    m = pk_max_u16(m, (uint32_t)dpp_mov<0x122>((int)m));
    m = pk_max_u16(m, (uint32_t)dpp_mov<0x121>((int)m));
    uint32_t a = m, b = m;
    swap32(a, b);
    a = b = pk_max_u16(a, b);
    swap16(a, b);
    a = pk_max_u16(a, b);
    const uint32_t lo = a & 0xFFFFu, hi = a >> 16;
    return lo > hi ? lo : hi;
}

// The scale of a row whose largest magnitude has the bits `mag`, and what its codes are made with.
//
// The quotient.  From 2^-100 up: t = x * r with r = fl(1 / s), then one step t + (x - t s) r in fused operations,
// which gives the correctly rounded quotient (the remainder is exact; every mantissa of x against every scale that an
// absolute maximum of the type can give is checked in the CPU tests).  No quotient rounds to more than 127 there.
// Below, where the remainder may be subnormal: through 64 bits, as div_bf16.
struct RowScale {
    float s, r;
    double rd;
    bool fine;  // the first way
};

template <int T>
__device__ __forceinline__ RowScale row_scale(uint32_t mag) {
    const uint32_t inf = T == kBf16 ? 0x7F80u : 0x7C00u;
    RowScale o;
    o.s = mag >= inf ? __uint_as_float(0x7FC00000u) : h_to_f32<T>(mag) / 127.0f;
    o.fine = o.s >= 0x1p-100f;
    o.r = o.fine ? 1.0f / o.s : 0.0f;
    o.rd = 0.0;
    if (!o.fine && mag != 0 && mag < inf) o.rd = 1.0 / (double)o.s;  // else the codes are 0
    return o;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {  // low bytes
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x04000C0Cu);
    return lo | hi;
}

// 8 values -> 8 codes
template <int T>
__device__ __forceinline__ uint2 codes8(const u32x4_t& v, const RowScale& o) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
    int q[8];
    if (o.fine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = h_to_f32<T>((e & 1) ? (d[e >> 1] >> 16) : (d[e >> 1] & 0xFFFFu));
            const float t = x * o.r;
            q[e] = (int)rintf(fmaf(fmaf(-t, o.s, x), o.r, t));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = h_to_f32<T>((e & 1) ? (d[e >> 1] >> 16) : (d[e >> 1] & 0xFFFFu));
            const float t = fminf(fmaxf(rintf(div_bf16(x, o.rd)), -127.0f), 127.0f);
            q[e] = o.rd == 0.0 ? 0 : (int)t;
        }
    }
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

// The first NT threads of a workgroup quantise a row: largest magnitude, then codes.  All threads call it (a barrier).
template <int T, int NT>
__device__ __forceinline__ void quantise_row_wg(const uint16_t* row, int64_t K, int8_t* out, float* scale) {
    constexpr int W = NT / 64, CACHED = 2;
    __shared__ uint32_t part[W];
    const int tid = threadIdx.x;
    const int64_t nvec = tid < NT ? K >> 3 : 0;
    u32x4_t cache[CACHED];
    uint32_t a = 0;
#pragma unroll
    for (int c = 0; c < CACHED; ++c) {
        const int64_t i = tid + c * NT;
        cache[c] = i < nvec ? ld16(row + i * 8) : u32x4_t{0, 0, 0, 0};
        a = mag8(cache[c], a);
    }
    for (int64_t i = tid + CACHED * NT; i < nvec; i += NT) a = mag8(ld16(row + i * 8), a);
    a = wave_mag(a);
    if ((tid & 63) == 0 && tid < NT) part[tid >> 6] = a;
    __syncthreads();
    uint32_t mag = part[0];
#pragma unroll
    for (int q = 1; q < W; ++q) mag = part[q] > mag ? part[q] : mag;
    const RowScale o = row_scale<T>(mag);
    if (tid == 0) *scale = o.s;
#pragma unroll
    for (int c = 0; c < CACHED; ++c) {
        const int64_t i = tid + c * NT;
        if (i < nvec) *(uint2*)(out + i * 8) = codes8<T>(cache[c], o);
    }
    for (int64_t i = tid + CACHED * NT; i < nvec; i += NT) *(uint2*)(out + i * 8) = codes8<T>(ld16(row + i * 8), o);
}

// act(g) u of the int32 sums of a gate and an up row
__device__ __forceinline__ float gated(int ag, int au, float xs, float sg, float su, int act) {
    float a, da;
    gate_act(((float)ag * xs) * sg, act, a, da);
    return a * (((float)au * xs) * su);
}

// ---------------------------------------------------------------- routing
constexpr int kRouteSelected = 0;  // values of the C ABI's route argument
constexpr int kRouteAll = 1;

// A logit as a whole number of the same order; 0 where the expert is masked (NaN or -inf).  -0 counts as 0.
__device__ __forceinline__ uint32_t route_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    return l > -INFINITY ? ((u >> 31) ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float route_logit(uint32_t key) {
    return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ float route_exp(float l, float top) { return l == top ? 1.0f : expf(l - top); }

__device__ __forceinline__ float wave_sum_f32(float v) {
    const uint32_t r = __float_as_uint(row_sum_f32(v));
    uint32_t a = r, b = r;
    swap32(a, b);
    a = b = __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    swap16(a, b);
    return __uint_as_float(a) + __uint_as_float(b);
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {  // uniform
    v = max_u32(v, (uint32_t)dpp_mov<0x128>((int)v));
    v = max_u32(v, (uint32_t)dpp_mov<0x124>((int)v));
    v = max_u32(v, (uint32_t)dpp_mov<0x122>((int)v));
    v = max_u32(v, (uint32_t)dpp_mov<0x121>((int)v));
    uint32_t a = v, b = v;
    swap32(a, b);
    a = b = max_u32(a, b);
    swap16(a, b);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)max_u32(a, b));
}

// One wave routes one token: its topk largest logits, largest first, equal ones
// to the lower expert.  Lane j < topk returns slot j's expert (-1: every
// expert left is masked) and weight exp(l_j - l_0) / sum, over the selected
// experts or over all.  NR x 64 >= E.
template <int NR>
__device__ __forceinline__ void route_token(const float* row, int E, int topk, int route, int lane, int& id, float& w) {
    uint32_t key[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int e = i * 64 + lane;
        const float l = row[e < E ? e : E - 1];  // no load under a branch: all are on their way at once
        key[i] = e < E ? route_key(l) : 0u;
    }
    uint32_t all[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) all[i] = key[i];
    id = -1;
    uint32_t mine = 0;
    for (int j = 0; j < topk; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < NR; ++i) best = key[i] > best ? key[i] : best;
        const uint32_t top = wave_max_u32(best);
        if (top == 0) break;  // uniform
        int e = -1;  // the first of the equal ones
#pragma unroll
        for (int i = NR - 1; i >= 0; --i) {
            const uint64_t at = __ballot(key[i] == top);
            if (at) e = i * 64 + __builtin_ctzll(at);
        }
        if (lane == j) {
            id = e;
            mine = top;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (e == i * 64 + lane) key[i] = 0;
    }
    const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)mine);
    const float top = route_logit(first);
    const float x = mine ? route_exp(route_logit(mine), top) : 0.0f;
    float part = x;
    if (route == kRouteAll) {
        part = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) part += all[i] ? route_exp(route_logit(all[i]), top) : 0.0f;
    }
    const float sum = wave_sum_f32(part);
    w = mine ? x / sum : 0.0f;
}

}  // namespace qlin
