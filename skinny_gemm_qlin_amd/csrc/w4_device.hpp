// w4_device.hpp -- number formats and epilogues of the 4-bit weight kernels.
//
// A weight is W[n,k] = ws[n,g] * (code[n,k] - wz[n,g]), g = k / group: codes
// 0..15 two a byte (element 2i in the low nibble of byte i), ws in the
// activations' 16-bit type, wz a byte 0..15 or the constant 8.
//
// Unpacking.  The byte 0x0n read as an E4M3 code is n * 2^-9: codes 0..7 are
// E4M3's subnormals and 8..15 its first binade, which continues them
// linearly.  v_cvt_scalef32_pk_{bf16,f16}_fp8 with scale 2^9 therefore turns
// two masked bytes into the two whole numbers in one instruction, exactly, and
// no magic-number offset has to be taken out of the sum afterwards.
#pragma once
#include "qlin_device.hpp"

namespace qlin {

constexpr int kBf16 = 0;  // values of the C ABI's dtype argument
constexpr int kFp16 = 1;
constexpr int kActSilu = 0;  // values of the C ABI's act argument
constexpr int kActGeluTanh = 1;

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v_t __attribute__((ext_vector_type(8)));
typedef float f32x2v_t __attribute__((ext_vector_type(2)));
typedef float f32x4v_t __attribute__((ext_vector_type(4)));
typedef float f32x16v_t __attribute__((ext_vector_type(16)));

// 16-bit storage <-> fp32
template <int T>
__device__ __forceinline__ float h_to_f32(uint32_t h) {
    if constexpr (T == kBf16) return bf16_to_f32(h);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

template <int T>
__device__ __forceinline__ uint16_t f32_to_h(float f) {  // nearest, ties to even
    if constexpr (T == kBf16) return f32_to_bf16(f);
    else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// two masked code bytes (HI: bytes 2 and 3 of d, else 0 and 1) -> two 16-bit whole numbers, exact
template <int T, bool HI>
__device__ __forceinline__ uint32_t codes2(uint32_t d) {
    if constexpr (T == kBf16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 512.0f, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d, 512.0f, HI));
}

// Eight codes (one dword) -> eight weights in element order, each rounded once
// to the 16-bit type.  bf16: (code - zero) * s in fp32 is exact (at most 5 + 8
// significant bits) and v_cvt_pk_bf16_f32 rounds it.  fp16: code - zero is a
// whole number, exact, and one packed multiplication by s rounds.
template <int T>
struct W4Scale;

template <>
struct W4Scale<kBf16> {
    float s, c;  // scale, -zero * scale
    __device__ __forceinline__ void set(uint32_t h, uint32_t z) {
        s = bf16_to_f32(h);
        c = -(float)z * s;
    }
    __device__ __forceinline__ u32x4_t weights8(uint32_t d) const {
        const uint32_t e = d & 0x0F0F0F0Fu, o = (d >> 4) & 0x0F0F0F0Fu;
        u32x4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2v_t v = {fmaf((float)((e >> (8 * i)) & 0xFFu), s, c), fmaf((float)((o >> (8 * i)) & 0xFFu), s, c)};
            r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
        }
        return r;
    }
};

template <>
struct W4Scale<kFp16> {
    f16x2_t s, z;
    __device__ __forceinline__ void set(uint32_t h, uint32_t zero) {
        const _Float16 sv = __builtin_bit_cast(_Float16, (uint16_t)h), zv = (_Float16)(float)zero;
        s = f16x2_t{sv, sv};
        z = f16x2_t{zv, zv};
    }
    __device__ __forceinline__ u32x4_t weights8(uint32_t d) const {
        const uint32_t e = d & 0x0F0F0F0Fu, o = (d >> 4) & 0x0F0F0F0Fu;
        // v_perm_b32: bytes e0 o0 e1 o1 / e2 o2 e3 o3 put the codes back in element order
        const uint32_t lo = __builtin_amdgcn_perm(o, e, 0x05010400u), hi = __builtin_amdgcn_perm(o, e, 0x07030602u);
        const uint32_t q[4] = {codes2<kFp16, false>(lo), codes2<kFp16, true>(lo), codes2<kFp16, false>(hi),
                               codes2<kFp16, true>(hi)};
        u32x4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = __builtin_bit_cast(uint32_t, (__builtin_bit_cast(f16x2_t, q[i]) - z) * s);
        return r;
    }
};

// 16 zero bytes: the source of direct-to-LDS loads past the end of a row
__device__ const u32x4_t kW4Zero16 = {0u, 0u, 0u, 0u};

// ---------------------------------------------------------------- matrix instructions on 16-bit storage
template <int T>
__device__ __forceinline__ f32x16v_t mfma32(const u32x4_t& a, const u32x4_t& b, const f32x16v_t& c) {
    if constexpr (T == kBf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v_t, a),
                                                       __builtin_bit_cast(bf16x8v_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
}

template <int T>
__device__ __forceinline__ f32x4v_t mfma16(const u32x4_t& a, const u32x4_t& b, const f32x4v_t& c) {
    if constexpr (T == kBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v_t, a),
                                                       __builtin_bit_cast(bf16x8v_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
}

// ---------------------------------------------------------------- operands and exchanges of the decode kernels
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

// ---------------------------------------------------------------- waits
// LDS writes of the workgroup become visible; outstanding global loads stay in flight
__device__ __forceinline__ void w4_lds_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int N_>
__device__ __forceinline__ void w4_wait_vmcnt() {  // s_waitcnt vmcnt(N_), other counters untouched
    static_assert(N_ >= 0 && N_ < 64, "vmcnt field");
    __builtin_amdgcn_s_waitcnt((N_ & 15) | ((N_ >> 4) << 14) | 0x70 | 0xF00);
}

// ---------------------------------------------------------------- gate activations
// p(g) with act(g) = g * p(g), and the derivative act'(g).  Both activations
// are g times a logistic function: silu p = 1/(1+e^-g); gelu in its tanh form
// 0.5 (1 + tanh z) = 1/(1+e^-2z), z = sqrt(2/pi) (g + 0.044715 g^3).  With
// q = 1 - p the derivative is p + g p q dv/dg, v the logistic's argument.
// v_exp_f32 and v_rcp_f32 (1 ulp) are well inside the 16-bit output rounding.
// |g| is cut at 30 for gelu's argument (p and q are 0 or 1 there to every
// digit, and g^3 cannot overflow), by comparisons that leave a NaN one.  Where
// p or q is 0 its product with g is 0 too: g may be infinite there, as a gate
// beyond fp16's range is once it has been kept.
__device__ __forceinline__ void gate_act(float g, int act, float& a, float& da) {
    float v, dv;
    if (act == kActSilu) {
        v = g;
        dv = 1.0f;
    } else {
        const float c = g > 30.0f ? 30.0f : (g < -30.0f ? -30.0f : g), cc = c * c;
        v = 1.5957691216057308f * (c + 0.044715f * c * cc);
        dv = 1.5957691216057308f * (1.0f + 0.134145f * cc);
    }
    const float e = __expf(-fabsf(v));                    // in (0, 1]
    const float r = __builtin_amdgcn_rcpf(1.0f + e);      // the larger of p and q
    const float p = v >= 0.0f ? r : e * r, q = v >= 0.0f ? e * r : r;
    a = p == 0.0f ? -0.0f : g * p;
    da = fmaf(q == 0.0f ? 0.0f : a * q, dv, p);
}

}  // namespace qlin
