// i8_device.h -- device-side pieces shared by the kernels of the 8-bit products
// with token and channel scales: the row rule, the rescale of an int32 sum and
// the store in the output's type.  Every kernel uses these, so an output's bits
// do not depend on which kernel computed its sum.
#pragma once

#include "q8_device.h"
#include "q8moe.h"

namespace q8 {

// Values of the three float types, as fp32 (exact).
template <int T> struct Elem;
template <> struct Elem<Q8_T_F32> { typedef float type; };
template <> struct Elem<Q8_T_F16> { typedef _Float16 type; };
template <> struct Elem<Q8_T_BF16> { typedef __bf16 type; };

// 4 (fp32) or 8 (16-bit types) consecutive values: one 16-byte load.
template <int T> constexpr int kVec = T == Q8_T_F32 ? 4 : 8;

template <int T>
__device__ __forceinline__ void unpack16(u32x4 r, float (&v)[kVec<T>])
{
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};   // (a bit cast of r.y itself reads element 0)
    if constexpr (T == Q8_T_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(float, d[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == Q8_T_F16) {
                v[2 * i] = half_bits_to_float(d[i]);
                v[2 * i + 1] = half_bits_to_float(d[i] >> 16);
            } else {
                v[2 * i] = __builtin_bit_cast(float, d[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, d[i] & 0xffff0000u);
            }
        }
    }
}

// |v| as ordered bits: finite < infinity (0x7f800000) < NaN.
__device__ __forceinline__ uint32_t abs_bits(float v)
{
    return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// The scale of a row from the largest abs_bits of its values.
__device__ __forceinline__ float row_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return __builtin_nanf("");
    return __builtin_bit_cast(float, amax_bits) / 127.0f;
}

// Codes of a row with scale s, as the exact quotient x / s decides them.  With
// a = |x| * (1/s), at most 2e-5 off the quotient v (v <= 127, two roundings),
// q = floor(a + 0.4999) is floor(v + 0.5) or one less; which, is the sign of
// |x| - (q + 0.5) * s, and a fused multiply-add rounds that difference once,
// which keeps its sign.  (5 operations against about 10 of an IEEE division,
// whose rounded quotient would also move exact ties.)  A scale below 2^-60 is
// lifted with the values by 2^64, so that neither 1/s overflows nor the
// difference underflows.
struct RowCoder {
    float s, inv, lift;
    uint32_t live;                                      // all ones, or 0: zero codes
    __device__ __forceinline__ explicit RowCoder(float scale)
    {
        live = scale > 0.0f ? ~0u : 0u;                 // 0 for s = 0 and NaN
        lift = live && scale < 0x1p-60f ? 0x1p64f : 1.0f;
        s = live ? scale * lift : 1.0f;
        inv = 1.0f / s;
    }
    __device__ __forceinline__ uint32_t code(float x) const
    {
        const float ax = fabsf(x) * lift;
        const float q = floorf(fmaf(ax, inv, 0.4999f));
        float c = fmaf(-(q + 0.5f), s, ax) >= 0.0f ? q + 1.0f : q;
        c = fminf(c, 127.0f);
        return (uint32_t)(int)__builtin_copysignf(c, x) & 255u;
    }
    __device__ __forceinline__ uint32_t code4(const float *v) const
    {
        return (code(v[0]) | code(v[1]) << 8 | code(v[2]) << 16 | code(v[3]) << 24) & live;
    }
};

// The fp32 value of an int32 sum: two products, or a product and a fused
// multiply-add with the bias (spelled out: one rounding order in every kernel).
__device__ __forceinline__ float i8_rescale(int sum, float sx, float sw)
{
    return ((float)sum * sx) * sw;
}

__device__ __forceinline__ float i8_rescale(int sum, float sx, float sw, float bias)
{
    return fmaf((float)sum * sx, sw, bias);
}

// silu(g) * u = g / (1 + exp(-g)) * u.  exp(-g) as 2^t with t = -g*log2(e) and
// the rounding error r of t put back as a factor 1 + r*ln 2 (t alone would cost
// |t| * 2^-24 relative); the clamp keeps infinities of g from making NaN there.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float c = fminf(fmaxf(-g, -104.0f), 104.0f);
    constexpr float kL2E = 1.44269504088896341f, kL2ELo = 1.925963033500e-8f;
    const float t = c * kL2E;
    const float r = fmaf(c, kL2E, -t) + c * kL2ELo;
    const float e0 = __builtin_amdgcn_exp2f(t);
    const float e = fmaf(e0, r * 0.693147180559945f, e0);
    const float d = 1.0f + (e0 < 3.0e38f ? e : e0);
    return g * __builtin_amdgcn_rcpf(d) * u;
}

// A value rounded to nearest even to the output's type.  (It is pinned as fp32
// first: a last product merged with the conversion, as v_fma_mixlo_f16 does,
// would round once where another kernel rounds twice.)
template <int T>
__device__ __forceinline__ typename Elem<T>::type round_out(float v)
{
    if constexpr (T == Q8_T_F16) asm("" : "+v"(v));
    return (typename Elem<T>::type)v;
}

template <int T>
__device__ __forceinline__ void store_out(void *y, int64_t i, float v)
{
    ((typename Elem<T>::type *)y)[i] = round_out<T>(v);
}

// Two values of a 16-bit type in a dword (one instruction for both).
template <int T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    if constexpr (T == Q8_T_BF16) {
        typedef __bf16 e2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(((f2){lo, hi}), e2));
    } else if constexpr (T == Q8_T_F16) {
        typedef _Float16 e2 __attribute__((ext_vector_type(2)));
        asm("" : "+v"(lo), "+v"(hi));              // (as in round_out)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(((f2){lo, hi}), e2));
    } else
        return 0;
}

// 16 bytes of outputs, the first `left` elements of them (element alignment is
// enough); STREAM: past the caches.
template <int T, bool STREAM>
__device__ __forceinline__ void store16(uint8_t *y, u32x4 v, int left)
{
    typedef u32x4 __attribute__((aligned(2))) u32x4_any;
    constexpr int V = kVec<T>;
    if (left >= V) {
        if constexpr (STREAM)
            __builtin_nontemporal_store((u32x4_any)v, (u32x4_any *)y);
        else
            *(u32x4_any *)y = v;
        return;
    }
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int r = 0; r < V - 1; ++r)
        if (r < left) {
            if constexpr (T == Q8_T_F32)
                ((uint32_t *)y)[r] = d[r];
            else
                ((uint16_t *)y)[r] = (uint16_t)(d[r / 2] >> (16 * (r & 1)));
        }
}

// Up to 4 consecutive values.
template <int T>
__device__ __forceinline__ void store_run(void *y, int64_t i, const float (&v)[4], int left)
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (r < left) store_out<T>(y, i + r, v[r]);
}

}  // namespace q8
