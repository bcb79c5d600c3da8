// i8_device.h -- device helpers of the int8 kernels (gfx950).
//
// A row's codes are q = 127 x / max|x| rounded to the nearest whole number, halves to even,
// decided as if in exact arithmetic: x = max|x| / 2 is a tie in every row (63.5), so a
// quotient rounded first would fall on either side.  The quotient in binary32 is off by less
// than 127 * 2^-23 < 2^-16; only where it lies within 2^-12 of a half (one value in 2000) is
// it formed again in binary64, where 127 x is exact and the quotient of two binary32
// numbers that is not a half itself lies 2^-33 or more from one.
#pragma once

#include "gq_device.h"
#include "i8_internal.h"
#include "mxfp4_device.h"

namespace gq {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

// An address that is the same in all lanes, for scalar registers.
__device__ __forceinline__ const int8_t *uniform(const int8_t *p)
{
    const uint64_t a = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return (const int8_t *)((uint64_t)hi << 32 | lo);
}

// The dword at a byte offset from such an address.
__device__ __forceinline__ uint32_t load_dword(const int8_t *base, uint32_t off)
{
    typedef const __attribute__((address_space(1))) int8_t *Global;
    typedef const __attribute__((address_space(1))) uint32_t *GlobalWord;
    return *(GlobalWord)((Global)(uint64_t)uniform(base) + off);
}

// What quantising a row takes: its largest magnitude, the scale (NaN for a row with an
// infinity or a NaN, whose codes are zero) and the factor of the quotient; r < 0 for rows of
// very small values, where 127 / max could be infinite: all their codes come from binary64.
struct I8Row {
    float top, s, r;
    __device__ __forceinline__ explicit I8Row(uint32_t max_bits)
    {
        const bool bad = max_bits >= 0x7f800000u;
        top = __builtin_bit_cast(float, max_bits);
        s = bad ? __builtin_nanf("") : top / 127.0f;
        r = bad || top == 0.0f ? 0.0f : top < 0x1p-60f ? -1.0f : 127.0f / top;
    }
    __device__ __forceinline__ I8Row(float top_, float s_, float r_) : top(top_), s(s_), r(r_) {}
};

template <int TYPE>
__device__ __forceinline__ float i8_load(const void *x, int64_t i)
{
    if constexpr (TYPE == kF32)
        return reinterpret_cast<const float *>(x)[i];
    const uint32_t u = reinterpret_cast<const uint16_t *>(x)[i];
    return TYPE == kBF16 ? __builtin_bit_cast(float, u << 16) : half_to_float(u);
}

// Eight consecutive values of a row (any alignment), of which n exist; the others are zero.
template <int TYPE>
struct I8Load8 { // kF16, kBF16
    uint4 u;
    __device__ __forceinline__ void load(const void *x, int64_t i, int n)
    {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + i;
        if (n >= 8) {
            __builtin_memcpy(&u, p, 16);
        } else {
            uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n)
                    t[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            u = make_uint4(t[0], t[1], t[2], t[3]);
        }
    }
    // the largest magnitude, as bits of a binary32 number; infinities and NaN above all others
    __device__ __forceinline__ uint32_t max_bits() const
    {
        const uint32_t t[4] = {u.x, u.y, u.z, u.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = max(m, max(t[j] & 0x7fffu, (t[j] >> 16) & 0x7fffu));
        return TYPE == kBF16 ? m << 16 : __builtin_bit_cast(uint32_t, half_to_float(m));
    }
    __device__ __forceinline__ float value(int j) const
    {
        const uint32_t t[4] = {u.x, u.y, u.z, u.w};
        const uint32_t b = t[j >> 1] >> (16 * (j & 1)) & 0xffffu;
        return TYPE == kBF16 ? __builtin_bit_cast(float, b << 16) : half_to_float(b);
    }
};
template <>
struct I8Load8<kF32> {
    float v[8];
    __device__ __forceinline__ void load(const void *x, int64_t i, int n)
    {
        const float *p = reinterpret_cast<const float *>(x) + i;
        if (n >= 8) {
            __builtin_memcpy(v, p, 32);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = j < n ? p[j] : 0.0f;
        }
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ float value(int j) const { return v[j]; }
};

// Eight codes of a row, packed.  1.5 * 2^23 added to a quotient leaves the nearest whole number
// in the low bits, its lowest byte the code.
template <int TYPE>
__device__ __forceinline__ uint2 i8_codes8(const I8Load8<TYPE> &v, const I8Row &row)
{
    constexpr float magic = 0x1.8p23f;
    uint32_t b[8];
    float off = 0.0f; // largest distance from a whole number
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = v.value(j) * row.r, m = t + magic;
        off = fmaxf(off, fabsf(t - (m - magic)));
        b[j] = __builtin_bit_cast(uint32_t, m);
    }
    if (__builtin_expect(off > 0.5f - 0x1p-12f || row.r < 0.0f, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            b[j] = (uint32_t)(int)rint(127.0 * (double)v.value(j) / (double)row.top);
    }
    const uint32_t keep = row.r == 0.0f ? 0u : ~0u; // zero rows, and those with NaN
    auto pack = [&](int j) {
        const uint32_t lo = __builtin_amdgcn_perm(b[j + 1], b[j], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[j + 3], b[j + 2], 0x04000c0cu);
        return (lo | hi) & keep;
    };
    return make_uint2(pack(0), pack(4));
}

// A binary32 value as it stands: without this the compiler may merge its last operation and the
// rounding to binary16 into one instruction with one rounding, and results would depend on
// which kernel, and which type, they were formed in.
__device__ __forceinline__ float as_is(float v)
{
    asm("" : "+v"(v));
    return v;
}

// act(z) = z sigmoid(p(z)), p = z (SiLU) or 2 sqrt(2/pi) (z + 0.044715 z^3) (GELU's tanh
// form: 0.5 (1 + tanh(p / 2)) = sigmoid(p)), and its derivative
// sigmoid(p) + z p'(z) sigmoid(p) (1 - sigmoid(p)).  e^-p may overflow: the sigmoid is then
// zero, as it should be; z in the derivative's second term is cut at 64, where that term is
// long zero, so that no zero meets an infinity.
struct Gate {
    float a, da;
};
__device__ __forceinline__ float gate_poly(float z, int act)
{
    constexpr float c = 1.5957691216057308f, a = 0.044715f;
    return act == kSilu ? z : c * fmaf(a * z * z, z, z);
}
__device__ __forceinline__ float gated_value(float g, float u, int act)
{
    return as_is(g / (1.0f + __expf(-gate_poly(g, act))) * u);
}
__device__ __forceinline__ Gate gate_grad(float z, int act)
{
    constexpr float c = 1.5957691216057308f, a = 0.044715f;
    const float sig = 1.0f / (1.0f + __expf(-gate_poly(z, act)));
    const float zc = fminf(fmaxf(z, -64.0f), 64.0f);
    const float dp = act == kSilu ? 1.0f : c * fmaf(3.0f * a * zc, zc, 1.0f);
    return {z * sig, fmaf(zc * dp, sig * (1.0f - sig), sig)};
}

// A sum of products of codes as a value: the weight's scale first, then the token's (their
// product could leave the range of binary32 where the value does not).  Three roundings.
__device__ __forceinline__ float i8_scaled(int sum, float ws, float xs)
{
    return as_is((float)sum * ws * xs);
}

// A weight row's scale as f P, P a power of two and f in [1/2, 1): codes times P are exact in
// both 16-bit types (in binary16 for scales from 2^-25 to 2^8), so that where f can go into
// the other operand before its rounding, a product rounds one operand only.  P stays between
// 2^-126 and 2^127; what that leaves (zero, subnormal and the largest scales, infinity, NaN)
// is f's.
__device__ __forceinline__ float scale_pow2(float s)
{
    const uint32_t e = __builtin_bit_cast(uint32_t, s) & 0x7f800000u;
    return __builtin_bit_cast(float, min(e + 0x00800000u, 0x7f000000u));
}
__device__ __forceinline__ float scale_fraction(float s) { return s * (1.0f / scale_pow2(s)); }

// Four consecutive 16-bit values from element i (any alignment), of which n exist.
__device__ __forceinline__ float4_t load4(const uint16_t *x, int64_t i, int64_t n, int type)
{
    uint2 u = make_uint2(0, 0);
    if (n >= 4) {
        __builtin_memcpy(&u, x + i, 8);
    } else {
        if (n > 0)
            u.x = x[i];
        if (n > 1)
            u.x |= (uint32_t)x[i + 1] << 16;
        if (n > 2)
            u.y = x[i + 2];
    }
    if (type == kBF16)
        return {__builtin_bit_cast(float, u.x << 16), __builtin_bit_cast(float, u.x & 0xffff0000u),
                __builtin_bit_cast(float, u.y << 16), __builtin_bit_cast(float, u.y & 0xffff0000u)};
    return {half_to_float(u.x), half_to_float(u.x >> 16), half_to_float(u.y), half_to_float(u.y >> 16)};
}

// y[i] = v, rounded to `type`.
__device__ __forceinline__ void i8_store(void *y, int64_t i, int type, float v)
{
    if (type == kF32)
        reinterpret_cast<float *>(y)[i] = v;
    else
        reinterpret_cast<uint16_t *>(y)[i] =
            (uint16_t)(type == kBF16 ? mx_pack2<true>(v, 0.f) : mx_pack2<false>(v, 0.f));
}

} // namespace gq
