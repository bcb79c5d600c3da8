// i8_device.h -- device helpers of the int8 kernels (gfx950).
//
// A row's codes are q = 127 x / max|x| rounded to the nearest whole number, halves to even,
// decided as if in exact arithmetic: x = max|x| / 2 is a tie in every row (63.5), so a
// quotient rounded first would fall on either side.  The quotient in binary32 is off by less
// than 127 * 2^-23 < 2^-16; only where it lies within 2^-15 of a half (one value in 16000, and
// the ties of short types) is 254 x compared with the odd multiple of max|x| that the half
// stands for.
#pragma once

#include <type_traits>

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
// very small values, where 127 / max could be infinite: their codes take the exact way.
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

// A binary32 value as it stands: without this the compiler may merge its last operation and the
// rounding to binary16 into one instruction with one rounding, and results would depend on
// which kernel, and which type, they were formed in.
__device__ __forceinline__ float as_is(float v)
{
    asm("" : "+v"(v));
    return v;
}

// The largest of a wave's values, in a scalar register: six dependent vector instructions, where
// exchanges through LDS would take six of its latencies.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto step = [&](auto ctrl, auto rows) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                         decltype(rows)::value, 0xF, false));
    };
    using std::integral_constant;
    step(integral_constant<int, 0xB1>{}, integral_constant<int, 0xF>{});  // lane ^ 1
    step(integral_constant<int, 0x4E>{}, integral_constant<int, 0xF>{});  // lane ^ 2
    step(integral_constant<int, 0x141>{}, integral_constant<int, 0xF>{}); // mirrored in 8
    step(integral_constant<int, 0x140>{}, integral_constant<int, 0xF>{}); // mirrored in 16
    step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{}); // rows 0, 2 to 1, 3
    step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{}); // rows 0, 1 to 2, 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
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

// The code of x, exactly.  The quotient lies between two halves of codes; h is the one nearer to
// it, and 254 x - 2 h top decides on which side of h it is: 2 h is odd and at most 255, so
// 2 h top is p + e of two binary32 numbers, and 254 x - p is exact where the two are close
// (elsewhere its sign is).  x and top are scaled so that none of it overflows or vanishes.
__device__ __forceinline__ int i8_code_exact(float x, float top)
{
    const float f = top < 0x1p-60f ? 0x1p100f : top > 1.0f ? 0x1p-16f : 1.0f;
    x *= f;
    top *= f;
    const float t = x * (127.0f / top), q = rintf(t);
    const float h = q + copysignf(0.5f, t - q), odd = 2.0f * h;
    const float p = as_is(odd * top), e = fmaf(odd, top, -p), d = fmaf(254.0f, x, -p) - e;
    const int lo = (int)(h - 0.5f); // h lies between lo and lo + 1
    return d > 0.0f ? lo + 1 : d < 0.0f ? lo : lo + (lo & 1);
}

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
    if (__builtin_expect(off > 0.5f - 0x1p-15f || row.r < 0.0f, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            b[j] = (uint32_t)i8_code_exact(v.value(j), row.top);
    }
    const uint32_t keep = row.r == 0.0f ? 0u : ~0u; // zero rows, and those with NaN
    auto pack = [&](int j) {
        const uint32_t lo = __builtin_amdgcn_perm(b[j + 1], b[j], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[j + 3], b[j + 2], 0x04000c0cu);
        return (lo | hi) & keep;
    };
    return make_uint2(pack(0), pack(4));
}

// act(z) = z sigmoid(p(z)), p = z (SiLU) or 2 sqrt(2/pi) (z + 0.044715 z^3) (GELU's tanh
// form: 0.5 (1 + tanh(p / 2)) = sigmoid(p)), and its derivative
// sigmoid(p) + z p'(z) sigmoid(p) (1 - sigmoid(p)).  Where the result has 16 bits the exponential
// and the reciprocal are the instructions': e^-p is off by |p| 2^-24 and more of it, two hundred
// times less than the result's rounding at p = -20, and a sigmoid below 2^-126 is zero.  Binary32
// results take the exponential to its last bits, of -|p|, so that it cannot overflow, and a division
// (for all types: gate and up 14336 x 4096 by 1024 rows 112 -> 121 us).  z in the derivative's
// second term is cut at 64, where that term is long zero, so that no zero meets an infinity.
struct Gate {
    float a, da;
};
__device__ __forceinline__ float gate_poly(float z, int act)
{
    constexpr float c = 1.5957691216057308f, a = 0.044715f;
    return act == kSilu ? z : c * fmaf(a * z * z, z, z);
}
template <bool F32>
__device__ __forceinline__ float gated_value(float g, float u, int act)
{
    const float p = gate_poly(g, act);
    if constexpr (F32) {
        const float e = expf(-fabsf(p));
        return as_is(g * ((p < 0.0f ? e : 1.0f) / (1.0f + e)) * u);
    } else {
        return as_is(g * __builtin_amdgcn_rcpf(1.0f + __expf(-p)) * u);
    }
}
__device__ __forceinline__ Gate gate_grad(float z, int act)
{
    constexpr float c = 1.5957691216057308f, a = 0.044715f;
    const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-gate_poly(z, act)));
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

// Four consecutive 16-bit values from element i (any alignment), of which n exist, as they lie,
// and as binary32.
__device__ __forceinline__ uint2 load4(const uint16_t *x, int64_t i, int64_t n)
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
    return u;
}
__device__ __forceinline__ float4_t values4(uint2 u, int type)
{
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
