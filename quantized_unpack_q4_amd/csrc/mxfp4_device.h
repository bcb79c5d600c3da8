// mxfp4_device.h -- device helpers of the microscaled 4-bit kernels (gfx950).
//
// A block is 32 consecutive values of a row, value = e2m1(code) * 2^(s - 127).
// Codes lie two to a byte, the even column in the low nibble, so the 16 bytes
// of a block are the operand order of the scaled matrix instructions: lane l of
// v_mfma_scale_f32_16x16x128 (32x32x64) takes one whole block of row l % 16
// (l % 32) as four registers and its scale as one byte.
//
// The scaled conversions take the scale as a binary32 number of which only the
// exponent counts: s << 23.  Checked over all 256 codes pairs and scales: exact
// in binary32 and bfloat16 (subnormals included), rounded to nearest even with
// overflow to infinity in binary16, NaN for s = 255.
#pragma once

#include "gq_device.h"
#include "mxfp4_internal.h"

namespace gq {

typedef _Float16 h2v __attribute__((ext_vector_type(2)));
typedef __bf16 b2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef int i8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float mx_scale(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

// The eight values of four code bytes as packed 16-bit numbers.
template <bool BF16>
__device__ __forceinline__ uint4 mx_values8(uint32_t q, float sc)
{
    if constexpr (BF16)
        return make_uint4(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 3)));
    else
        return make_uint4(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 3)));
}

// 16 x 16 x 32 product of packed 16-bit operands.
template <bool BF16>
__device__ __forceinline__ float4_t mx_mfma16(uint4 a, uint4 b, float4_t c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a),
                                                       __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                      __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// 16 x 16 x 128 product of MXFP4 operands: a block of 32 codes per lane and its
// scale in the low byte of sa, sb.
__device__ __forceinline__ float4_t mx_mfma16_fp4(uint4 a, uint32_t sa, uint4 b, uint32_t sb,
                                                  float4_t c)
{
    const i8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0,
                                                            (int)sb);
}

// Lanes of a wave hand values on through LDS without a barrier: the LDS keeps the order of a
// wave's accesses, and this keeps it in the compiled code, which knows one lane's addresses
// only.
__device__ __forceinline__ void lds_wave_order() { asm volatile("" ::: "memory"); }

// Two binary32 values rounded (nearest even) to the 16-bit type, packed.
template <bool BF16>
__device__ __forceinline__ uint32_t mx_pack2(float lo, float hi)
{
    if constexpr (BF16) {
        const b2v v = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        return pack_half2(lo, hi);
    }
}

// The scales of 4 Q consecutive blocks of a row from block b0 (a multiple of 4), as Q words;
// blocks past the row's nblk have scale 1.  One load a row instead of one a block: a load
// of single bytes from 16 rows costs the L2 as much as one of whole blocks (without it the
// weight-streaming products took 25-35% less).  Rows need no alignment.
template <int Q>
struct MxScales {
    uint32_t w[Q];
    __device__ __forceinline__ void load(const uint8_t *row, int b0, int nblk)
    {
        if (b0 + 4 * Q <= nblk) {
            __builtin_memcpy(w, row + b0, 4 * Q);
        } else {
#pragma unroll
            for (int u = 0; u < Q; ++u) {
                w[u] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[u] |= (b0 + 4 * u + i < nblk ? (uint32_t)row[b0 + 4 * u + i] : 127u) << (8 * i);
            }
        }
    }
};

// Four consecutive outputs y[0..3] of a row, of which `n` exist; vec: 16-byte
// (8-byte for the 16-bit types) aligned.
__device__ __forceinline__ void mx_store4(void *y, int64_t idx, int type, float4_t v, int n,
                                          bool vec)
{
    if (type == kF32) {
        float *p = reinterpret_cast<float *>(y) + idx;
        if (vec && n >= 4) {
            *reinterpret_cast<float4_t *>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n)
                    p[i] = v[i];
        }
        return;
    }
    const uint32_t a = type == kBF16 ? mx_pack2<true>(v[0], v[1]) : mx_pack2<false>(v[0], v[1]);
    const uint32_t b = type == kBF16 ? mx_pack2<true>(v[2], v[3]) : mx_pack2<false>(v[2], v[3]);
    uint16_t *p = reinterpret_cast<uint16_t *>(y) + idx;
    if (vec && n >= 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
    } else {
        const uint32_t t[2] = {a, b};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n)
                p[i] = (uint16_t)(t[i >> 1] >> (16 * (i & 1)));
    }
}

} // namespace gq
