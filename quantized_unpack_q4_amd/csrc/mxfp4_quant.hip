// mxfp4_quant.hip -- microscaled 4-bit quantisation of activations (or weights)
// and its inverse.
//
// Per block of 32 values: s = max(E - 2, 0), with E the binary32 exponent field
// of the largest magnitude, i.e. the scale 2^(floor(log2 max|x|) - 2) clamped at
// 2^-127 (the e2m1 grid's largest binade starts at 4 = 2^2), and code = x / scale
// rounded to nearest even on the grid 0, 0.5, 1, 1.5, 2, 3, 4, 6 and saturated at
// 6: one scaled conversion per two values.  A block holding an infinity or a NaN
// has s = 255 (NaN) and zero codes: largest magnitudes are compared as integers,
// where every such pattern sorts above the finite ones.
//
// Both passes move bytes and little else.  A lane takes 8 values (16 bytes of a
// 16-bit type, one dword of codes), four neighbouring lanes share a block.
#include "mxfp4_device.h"

namespace gq {

namespace {

// 8 values of row-major x at element offset `i`, as binary32.
template <int TYPE>
struct Load8 { // kF16, kBF16
    uint4 u;
    __device__ __forceinline__ void load(const void *x, int64_t i)
    {
        u = ld16(reinterpret_cast<const uint16_t *>(x) + i);
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        const uint32_t t[4] = {u.x, u.y, u.z, u.w};
        uint32_t m = 0; // largest 16-bit magnitude pattern
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = max(m, max(t[j] & 0x7fffu, (t[j] >> 16) & 0x7fffu));
        if constexpr (TYPE == kBF16)
            return m << 16;
        else // exact; infinity and NaN stay so
            return __builtin_bit_cast(uint32_t, half_to_float(m));
    }
    __device__ __forceinline__ uint32_t codes(float sc) const
    {
        const uint32_t t[4] = {u.x, u.y, u.z, u.w};
        uint32_t r = 0;
        if constexpr (TYPE == kBF16) {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2v, t[0]), sc, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2v, t[1]), sc, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2v, t[2]), sc, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2v, t[3]), sc, 3);
        } else {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2v, t[0]), sc, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2v, t[1]), sc, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2v, t[2]), sc, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2v, t[3]), sc, 3);
        }
        return r;
    }
};
template <>
struct Load8<kF32> {
    float v[8];
    __device__ __forceinline__ void load(const void *x, int64_t i)
    {
        const float *p = reinterpret_cast<const float *>(x) + i;
        const float4 a = ldf4(p), b = ldf4(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float sc) const
    {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], sc, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], sc, 3);
        return r;
    }
};

// Thread t takes values 8t .. 8t+7 of the N*K in row-major order; rows of x start
// ldx elements apart.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void *__restrict__ x,
                                                             int64_t ldx,
                                                             uint32_t *__restrict__ q,
                                                             uint8_t *__restrict__ s,
                                                             int64_t n8, int k8)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n8) // whole blocks leave together: n8 is a multiple of 4
        return;
    int64_t src = t * 8;
    if (ldx != (int64_t)k8 * 8) {
        const int64_t row = t / k8;
        src = row * ldx + (t - row * k8) * 8;
    }
    Load8<TYPE> v;
    v.load(x, src);
    uint32_t m = v.max_bits();
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true)); // lane ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true)); // lane ^ 2
    const uint32_t e = m >> 23;
    const uint32_t sb = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
    const uint32_t c = v.codes(mx_scale(sb == 255u ? 127u : sb));
    q[t] = sb == 255u ? 0u : c;
    if ((t & 3) == 0)
        s[t >> 2] = (uint8_t)sb;
}

// Thread t writes the values of code dword t.
template <int TYPE>
__global__ __launch_bounds__(256) void dequant_mxfp4_kernel(const uint32_t *__restrict__ q,
                                                            const uint8_t *__restrict__ s,
                                                            void *__restrict__ out, int64_t n8)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= n8)
        return;
    const uint32_t c = q[t];
    const float sc = mx_scale(s[t >> 2]);
    if constexpr (TYPE == kF32) {
        typedef float f2v __attribute__((ext_vector_type(2)));
        const f2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 0);
        const f2v b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 1);
        const f2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 2);
        const f2v e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 3);
        float4_t *o = reinterpret_cast<float4_t *>(reinterpret_cast<float *>(out) + t * 8);
        o[0] = float4_t{a.x, a.y, b.x, b.y};
        o[1] = float4_t{d.x, d.y, e.x, e.y};
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + t * 8) =
            mx_values8<TYPE == kBF16>(c, sc);
    }
}

} // namespace

hipError_t launch_quantize_mxfp4(const void *x, int type, int64_t ldx, uint8_t *q, uint8_t *s,
                                 int64_t N, int64_t K, hipStream_t st)
{
    const int64_t n8 = N * (K / 8);
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    uint32_t *qd = reinterpret_cast<uint32_t *>(q);
    const int k8 = (int)(K / 8);
    if (type == kF32)
        hipLaunchKernelGGL((quantize_mxfp4_kernel<kF32>), grid, block, 0, st, x, ldx, qd, s, n8, k8);
    else if (type == kF16)
        hipLaunchKernelGGL((quantize_mxfp4_kernel<kF16>), grid, block, 0, st, x, ldx, qd, s, n8, k8);
    else
        hipLaunchKernelGGL((quantize_mxfp4_kernel<kBF16>), grid, block, 0, st, x, ldx, qd, s, n8, k8);
    return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(MxMat w, void *out, int type, int64_t M, int64_t K, hipStream_t st)
{
    const int64_t n8 = M * (K / 8);
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    const uint32_t *qd = reinterpret_cast<const uint32_t *>(w.q);
    if (type == kF32)
        hipLaunchKernelGGL((dequant_mxfp4_kernel<kF32>), grid, block, 0, st, qd, w.s, out, n8);
    else if (type == kF16)
        hipLaunchKernelGGL((dequant_mxfp4_kernel<kF16>), grid, block, 0, st, qd, w.s, out, n8);
    else
        hipLaunchKernelGGL((dequant_mxfp4_kernel<kBF16>), grid, block, 0, st, qd, w.s, out, n8);
    return hipGetLastError();
}

} // namespace gq
