// i8_quant.hip -- 8-bit codes and a scale for every row (token or output channel), and back.
//
// scale = max|x| / 127, code = 127 x / max|x| to the nearest (i8_device.h).  A row with an
// infinity or a NaN has a NaN scale and zero codes; a zero row has scale zero.
#include "i8_device.h"

#include <algorithm>

namespace gq {

namespace {

// One workgroup per row.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_i8_kernel(const void *__restrict__ x, int64_t ldx,
                                                          int8_t *__restrict__ q, int64_t ldq,
                                                          float *__restrict__ s, int64_t N,
                                                          int64_t K)
{
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x;
    for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const int64_t x0 = n * ldx;
    uint32_t m = 0;
    for (int64_t k = 8 * tid; k < K; k += 8 * 256) {
        I8Load8<TYPE> v;
        v.load(x, x0 + k, (int)min(K - k, (int64_t)8));
        m = max(m, v.max_bits());
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if ((tid & 63) == 0)
        part[tid >> 6] = m;
    __syncthreads();
    const I8Row row(max(max(part[0], part[1]), max(part[2], part[3])));
    if (tid == 0)
        s[n] = row.s;
    int8_t *dst = q + n * ldq;
    for (int64_t k = 8 * tid; k < K; k += 8 * 256) {
        I8Load8<TYPE> v;
        const int c = (int)min(K - k, (int64_t)8);
        v.load(x, x0 + k, c);
        const uint2 b = i8_codes8(v, row);
        if (c == 8) {
            *reinterpret_cast<uint2 *>(dst + k) = b;
        } else {
            for (int j = 0; j < c; ++j)
                dst[k + j] = (int8_t)((j < 4 ? b.x : b.y) >> (8 * (j & 3)));
        }
    }
    __syncthreads();
    }
}

template <int TYPE>
__global__ __launch_bounds__(256) void dequant_i8_kernel(const int8_t *__restrict__ q, int64_t ldq,
                                                         const float *__restrict__ s,
                                                         void *__restrict__ out, int64_t K,
                                                         int64_t total)
{
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t m = t / K, k = t - m * K;
        i8_store(out, t, TYPE, as_is((float)q[m * ldq + k] * s[m]));
    }
}

} // namespace

hipError_t launch_quantize_i8(const void *x, int type, int64_t ldx, int8_t *q, int64_t ldq,
                              float *s, int64_t N, int64_t K, hipStream_t st)
{
    const dim3 grid((unsigned)std::min(N, (int64_t)1 << 16)), block(256);
    if (type == kF32)
        hipLaunchKernelGGL(quantize_i8_kernel<kF32>, grid, block, 0, st, x, ldx, q, ldq, s, N, K);
    else if (type == kF16)
        hipLaunchKernelGGL(quantize_i8_kernel<kF16>, grid, block, 0, st, x, ldx, q, ldq, s, N, K);
    else
        hipLaunchKernelGGL(quantize_i8_kernel<kBF16>, grid, block, 0, st, x, ldx, q, ldq, s, N, K);
    return hipGetLastError();
}

hipError_t launch_dequant_i8(I8Mat w, void *out, int type, int64_t M, int64_t K, hipStream_t st)
{
    const int64_t total = M * K;
    const dim3 grid((unsigned)std::min((total + 255) / 256, (int64_t)1 << 16)), block(256);
    if (type == kF32)
        hipLaunchKernelGGL(dequant_i8_kernel<kF32>, grid, block, 0, st, w.q, w.ld, w.s, out, K, total);
    else if (type == kF16)
        hipLaunchKernelGGL(dequant_i8_kernel<kF16>, grid, block, 0, st, w.q, w.ld, w.s, out, K, total);
    else
        hipLaunchKernelGGL(dequant_i8_kernel<kBF16>, grid, block, 0, st, w.q, w.ld, w.s, out, K, total);
    return hipGetLastError();
}

} // namespace gq
