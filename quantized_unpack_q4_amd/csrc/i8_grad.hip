// i8_grad.hip -- gradients through int8 matrices, one output a thread.
#include "i8_device.h"

namespace gq {

namespace {

__global__ __launch_bounds__(256) void grad_i8_kernel(I8GradPart p0, I8GradPart p1, int nparts, bool split,
                                                      int64_t ldd, uint16_t *dx, int type, int M,
                                                      int K, int64_t total)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= total)
        return;
    const int64_t n = t / K, k = t - n * K;
    float s = 0;
    for (int p = 0; p < nparts; ++p) {
        const I8GradPart &a = p ? p1 : p0;
        for (int m = 0; m < M; ++m) {
            const float sc = split ? scale_split(a.w.s[m]).pow2 : a.w.s[m];
            const float wv = as_is((float)a.w.q[m * a.w.ld + k] * sc);
            const uint32_t r = type == kBF16 ? mx_pack2<true>(wv, 0.f) : mx_pack2<false>(wv, 0.f);
            const float w16 = type == kBF16 ? __builtin_bit_cast(float, r << 16) : half_to_float(r);
            s += w16 * (type == kBF16 ? i8_load<kBF16>(a.d, n * ldd + m) : i8_load<kF16>(a.d, n * ldd + m));
        }
    }
    i8_store(dx, t, type, s);
}

unsigned blocks(int64_t total) { return (unsigned)((total + 255) / 256); }

} // namespace

hipError_t launch_grad_i8(const I8GradPart *parts, int nparts, bool split, int64_t ldd,
                          uint16_t *dx, int type, int64_t M, int64_t K, int64_t N, hipStream_t st)
{
    hipLaunchKernelGGL(grad_i8_kernel, dim3(blocks(K * N)), dim3(256), 0, st, parts[0],
                       parts[nparts - 1], nparts, split, ldd, dx, type, (int)M, (int)K, K * N);
    return hipGetLastError();
}

} // namespace gq
