// i8_products.hip -- products of int8 matrices, one output a thread.
#include "i8_device.h"

namespace gq {

namespace {

__device__ __forceinline__ int dot(const int8_t *a, const int8_t *b, int K)
{
    int s = 0;
    for (int k = 0; k < K; ++k)
        s += (int)a[k] * (int)b[k];
    return s;
}

__global__ __launch_bounds__(256) void gemm_i8_kernel(I8Mat w, I8Mat x, void *y, int type, int M,
                                                      int K, int64_t total)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= total)
        return;
    const int64_t n = t / M, m = t - n * M;
    i8_store(y, t, type, i8_scaled(dot(w.q + m * w.ld, x.q + n * x.ld, K), w.s[m], x.s[n]));
}

// grads: dh -> gradients of g and u; else h
__global__ __launch_bounds__(256) void gated_i8_kernel(I8Mat gate, I8Mat up, I8Mat x, void *h,
                                                       const uint16_t *dh, int64_t ldd, int type,
                                                       int act, int I, int H, int64_t total)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= total)
        return;
    const int64_t n = t / I, i = t - n * I;
    const int8_t *xq = x.q + n * x.ld;
    const float g = i8_scaled(dot(gate.q + i * gate.ld, xq, H), gate.s[i], x.s[n]);
    const float u = i8_scaled(dot(up.q + i * up.ld, xq, H), up.s[i], x.s[n]);
    if (!dh) {
        i8_store(h, t, type, gated_value(g, u, act));
        return;
    }
    const float d = type == kBF16 ? i8_load<kBF16>(dh, t) : i8_load<kF16>(dh, t);
    const Gate a = gate_grad(g, act);
    i8_store(h, (2 * n) * ldd + i, type, d * u * a.da);
    i8_store(h, (2 * n + 1) * ldd + i, type, d * a.a);
}

__global__ __launch_bounds__(256) void grad_i8_kernel(I8GradPart p0, I8GradPart p1, int nparts,
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
            const float wv = as_is((float)a.w.q[m * a.w.ld + k] * a.w.s[m]);
            const uint32_t r = type == kBF16 ? mx_pack2<true>(wv, 0.f) : mx_pack2<false>(wv, 0.f);
            const float w16 = type == kBF16 ? __builtin_bit_cast(float, r << 16) : half_to_float(r);
            s += w16 * (type == kBF16 ? i8_load<kBF16>(a.d, n * ldd + m) : i8_load<kF16>(a.d, n * ldd + m));
        }
    }
    i8_store(dx, t, type, s);
}

// One workgroup per activation row quantises it into LDS pieces and multiplies 256 rows at a time.
template <int TYPE>
__global__ __launch_bounds__(256) void gemv_i8_kernel(I8Mat w, I8Mat w2, const void *x, void *y,
                                                      int act, int M, int K)
{
    __shared__ uint32_t part[4];
    __shared__ __attribute__((aligned(16))) int8_t codes[2048];
    const int tid = threadIdx.x, b = blockIdx.y;
    const int64_t x0 = (int64_t)b * K;
    uint32_t mx = 0;
    for (int k = 8 * tid; k < K; k += 2048) {
        I8Load8<TYPE> v;
        v.load(x, x0 + k, min(K - k, 8));
        mx = max(mx, v.max_bits());
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, off, 64));
    if ((tid & 63) == 0)
        part[tid >> 6] = mx;
    __syncthreads();
    const I8Row row(max(max(part[0], part[1]), max(part[2], part[3])));
    const int64_t m = (int64_t)blockIdx.x * 256 + tid;
    int s0 = 0, s1 = 0;
    for (int k0 = 0; k0 < K; k0 += 2048) {
        I8Load8<TYPE> v;
        if (k0 + 8 * tid < K) {
            v.load(x, x0 + k0 + 8 * tid, min(K - k0 - 8 * tid, 8));
            *reinterpret_cast<uint2 *>(codes + 8 * tid) = i8_codes8(v, row);
        }
        __syncthreads();
        if (m < M) {
            s0 += dot(w.q + m * w.ld + k0, codes, min(K - k0, 2048));
            if (w2.q)
                s1 += dot(w2.q + m * w2.ld + k0, codes, min(K - k0, 2048));
        }
        __syncthreads();
    }
    if (m >= M)
        return;
    float v = i8_scaled(s0, w.s[m], row.s);
    if (w2.q)
        v = gated_value(v, i8_scaled(s1, w2.s[m], row.s), act);
    i8_store(y, (int64_t)b * M + m, TYPE, v);
}

unsigned blocks(int64_t total) { return (unsigned)((total + 255) / 256); }

hipError_t gemv(I8Mat w, I8Mat w2, const void *x, void *y, int type, int act, int64_t M, int64_t K,
                int B, hipStream_t st)
{
    const dim3 grid(blocks(M), B), block(256);
    if (type == kF32)
        hipLaunchKernelGGL(gemv_i8_kernel<kF32>, grid, block, 0, st, w, w2, x, y, act, (int)M, (int)K);
    else if (type == kF16)
        hipLaunchKernelGGL(gemv_i8_kernel<kF16>, grid, block, 0, st, w, w2, x, y, act, (int)M, (int)K);
    else
        hipLaunchKernelGGL(gemv_i8_kernel<kBF16>, grid, block, 0, st, w, w2, x, y, act, (int)M, (int)K);
    return hipGetLastError();
}

} // namespace

hipError_t launch_gemv_i8(I8Mat w, const void *x, void *y, int type, int64_t M, int64_t K, int B,
                          hipStream_t st)
{
    return gemv(w, I8Mat{}, x, y, type, kSilu, M, K, B, st);
}

hipError_t launch_gated_gemv_i8(I8Mat gate, I8Mat up, const void *x, void *h, int type, int act,
                                int64_t I, int64_t H, int N, hipStream_t st)
{
    return gemv(gate, up, x, h, type, act, I, H, N, st);
}

hipError_t launch_gemm_i8(I8Mat w, I8Mat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                          hipStream_t st)
{
    hipLaunchKernelGGL(gemm_i8_kernel, dim3(blocks(M * N)), dim3(256), 0, st, w, x, y, type, (int)M,
                       (int)K, M * N);
    return hipGetLastError();
}

hipError_t launch_gated_i8(I8Mat gate, I8Mat up, I8Mat x, void *h, int type, int act, int64_t I,
                           int64_t H, int64_t N, hipStream_t st)
{
    hipLaunchKernelGGL(gated_i8_kernel, dim3(blocks(I * N)), dim3(256), 0, st, gate, up, x, h,
                       (const uint16_t *)nullptr, (int64_t)0, type, act, (int)I, (int)H, I * N);
    return hipGetLastError();
}

hipError_t launch_gated_grads_i8(I8Mat gate, I8Mat up, I8Mat x, const uint16_t *dh, uint16_t *d,
                                 int64_t ldd, int type, int act, int64_t I, int64_t H, int64_t N,
                                 hipStream_t st)
{
    hipLaunchKernelGGL(gated_i8_kernel, dim3(blocks(I * N)), dim3(256), 0, st, gate, up, x, d, dh,
                       ldd, type, act, (int)I, (int)H, I * N);
    return hipGetLastError();
}

hipError_t launch_grad_i8(const I8GradPart *parts, int nparts, int64_t ldd, uint16_t *dx, int type,
                          int64_t M, int64_t K, int64_t N, hipStream_t st)
{
    hipLaunchKernelGGL(grad_i8_kernel, dim3(blocks(K * N)), dim3(256), 0, st, parts[0],
                       parts[nparts - 1], nparts, ldd, dx, type, (int)M, (int)K, K * N);
    return hipGetLastError();
}

hipError_t launch_ffn_i8(const I8FfnArgs &a, hipStream_t st)
{
    int8_t *xq = reinterpret_cast<int8_t *>(a.ws + a.off[0]), *hq = reinterpret_cast<int8_t *>(a.ws + a.off[3]);
    float *xs = reinterpret_cast<float *>(a.ws + a.off[1]), *hs = reinterpret_cast<float *>(a.ws + a.off[4]);
    void *h = a.ws + a.off[2];
    const int64_t ldx = (a.H + 15) / 16 * 16, ldh = (a.I + 15) / 16 * 16;
    hipError_t e = launch_quantize_i8(a.x, a.type, a.H, xq, ldx, xs, a.T, a.H, st);
    if (e == hipSuccess)
        e = launch_gated_i8(a.gate, a.up, {xq, ldx, xs}, h, a.type, a.act, a.I, a.H, a.T, st);
    if (e == hipSuccess)
        e = launch_quantize_i8(h, a.type, a.I, hq, ldh, hs, a.T, a.I, st);
    if (e == hipSuccess)
        e = launch_gemm_i8(a.down, {hq, ldh, hs}, a.out, a.type, a.H, a.I, a.T, st);
    return e;
}

} // namespace gq
