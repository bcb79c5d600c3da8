// i8_quant.hip -- 8-bit codes and a scale for every row (token or output channel), and back.
//
// scale = max|x| / 127, code = 127 x / max|x| to the nearest (i8_device.h).  A row with an
// infinity or a NaN has a NaN scale and zero codes; a zero row has scale zero.
//
// Both move bytes and little else.  A workgroup of T threads quantises a row and holds 16 T values
// of it in registers, 16 (one 16-byte store of codes) a thread; the rest of a longer row is read
// twice, from a cache the second time.  T goes by the row's length, up to 256 (4096 values); rows
// longer than that get 1024 threads, 16384 values, where no more than a row a CU is there
// to hide the second reading: by 256 rows of 14336 bfloat16 values 6.0 us (with 256 threads 9.5), of
// 8192 5.0 (5.9), 16 rows of 5000 4.9 (6.0).  With more rows the small workgroups, which wait less
// for each other, make up for it: by 4096 rows of 14336 40.8 us (45.9 with 1024 threads), of 8192 21.8
// (35.9), by 1024 of 14336 13.7 (15.5); from 257 to 512 of 14336 it is the other way round by up to a
// fifth, 9.5 (7.8) to 10.1 (9.6), and by 1024 rows of 60000, past what either holds, 50 (43).
#include "gq_internal.h"
#include "i8_device.h"

#include <algorithm>
#include <type_traits>

namespace gq {

namespace {

// The largest of all threads' values; `part` is not the one of the call before.
template <int T>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t (&part)[T / 64])
{
    m = wave_max(m);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int i = 1; i < T / 64; ++i)
            m = max(m, part[i]);
    }
    return m;
}

// 16 values from column k of a row, and their codes.
template <int TYPE>
struct Load16 {
    I8Load8<TYPE> v[2];
    __device__ __forceinline__ void load(const void *x, int64_t row, int64_t k, int64_t K)
    {
        const int n = (int)max(min(K - k, (int64_t)16), (int64_t)0);
        v[0].load(x, row + k, min(n, 8));
        v[1].load(x, row + k + 8, max(n - 8, 0));
    }
    __device__ __forceinline__ uint32_t max_bits() const { return max(v[0].max_bits(), v[1].max_bits()); }
    __device__ __forceinline__ void store(int8_t *q, int64_t k, int64_t K, const I8Row &row) const
    {
        if (k >= K)
            return;
        const uint2 a = i8_codes8(v[0], row), b = i8_codes8(v[1], row);
        if (k + 16 <= K) {
            *reinterpret_cast<uint4 *>(q + k) = make_uint4(a.x, a.y, b.x, b.y);
        } else { // what lies behind the row's codes stays
            const uint32_t t[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k + j < K)
                    q[k + j] = (int8_t)(t[j >> 2] >> (8 * (j & 3)));
        }
    }
};

// One workgroup of T threads per row, up to 16 T values of it in registers.
template <int TYPE, int T>
__global__ __launch_bounds__(T) void quantize_i8_kernel(const void *__restrict__ x, int64_t ldx,
                                                        int8_t *__restrict__ q, int64_t ldq,
                                                        float *__restrict__ s, int64_t N, int64_t K)
{
    __shared__ uint32_t part[2][T / 64];
    const int tid = threadIdx.x;
    Load16<TYPE> next;
    next.load(x, blockIdx.x * ldx, 16 * tid, K);
    int turn = 0;
    for (int64_t n = blockIdx.x; n < N; n += gridDim.x, turn ^= 1) {
        const Load16<TYPE> v = next;
        uint32_t m = v.max_bits();
        for (int64_t k = 16 * (T + tid); k < K; k += 16 * T) {
            Load16<TYPE> w;
            w.load(x, n * ldx, k, K);
            m = max(m, w.max_bits());
        }
        if (n + gridDim.x < N) // the next row, while this one is compared and stored
            next.load(x, (n + gridDim.x) * ldx, 16 * tid, K);
        const I8Row row(block_max<T>(m, part[turn]));
        if (tid == 0)
            s[n] = row.s;
        int8_t *dst = q + n * ldq;
        v.store(dst, 16 * tid, K, row);
        for (int64_t k = 16 * (T + tid); k < K; k += 16 * T) {
            Load16<TYPE> w;
            w.load(x, n * ldx, k, K);
            w.store(dst, k, K, row);
        }
    }
}

// V consecutive values a thread, 2^tpr threads a row at a time, 256 / 2^tpr rows a workgroup.
// NT: past the caches (4096 x 14336 to binary32, 294 MB: 42 us against 58).
template <int TYPE, int V, bool NT>
__global__ __launch_bounds__(256) void dequant_i8_kernel(const int8_t *__restrict__ q, int64_t ldq,
                                                         const float *__restrict__ s,
                                                         void *__restrict__ out, int64_t M, int64_t K,
                                                         int tpr)
{
    constexpr int ES = TYPE == kF32 ? 4 : 2;
    const int64_t k0 = ((int64_t)blockIdx.x << tpr | (threadIdx.x & ((1 << tpr) - 1))) * V;
    const int64_t kstep = ((int64_t)gridDim.x << tpr) * V, mstep = (int64_t)gridDim.y << (8 - tpr);
    for (int64_t m = (int64_t)blockIdx.y << (8 - tpr) | threadIdx.x >> tpr; m < M; m += mstep) {
        const float sc = s[m];
        for (int64_t k = k0; k < K; k += kstep) {
            const int8_t *src = q + m * ldq + k;
            uint8_t *dst = reinterpret_cast<uint8_t *>(out) + (m * K + k) * ES;
            uint32_t w[V / 4]; // (every row has the bytes up to the next multiple of 16)
            __builtin_memcpy(w, src, V);
            uint32_t o[V * ES / 4];
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float a = as_is((float)(int8_t)(w[j / 4] >> (8 * (j & 3))) * sc);
                const float b = as_is((float)(int8_t)(w[j / 4] >> (8 * (j & 3) + 8)) * sc);
                if constexpr (TYPE == kF32) {
                    o[j] = __builtin_bit_cast(uint32_t, a);
                    o[j + 1] = __builtin_bit_cast(uint32_t, b);
                } else {
                    o[j / 2] = mx_pack2<TYPE == kBF16>(a, b);
                }
            }
            if (k + V <= K) {
                typedef uint32_t Chunk __attribute__((ext_vector_type(4), aligned(2)));
                const Chunk c = {o[0], o[1], o[2], o[3]};
                if constexpr (NT)
                    __builtin_nontemporal_store(c, reinterpret_cast<Chunk *>(dst));
                else
                    *reinterpret_cast<Chunk *>(dst) = c;
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (k + j < K) {
                        if constexpr (TYPE == kF32)
                            reinterpret_cast<uint32_t *>(dst)[j] = o[j];
                        else
                            reinterpret_cast<uint16_t *>(dst)[j] = (uint16_t)(o[j / 2] >> (16 * (j & 1)));
                    }
            }
        }
    }
}

template <int TYPE>
hipError_t quantize(const void *x, int64_t ldx, int8_t *q, int64_t ldq, float *s, int64_t N, int64_t K,
                    hipStream_t st)
{
    auto launch = [&](auto t) {
        constexpr int T = decltype(t)::value;
        const dim3 grid((unsigned)std::min(N, (int64_t)std::max(24 * 64 / T, 1) * device_cus()));
        hipLaunchKernelGGL((quantize_i8_kernel<TYPE, T>), grid, dim3(T), 0, st, x, ldx, q, ldq, s, N, K);
        return hipGetLastError();
    };
    using std::integral_constant; // (1024 threads: see above)
    return K <= 1024              ? launch(integral_constant<int, 64>{})
           : K <= 2048            ? launch(integral_constant<int, 128>{})
           : K <= 4096 || N > 256 ? launch(integral_constant<int, 256>{})
                                  : launch(integral_constant<int, 1024>{});
}

template <int TYPE>
hipError_t dequant(I8Mat w, void *out, int64_t M, int64_t K, hipStream_t st)
{
    constexpr int V = TYPE == kF32 ? 4 : 8; // a 16-byte store
    int tpr = 0;
    while (tpr < 8 && ((int64_t)V << tpr) < K)
        ++tpr;
    const dim3 grid((unsigned)std::min((K + 256 * V - 1) / (256 * V), (int64_t)64),
                    (unsigned)std::min((M + (256 >> tpr) - 1) / (256 >> tpr), (int64_t)65535));
    // outputs that the L2 caches (32 MB) could not hold for what comes next
    if (M * K * (TYPE == kF32 ? 4 : 2) > (int64_t)32 << 20)
        hipLaunchKernelGGL((dequant_i8_kernel<TYPE, V, true>), grid, dim3(256), 0, st, w.q, w.ld, w.s, out,
                           M, K, tpr);
    else
        hipLaunchKernelGGL((dequant_i8_kernel<TYPE, V, false>), grid, dim3(256), 0, st, w.q, w.ld, w.s, out,
                           M, K, tpr);
    return hipGetLastError();
}

} // namespace

hipError_t launch_quantize_i8(const void *x, int type, int64_t ldx, int8_t *q, int64_t ldq,
                              float *s, int64_t N, int64_t K, hipStream_t st)
{
    return type == kF32   ? quantize<kF32>(x, ldx, q, ldq, s, N, K, st)
           : type == kF16 ? quantize<kF16>(x, ldx, q, ldq, s, N, K, st)
                          : quantize<kBF16>(x, ldx, q, ldq, s, N, K, st);
}

hipError_t launch_dequant_i8(I8Mat w, void *out, int type, int64_t M, int64_t K, hipStream_t st)
{
    return type == kF32   ? dequant<kF32>(w, out, M, K, st)
           : type == kF16 ? dequant<kF16>(w, out, M, K, st)
                          : dequant<kBF16>(w, out, M, K, st);
}

} // namespace gq
