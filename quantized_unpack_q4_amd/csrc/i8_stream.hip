// i8_stream.hip -- int8 products by up to 16 activation rows, weights streamed once.
//
// A workgroup takes tiles of 16 weight rows (of each matrix in the gate/up form); its W waves
// share K, a contiguous run each, and multiply on the 16x16x64 product, whose operand is 16
// codes (16 bytes) of a row per lane as they lie in memory.  The waves' sums are whole numbers:
// joined through LDS they are the same in any order.
//
// Activations are codes, read from memory in the same form, or floats, which every workgroup
// quantises itself: the largest magnitude of each row over all waves, then each wave the codes
// of its own run into LDS, once for all of a workgroup's tiles.  Columns past K get zero codes,
// so that what lies there in the weights counts nothing.
#include <algorithm>

#include "gq_internal.h"
#include "i8_device.h"

namespace gq {

namespace {

constexpr int kCodes = 3; // activations are codes (else a type)

struct I8StreamArgs {
    I8Mat w, w2; // gate/up: gate, up
    const void *x;
    I8Mat xc;
    void *y;
    int type, act;
    int M, K, B;
    int run; // columns of a wave, a multiple of 64
};

__device__ __forceinline__ int4v mfma16_i8(uint4 a, uint4 b, int4v c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(int4v, a),
                                                 __builtin_bit_cast(int4v, b), c, 0, 0, 0);
}

// Bytes of LDS for codes: rows of a run are 16 bytes further apart than the run is long, so
// that 16 rows' reads touch distinct banks.
constexpr int64_t codes_bytes(int W, int64_t B, int64_t run) { return W * B * (run + 16); }

template <int SRC, bool PAIR, int W, int LDSB>
__global__ __launch_bounds__(64 * W) void i8_stream_kernel(I8StreamArgs p)
{
    constexpr int P = PAIR ? 2 : 1, U = 8;
    constexpr bool FLOATS = SRC != kCodes;
    __shared__ __attribute__((aligned(16))) uint8_t codes[FLOATS ? LDSB : 16];
    __shared__ uint32_t part[16][W];
    __shared__ float xscale[16];
    __shared__ int4v red[W][P][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int M = p.M, K = p.K, B = p.B;
    const int k0 = wave * p.run, cols = max(0, min(K - k0, p.run));
    const int steps = (cols + 63) >> 6; // of 64 columns
    const int lastc = ((K + 15) >> 4) - 1; // last chunk of 16 codes of a row
    const int pitch = p.run + 16;
    uint8_t *mine = codes + (FLOATS ? wave * B * pitch : 0);

    if constexpr (FLOATS) {
        for (int b = 0; b < B; ++b) {
            uint32_t m = 0;
            for (int k = 8 * lane; k < cols; k += 512) {
                I8Load8<SRC> v;
                v.load(p.x, (int64_t)b * K + k0 + k, min(cols - k, 8));
                m = max(m, v.max_bits());
            }
            m = wave_max(m);
            if (lane == 0)
                part[b][wave] = m;
        }
        __syncthreads();
        uint32_t m = 0;
        if (lane < B)
#pragma unroll
            for (int i = 0; i < W; ++i)
                m = max(m, part[lane][i]);
        const I8Row row(m); // lane b: row b
        if (wave == 0 && lane < B)
            xscale[lane] = row.s;
        const int nb = 8 * steps; // blocks of 8 columns of a row
        for (int b = 0; b < B; ++b) {
            const I8Row rb(__shfl(row.top, b, 64), __shfl(row.s, b, 64), __shfl(row.r, b, 64));
            for (int c = lane; c < nb; c += 64) {
                I8Load8<SRC> v;
                v.load(p.x, (int64_t)b * K + k0 + 8 * c, max(min(cols - 8 * c, 8), 0));
                *reinterpret_cast<uint2 *>(mine + b * pitch + 8 * c) = i8_codes8(v, rb);
            }
        }
        lds_wave_order();
    }

    const int tiles = (M + 15) >> 4;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int m0 = 16 * tile;
        const int64_t wr = min(m0 + r, M - 1);
        const int8_t *wp[2] = {p.w.q + wr * p.w.ld, PAIR ? p.w2.q + wr * p.w2.ld : nullptr};
        const int xr = min(r, B - 1);
        const int8_t *xp = FLOATS ? nullptr : p.xc.q + xr * p.xc.ld;
        int4v acc[P];
#pragma unroll
        for (int i = 0; i < P; ++i)
            acc[i] = int4v{0, 0, 0, 0};
        for (int s0 = 0; s0 < steps; s0 += U) {
            uint4 a[P][U], xv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ch = min((k0 >> 4) + 4 * (s0 + u) + q, lastc);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    a[i][u] = ld16(wp[i] + 16 * ch);
                if (!FLOATS)
                    xv[u] = ld16(xp + 16 * ch);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s0 + u >= steps)
                    break;
                if constexpr (FLOATS) {
                    xv[u] = ld16(mine + xr * pitch + 64 * (s0 + u) + 16 * q);
                } else {
                    const int left = K - (k0 + 64 * (s0 + u) + 16 * q); // codes past K are zero
                    if (__builtin_expect(left < 16, 0)) {
                        uint32_t t[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int n = min(max(left - 4 * j, 0), 4);
                            t[j] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
                        }
                        xv[u] = make_uint4(t[0], t[1], t[2], t[3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < P; ++i)
                    acc[i] = mfma16_i8(a[i][u], xv[u], acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            red[wave][i][lane] = acc[i];
        __syncthreads();
        // output t: weight row t % 16, activation row t / 16; in the accumulators lane
        // 16 (row / 4) + activation row, element row % 4
        if (tid < 256 && tid >> 4 < B && m0 + (tid & 15) < M) {
            const int m = tid & 15, b = tid >> 4, from = 16 * (m >> 2) + b;
            int sum[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sum[i] = 0;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    sum[i] += red[j][i][from][m & 3];
            }
            const float xs = FLOATS ? xscale[b] : p.xc.s[b];
            float v = i8_scaled(sum[0], p.w.s[m0 + m], xs);
            if constexpr (PAIR)
                v = gated_value(v, i8_scaled(sum[P - 1], p.w2.s[m0 + m], xs), p.act);
            i8_store(p.y, (int64_t)b * M + m0 + m, p.type, v);
        }
        __syncthreads();
    }
}

// Sixteen waves where K is long enough to keep eight waiting for their weights.
constexpr int64_t kLongK = 8192;
// Values a workgroup quantises itself.
constexpr int64_t kFused = 16384;

template <int SRC, bool PAIR, int W>
hipError_t launch_waves(I8StreamArgs p, int64_t grid, hipStream_t st)
{
    // a run is at most K / W + 64 columns, and where K is long one row is quantised at most
    constexpr int B = W == 8 ? 16 : 1;
    constexpr int LDSB = SRC == kCodes ? 16 : (int)(kFused + W * B * (64 + 16));
    static_assert(W == 8 || 2 * kLongK >= kFused, "one row");
    p.run = ((p.K + W - 1) / W + 63) / 64 * 64;
    if (SRC != kCodes && codes_bytes(W, p.B, p.run) > LDSB)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((i8_stream_kernel<SRC, PAIR, W, LDSB>), dim3((unsigned)grid), dim3(64 * W), 0, st,
                       p);
    return hipGetLastError();
}

template <int SRC, bool PAIR>
hipError_t launch_stream(const I8StreamArgs &p, hipStream_t st)
{
    const int64_t tiles = ((int64_t)p.M + 15) / 16;
    return p.K > kLongK ? launch_waves<SRC, PAIR, 16>(p, tiles, st) : launch_waves<SRC, PAIR, 8>(p, tiles, st);
}

template <bool PAIR>
hipError_t stream_floats(const I8StreamArgs &p, hipStream_t st)
{
    return p.type == kF32   ? launch_stream<kF32, PAIR>(p, st)
           : p.type == kF16 ? launch_stream<kF16, PAIR>(p, st)
                            : launch_stream<kBF16, PAIR>(p, st);
}

I8StreamArgs args(I8Mat w, I8Mat w2, void *y, int type, int act, int64_t M, int64_t K, int64_t B)
{
    I8StreamArgs p{};
    p.w = w;
    p.w2 = w2;
    p.y = y;
    p.type = type;
    p.act = act;
    p.M = (int)M;
    p.K = (int)K;
    p.B = (int)B;
    return p;
}

} // namespace

bool i8_fused(int64_t K, int64_t B) { return B <= 16 && B * K <= kFused; }

hipError_t launch_gemv_i8(I8Mat w, const void *x, void *y, int type, int64_t M, int64_t K, int B,
                          hipStream_t st)
{
    I8StreamArgs p = args(w, {}, y, type, kSilu, M, K, B);
    p.x = x;
    return stream_floats<false>(p, st);
}

hipError_t launch_gated_gemv_i8(I8Mat gate, I8Mat up, const void *x, void *h, int type, int act,
                                int64_t I, int64_t H, int N, hipStream_t st)
{
    I8StreamArgs p = args(gate, up, h, type, act, I, H, N);
    p.x = x;
    return stream_floats<true>(p, st);
}

hipError_t launch_gemm_i8(I8Mat w, I8Mat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                          hipStream_t st)
{
    if (N > 16)
        return launch_i8_tiles(w, x, y, type, M, K, N, st);
    I8StreamArgs p = args(w, {}, y, type, kSilu, M, K, N);
    p.xc = x;
    return launch_stream<kCodes, false>(p, st);
}

hipError_t launch_gated_i8(I8Mat gate, I8Mat up, I8Mat x, void *h, int type, int act, int64_t I,
                           int64_t H, int64_t N, hipStream_t st)
{
    if (N > 16)
        return launch_gated_tiles(gate, up, x, h, type, act, I, H, N, st);
    I8StreamArgs p = args(gate, up, h, type, act, I, H, N);
    p.xc = x;
    return launch_stream<kCodes, true>(p, st);
}

hipError_t launch_ffn_i8(const I8FfnArgs &a, hipStream_t st)
{
    int8_t *xq = reinterpret_cast<int8_t *>(a.ws + a.off[0]), *hq = reinterpret_cast<int8_t *>(a.ws + a.off[3]);
    float *xs = reinterpret_cast<float *>(a.ws + a.off[1]), *hs = reinterpret_cast<float *>(a.ws + a.off[4]);
    void *h = a.ws + a.off[2];
    const int64_t ldx = (a.H + 15) / 16 * 16, ldh = (a.I + 15) / 16 * 16;
    hipError_t e;
    if (i8_fused(a.H, a.T)) {
        e = launch_gated_gemv_i8(a.gate, a.up, a.x, h, a.type, a.act, a.I, a.H, (int)a.T, st);
    } else {
        e = launch_quantize_i8(a.x, a.type, a.H, xq, ldx, xs, a.T, a.H, st);
        if (e == hipSuccess)
            e = launch_gated_i8(a.gate, a.up, {xq, ldx, xs}, h, a.type, a.act, a.I, a.H, a.T, st);
    }
    if (e != hipSuccess)
        return e;
    if (i8_fused(a.I, a.T))
        return launch_gemv_i8(a.down, h, a.out, a.type, a.H, a.I, (int)a.T, st);
    e = launch_quantize_i8(h, a.type, a.I, hq, ldh, hs, a.T, a.I, st);
    if (e == hipSuccess)
        e = launch_gemm_i8(a.down, {hq, ldh, hs}, a.out, a.type, a.H, a.I, a.T, st);
    return e;
}

} // namespace gq
