// i8_stream.hip -- int8 products by up to 16 activation rows, weights streamed once.
//
// What bounds them is the weight stream: from HBM, 14336 x 4096 takes 14.3 us by one bfloat16 row
// (4.1 TB/s), gate and up of that size 24.5 (4.8 TB/s; a large copy 5.1), 4096 x 14336 14.4; by 16
// rows of codes 18.1 and 18.6.  Matrices of 4096 x 4096 and less take 7 us, most of it start, one
// latency of memory and the join.
//
// A workgroup takes tiles of 16 or 32 weight rows (of each matrix in the gate/up form); its W waves
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
constexpr int codes_bytes(int W, int B, int run) { return W * B * (run + 16); }

template <int SRC, bool PAIR, int W, int R, int LDSB>
__global__ __launch_bounds__(64 * W) void i8_stream_kernel(I8StreamArgs p)
{
    constexpr bool FLOATS = SRC != kCodes;
    constexpr int P = PAIR ? 2 : 1, TR = 16 * R; // matrices, weight rows of a tile
    // Steps loaded at once.  With the next tile's on their way while a tile is joined, few are
    // enough, and the registers go to more waves: gate and up of 14336 x 4096 by one row, from
    // HBM, 24.3 us with two, 25.3 with four, 30 with eight.
    constexpr int U = PAIR ? 2 : 4;
    __shared__ __attribute__((aligned(16))) uint8_t codes[FLOATS ? LDSB : 16];
    __shared__ uint32_t part[4][W];
    __shared__ float xscale[4];
    __shared__ int4v red[W][P][R][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int M = p.M, K = p.K, B = p.B;
    const int k0 = wave * p.run, cols = max(0, min(K - k0, p.run));
    const int steps = (cols + 63) >> 6; // of 64 columns
    const int lastc = ((K + 15) >> 4) - 1; // last chunk of 16 codes of a row
    const int pitch = p.run + 16;
    uint8_t *mine = codes + (FLOATS ? wave * B * pitch : 0);

    const int tiles = (M + TR - 1) / TR;
    const int xr = min(r, B - 1);
    const int8_t *xp = FLOATS ? nullptr : p.xc.q + xr * p.xc.ld;
    // weights (and codes of activations) of U steps from s0
    struct Batch {
        uint4 a[P][R][U], x[FLOATS ? 1 : U];
    };
    auto load = [&](int tile, int s0, Batch &t) {
        const int8_t *wp[P][R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t wr = min(TR * tile + 16 * j + r, M - 1);
            wp[0][j] = p.w.q + wr * p.w.ld;
            if constexpr (PAIR)
                wp[P - 1][j] = p.w2.q + wr * p.w2.ld;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u >= steps)
                break;
            const int ch = min((k0 >> 4) + 4 * (s0 + u) + q, lastc);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < R; ++j)
                    t.a[i][j][u] = ld16(wp[i][j] + 16 * ch);
            if constexpr (!FLOATS)
                t.x[u] = ld16(xp + 16 * ch);
        }
    };
    Batch now;
    if constexpr (FLOATS) {
        // All values, before the first weights, which then come while they are quantised: two
        // pieces of 512 columns of one or two rows, or one of up to four.
        const bool two = B <= 2;
        const int pieces = two ? (p.run > 512 ? 2 * B : 2 * B - 1) : B; // (the last may be empty)
        I8Load8<SRC> x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= pieces)
                break;
            const int b = two ? i >> 1 : i, c = 8 * lane + (two ? 512 * (i & 1) : 0);
            x[i].load(p.x, (int64_t)b * K + k0 + c, max(min(cols - c, 8), 0));
        }
        load(blockIdx.x, 0, now);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = i < pieces ? wave_max(x[i].max_bits()) : 0;
            if (lane == 0)
                part[i][wave] = m;
        }
        __syncthreads();
        uint32_t m = 0;
        if (lane < 4)
#pragma unroll
            for (int i = 0; i < W; ++i)
                m = max(m, part[lane][i]);
        if (two)
            m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
        const I8Row row(m); // lane i: piece i's
        if (wave == 0 && lane < 4)
            xscale[two ? lane >> 1 : lane] = row.s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= pieces)
                break;
            const I8Row rb(__shfl(row.top, i, 64), __shfl(row.s, i, 64), __shfl(row.r, i, 64));
            const int b = two ? i >> 1 : i, c = 8 * lane + (two ? 512 * (i & 1) : 0);
            if (c < 64 * steps)
                *reinterpret_cast<uint2 *>(mine + b * pitch + c) = i8_codes8(x[i], rb);
        }
        lds_wave_order();
    } else {
        load(blockIdx.x, 0, now);
    }

    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int m0 = TR * tile;
        int4v acc[P][R];
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < R; ++j)
                acc[i][j] = int4v{0, 0, 0, 0};
        for (int s0 = 0; s0 < steps; s0 += U) {
            if (s0 > 0)
                load(tile, s0, now);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s0 + u >= steps)
                    break;
                uint4 xv;
                if constexpr (FLOATS) {
                    xv = ld16(mine + xr * pitch + 64 * (s0 + u) + 16 * q);
                } else {
                    xv = now.x[u];
                    const int left = K - (k0 + 64 * (s0 + u) + 16 * q); // codes past K are zero
                    if (__builtin_expect(left < 16, 0)) {
                        uint32_t t[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int n = min(max(left - 4 * j, 0), 4);
                            t[j] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
                        }
                        xv = make_uint4(t[0], t[1], t[2], t[3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int j = 0; j < R; ++j)
                        acc[i][j] = mfma16_i8(now.a[i][j][u], xv, acc[i][j]);
            }
        }
        if (tile + (int)gridDim.x < tiles) // while this tile's sums are joined
            load(tile + gridDim.x, 0, now);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < R; ++j)
                red[wave][i][j][lane] = acc[i][j];
        __syncthreads();
        // output t: weight row t % 16 of group t / 256, activation row t / 16 % 16; in the
        // accumulators lane 16 (row / 4) + activation row, element row % 4
        const int m = tid & 15, b = tid >> 4 & 15, g = tid >> 8, from = 16 * (m >> 2) + b;
        const int row = m0 + 16 * g + m;
        static_assert(W * 64 >= 256 * R, "a thread for every output");
        if (g < R && b < B && row < M) {
            int sum[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sum[i] = 0;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    sum[i] += red[j][i][g][from][m & 3];
            }
            const float xs = FLOATS ? xscale[b] : p.xc.s[b];
            float v = i8_scaled(sum[0], p.w.s[row], xs);
            if constexpr (PAIR) {
                const float u = i8_scaled(sum[P - 1], p.w2.s[row], xs);
                v = p.type == kF32 ? gated_value<true>(v, u, p.act) : gated_value<false>(v, u, p.act);
            }
            i8_store(p.y, (int64_t)b * M + row, p.type, v);
        }
        __syncthreads();
    }
}

// Sixteen waves where K is long enough to keep eight waiting for their weights.
constexpr int64_t kLongK = 8192;

template <int SRC, bool PAIR, int W, int R>
hipError_t launch_waves(I8StreamArgs p, hipStream_t st)
{
    // codes of up to four rows: see i8_fused
    constexpr int LDSB = SRC == kCodes ? 16 : std::max(codes_bytes(W, 4, 512), codes_bytes(W, 1, 1024));
    p.run = ((p.K + W - 1) / W + 63) / 64 * 64;
    if (SRC != kCodes && (!i8_fused(p.K, p.B) || codes_bytes(W, p.B, p.run) > LDSB))
        return hipErrorInvalidValue;
    // As many workgroups as the CUs hold at once, which quantise once for all of their tiles
    // (14336 x 4096, batch 4: 17 us, with a workgroup a tile 24), equally many each (gate and up
    // of 14336 rows, 896 tiles, on 448 workgroups instead of 512: 27.6 us, 30.3).
    const int64_t tiles = ((int64_t)p.M + 16 * R - 1) / (16 * R);
    const int64_t most = (W == 8 ? 2 : 1) * device_cus(), each = (tiles + most - 1) / most;
    const int64_t grid = (tiles + each - 1) / each;
    hipLaunchKernelGGL((i8_stream_kernel<SRC, PAIR, W, R, LDSB>), dim3((unsigned)grid), dim3(64 * W), 0, st,
                       p);
    return hipGetLastError();
}

template <int SRC, bool PAIR>
hipError_t launch_stream(const I8StreamArgs &p, hipStream_t st)
{
    // Codes of activations are read once a tile: tiles of 32 rows where they fill the device
    // (14336 x 4096 by 16 rows 20.7 -> 18.1 us).
    if constexpr (SRC == kCodes)
        if (p.M >= 32 * device_cus())
            return p.K > kLongK ? launch_waves<SRC, PAIR, 16, 2>(p, st) : launch_waves<SRC, PAIR, 8, 2>(p, st);
    return p.K > kLongK ? launch_waves<SRC, PAIR, 16, 1>(p, st) : launch_waves<SRC, PAIR, 8, 1>(p, st);
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

// What four pieces of 512 columns for each of eight (one row: sixteen) waves hold.  More rows
// are better quantised once: four rows of 4096 take 17 us against 14336 weight rows, 18.6 with
// codes from a launch before, which sixteen rows of 1024, one after another, took too.
bool i8_fused(int64_t K, int64_t B)
{
    return B == 1 ? K <= 2 * kLongK : B == 2 ? K <= kLongK : B <= 4 && K <= kLongK / 2;
}

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
