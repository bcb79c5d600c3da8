// mxfp4_skinny.hip -- products over MXFP4 weights with up to 16 activation rows, 16-bit
// or MXFP4, dense or of the experts of a mixture-of-experts layer.
//
// Y[n][r] = sum_k w[r][k] x[n][k].  The weights are read once and everything else is
// small: the latency and rate of the weight loads bound the kernel.  A workgroup owns R
// tiles of 16 weight rows; its waves split K in steps of 128, each issuing the loads of
// several steps and tiles before it uses them, and the workgroup joins their sums in wave
// order (a fixed order: results do not vary).
//
// In a step a lane takes one whole block (32 weights, 16 bytes, one scale) of weight row
// lane % 16: block lane / 16 of the step's four.  With 16-bit activations it converts the
// block to 16-bit weights, scale included, and feeds four 16x16x32 products, whose k order
// inside the step is permuted alike for both operands (product i takes columns 8i .. 8i+7
// of each of the four blocks).  With MXFP4 activations the block and its scale are the
// operand of one scaled 16x16x128 product.
#include "gq_internal.h"
#include "mxfp4_device.h"

namespace gq {

namespace {

enum { kActF16 = 1, kActBF16 = 2, kActMx = 3 };
enum { kDense = 0, kGateUp = 1, kDown = 2 };

struct SkinnyArgs {
    MxMat w, w2; // gate/up: gate, up
    const void *x;
    const uint8_t *xs; // scales of MXFP4 activations
    void *y;
    int ytype;
    int M, K, N;
    // grouped experts
    const int32_t *sorted, *tiles, *offsets;
    int max_tiles, topk, E;
    int64_t eq, es; // code and scale bytes per expert
    const float *wts;
    int weight_input;
};

// R tiles of 16 weight rows (gate/up: of each matrix).
template <int ACT, int MODE, int R, int NW>
__global__ __launch_bounds__(64 * NW) void mxfp4_skinny_kernel(SkinnyArgs p)
{
    constexpr int NMAT = MODE == kGateUp ? 2 : 1, NR = NMAT * R;
    constexpr int U = NR > 2 ? 8 / NR : 4; // steps whose loads are issued together
    constexpr int NX = ACT == kActMx ? 1 : 4;
    constexpr bool BF = ACT != kActF16;
    __shared__ float4_t red[NW][NR][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int M = p.M, K = p.K;
    const int m0 = blockIdx.x * (16 * R);
    int n0 = 0, nvalid = p.N, e = 0;
    if constexpr (MODE != kDense) {
        const int t = blockIdx.y;
        if (t >= p.offsets[p.E + 1])
            return;
        e = p.tiles[t];
        n0 = p.tiles[p.max_tiles + t];
        nvalid = min(p.offsets[e + 1] - n0, 16);
    }

    // rows past the last repeat it and are not stored; tile i of matrix m is NMAT i + m
    const uint8_t *qrow[NR], *srow[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const MxMat &w = i % NMAT ? p.w2 : p.w;
        const int64_t row = min(m0 + 16 * (i / NMAT) + c, M - 1);
        qrow[i] = w.q + e * p.eq + row * (K >> 1);
        srow[i] = w.s + e * p.es + row * (K >> 5);
    }
    const int nl = n0 + min(c, nvalid - 1);
    const int64_t xrow = MODE == kGateUp ? p.sorted[nl] / p.topk : nl;

    float4_t acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};

    const int nblk = K >> 5, steps = (nblk + 3) >> 2;
    for (int st0 = wave; st0 < steps; st0 += NW * U) {
        uint4 q[U][NR], xv[U][NX];
        uint32_t s[U][NR], sx[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = st0 + NW * u;
            if (st >= steps)
                break;
            // past the last block: that one again, taken as zeros of scale 1
            const int blk = min(4 * st + h, nblk - 1);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                q[u][i] = ld16(qrow[i] + 16 * blk);
                s[u][i] = srow[i][blk];
            }
            if constexpr (ACT == kActMx) {
                xv[u][0] = ld16(reinterpret_cast<const uint8_t *>(p.x) + xrow * (K >> 1) + 16 * blk);
                sx[u] = p.xs[xrow * nblk + blk];
            } else {
#pragma unroll
                for (int n = 0; n < NX; ++n)
                    xv[u][n] = ld16(reinterpret_cast<const uint16_t *>(p.x) + xrow * K + 32 * blk + 8 * n);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = st0 + NW * u;
            if (st >= steps)
                break;
            if (4 * st + h >= nblk) {
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    q[u][i] = make_uint4(0, 0, 0, 0);
                    s[u][i] = 127;
                }
#pragma unroll
                for (int n = 0; n < NX; ++n)
                    xv[u][n] = make_uint4(0, 0, 0, 0);
                sx[u] = 127;
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if constexpr (ACT == kActMx) {
                    acc[i] = mx_mfma16_fp4(q[u][i], s[u][i], xv[u][0], sx[u], acc[i]);
                } else {
                    const float sc = mx_scale(s[u][i]);
                    const uint32_t d[4] = {q[u][i].x, q[u][i].y, q[u][i].z, q[u][i].w};
#pragma unroll
                    for (int n = 0; n < NX; ++n)
                        acc[i] = mx_mfma16<BF>(mx_values8<BF>(d[n], sc), xv[u][n], acc[i]);
                }
            }
        }
    }

    // lane l holds rows 4 (l / 16) + 0..3 of a tile, of column l % 16
#pragma unroll
    for (int i = 0; i < NR; ++i)
        red[wave][i][lane] = acc[i];
    __syncthreads();
    for (int idx = tid; idx < R * 64; idx += 64 * NW) {
        const int i = idx >> 6, ln = idx & 63;
        const int n = ln & 15, m = m0 + 16 * i + 4 * (ln >> 4);
        if (n >= nvalid || m >= M)
            continue;
        float4_t a[NMAT];
#pragma unroll
        for (int t = 0; t < NMAT; ++t) {
            a[t] = red[0][NMAT * i + t][ln];
            for (int w = 1; w < NW; ++w)
                a[t] += red[w][NMAT * i + t][ln];
        }
        if constexpr (MODE == kGateUp) {
            const float pw = p.weight_input ? p.wts[p.sorted[n0 + n]] : 1.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[0][k] = silu(pw * a[0][k]) * (pw * a[1][k]);
        }
        mx_store4(p.y, (int64_t)(n0 + n) * M + m, p.ytype, a[0], M - m, (M & 3) == 0);
    }
}

template <int ACT, int MODE, int R, int NW>
hipError_t launch(const SkinnyArgs &p, unsigned gy, hipStream_t st)
{
    const dim3 grid((unsigned)((p.M + 16 * R - 1) / (16 * R)), gy);
    hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, R, NW>), grid, dim3(64 * NW), 0, st, p);
    return hipGetLastError();
}

// N <= 16
template <int ACT>
hipError_t launch_dense(MxMat w, const void *x, const uint8_t *xs, void *y, int ytype, int64_t M,
                        int64_t K, int64_t N, hipStream_t st)
{
    SkinnyArgs p{};
    p.w = w;
    p.x = x;
    p.xs = xs;
    p.y = y;
    p.ytype = ytype;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    // row tiles shared out among the CUs, up to four to a workgroup (the activations are
    // read once for them).  Measured, us at one, two and four: bfloat16 by 16 rows 4096 x
    // 4096 8.5, 10.3, 14.4; 14336 x 4096 24, 19, 15; 4096 x 14336 23, 30, 43; by 1 row 14336 x
    // 4096 14.0, 13.7, 13.1; MXFP4 by 16 rows 14336 x 4096 16.9, 13.6, 12.8
    const int64_t tiles = (M + 15) / 16, cus = device_cus();
    return tiles > 2 * cus ? launch<ACT, kDense, 4, 8>(p, 1, st)
           : tiles > cus   ? launch<ACT, kDense, 2, 8>(p, 1, st)
                           : launch<ACT, kDense, 1, 8>(p, 1, st);
}

// One expert product, weights streamed once per 16 tokens.  Two or four row tiles a
// workgroup of four waves: four once that still gives every CU one.  Measured, us for the
// layer of 64 experts, top-8, hidden 2048, intermediate 1024 with one tile (eight waves), two
// and four: 1 token 33, 24, 28; 4 tokens 67, 44, 43; 32 tokens -, 78, 71.
template <int MODE>
hipError_t launch_expert(const SkinnyArgs &p, bool bf16, int64_t A, hipStream_t st)
{
    const unsigned gy = (unsigned)p.max_tiles;
    const int64_t hit = A < p.E ? A : p.E; // experts with a token, at most
    if ((p.M + 63) / 64 * hit > device_cus())
        return bf16 ? launch<kActBF16, MODE, 4, 4>(p, gy, st) : launch<kActF16, MODE, 4, 4>(p, gy, st);
    return bf16 ? launch<kActBF16, MODE, 2, 4>(p, gy, st) : launch<kActF16, MODE, 2, 4>(p, gy, st);
}

hipError_t launch_moe_skinny(const MxMoeArgs &a, int max_tiles, hipStream_t st)
{
    SkinnyArgs p{};
    p.offsets = reinterpret_cast<const int32_t *>(a.ws + a.off[0]);
    p.sorted = reinterpret_cast<const int32_t *>(a.ws + a.off[1]);
    p.tiles = reinterpret_cast<const int32_t *>(a.ws + a.off[3]);
    p.max_tiles = max_tiles;
    p.topk = (int)a.topk;
    p.E = (int)a.E;
    p.wts = a.wts;
    p.weight_input = a.weight_input;
    p.eq = a.H * a.I / 2;
    p.es = a.H * a.I / 32;

    p.w = a.gate;
    p.w2 = a.up;
    p.x = a.x;
    p.y = a.ws + a.off[4];
    p.ytype = a.type;
    p.M = (int)a.I;
    p.K = (int)a.H;
    hipError_t err = launch_expert<kGateUp>(p, a.type == kBF16, a.T * a.topk, st);
    if (err != hipSuccess)
        return err;
    p.w = a.down;
    p.x = a.ws + a.off[4];
    p.y = a.ws + a.off[5];
    p.ytype = kF32;
    p.M = (int)a.H;
    p.K = (int)a.I;
    return launch_expert<kDown>(p, a.type == kBF16, a.T * a.topk, st);
}

} // namespace

hipError_t launch_gemm_mxfp4(MxMat w, const uint16_t *x, uint16_t *y, int type, int64_t M,
                             int64_t K, int64_t N, hipStream_t st)
{
    if (N > 16)
        return launch_gemm_tiles16(w, x, y, type, M, K, N, st);
    return type == kF16 ? launch_dense<kActF16>(w, x, nullptr, y, type, M, K, N, st)
                        : launch_dense<kActBF16>(w, x, nullptr, y, type, M, K, N, st);
}

hipError_t launch_gemm_mxfp4_mxfp4(MxMat w, MxMat x, void *y, int type, int64_t M, int64_t K,
                                   int64_t N, hipStream_t st)
{
    if (N > 16)
        return launch_mx_tiles(w, x, y, type, M, K, N, st);
    return launch_dense<kActMx>(w, x.q, x.s, y, type, M, K, N, st);
}

hipError_t launch_moe_mxfp4(const MxMoeArgs &a, hipStream_t st)
{
    const int64_t A = a.T * a.topk;
    const int tokens = moe_tile16_tokens(a.T, a.E, a.topk);
    const int bn = tokens ? tokens : 16;
    const int max_tiles = (int)((A + bn - 1) / bn + a.E);
    hipError_t err = launch_moe_group(a.ids, a.ws, a.off, A, a.E, bn, max_tiles, st);
    if (err != hipSuccess)
        return err;
    err = tokens ? launch_moe_tiles16(a, tokens, max_tiles, st) : launch_moe_skinny(a, max_tiles, st);
    if (err != hipSuccess)
        return err;
    return launch_moe_combine(reinterpret_cast<const float *>(a.ws + a.off[5]),
                              reinterpret_cast<const int32_t *>(a.ws + a.off[2]), a.wts, a.out,
                              a.type == kBF16, a.T, a.H, a.topk, a.weight_input != 0, st);
}

} // namespace gq
