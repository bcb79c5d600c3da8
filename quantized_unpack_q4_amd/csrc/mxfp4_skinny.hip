// mxfp4_skinny.hip -- products over MXFP4 weights with few activation rows.
//
// Y[n][r] = sum_k w[r][k] x[n][k].  The weights are streamed once per group of up
// to 64 activation rows and everything else is small, so the kernel is bound by
// the latency and rate of the weight loads: a workgroup owns 16 weight rows, its
// waves split K in steps of 128, and every wave keeps its own accumulators, which
// the workgroup adds in wave order (a fixed order: results do not vary).
//
// In a step a lane takes one whole block (32 weights, 16 bytes, one scale) of
// weight row lane % 16: block lane / 16 of the step's four.  With 16-bit
// activations it converts the block to 16-bit weights, scale included,
// and feeds four 16x16x32 products, whose k order inside the step is permuted
// alike for both operands (product i takes columns 8i .. 8i+7 of each of the four
// blocks).  With MXFP4 activations the block and its scale are the operand of one
// scaled 16x16x128 product.
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

template <int ACT, int MODE, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void mxfp4_skinny_kernel(SkinnyArgs p)
{
    constexpr int NMAT = MODE == kGateUp ? 2 : 1;
    constexpr bool BF = ACT != kActF16;
    __shared__ float4_t red[NW][NMAT * NT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int M = p.M, K = p.K;
    const int m0 = blockIdx.x * 16;
    int n0, nvalid, e = 0;
    if constexpr (MODE == kDense) {
        n0 = blockIdx.y * (16 * NT);
        nvalid = p.N - n0;
    } else {
        const int t = blockIdx.y;
        if (t >= p.offsets[p.E + 1])
            return;
        e = p.tiles[t];
        n0 = p.tiles[p.max_tiles + t];
        nvalid = p.offsets[e + 1] - n0;
    }
    nvalid = nvalid < 16 * NT ? nvalid : 16 * NT;

    // rows past the last repeat it and are not stored
    const int64_t row = m0 + c < M ? m0 + c : M - 1;
    const uint8_t *qrow[NMAT], *srow[NMAT];
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
        const MxMat &w = m ? p.w2 : p.w;
        qrow[m] = w.q + e * p.eq + row * (K >> 1);
        srow[m] = w.s + e * p.es + row * (K >> 5);
    }
    int64_t xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int nl = 16 * j + c < nvalid ? 16 * j + c : nvalid - 1;
        xrow[j] = MODE == kGateUp ? p.sorted[n0 + nl] / p.topk : n0 + nl;
    }

    float4_t acc[NMAT][NT];
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[m][j] = float4_t{0.f, 0.f, 0.f, 0.f};

    const int nblk = K >> 5, steps = (nblk + 3) >> 2;
    for (int st = wave; st < steps; st += NW) {
        const bool ok = 4 * st + h < nblk; // past the last block: zeros of scale 1
        const int blk = ok ? 4 * st + h : nblk - 1;
        uint4 q[NMAT];
        uint32_t s[NMAT];
#pragma unroll
        for (int m = 0; m < NMAT; ++m) {
            q[m] = ld16(qrow[m] + 16 * (int64_t)blk);
            s[m] = srow[m][blk];
            if (!ok) {
                q[m] = make_uint4(0, 0, 0, 0);
                s[m] = 127;
            }
        }
        if constexpr (ACT == kActMx) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint4 xq = ld16(reinterpret_cast<const uint8_t *>(p.x) + xrow[j] * (K >> 1) +
                                16 * (int64_t)blk);
                uint32_t sx = p.xs[xrow[j] * (K >> 5) + blk];
                if (!ok) {
                    xq = make_uint4(0, 0, 0, 0);
                    sx = 127;
                }
#pragma unroll
                for (int m = 0; m < NMAT; ++m)
                    acc[m][j] = mx_mfma16_fp4(q[m], s[m], xq, sx, acc[m][j]);
            }
        } else {
            uint4 w[NMAT][4];
#pragma unroll
            for (int m = 0; m < NMAT; ++m) {
                const float sc = mx_scale(s[m]);
                const uint32_t d[4] = {q[m].x, q[m].y, q[m].z, q[m].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[m][i] = mx_values8<BF>(d[i], sc);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int64_t xi = xrow[j] * K + 32 * (int64_t)blk;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 xv = ld16(reinterpret_cast<const uint16_t *>(p.x) + xi + 8 * i);
                    if (!ok)
                        xv = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int m = 0; m < NMAT; ++m)
                        acc[m][j] = mx_mfma16<BF>(w[m][i], xv, acc[m][j]);
                }
            }
        }
    }

    // lane l holds rows m0 + 4 (l / 16) + 0..3 of column l % 16
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            red[wave][m * NT + j][lane] = acc[m][j];
    __syncthreads();
    for (int idx = tid; idx < NT * 64; idx += 64 * NW) {
        const int j = idx >> 6, ln = idx & 63;
        const int n = 16 * j + (ln & 15), m = m0 + 4 * (ln >> 4);
        if (n >= nvalid || m >= M)
            continue;
        float4_t a[NMAT];
#pragma unroll
        for (int t = 0; t < NMAT; ++t) {
            a[t] = red[0][t * NT + j][ln];
            for (int w = 1; w < NW; ++w)
                a[t] += red[w][t * NT + j][ln];
        }
        if constexpr (MODE == kGateUp) {
            const float pw = p.weight_input ? p.wts[p.sorted[n0 + n]] : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[0][i] = silu(pw * a[0][i]) * (pw * a[1][i]);
        }
        mx_store4(p.y, (int64_t)(n0 + n) * M + m, p.ytype, a[0], M - m, (M & 3) == 0);
    }
}

template <int ACT, int MODE>
hipError_t launch(const SkinnyArgs &p, int nt, unsigned gy, hipStream_t st)
{
    const dim3 grid((unsigned)((p.M + 15) / 16), gy);
    if (nt == 1)
        hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, 1, 8>), grid, dim3(512), 0, st, p);
    else if (nt == 2)
        hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, 2, 8>), grid, dim3(512), 0, st, p);
    else
        hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, 4, 8>), grid, dim3(512), 0, st, p);
    return hipGetLastError();
}

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
    const int nt = N <= 16 ? 1 : N <= 32 ? 2 : 4;
    return launch<ACT, kDense>(p, nt, (unsigned)((N + 16 * nt - 1) / (16 * nt)), st);
}

} // namespace

hipError_t launch_gemm_mxfp4(MxMat w, const uint16_t *x, uint16_t *y, int type, int64_t M,
                             int64_t K, int64_t N, hipStream_t st)
{
    if (N > 16 && tiles16_fit(K))
        return launch_gemm_tiles16(w, x, y, type, M, K, N, st);
    return type == kF16 ? launch_dense<kActF16>(w, x, nullptr, y, type, M, K, N, st)
                        : launch_dense<kActBF16>(w, x, nullptr, y, type, M, K, N, st);
}

hipError_t launch_gemm_mxfp4_mxfp4(MxMat w, MxMat x, void *y, int type, int64_t M, int64_t K,
                                   int64_t N, hipStream_t st)
{
    if (N > 16 && mx_tiles_fit(K))
        return launch_mx_tiles(w, x, y, type, M, K, N, st);
    return launch_dense<kActMx>(w, x.q, x.s, y, type, M, K, N, st);
}

// Gate/up and down of the experts, weights streamed once per 16 nt tokens.
static hipError_t launch_moe_skinny16(const MxMoeArgs &a, int nt, int max_tiles, hipStream_t st)
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
    hipError_t err = a.type == kF16 ? launch<kActF16, kGateUp>(p, nt, (unsigned)max_tiles, st)
                                    : launch<kActBF16, kGateUp>(p, nt, (unsigned)max_tiles, st);
    if (err != hipSuccess)
        return err;
    p.w = a.down;
    p.x = a.ws + a.off[4];
    p.y = a.ws + a.off[5];
    p.ytype = kF32;
    p.M = (int)a.H;
    p.K = (int)a.I;
    return a.type == kF16 ? launch<kActF16, kDown>(p, nt, (unsigned)max_tiles, st)
                          : launch<kActBF16, kDown>(p, nt, (unsigned)max_tiles, st);
}

hipError_t launch_moe_mxfp4(const MxMoeArgs &a, hipStream_t st)
{
    const int64_t A = a.T * a.topk;
    const int tokens = moe_tile16_tokens(a.T, a.H, a.I, a.E, a.topk);
    // (activations past the tiles' 32-bit offsets: groups of 64 tokens)
    const int nt = A / a.E < 2 ? 1 : 4, bn = tokens ? tokens : 16 * nt;
    const int max_tiles = (int)((A + bn - 1) / bn + a.E);
    hipError_t err = launch_moe_group(a.ids, a.ws, a.off, A, a.E, bn, max_tiles, st);
    if (err != hipSuccess)
        return err;
    err = tokens ? launch_moe_tiles16(a, tokens, max_tiles, st) : launch_moe_skinny16(a, nt, max_tiles, st);
    if (err != hipSuccess)
        return err;
    return launch_moe_combine(reinterpret_cast<const float *>(a.ws + a.off[5]),
                              reinterpret_cast<const int32_t *>(a.ws + a.off[2]), a.wts, a.out,
                              a.type == kBF16, a.T, a.H, a.topk, a.weight_input != 0, st);
}

} // namespace gq
