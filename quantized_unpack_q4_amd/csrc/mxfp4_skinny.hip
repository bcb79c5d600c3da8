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

// R tiles of 16 weight rows (gate/up: of each matrix); a wave takes Q steps of K at a time.
template <int ACT, int MODE, int R, int NW, int Q>
__global__ __launch_bounds__(64 * NW) void mxfp4_skinny_kernel(SkinnyArgs p)
{
    constexpr int NMAT = MODE == kGateUp ? 2 : 1, NR = NMAT * R;
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
    const int nblk = K >> 5;
    const uint8_t *qrow[NR], *srow[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const MxMat &w = i % NMAT ? p.w2 : p.w;
        const int64_t row = min(m0 + 16 * (i / NMAT) + c, M - 1);
        qrow[i] = w.q + e * p.eq + row * (K >> 1);
        srow[i] = w.s + e * p.es + row * nblk;
    }
    const int nl = n0 + min(c, nvalid - 1);
    const int64_t xrow = MODE == kGateUp ? p.sorted[nl] / p.topk : nl;

    struct Unit {
        uint4 q[Q][NR], x[Q][NX];
        MxScales<Q> s[NR], sx;
    };
    auto load = [&](int un, Unit &b) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            // past the last block: that one again, taken as zeros
            const int blk = min(4 * (Q * un + u) + h, nblk - 1);
#pragma unroll
            for (int i = 0; i < NR; ++i)
                b.q[u][i] = ld16(qrow[i] + 16 * blk);
            if constexpr (ACT == kActMx) {
                b.x[u][0] = ld16(reinterpret_cast<const uint8_t *>(p.x) + xrow * (K >> 1) + 16 * blk);
            } else {
#pragma unroll
                for (int n = 0; n < NX; ++n)
                    b.x[u][n] = ld16(reinterpret_cast<const uint16_t *>(p.x) + xrow * K + 32 * blk + 8 * n);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
            b.s[i].load(srow[i], 4 * Q * un, nblk);
        if constexpr (ACT == kActMx)
            b.sx.load(p.xs + xrow * nblk, 4 * Q * un, nblk);
    };
    float4_t acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int un, Unit &b) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            const bool none = 4 * (Q * un + u) + h >= nblk;
            if (none) {
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    b.q[u][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int n = 0; n < NX; ++n)
                    b.x[u][n] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const uint32_t s = b.s[i].w[u] >> (8 * h); // (its low byte)
                if constexpr (ACT == kActMx) {
                    acc[i] = mx_mfma16_fp4(b.q[u][i], s, b.x[u][0], b.sx.w[u] >> (8 * h), acc[i]);
                } else {
                    const float sc = mx_scale(s & 255u);
                    const uint32_t d[4] = {b.q[u][i].x, b.q[u][i].y, b.q[u][i].z, b.q[u][i].w};
#pragma unroll
                    for (int n = 0; n < NX; ++n)
                        acc[i] = mx_mfma16<BF>(mx_values8<BF>(d[n], sc), b.x[u][n], acc[i]);
                }
            }
        }
    };

    const int units = ((nblk + 3) / 4 + Q - 1) / Q;
    if constexpr (Q * (NR + NX) <= 20) { // registers for the next unit's loads too
        Unit b0, b1;
        int un = wave;
        if (un < units)
            load(un, b0);
        for (; un < units; un += 2 * NW) {
            if (un + NW < units)
                load(un + NW, b1);
            compute(un, b0);
            if (un + NW < units) {
                if (un + 2 * NW < units)
                    load(un + 2 * NW, b0);
                compute(un + NW, b1);
            }
        }
    } else {
        for (int un = wave; un < units; un += NW) {
            Unit b;
            load(un, b);
            compute(un, b);
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
        if constexpr (MODE == kGateUp) { // (h goes to 16 bits: see mxfp4_tiles16.hip)
            const float pw = p.weight_input ? p.wts[p.sorted[n0 + n]] : 1.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[0][k] = silu(pw * a[0][k]) * (pw * a[1][k]);
        }
        mx_store4(p.y, (int64_t)(n0 + n) * M + m, p.ytype, a[0], M - m, (M & 3) == 0);
    }
}

// As many steps at a time, up to QMAX, as leave every wave some.
template <int ACT, int MODE, int R, int NW, int QMAX>
hipError_t launch(const SkinnyArgs &p, unsigned gy, hipStream_t st)
{
    const dim3 grid((unsigned)((p.M + 16 * R - 1) / (16 * R)), gy), block(64 * NW);
    const int steps = (p.K + 127) / 128;
    if constexpr (QMAX >= 4) {
        if (steps >= 4 * NW) {
            hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, R, NW, 4>), grid, block, 0, st, p);
            return hipGetLastError();
        }
    }
    if (steps >= 2 * NW)
        hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, R, NW, 2>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((mxfp4_skinny_kernel<ACT, MODE, R, NW, 1>), grid, block, 0, st, p);
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
    // Row tiles shared out among the CUs, up to four to a workgroup (the activations are
    // read once for them).  Measured, us at one, two and four: bfloat16 by 16 rows 4096 x
    // 4096 7.8, 9.2, 12.2; 14336 x 4096 26, 17, 13.4; 4096 x 14336 21, 26, 36; by 1 row 14336 x
    // 4096 15.7, 11.6, 11.0; MXFP4 by 16 rows 14336 x 4096 12.6, 12.4, 10.6.  Four, two and
    // one step at a time: bfloat16 by 1 row 14336 x 14336 29, 31, 37.
    const int64_t tiles = (M + 15) / 16, cus = device_cus();
    return tiles > 2 * cus ? launch<ACT, kDense, 4, 8, 4>(p, 1, st)
           : tiles > cus   ? launch<ACT, kDense, 2, 8, 4>(p, 1, st)
                           : launch<ACT, kDense, 1, 8, 4>(p, 1, st);
}

// One expert product, weights streamed once per 16 tokens: two row tiles a workgroup of four
// waves, up to two steps at a time.  Measured, us for the layer of 64 experts, top-8, hidden
// 2048, intermediate 1024, weights from HBM: 1 token 22.5 (one tile 22.9, four 26), 4 tokens
// 41 (37, 41), 16 tokens 68 (67, 70), 64 tokens 78 (85, 75); with eight waves 26, 54, 93, 109.
template <int MODE>
hipError_t launch_expert(const SkinnyArgs &p, bool bf16, hipStream_t st)
{
    const unsigned gy = (unsigned)p.max_tiles;
    return bf16 ? launch<kActBF16, MODE, 2, 4, 2>(p, gy, st) : launch<kActF16, MODE, 2, 4, 2>(p, gy, st);
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
    hipError_t err = launch_expert<kGateUp>(p, a.type == kBF16, st);
    if (err != hipSuccess)
        return err;
    p.w = a.down;
    p.x = a.ws + a.off[4];
    p.y = a.ws + a.off[5];
    p.ytype = kF32;
    p.M = (int)a.H;
    p.K = (int)a.I;
    return launch_expert<kDown>(p, a.type == kBF16, st);
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
