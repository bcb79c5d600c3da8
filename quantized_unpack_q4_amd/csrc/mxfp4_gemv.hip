// mxfp4_gemv.hip -- MXFP4 weights times 1 to 16 binary32 activation rows.
//
// y[b][r] = sum_k w[r][k] x[b][k].  The weights are read once and everything else is
// small: latency and the rate of the weight loads bound the kernel, so a lane loads
// whole blocks (16 bytes of codes, one scale) several steps ahead, the first before
// anything else.
//
// Binary32 activations are split into three bfloat16 parts, x = a + 2^-7 b + 2^-15 c exactly
// (8 + 8 + 8 significant bits, each part cut toward zero from what is left; of subnormal
// activations the last bit, 2^-149, may be lost), and an MXFP4 weight is a bfloat16 number
// exactly (s <= 252), so the products are exact and only the binary32 sums of the matrix
// cores round.  An infinite or NaN activation leaves a NaN in the second part (infinity
// minus infinity), so its row's results are NaN.  The factors keep the parts of activations
// below 2^-109 above the last place of bfloat16, 2^-133 (unscaled, 1e-36 is off by 2e-5 of
// itself and 1e-40 by 4 %), and no part above x itself, so that the parts' sums overflow
// only where the whole may; they cost a sum for each part and 6 to 12 % of the time at batch 6
// to 16 (4096 x 14336 batch 16 26.4 -> 28.6 us, weights from HBM), nothing up to five rows,
// whose parts are columns with sums of their own.
//
// In a step of 128 columns lane (c, h) takes block h of weight row c, converted with its
// scale, and feeds four 16x16x32 products whose k order is permuted alike for both operands
// (product i takes columns 8i .. 8i+7 of the step's four blocks).  A workgroup of NW waves
// owns RT tiles of 16 weight rows; its waves take units of Q consecutive steps, every NW-th,
// and join their sums through LDS in wave order.
//
// Up to five activation rows the three parts of a row are three columns of one product
// (column 3b + p), joined at the end: the parts of a chunk of x (1024 NW values, all rows of
// it) lie in LDS as rows of bfloat16, split once for the workgroup.  Above five rows each
// part has a product of its own and every wave splits what it needs itself.
#include "gq_internal.h"
#include "mxfp4_device.h"

namespace gq {

namespace {

// A workgroup of NW waves stages 1024 NW activations at a time, four each four values a
// thread: this many columns, whole steps of 128.  Their parts take 3 B rows of two bytes a
// column and 16 more, at most x_bytes(NW).
__host__ __device__ constexpr int chunk_columns(int NW, int B) { return 1024 * NW / B / 128 * 128; }
constexpr int x_bytes(int NW) { return 6 * 1024 * NW + 15 * 16; }

// What the second and third part are worth.
constexpr float kPart2 = 0x1p-7f, kPart3 = 0x1p-15f;

// The three bfloat16 parts of four binary32 values, packed.
__device__ __forceinline__ void split3(const float4 v, uint2 &a, uint2 &b, uint2 &c)
{
    const float x[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) { // (a rest is below the last place of the part before it)
        hi[j] = __builtin_bit_cast(uint32_t, x[j]);
        const float r = (x[j] - __builtin_bit_cast(float, hi[j] & 0xffff0000u)) * 0x1p7f;
        mid[j] = __builtin_bit_cast(uint32_t, r);
        lo[j] = __builtin_bit_cast(uint32_t, (r - __builtin_bit_cast(float, mid[j] & 0xffff0000u)) * 0x1p8f);
    }
    // the upper halves of a pair
    a = make_uint2(__builtin_amdgcn_perm(hi[1], hi[0], 0x07060302u),
                   __builtin_amdgcn_perm(hi[3], hi[2], 0x07060302u));
    b = make_uint2(__builtin_amdgcn_perm(mid[1], mid[0], 0x07060302u),
                   __builtin_amdgcn_perm(mid[3], mid[2], 0x07060302u));
    c = make_uint2(__builtin_amdgcn_perm(lo[1], lo[0], 0x07060302u),
                   __builtin_amdgcn_perm(lo[3], lo[2], 0x07060302u));
}

// The sum of the parts' products.
__device__ __forceinline__ float join3(float a, float b, float c)
{
    return fmaf(b, kPart2, c * kPart3) + a;
}

// 1 <= B <= 5.
template <int RT, int NW, int Q>
__global__ __launch_bounds__(64 * NW) void mxfp4_gemv_kernel(MxMat w, const float *__restrict__ x,
                                                             float *__restrict__ y, int M, int K,
                                                             int B)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[x_bytes(NW)];
    static_assert(NW * RT * 1024 <= x_bytes(NW), "sums fit");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int m0 = blockIdx.x * (16 * RT);
    const int nblk = K >> 5, steps = (nblk + 3) >> 2;
    const int kc = chunk_columns(NW, B), cs = kc >> 7, upc = (cs + Q * NW - 1) / (Q * NW);
    const int chunks = (steps + cs - 1) / cs, total = chunks * upc;
    const int xstride = 2 * kc + 16;

    const uint8_t *qrow[RT], *srow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) { // rows past the last repeat it and are not stored
        const int64_t row = min(m0 + 16 * t + c, M - 1);
        qrow[t] = w.q + row * (K >> 1);
        srow[t] = w.s + row * nblk;
    }
    // this wave's units: upc in every chunk, at first (in the chunk) = its number and then
    // every NW-th; not all of their steps exist
    struct Walk {
        int n = 0, first = 0; // units taken in this chunk, the chunk's first step
    };
    auto next = [&](Walk &k) {
        if (++k.n == upc) {
            k.n = 0;
            k.first += cs;
        }
    };
    // step u of the unit, in the chunk; -1: none
    auto step_of = [&](const Walk &k, int u) {
        const int in = Q * (wave + NW * k.n) + u;
        return in < cs && k.first + in < steps ? in : -1;
    };
    Walk ahead, now;
    struct Unit {
        uint4 q[Q][RT];
        MxScales<Q> s[RT];
    };
    auto load = [&](Unit &g) {
        const int b0 = 4 * (ahead.first + Q * (wave + NW * ahead.n));
        if (step_of(ahead, 0) >= 0) {
#pragma unroll
            for (int u = 0; u < Q; ++u) {
                // past the last block: that one again, taken as zeros
                const int blk = min(b0 + 4 * u + h, nblk - 1);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    g.q[u][t] = ld16(qrow[t] + 16 * blk);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
                g.s[t].load(srow[t], b0, nblk);
        }
        next(ahead);
    };
    float4 xr[4];
    auto load_x = [&](int ch) {
        const int kq = kc >> 2; // float4 of a row in the chunk
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int f = tid + 64 * NW * j, b = f / kq;
            const int64_t k = (int64_t)ch * kc + 4 * (f - b * kq);
            xr[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b < B && k < K)
                xr[j] = ldf4(x + (int64_t)b * K + k);
        }
    };
    auto stage_x = [&]() {
        const int kq = kc >> 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int f = tid + 64 * NW * j, b = f / kq;
            if (b >= B)
                continue;
            uint2 p0, p1, p2;
            split3(xr[j], p0, p1, p2);
            uint8_t *d = lds + 3 * b * xstride + 8 * (f - b * kq);
            *reinterpret_cast<uint2 *>(d) = p0;
            *reinterpret_cast<uint2 *>(d + xstride) = p1;
            *reinterpret_cast<uint2 *>(d + 2 * xstride) = p2;
        }
    };

    float4_t acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
        acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    // columns past the last repeat it and are not stored
    const int xrow = min(c, 3 * B - 1);
    auto compute = [&](Unit &g) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            const int in = step_of(now, u);
            if (in < 0) // the whole wave
                break;
            const bool ok = 4 * (now.first + in) + h < nblk;
            const uint8_t *xp = lds + xrow * xstride + 64 * h + 256 * in;
            float sc[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                sc[t] = mx_scale((g.s[t].w[u] >> (8 * h)) & 255u);
                if (!ok)
                    g.q[u][t] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint4 xv = ld16(xp + 16 * n);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint4 &q = g.q[u][t];
                    const uint4 wv = mx_values8<true>(n == 0 ? q.x : n == 1 ? q.y : n == 2 ? q.z : q.w, sc[t]);
                    acc[t] = mx_mfma16<true>(wv, xv, acc[t]);
                }
            }
        }
        next(now);
    };

    Unit g0, g1;
    load(g0);
    load_x(0);
    int chunk = 0;
    auto half = [&](Unit &cur, Unit &nxt) {
        load(nxt);
        if (now.n == 0) { // the first unit of a chunk, for all waves alike
            if (chunk > 0)
                __syncthreads(); // the chunk before has been read
            stage_x();
            if (++chunk < chunks)
                load_x(chunk);
            __syncthreads();
        }
        compute(cur);
    };
    for (int i = 0; i < total; i += 2) {
        half(g0, g1);
        if (i + 1 < total)
            half(g1, g0);
    }

    // lane l of a wave holds rows 4 (l / 16) + 0..3 of column l % 16
    __syncthreads();
    float4_t *red = reinterpret_cast<float4_t *>(lds);
#pragma unroll
    for (int t = 0; t < RT; ++t)
        red[(wave * RT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int o = tid; o < RT * 16 * B; o += 64 * NW) {
        const int r = o % (16 * RT), b = o / (16 * RT);
        const int t = r >> 4, m = r & 15;
        if (m0 + r >= M)
            continue;
        const float *f = reinterpret_cast<const float *>(lds) + 256 * t + 64 * (m >> 2) + (m & 3);
        float sum = 0.f;
        for (int v = 0; v < NW; ++v) {
            const float *fv = f + v * RT * 256;
            sum += join3(fv[4 * (3 * b)], fv[4 * (3 * b + 1)], fv[4 * (3 * b + 2)]);
        }
        y[(int64_t)b * M + m0 + r] = sum;
    }
}

// More than five activation rows: a wave splits what it needs of x itself.  In a unit of two
// steps it loads 256 columns of the B rows (1 KB of a row per load), turns them in LDS of its
// own (rows padded by 16 bytes, so that the 16 rows of a read phase meet 16 distinct bank
// groups) and splits the eight values a lane feeds to a product: no barriers, and the loads
// of the next unit are in flight meanwhile.
template <int RT, int NW>
__global__ __launch_bounds__(64 * NW) void mxfp4_gemv_wide_kernel(MxMat w, const float *__restrict__ x,
                                                                  float *__restrict__ y, int M,
                                                                  int K, int B)
{
    constexpr int Q = 2, kRow = 1024 + 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[NW][16 * kRow];
    static_assert(RT * 1024 <= 16 * kRow, "sums fit");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int m0 = blockIdx.x * (16 * RT);
    const int nblk = K >> 5, units = (nblk + 4 * Q - 1) / (4 * Q);

    const uint8_t *qrow[RT], *srow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) { // rows past the last repeat it and are not stored
        const int64_t row = min(m0 + 16 * t + c, M - 1);
        qrow[t] = w.q + row * (K >> 1);
        srow[t] = w.s + row * nblk;
    }
    struct Unit {
        uint4 q[Q][RT];
        MxScales<Q> s[RT];
    };
    auto load = [&](int un, Unit &g) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            // past the last block: that one again, taken as zeros
            const int blk = min(4 * (Q * un + u) + h, nblk - 1);
#pragma unroll
            for (int t = 0; t < RT; ++t)
                g.q[u][t] = ld16(qrow[t] + 16 * blk);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
            g.s[t].load(srow[t], 4 * Q * un, nblk);
    };
    float4 xr[16];
    auto load_x = [&](int un) {
        const int k = 256 * un + 4 * lane;
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (b < B)
                xr[b] = k < K ? ldf4(x + (int64_t)b * K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto turn_x = [&]() {
        uint8_t *d = lds[wave] + 16 * lane;
        lds_wave_order(); // after the reads of the unit before
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (b < B)
                *reinterpret_cast<float4 *>(d + b * kRow) = xr[b];
        lds_wave_order();
    };

    float4_t acc[RT], acc2[RT], acc3[RT]; // of the three parts
#pragma unroll
    for (int t = 0; t < RT; ++t)
        acc[t] = acc2[t] = acc3[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    // columns past the last repeat it and are not stored
    const uint8_t *xp = lds[wave] + min(c, B - 1) * kRow + 128 * h;
    auto compute = [&](int un, Unit &g) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            const bool ok = 4 * (Q * un + u) + h < nblk;
            float sc[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                sc[t] = mx_scale((g.s[t].w[u] >> (8 * h)) & 255u);
                if (!ok)
                    g.q[u][t] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float *v = reinterpret_cast<const float *>(xp + 512 * u + 32 * n);
                uint2 a0, b0, c0, a1, b1, c1;
                split3(ldf4(v), a0, b0, c0);
                split3(ldf4(v + 4), a1, b1, c1);
                const uint4 xa = make_uint4(a0.x, a0.y, a1.x, a1.y);
                const uint4 xb = make_uint4(b0.x, b0.y, b1.x, b1.y);
                const uint4 xc = make_uint4(c0.x, c0.y, c1.x, c1.y);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint4 &q = g.q[u][t];
                    const uint4 wv = mx_values8<true>(n == 0 ? q.x : n == 1 ? q.y : n == 2 ? q.z : q.w, sc[t]);
                    acc3[t] = mx_mfma16<true>(wv, xc, acc3[t]);
                    acc2[t] = mx_mfma16<true>(wv, xb, acc2[t]);
                    acc[t] = mx_mfma16<true>(wv, xa, acc[t]);
                }
            }
        }
    };

    Unit g0, g1;
    int un = wave;
    if (un < units) {
        load(un, g0);
        load_x(un);
    }
    auto half = [&](Unit &cur, Unit &nxt) {
        turn_x();
        if (un + NW < units) {
            load(un + NW, nxt);
            load_x(un + NW);
        }
        compute(un, cur);
        un += NW;
    };
    while (un < units) {
        half(g0, g1);
        if (un < units)
            half(g1, g0);
    }

    // lane l of a wave holds rows 4 (l / 16) + 0..3 of column l % 16
    lds_wave_order();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[t][i] = join3(acc[t][i], acc2[t][i], acc3[t][i]);
        *reinterpret_cast<float4_t *>(lds[wave] + 1024 * t + 16 * lane) = acc[t];
    }
    __syncthreads();
    for (int o = tid; o < RT * 16 * B; o += 64 * NW) {
        const int r = o % (16 * RT), b = o / (16 * RT), m = r & 15;
        if (m0 + r >= M)
            continue;
        float sum = 0.f;
        for (int v = 0; v < NW; ++v)
            sum += reinterpret_cast<const float *>(lds[v])[256 * (r >> 4) + 64 * (m >> 2) + 4 * b + (m & 3)];
        y[(int64_t)b * M + m0 + r] = sum;
    }
}

template <int RT, int NW, int Q>
hipError_t launch(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B, hipStream_t st)
{
    hipLaunchKernelGGL((mxfp4_gemv_kernel<RT, NW, Q>), dim3((unsigned)((M + 16 * RT - 1) / (16 * RT))),
                       dim3(64 * NW), 0, st, w, x, y, (int)M, (int)K, B);
    return hipGetLastError();
}

template <int RT>
hipError_t launch_wide(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B, hipStream_t st)
{
    hipLaunchKernelGGL((mxfp4_gemv_wide_kernel<RT, 8>), dim3((unsigned)((M + 16 * RT - 1) / (16 * RT))),
                       dim3(512), 0, st, w, x, y, (int)M, (int)K, B);
    return hipGetLastError();
}

} // namespace

hipError_t launch_gemv_mxfp4(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B,
                             hipStream_t st)
{
    // Tiles of 16 rows shared out among the CUs (the activations are split once for a
    // workgroup's or wave's).  Measured, us, weights from HBM.  Up to five rows, units of two
    // steps, one tile of 8 waves, of 16 waves, two tiles of 8 waves: 4096 x 4096 batch 1 6.5,
    // 6.5, 7.7, batch 4 7.3, 6.7, 8.7; 4096 x 14336 batch 1 13.6, 11.4, 17.6, batch 4 18, 15.5,
    // 23; 14336 x 4096 batch 1 13.7, 20.9, 12.1, batch 4 16.7, 21, 14.0.  Units of four, two
    // and one steps, one tile of 8 waves, batch 1: 4096 x 4096 5.9, 6.5, 7.6; 4096 x 2048 4.8, 4.7,
    // 5.9.  More rows, one, two and four tiles, batch 16: 4096 x 14336 30, 34, 48; 6144 x 4096
    // 20.7, 14.2, 17.9; 14336 x 4096 39, 26, 19.4.
    const int64_t tiles = (M + 15) / 16, cus = device_cus();
    if (B > 5)
        return tiles > 2 * cus ? launch_wide<4>(w, x, y, M, K, B, st)
               : tiles > cus   ? launch_wide<2>(w, x, y, M, K, B, st)
                               : launch_wide<1>(w, x, y, M, K, B, st);
    if (tiles > cus)
        return launch<2, 8, 2>(w, x, y, M, K, B, st);
    if (B * K > 8192) // x is not staged at once by eight waves
        return launch<1, 16, 2>(w, x, y, M, K, B, st);
    return K >= 4096 ? launch<1, 8, 4>(w, x, y, M, K, B, st) : launch<1, 8, 2>(w, x, y, M, K, B, st);
}

} // namespace gq
