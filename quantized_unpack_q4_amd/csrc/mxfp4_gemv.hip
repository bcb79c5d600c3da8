// mxfp4_gemv.hip -- MXFP4 weights times 1 to 16 binary32 activation rows.
//
// y[b][r] = sum_k w[r][k] x[b][k].  The weights are read once and everything else is
// small: latency and the rate of the weight loads bound the kernel, so a lane loads
// whole blocks (16 bytes of codes, one scale) several steps ahead, the first before
// anything else.
//
// Binary32 activations are split into three bfloat16 parts, x = a + b + c exactly
// (8 + 8 + 8 significant bits, each part cut toward zero from what is left), and an
// MXFP4 weight is a bfloat16 number exactly (s <= 252), so the products are exact and
// only the binary32 sums of the matrix cores round.  Infinite and NaN activations stay
// in the first part alone.
//
// A workgroup of NW waves owns RT tiles of 16 weight rows; its waves take every NW-th
// step of 128 columns and join their sums through LDS in wave order.  The parts of a
// chunk of x (1024 NW values, all rows of it) lie in LDS as rows of bfloat16.  In a step
// lane (c, h) takes block h of weight row c, converted with its scale, and feeds four
// 16x16x32 products whose k order is permuted alike for both operands (product i takes
// columns 8i .. 8i+7 of the step's four blocks).  Up to five activation rows the three
// parts of a row are three columns of one product (column 3b + p), added at the end;
// above that each part has a product of its own.
#include "gq_internal.h"
#include "mxfp4_device.h"

namespace gq {

namespace {

// A workgroup of NW waves stages 1024 NW activations at a time, four each four values a
// thread: this many columns, whole steps of 128.  Their parts take 3 B rows of two bytes a
// column and 16 more, at most x_bytes(NW).
__host__ __device__ constexpr int chunk_columns(int NW, int B) { return 1024 * NW / B / 128 * 128; }
constexpr int x_bytes(int NW) { return 6 * 1024 * NW + 48 * 16; }

// The three bfloat16 parts of four binary32 values, packed.
__device__ __forceinline__ void split3(const float4 v, uint2 &a, uint2 &b, uint2 &c)
{
    const float x[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = __builtin_bit_cast(uint32_t, x[j]);
        const float r = x[j] - __builtin_bit_cast(float, hi[j] & 0xffff0000u);
        mid[j] = __builtin_bit_cast(uint32_t, r);
        lo[j] = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, mid[j] & 0xffff0000u));
        if ((hi[j] & 0x7f800000u) == 0x7f800000u) {
            hi[j] |= (hi[j] & 0x7fffffu) ? 0x400000u : 0u; // a NaN stays one when cut
            mid[j] = lo[j] = 0;
        }
    }
    // the upper halves of a pair
    a = make_uint2(__builtin_amdgcn_perm(hi[1], hi[0], 0x07060302u),
                   __builtin_amdgcn_perm(hi[3], hi[2], 0x07060302u));
    b = make_uint2(__builtin_amdgcn_perm(mid[1], mid[0], 0x07060302u),
                   __builtin_amdgcn_perm(mid[3], mid[2], 0x07060302u));
    c = make_uint2(__builtin_amdgcn_perm(lo[1], lo[0], 0x07060302u),
                   __builtin_amdgcn_perm(lo[3], lo[2], 0x07060302u));
}

// SETS 1: 3 B <= 16; SETS 3: B <= 16.
template <int SETS, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void mxfp4_gemv_kernel(MxMat w, const float *__restrict__ x,
                                                             float *__restrict__ y, int M, int K,
                                                             int B)
{
    constexpr int GS = 4 / RT; // steps per group of loads, two groups in registers
    __shared__ __attribute__((aligned(16))) uint8_t lds[x_bytes(NW)];
    static_assert(NW * RT * 1024 <= x_bytes(NW), "sums fit");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int m0 = blockIdx.x * (16 * RT);
    const int nblk = K >> 5, steps = (nblk + 3) >> 2;
    const int kc = chunk_columns(NW, B), cs = kc >> 7, spc = (cs + NW - 1) / NW;
    const int chunks = (steps + cs - 1) / cs, total = chunks * spc;
    const int xstride = 2 * kc + 16;

    const uint8_t *qrow[RT], *srow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) { // rows past the last repeat it and are not stored
        const int64_t row = min(m0 + 16 * t + c, M - 1);
        qrow[t] = w.q + row * (K >> 1);
        srow[t] = w.s + row * nblk;
    }
    // this wave's steps: spc in every chunk, at first (in the chunk) = its number and then
    // every NW-th; not all of them exist
    struct Walk {
        int n = 0, first = 0; // steps taken in this chunk, its first step
    };
    auto step_of = [&](const Walk &k) {
        const int in = wave + NW * k.n, st = k.first + in;
        return in < cs && st < steps ? st : -1;
    };
    auto next = [&](Walk &k) {
        if (++k.n == spc) {
            k.n = 0;
            k.first += cs;
        }
    };
    Walk ahead, now;
    struct Group {
        uint4 q[GS][RT];
        uint32_t s[GS][RT];
    };
    auto load = [&](Group &g) {
#pragma unroll
        for (int u = 0; u < GS; ++u) {
            const int st = step_of(ahead);
            next(ahead);
            if (st < 0)
                continue;
            const bool ok = 4 * st + h < nblk; // past the last block: zeros of scale 1
            const int blk = ok ? 4 * st + h : nblk - 1;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                g.q[u][t] = ld16(qrow[t] + 16 * (int64_t)blk);
                g.s[u][t] = srow[t][blk];
            }
        }
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
            uint8_t *d = lds + (SETS == 1 ? 3 * b : b) * xstride + 8 * (f - b * kq);
            const int ps = (SETS == 1 ? 1 : B) * xstride;
            *reinterpret_cast<uint2 *>(d) = p0;
            *reinterpret_cast<uint2 *>(d + ps) = p1;
            *reinterpret_cast<uint2 *>(d + 2 * ps) = p2;
        }
    };

    float4_t acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
        acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    // columns past the last repeat it and are not stored
    const int xrow = SETS == 1 ? min(c, 3 * B - 1) : min(c, B - 1);
    auto compute = [&](int u, Group &g) {
        const int st = step_of(now);
        if (st < 0) // the whole wave
            return;
        const bool ok = 4 * st + h < nblk;
        const uint8_t *xp = lds + xrow * xstride + 64 * h + 256 * (st - now.first);
        float sc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            sc[t] = mx_scale(ok ? g.s[u][t] : 127u);
            if (!ok)
                g.q[u][t] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            uint4 xv[SETS];
#pragma unroll
            for (int p = 0; p < SETS; ++p)
                xv[p] = ld16(xp + p * B * xstride + 16 * n);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const uint4 &q = g.q[u][t];
                const uint4 wv = mx_values8<true>(n == 0 ? q.x : n == 1 ? q.y : n == 2 ? q.z : q.w, sc[t]);
#pragma unroll
                for (int p = 0; p < SETS; ++p)
                    acc[t] = mx_mfma16<true>(wv, xv[p], acc[t]);
            }
        }
    };

    Group g0, g1;
    load(g0);
    load_x(0);
    int chunk = 0;
    auto half = [&](int i0, Group &cur, Group &nxt) {
        load(nxt);
#pragma unroll
        for (int u = 0; u < GS; ++u) {
            const int i = i0 + u;
            if (i >= total)
                break;
            if (now.n == 0) { // the first step of a chunk, for all waves alike
                if (chunk > 0)
                    __syncthreads(); // the chunk before has been read
                stage_x();
                if (++chunk < chunks)
                    load_x(chunk);
                __syncthreads();
            }
            compute(u, cur);
            next(now);
        }
    };
    for (int i = 0; i < total; i += 2 * GS) {
        half(i, g0, g1);
        half(i + GS, g1, g0);
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
            if constexpr (SETS == 1)
                sum += (fv[4 * (3 * b + 2)] + fv[4 * (3 * b + 1)]) + fv[4 * (3 * b)];
            else
                sum += fv[4 * b];
        }
        y[(int64_t)b * M + m0 + r] = sum;
    }
}

template <int SETS, int RT, int NW>
hipError_t launch(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B, hipStream_t st)
{
    hipLaunchKernelGGL((mxfp4_gemv_kernel<SETS, RT, NW>), dim3((unsigned)((M + 16 * RT - 1) / (16 * RT))),
                       dim3(64 * NW), 0, st, w, x, y, (int)M, (int)K, B);
    return hipGetLastError();
}

} // namespace

hipError_t launch_gemv_mxfp4(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B,
                             hipStream_t st)
{
    // Tiles of 16 rows shared out among the CUs, up to four to a workgroup (the
    // activations are split once for them).  Eight waves where two or three such
    // workgroups share a CU or all of x is staged at once, sixteen where one has a CU to
    // itself.  Measured, us, K-split over 8 and 16 waves: 4096 x 4096 batch 1 6.7, 7.9,
    // batch 16 17.0, 14.7; 4096 x 14336 batch 1 16.7, 15.4, batch 16 54, 44; 14336 x 4096
    // with four tiles a workgroup batch 1 14.3, 16.8 (one tile: 15.0, 26), batch 16 26.5,
    // 29.9 (one tile: 43, 50); with two tiles batch 4 15.9, 18.2, batch 16 38, 31.5.
    const int64_t tiles = (M + 15) / 16, cus = device_cus();
    const bool columns = 3 * B <= 16;
    if (tiles > 2 * cus)
        return columns ? launch<1, 4, 8>(w, x, y, M, K, B, st) : launch<3, 4, 8>(w, x, y, M, K, B, st);
    if (tiles > cus)
        return columns ? launch<1, 2, 8>(w, x, y, M, K, B, st) : launch<3, 2, 16>(w, x, y, M, K, B, st);
    if (!columns)
        return launch<3, 1, 16>(w, x, y, M, K, B, st);
    return B * K <= 8192 ? launch<1, 1, 8>(w, x, y, M, K, B, st) : launch<1, 1, 16>(w, x, y, M, K, B, st);
}

} // namespace gq
