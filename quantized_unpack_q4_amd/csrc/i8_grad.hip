// i8_grad.hip -- gradients through int8 matrices: dx[n][k] = sum_m d[n][m] w16[m][k], 16-bit
// gradients, weights converted to their type on the way.
//
// The sum runs over the weights' rows, so an operand of the matrix product is a column piece.
// A workgroup of WM x WN waves owns 128 WM columns of the weights by 32 FN WN rows of d, and
// takes 64 weight rows a stage.  A thread loads a dword (four columns) of eight consecutive
// rows, straight to registers, forms q s of each column in binary32, rounds and packs the eight
// rows' values of a column, 16 bytes, and stores them as one chunk of that column's LDS row: the
// transposition costs nothing, each weight is converted once a workgroup, and both operands of
// the 32x32x16 products are then read as 16-byte chunks of 128-byte LDS rows.  d goes global ->
// LDS by direct copies.
//
// Column 4 l + i of the tile lies in LDS row (32 WM) i + l: the chunks that a wave stores at a
// time go to consecutive rows (distinct banks), and a wave's four fragments, i = 0 .. 3 of the
// same l, hold 128 consecutive columns, sixteen of them consecutive in a lane's accumulators,
// which are stored as they lie.
//
// SCALED, for the gated half: d's rows hold the weights' scales and a power of two already
// (i8_tiles.hip), the weights' operands are their codes, which both 16-bit types hold exactly, and
// the power of two is taken back from the sums.
//
// Where tiles are too few to fill the device the sum is cut into runs, a workgroup each, whose
// binary32 sums a second launch adds in run order.
//
// What bounds it on 256 x 256 tiles: 4096 x 14336 by 2048 rows takes 233 us (1.03 PFLOP/s; the
// library's bfloat16 products of 16384 x 16384 matrices reach 1.60), 4096 x 4096 by 4096 rows, one
// full round, 118 (1.16).  Of those 118, products, operand reads and barriers alone take 93; copies
// and loads add 11, conversions and their stores 12.  Steps that got there: conversions from
// unsigned bytes with a fused step and per-stage selections of what becomes of a scale 172 us,
// signed ones (two instructions a weight), scales in scalar registers, masks in the last stage
// only 124; conversions between the products and the last products after the barrier 118.
// Tried and not kept: 128 x 128 per wave on four waves (spills), weights loaded two stages ahead
// (130 us: registers).
#include <algorithm>
#include <type_traits>

#include "gq_internal.h"
#include "gq_lds_dma.h"
#include "i8_device.h"
#include "i8_plan.h"
#include "mxfp4_tile.h"

namespace gq {

namespace {

struct GradArgs {
    I8GradPart part[2];
    uint16_t *dx;
    int64_t ldd;
    int nparts;
    int M, K, N; // d has zeros from M to the next multiple of 8
    int tiles_k, tiles_total;
    const int *e;   // SCALED: the rows' exponents
    int splits;     // runs of the sum, a workgroup each
    float *partial; // their sums where there are several: [splits][N][ldp]
    int64_t ldp;
};

template <bool BF16>
__device__ __forceinline__ float16_t mfma32_16(uint4 a, uint4 b, float16_t c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, a),
                                                       __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                                      __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// SCALED: operands are binary16 whatever the result's type.
template <bool BF16, bool SCALED, int WM, int WN, int FN, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN, 2) void grad_tile_kernel(GradArgs p)
{
    constexpr int NW = WM * WN, NT = 64 * NW, BK = 128 * WM, BN = 32 * FN * WN;
    constexpr int UN = 8 * (BK / 4) / NT; // 8-row, 4-column units of a thread and stage
    constexpr int CX = BN / 8 / NW;       // 1 KB copies of d per wave and stage
    constexpr int kD = 2 * BK * 128;      // byte offset of d in LDS
    constexpr bool OP_BF16 = BF16 && !SCALED; // type of the operands
    static_assert(UN * NT == 8 * (BK / 4) && CX * 8 * NW == BN, "whole units and copies");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (BK + BN) * 128];
    const TileWork work = tile_work(p.tiles_total * p.splits, p.tiles_total * p.splits);
    if (work.tile < 0)
        return;
    const int split = work.tile / p.tiles_total;
    int tk, tn;
    tile_pos(work.tile % p.tiles_total, p.tiles_k, p.tiles_total / p.tiles_k, tk, tn);
    const int k0 = tk * BK, n0 = tn * BN;
    const int M = p.M, K = p.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 31, h = lane >> 5;
    const int nv = min(p.N - n0, BN);
    const int nch = (M + 7) >> 3, nst = (nch + 7) >> 3; // chunks of 8 weight rows, stages of a part
    // this workgroup's run of the stages of all parts
    const int all = p.nparts * nst, first = (int)((int64_t)all * split / p.splits);
    const int total = (int)((int64_t)all * (split + 1) / p.splits) - first;

    // d: copy i of this wave: rows 8 (CX wave + i) + lane / 8, slot lane % 8
    uint32_t doff[CX], dchk[CX];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const int row = 8 * (CX * wave + i) + (lane >> 3);
        doff[i] = (uint32_t)min(row, nv - 1) * (uint32_t)p.ldd * 2u;
        dchk[i] = (lane & 7) ^ swz8(row);
    }
    const uint32_t base = lds_addr(lds);
    // d, stage after stage of the run (past the last: the last again)
    int dst = first >= nst ? first - nst : first, dleft = total;
    const uint16_t *dq = (first >= nst ? p.part[1].d + 0 : p.part[0].d + 0) + (int64_t)n0 * p.ldd +
                         (int64_t)dst * 64;
    auto copy_d = [&](int b, int i) {
        const uint32_t last = (uint32_t)(nch - 1 - 8 * dst); // chunks past it repeat it
        load_lds16(dq, doff[i] + 16u * (TAIL ? min(dchk[i], last) : dchk[i]),
                   __builtin_amdgcn_readfirstlane(base + kD + b * (BN * 128) + 1024u * (CX * wave + i)));
    };
    auto next_d = [&] {
        if (--dleft <= 0)
            return;
        dq += 64;
        if (++dst == nst) {
            dst = 0;
            dq = p.part[1].d + (int64_t)n0 * p.ldd;
        }
    };
    // weights: unit u of this thread, rows 8 c .. 8 c + 7 of columns 4 l .. 4 l + 3
    struct Raw {
        uint32_t w[8];
        float s[8];
    };
    int urow[UN], ucol[UN], uput[UN][4];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int id = tid + NT * u, c = id / (BK / 4), l = id % (BK / 4);
        urow[u] = 8 * c;
        ucol[u] = min(k0 + 4 * l, ((K + 15) & ~15) - 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (BK / 4) * i + l;
            uput[u][i] = row * 128 + 16 * (c ^ swz8(row));
        }
    }
    int wst, wleft = total;
    const int8_t *wq;
    const float *wsc;
    uint32_t ld, uoff[UN][8];
    auto enter = [&](const I8Mat &w, int st) { // stage st of a matrix
        wst = st;
        ld = (uint32_t)w.ld;
        wq = w.q + 64 * (int64_t)st * ld;
        wsc = w.s + 64 * (int64_t)st;
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                uoff[u][i] = (uint32_t)(urow[u] + i) * ld + (uint32_t)ucol[u];
    };
    if (first >= nst)
        enter(p.part[1].w, first - nst);
    else
        enter(p.part[0].w, first);
    auto load_w = [&](Raw (&raw)[UN]) {
        const int left = M - 64 * wst; // rows past it repeat the last
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (!TAIL || left >= 64) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    raw[u].w[i] = load_dword(wq, uoff[u][i]);
                if constexpr (!SCALED) {
                    *reinterpret_cast<float4 *>(raw[u].s) = ldf4(wsc + urow[u]);
                    *reinterpret_cast<float4 *>(raw[u].s + 4) = ldf4(wsc + urow[u] + 4);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int m = min(urow[u] + i, left - 1);
                    raw[u].w[i] = load_dword(wq, (uint32_t)m * ld + (uint32_t)ucol[u]);
                    if constexpr (!SCALED)
                        raw[u].s[i] = wsc[m];
                }
            }
        }
        if (--wleft <= 0) // (past the last stage: the last again)
            return;
        wq += 64 * (int64_t)ld;
        wsc += 64;
        if (++wst == nst)
            enter(p.part[1].w, 0);
    };
    // Once loaded (the compiler waits here, where nothing else is in flight): a tile of 256
    // columns has one unit's rows in all lanes of a wave, their scales then go to scalar
    // registers.
    auto ready = [&](Raw (&raw)[UN]) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                asm volatile("" : "+v"(raw[u].w[i]));
                if constexpr (!SCALED) {
                    asm volatile("" : "+v"(raw[u].s[i]));
                    if constexpr (BK == 256)
                        raw[u].s[i] = __builtin_bit_cast(
                            float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, raw[u].s[i])));
                }
            }
    };
    // Column i of the units into buffer b, in NM pieces, one after each product of a step: q s of
    // a piece's rows, rounded to binary32 and then to the type; a unit's eight are 16 bytes.
    constexpr int NM = 4 * FN, PW = 8 * UN / NM;
    static_assert(PW * NM == 8 * UN, "whole pieces");
    float pv[4];
    uint32_t pk[4][4];
    auto put_w = [&](const Raw (&raw)[UN], auto ic, int b, int piece) {
        constexpr int i = decltype(ic)::value;
#pragma unroll
        for (int e = piece * PW; e < piece * PW + PW; ++e) {
            const int u = e / 8, j = e % 8;
            float v = (float)(int8_t)(raw[u].w[j] >> (8 * i));
            if constexpr (!SCALED)
                v = as_is(v * raw[u].s[j]);
            if (j % 2)
                pk[i][j / 2] = mx_pack2<OP_BF16>(pv[i], v);
            else
                pv[i] = v;
            if (j == 7)
                *reinterpret_cast<uint4 *>(lds + b * (BK * 128) + uput[u][i]) =
                    make_uint4(pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
        }
    };

    float16_t acc[4][FN];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = float16_t{};
    struct Frag {
        uint4 a[4], b[FN];
    };
    uint32_t rof[4]; // (the swizzle of row 32 i + r is that of r)
#pragma unroll
    for (int s = 0; s < 4; ++s)
        rof[s] = r * 128 + 16 * ((2 * s + h) ^ swz8(r));
    auto read = [&](int t, int s, Frag &f) {
        const uint8_t *W = lds + (t & 1) * (BK * 128) + 32 * wm * 128 + rof[s];
        const uint8_t *D = lds + kD + (t & 1) * (BN * 128) + 32 * FN * wn * 128 + rof[s];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f.a[i] = ld16(W + (BK / 4) * i * 128);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            f.b[j] = ld16(D + 32 * j * 128);
        __builtin_amdgcn_sched_barrier(0);
    };
    // the products of a step; between(u) after each of them, in the shadow of the matrix
    // instruction
    auto multiply = [&](int t, int s, Frag &f, auto between) {
        if constexpr (TAIL) {
            const int st = first + t >= nst ? first + t - nst : first + t;
            if (st == nst - 1) { // gradients past M are zero (they may be anything)
                asm volatile(""); // (a branch, not a selection in every stage)
                const bool none = 8 * st + 2 * s + h >= nch;
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    f.b[j].x = none ? 0 : f.b[j].x;
                    f.b[j].y = none ? 0 : f.b[j].y;
                    f.b[j].z = none ? 0 : f.b[j].z;
                    f.b[j].w = none ? 0 : f.b[j].w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = mfma32_16<OP_BF16>(f.a[i], f.b[j], acc[i][j]);
                asm volatile("" : "+v"(acc[i][j]));
                between(i * FN + j);
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;

    // Stage t: the products of its buffers; its waves put the weights of stage t + 1, loaded
    // a stage ago, into the other buffers, and start the copies of d of stage t + 1 and the loads
    // of stage t + 2.
    Frag f0, f1;
    auto stage = [&](int t, const Raw (&put)[UN], Raw (&load)[UN]) {
        const int b = (t + 1) & 1;
#pragma unroll
        for (int i = 0; i < CX; ++i)
            copy_d(b, i);
        next_d();
        load_w(load);
        read(t, 1, f1);
        multiply(t, 0, f0, [&](int u) { put_w(put, I0{}, b, u); });
        read(t, 2, f0);
        multiply(t, 1, f1, [&](int u) {
            put_w(put, I1{}, b, u);
            put_w(put, I2{}, b, u);
        });
        read(t, 3, f1);
        multiply(t, 2, f0, [&](int u) { put_w(put, I3{}, b, u); });
        // the next stage is converted and copied, and every wave has read this one; its last
        // products run while the next one's first operands are read
        wait_copies<0>();
        read(t + 1, 0, f0); // (after the last stage: read and not used)
        multiply(t, 3, f1, [](int) {});
        ready(load);
    };
    Raw r0[UN], r1[UN];
    load_w(r0);
    load_w(r1);
    ready(r0);
#pragma unroll
    for (int u = 0; u < NM; ++u)
        put_w(r0, I0{}, 0, u);
#pragma unroll
    for (int u = 0; u < NM; ++u)
        put_w(r0, I1{}, 0, u);
#pragma unroll
    for (int u = 0; u < NM; ++u)
        put_w(r0, I2{}, 0, u);
#pragma unroll
    for (int u = 0; u < NM; ++u)
        put_w(r0, I3{}, 0, u);
#pragma unroll
    for (int i = 0; i < CX; ++i)
        copy_d(0, i);
    next_d();
    wait_copies<0>();
    ready(r1);
    read(0, 0, f0);
    for (int t = 0; t < total; t += 2) {
        stage(t, r1, r0);
        if (t + 1 < total)
            stage(t + 1, r0, r1);
    }
    wait_copies<0>();

    // element v of accumulator i: column 4 (8 (v / 4) + 4 h + v % 4) + i, row r
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = 32 * (FN * wn + j) + r;
        if (n >= nv)
            break;
        if (p.splits > 1) { // (rows hold a multiple of 16 columns)
            float *sum = p.partial + ((int64_t)split * p.N + n0 + n) * p.ldp;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int k = k0 + 128 * wm + 32 * g + 16 * h;
                if (k < K)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<float4_t *>(sum + k + 4 * c) =
                            float4_t{acc[0][j][4 * g + c], acc[1][j][4 * g + c], acc[2][j][4 * g + c],
                                     acc[3][j][4 * g + c]};
            }
            continue;
        }
        if constexpr (SCALED) {
            const int e = p.e[n0 + n];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][j][v] = as_is(__builtin_amdgcn_ldexpf(acc[i][j][v], e));
        }
        uint16_t *out = p.dx + (int64_t)(n0 + n) * K;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int k = k0 + 128 * wm + 32 * g + 16 * h;
            uint32_t o[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[2 * c] = mx_pack2<BF16>(acc[0][j][4 * g + c], acc[1][j][4 * g + c]);
                o[2 * c + 1] = mx_pack2<BF16>(acc[2][j][4 * g + c], acc[3][j][4 * g + c]);
            }
            if (k + 16 <= K) { // (rows need not start 16-byte aligned)
                __builtin_memcpy(out + k, o, 32);
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (k + c < K)
                        out[k + c] = (uint16_t)(o[c >> 1] >> (16 * (c & 1)));
            }
        }
    }
}

// The runs' sums added in run order, multiplied by 2^e of their row where there are such, and
// rounded once.
template <bool BF16>
__global__ __launch_bounds__(256) void grad_sum_kernel(const float *__restrict__ partial, int splits,
                                                       int64_t ldp, const int *__restrict__ e,
                                                       uint16_t *__restrict__ dx, int K, int64_t N)
{
    const int64_t row4 = (K + 3) / 4, total = N * row4, step = (int64_t)gridDim.x * 256;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
        const int64_t n = t / row4;
        const int k = (int)(t - n * row4) * 4;
        const float *s = partial + n * ldp + k;
        float4_t v = *reinterpret_cast<const float4_t *>(s);
        for (int i = 1; i < splits; ++i)
            v += *reinterpret_cast<const float4_t *>(s + i * N * ldp);
        if (e) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = as_is(__builtin_amdgcn_ldexpf(v[c], e[n]));
        }
        mx_store4(dx, n * K + k, BF16 ? kBF16 : kF16, v, K - k, K % 4 == 0);
    }
}

// Rows of d with M elements of any alignment into rows of ldo (a multiple of 8), zeros behind
// them.
__global__ __launch_bounds__(256) void align_rows_kernel(const uint16_t *__restrict__ d, int64_t ldd,
                                                         uint16_t *__restrict__ out, int ldo, int M,
                                                         int64_t total)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
        const int64_t n = t / (ldo / 8);
        const int m = (int)(t - n * (ldo / 8)) * 8;
        I8Load8<kF16> v;
        v.load(d, n * ldd + m, max(min(M - m, 8), 0));
        *reinterpret_cast<uint4 *>(out + n * ldo + m) = v.u;
    }
}

template <bool SCALED, int WM, int WN, int FN>
hipError_t launch_grad_tiles(GradArgs p, int type, hipStream_t st)
{
    constexpr int BK = 128 * WM, BN = 32 * FN * WN;
    p.tiles_k = (p.K + BK - 1) / BK;
    p.tiles_total = p.tiles_k * ((p.N + BN - 1) / BN);
    const dim3 grid(tile_grid((int64_t)p.tiles_total * p.splits, (int64_t)p.tiles_total * p.splits)), block(64 * WM * WN);
    auto launch = [&](auto bf16, auto tail) {
        hipLaunchKernelGGL((grad_tile_kernel<decltype(bf16)::value, SCALED, WM, WN, FN, decltype(tail)::value>),
                           grid, block, 0, st, p);
    };
    if (type == kBF16)
        p.M % 64 ? launch(std::true_type{}, std::true_type{}) : launch(std::true_type{}, std::false_type{});
    else
        p.M % 64 ? launch(std::false_type{}, std::true_type{}) : launch(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

template <bool SCALED>
hipError_t launch_grad(const GradArgs &p, int tile, int type, hipStream_t st)
{
    switch (tile) {
    case 0: return launch_grad_tiles<SCALED, 2, 4, 2>(p, type, st);
    case 1: return launch_grad_tiles<SCALED, 2, 4, 1>(p, type, st);
    default: return launch_grad_tiles<SCALED, 1, 2, 1>(p, type, st);
    }
}

int64_t partial_ld(int64_t K) { return (K + 15) / 16 * 16; }

} // namespace

hipError_t launch_align_rows(const uint16_t *d, int64_t ldd, uint16_t *out, int64_t ldo, int64_t M,
                             int64_t N, hipStream_t st)
{
    const int64_t total = N * (ldo / 8);
    hipLaunchKernelGGL(align_rows_kernel, dim3((unsigned)std::min((total + 255) / 256, (int64_t)1 << 16)), dim3(256), 0, st, d,
                       ldd, out, (int)ldo, (int)M, total);
    return hipGetLastError();
}

size_t grad_partial_bytes(int nparts, int64_t M, int64_t K, int64_t N)
{
    const int splits = grad_plan(nparts, M, K, N).splits;
    const size_t e = nparts > 1 ? (size_t)grad_exponent_bytes(N) : 0;
    return e + (splits > 1 ? (size_t)splits * N * partial_ld(K) * 4 : 0);
}

hipError_t launch_grad_i8(const I8GradPart *parts, int nparts, bool scaled, int64_t ldd,
                          uint16_t *dx, int type, int64_t M, int64_t K, int64_t N, void *partial,
                          hipStream_t st)
{
    const GradPlan plan = grad_plan(nparts, M, K, N);
    GradArgs p{};
    p.part[0] = parts[0];
    p.part[1] = parts[nparts - 1];
    p.nparts = nparts;
    p.ldd = ldd;
    p.dx = dx;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    p.splits = plan.splits;
    p.e = scaled ? (const int *)partial : nullptr;
    p.partial = (float *)((char *)partial + (scaled ? grad_exponent_bytes(N) : 0));
    p.ldp = partial_ld(K);
    const hipError_t e = scaled ? launch_grad<true>(p, plan.tile, type, st)
                                : launch_grad<false>(p, plan.tile, type, st);
    if (e != hipSuccess || p.splits == 1)
        return e;
    const dim3 grid((unsigned)std::min((N * ((K + 3) / 4) + 255) / 256, (int64_t)1 << 14)), block(256);
    if (type == kBF16)
        hipLaunchKernelGGL(grad_sum_kernel<true>, grid, block, 0, st, p.partial, p.splits, p.ldp,
                           p.e, dx, (int)K, N);
    else
        hipLaunchKernelGGL(grad_sum_kernel<false>, grid, block, 0, st, p.partial, p.splits, p.ldp,
                           p.e, dx, (int)K, N);
    return hipGetLastError();
}

} // namespace gq
