// i8_tiles.hip -- products of int8 matrices on workgroup tiles.
//
// sum_k w[r][k] x[n][k] in whole numbers.  A workgroup of WM x WN waves owns 32 FM WM weight
// rows by 32 FN WN activation rows; a wave holds FM x FN accumulators of the 32x32x32 product,
// whose operand is 16 codes (16 bytes) per lane as they lie in memory.  Codes go global -> LDS
// by direct copies, 128 columns (128 bytes of a row: whole cache lines) per stage, NB stages in
// turn; operands are read a step ahead of the products, copies are issued between them.
//
// What bounds it, on 256 x 256 tiles: the matrix cores under the power limit.  4096 x 14336 by 4096
// rows takes 190 us (2.5 POP/s; the library's product of 16384 x 16384 matrices 2.4), and the same
// products on unchanging registers, without copies and LDS reads, 150 to 180 (by the codes'
// values).  14336 x 4096 by 4096
// rows, 3.5 rounds of tiles, takes 208 (200 with the weights in a cache).  64 x 64 tiles are bound
// by what a CU reads from the L2 (4096 x 14336 by 130 rows 33 us from HBM, 26 again), two groups of
// waves with a run of K each took as long.  128 x 128 per wave (four waves) was 4% slower.
//
// Gate/up: half of a tile's weight rows are rows of the gate matrix, half the same rows of the
// up matrix, and a wave holds both of a row: h, or the gradients of g and u, is formed in
// registers: 14336 x 4096 by 1024 rows takes 116 us, with the gradients of g and u 128.  Those
// leave as binary16 operands of the product with the codes, times their weight row's scale and a
// power of two of their token: 11 bits, where bfloat16 had 8, at the exponents a token's gradients
// have, so that none leaves the type, as unscaled ones do (dg above 65504 for a dX of 100).
//
// The last stage of a K that is no multiple of 128: copies past a row's last 16 bytes repeat
// those, and the weights' codes past K are zeroed in registers (what lies there in the
// activations then counts nothing).
#include <algorithm>
#include <type_traits>

#include "gq_internal.h"
#include "gq_lds_dma.h"
#include "i8_device.h"
#include "i8_plan.h"
#include "mxfp4_tile.h"

namespace gq {

namespace {

enum { kPlain = 0, kGated = 1, kGrads = 2 };

struct I8TileArgs {
    I8Mat w, w2; // gate/up: gate, up
    I8Mat x;
    void *y;
    const uint16_t *dh; // kGrads: the gradient of h, of `type`
    int *e;             // kGrads: exponents of the rows of y, which is binary16
    int64_t ldy;        // elements between rows of y
    int64_t part;       // kGrads: elements from the gradient of g to that of u
    int type, act;
    int M, K, N; // M rows of each matrix
    int tiles_m, tiles_total, tiles_whole;
};

__device__ __forceinline__ int16v mfma_i8(uint4 a, uint4 b, int16v c)
{
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(int4v, a),
                                                 __builtin_bit_cast(int4v, b), c, 0, 0, 0);
}

// Groups of 8 weight rows that a wave stores at once: all of its rows, or a fragment's where two
// results are held.
constexpr int store_groups(int MODE, int FM) { return MODE == kPlain ? 4 * FM : MODE == kGated ? 2 * FM : 4; }

// After the stages LDS holds the waves' scratch for storing and, per weight row, the scales.
constexpr int scratch_bytes(int MODE, int NW, int FM) { return NW * store_scratch(store_groups(MODE, FM), 4); }

template <int MODE, int WM, int WN, int FM, int FN, int NB>
constexpr int i8_lds_bytes()
{
    constexpr int BM = 32 * FM * WM;
    return std::max(NB * (BM + 32 * FN * WN) * 128, scratch_bytes(MODE, WM * WN, FM) + BM * 4);
}

// The tile of weight rows m0 .. (of each matrix) and activation rows n0 ..: NB stages in LDS,
// of which NB - 1 are in flight when a stage begins.
template <int MODE, int WM, int WN, int FM, int FN, int NB, bool TAIL>
__device__ __forceinline__ void i8_tile(const I8TileArgs &p, int m0, int n0, uint8_t *lds)
{
    constexpr int NW = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN, BR = BM + BN;
    constexpr int NC = BR / 8 / NW; // 1 KB copies per wave and stage
    constexpr bool PAIR = MODE != kPlain;
    constexpr int BW = PAIR ? BM / 2 : BM, FW = PAIR ? FM / 2 : FM; // rows, fragments of a matrix
    // one wave a SIMD: the compiler keeps the accumulators in the other register file
    constexpr bool AGPR = NW <= 4 && i8_lds_bytes<MODE, WM, WN, FM, FN, NB>() > (80 << 10);
    static_assert(NC * 8 * NW == BR && BW % 8 == 0 && (!PAIR || FM % 2 == 0), "whole copies, pairs");
    const int M = p.M, K = p.K;
    const uint32_t ldw = (uint32_t)p.w.ld, ldw2 = (uint32_t)(PAIR ? p.w2.ld : p.w.ld), ldx = (uint32_t)p.x.ld;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 31, h = lane >> 5;
    const int mv = min(M - m0, BW), nv = min(p.N - n0, BN); // valid rows
    const int nch = (K + 15) >> 4, nst = (nch + 7) >> 3;     // chunks of 16 codes, stages
    const int8_t *aq = p.w.q + (int64_t)m0 * p.w.ld;
    const int8_t *aq2 = PAIR ? p.w2.q + (int64_t)m0 * p.w2.ld : aq;
    const int8_t *bq = p.x.q + (int64_t)n0 * p.x.ld;

    // what belongs to the matrix of a tile row: gate, up, activations
    auto pick = [](int row, auto gate, auto up, auto x) {
        return row >= BM ? x : PAIR && row >= BW ? up : gate;
    };
    // copy i of this wave: tile rows 8 (NC wave + i) + lane / 8 (weight rows first),
    // slot lane % 8; the 8 rows are of one matrix
    uint32_t off[NC], chk[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int row = 8 * (NC * wave + i) + (lane >> 3);
        const int rr = row < BM ? min(PAIR && row >= BW ? row - BW : row, mv - 1) : min(row - BM, nv - 1);
        const int row0 = 8 * (NC * wave + i);
        off[i] = (uint32_t)rr * pick(row0, ldw, ldw2, ldx);
        chk[i] = (lane & 7) ^ swz8(row);
    }
    const uint32_t base = lds_addr(lds);
    // Past the last stage the copies repeat it into the buffer whose turn it is, which no one
    // reads.
    auto copy1 = [&](int st, int i) {
        const int src = min(st, nst - 1);
        const uint32_t last = (uint32_t)(nch - 1 - 8 * src); // chunks past it repeat it
        const int row0 = 8 * (NC * wave + i);
        load_lds16(uniform(pick(row0, aq, aq2, bq) + (int64_t)src * 128), off[i] + 16u * (TAIL ? min(chk[i], last) : chk[i]),
                   __builtin_amdgcn_readfirstlane(base + (st % NB * BR + row0) * 128));
    };

    int16v acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = int16v{};

    struct Frag {
        uint4 a[FM], b[FN];
    };
    // operand addresses: the swizzle of row 32 i + r is that of r
    uint32_t rof[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        rof[t] = r * 128 + 16 * ((2 * t + h) ^ swz8(r));
    // first tile row of fragment i of this wave
    auto frow = [&](int i) { return i < FW ? 32 * (FW * wm + i) : BW + 32 * (FW * wm + i - FW); };
    const int brow = (BM + 32 * FN * wn) * 128;
    auto read = [&](int st, int t, Frag &f) {
        const uint8_t *S = lds + st % NB * BR * 128 + rof[t];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            f.a[i] = ld16(S + frow(i) * 128);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            f.b[j] = ld16(S + brow + 32 * j * 128);
        __builtin_amdgcn_sched_barrier(0);
    };
    // the products of step t of stage st; copies c0 .. c0 + CP - 1 of stage stc (uniform)
    // are issued between them
    constexpr int CP = (NC + 1) / 2, EV = FM * FN / CP > 0 ? FM * FN / CP : 1;
    auto multiply = [&](int st, auto tc, Frag &f, int stc, int c0, auto lastc) {
        constexpr int t = decltype(tc)::value;
        if constexpr (TAIL && decltype(lastc)::value) { // codes past K are zero
            const int left = K - (128 * st + 16 * (2 * t + h));
            uint32_t mask[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int n = min(max(left - 4 * u, 0), 4);
                mask[u] = n == 4 ? ~0u : (1u << (8 * n)) - 1u;
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
                f.a[i].x &= mask[0], f.a[i].y &= mask[1], f.a[i].z &= mask[2], f.a[i].w &= mask[3];
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = mfma_i8(f.a[i], f.b[j], acc[i][j]);
                // the products stay where they are written, between reads and copies
                if constexpr (AGPR)
                    asm volatile("" : "+a"(acc[i][j]));
                else
                    asm volatile("" : "+v"(acc[i][j]));
                const int u = i * FN + j;
                if (c0 >= 0 && u % EV == EV - 1 && u / EV < CP && c0 + u / EV < NC)
                    copy1(stc, c0 + u / EV);
            }
        if (c0 >= 0)
#pragma unroll
            for (int u = FM * FN / EV; u < CP; ++u)
                if (c0 + u < NC)
                    copy1(stc, c0 + u);
    };

#pragma unroll
    for (int g = 0; g < NB - 1; ++g)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            copy1(g, i);
    wait_copies<(NB - 2) * NC>();
    Frag f0, f1;
    read(0, 0, f0);
#pragma unroll
    for (int i = 0; i < CP; ++i)
        copy1(NB - 1, i);
    auto stage = [&](int st, auto lastc) {
        read(st, 1, f1);
        multiply(st, std::integral_constant<int, 0>{}, f0, st + NB - 1, CP, lastc);
        read(st, 2, f0);
        multiply(st, std::integral_constant<int, 1>{}, f1, 0, -1, lastc);
        read(st, 3, f1);
        multiply(st, std::integral_constant<int, 2>{}, f0, 0, -1, lastc);
        // the next stage's copies have landed and every wave has read this stage,
        // whose place the one after takes
        wait_copies<(NB - 2) * NC>();
        read(st + 1, 0, f0); // (after the last stage: read and not used)
        multiply(st, std::integral_constant<int, 3>{}, f1, st + NB, 0, lastc);
    };
    const int whole = TAIL ? nst - 1 : nst;
    for (int st = 0; st < whole; ++st)
        stage(st, std::false_type{});
    if constexpr (TAIL)
        stage(whole, std::true_type{});
    wait_copies<0>();

    // per weight row of the tile: the scales, of gate and up one after another
    constexpr int G = store_groups(MODE, FM);
    float *const sc = reinterpret_cast<float *>(lds + scratch_bytes(MODE, NW, FM));
    for (int i = tid; i < BW; i += 64 * NW) {
        const bool in = m0 + i < M; // (rows past the last: zeros, as their results then are)
        const float ws = in ? p.w.s[m0 + i] : 0.0f;
        sc[i] = ws;
        if constexpr (PAIR) {
            const float us = in ? p.w2.s[m0 + i] : 0.0f;
            sc[BW + i] = us;
        }
    }
    __syncthreads();

    // element v of an accumulator: weight row 8 (v / 4) + 4 h + v % 4, activation row r
    const int mw = 32 * FW * wm; // the wave's first row in the tile
    const int64_t m = m0 + mw;
    if (m >= M)
        return;
    uint8_t *scr = lds + wave * store_scratch(G, 4);
    auto scaled4 = [&](int i, int j, int v4, float4_t ws, float xs) {
        float4_t v;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = i8_scaled(acc[i][j][4 * v4 + c], ws[c], xs);
        return v;
    };
    // (gradients past the last row, up to a multiple of 8, are stored: zeros, as their dh is)
    const int64_t end = MODE == kGrads ? (M + 7) / 8 * 8 : M;
    auto store = [&](const float4_t(&v)[G], void *y, int64_t n, int left, int64_t m) {
        if (MODE != kGrads && p.type == kF32)
            store_rows<kF32>(scr, y, n, left, m, end, v, p.ldy);
        else if (MODE == kGrads || p.type == kF16)
            store_rows<kF16>(scr, y, n, left, m, end, v, p.ldy);
        else
            store_rows<kBF16>(scr, y, n, left, m, end, v, p.ldy);
    };
    const bool full = m + 32 * FW <= M; // (uniform)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = 32 * (FN * wn + j);
        if (n >= nv)
            break;
        const int64_t nr = n0 + min(n + r, nv - 1);
        const float xs = p.x.s[nr];
        const int e = MODE == kGrads ? p.e[nr] : 0;
        // all of a row's gradients of h at once: one wait for memory instead of one a piece
        uint2 dh[MODE == kGrads ? 4 * FW : 1];
        if constexpr (MODE == kGrads) {
            const uint16_t *src = p.dh + nr * M + m + 4 * h;
            if (full) {
#pragma unroll
                for (int i = 0; i < 4 * FW; ++i)
                    __builtin_memcpy(&dh[i], src + 8 * i, 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4 * FW; ++i)
                    dh[i] = load4(src, 8 * i, M - (m + 8 * i + 4 * h));
            }
        }
        float4_t v[G], v2[MODE == kGrads ? G : 1];
        auto form = [&](auto f32) {
            auto value = [&](float g, float u) { return gated_value<decltype(f32)::value>(g, u, p.act); };
#pragma unroll
            for (int i = 0; i < FW; ++i) {
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const float *row = sc + mw + 32 * i + 8 * v4 + 4 * h;
                    const float4_t ws = *reinterpret_cast<const float4_t *>(row);
                    const float4_t g = scaled4(i, j, v4, ws, xs);
                    if constexpr (MODE == kPlain) {
                        v[4 * i + v4] = g;
                    } else {
                        const float4_t us = *reinterpret_cast<const float4_t *>(row + BW);
                        const float4_t u = scaled4(FW + i, j, v4, us, xs);
                        if constexpr (MODE == kGated) {
                            v[4 * i + v4] = float4_t{value(g[0], u[0]), value(g[1], u[1]), value(g[2], u[2]), value(g[3], u[3])};
                        } else {
                            const float4_t d = values4(dh[4 * i + v4], p.type);
                            float4_t dg, du;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const Gate a = gate_grad(g[c], p.act);
                                dg[c] = __builtin_amdgcn_ldexpf(d[c] * u[c] * a.da * ws[c], -e);
                                du[c] = __builtin_amdgcn_ldexpf(d[c] * a.a * us[c], -e);
                            }
                            v[v4] = dg;
                            v2[v4] = du;
                        }
                    }
                }
                if constexpr (MODE == kGrads) {
                    if (m + 32 * i < M) {
                        store(v, p.y, n0 + n, nv - n, m + 32 * i);
                        store(v2, reinterpret_cast<uint16_t *>(p.y) + p.part, n0 + n, nv - n, m + 32 * i);
                    }
                }
            }
        };
        if (MODE == kGated && p.type == kF32)
            form(std::true_type{});
        else
            form(std::false_type{});
        if constexpr (MODE != kGrads)
            store(v, p.y, n0 + n, nv - n, m);
    }
}

// The exponent e of each row of gradients, so that dg ws 2^-e and du us 2^-e, the operands of the
// product after this one, are binary16 numbers: with |act'| < 1.13, |act(g)| <= |g| and
// |sum| <= 128 L, L the sum of the row's magnitudes of codes, both are at most
// 1.13 max_i |dh[i] ws[i] us[i]| |xs| 128 L, and e makes that, taken by the factors' exponents, at
// most 2^15.  The bound exceeds what a row really holds, by some 2^13 for sums of codes of both
// signs: the largest operands are then near 2^2, all that are down to 2^-16 of them have their 11
// bits, and smaller ones an error of 2^-27 of them.  A workgroup per row; 1024 rows of 14336
// gradients 12 us.
template <int TYPE>
__global__ __launch_bounds__(256) void grad_exponents_kernel(I8TileArgs p)
{
    __shared__ uint32_t part[2][4];
    const int tid = threadIdx.x;
    const int64_t n = blockIdx.x;
    // |v| < 2^(field(v) - 126)
    auto field = [](float v) { return __builtin_bit_cast(uint32_t, v) >> 23 & 0xffu; };
    uint32_t top = 0; // of the three factors' fields
    for (int i = 8 * tid; i < p.M; i += 8 * 256) {
        const int left = p.M - i;
        I8Load8<TYPE> d;
        d.load(p.dh, n * p.M + i, min(left, 8));
        float s[8], t[8];
        if (left >= 8) {
            *reinterpret_cast<float4 *>(s) = ldf4(p.w.s + i);
            *reinterpret_cast<float4 *>(s + 4) = ldf4(p.w.s + i + 4);
            *reinterpret_cast<float4 *>(t) = ldf4(p.w2.s + i);
            *reinterpret_cast<float4 *>(t + 4) = ldf4(p.w2.s + i + 4);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = j < left ? p.w.s[i + j] : 0.0f;
                t[j] = j < left ? p.w2.s[i + j] : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, field(d.value(j)) + field(s[j]) + field(t[j]));
    }
    uint32_t sum = 0;
    const int8_t *q = p.x.q + n * p.x.ld;
    for (int k = 16 * tid; k < p.K; k += 16 * 256) {
        const uint4 v = ld16(q + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) { // codes past K count as zeros
            const int c = min(max(p.K - k - 4 * j, 0), 4);
            const uint32_t mask = c == 4 ? ~0u : (1u << (8 * c)) - 1u;
            sum = __builtin_amdgcn_sad_u8((w[j] & mask) ^ 0x80808080u, 0x80808080u, sum);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off, 64);
    const uint32_t m = wave_max(top);
    if ((tid & 63) == 0) {
        part[0][tid >> 6] = m;
        part[1][tid >> 6] = sum;
    }
    __syncthreads();
    if (tid == 0) {
        const int most = (int)max(max(part[0][0], part[0][1]), max(part[0][2], part[0][3]));
        const uint32_t l = part[1][0] + part[1][1] + part[1][2] + part[1][3];
        const int e = most + (int)field(p.x.s[n]) + (int)field((float)l) - 5 * 126 + 8 - 15;
        p.e[n] = max(e, -100); // (rows of zeros, or of next to nothing)
    }
}

// Whether a launch of these tiles may cut its last ones: the 256-row ones.
constexpr bool cuts(int FM) { return FM == 4; }

template <int MODE, int WM, int WN, int FM, int FN, int NB, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN, 2) void i8_tile_kernel(I8TileArgs p)
{
    constexpr int BM = 32 * FM * WM / (MODE == kPlain ? 1 : 2), BN = 32 * FN * WN;
    __shared__ __attribute__((aligned(16))) uint8_t lds[std::max(
        i8_lds_bytes<MODE, WM, WN, FM, FN, NB>(),
        cuts(FM) ? i8_lds_bytes<MODE, WM, WN, FM, FN / 2, NB + 1>() : 0)]; // (halves: one stage more)
    const TileWork work = tile_work(p.tiles_total, p.tiles_whole);
    if (work.tile < 0)
        return;
    int tm, tn;
    tile_pos(work.tile, p.tiles_m, p.tiles_total / p.tiles_m, tm, tn);
    if constexpr (cuts(FM)) {
        if (work.half >= 0) {
            const int n0 = tn * BN + work.half * (BN / 2);
            if (n0 < p.N)
                i8_tile<MODE, WM, WN, FM, FN / 2, NB + 1, TAIL>(p, tm * BM, n0, lds);
            return;
        }
    }
    i8_tile<MODE, WM, WN, FM, FN, NB, TAIL>(p, tm * BM, tn * BN, lds);
}

template <int MODE, int WM, int WN, int FM, int FN, int NB>
hipError_t launch_tiles(I8TileArgs p, hipStream_t st)
{
    constexpr int BM = 32 * FM * WM / (MODE == kPlain ? 1 : 2), BN = 32 * FN * WN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_total = p.tiles_m * ((p.N + BN - 1) / BN);
    p.tiles_whole = cuts(FM) ? tiles_whole(p.tiles_total, device_cus()) : p.tiles_total;
    const dim3 grid(tile_grid(p.tiles_total, p.tiles_whole)), block(64 * WM * WN);
    if (p.K % 128 == 0)
        hipLaunchKernelGGL((i8_tile_kernel<MODE, WM, WN, FM, FN, NB, false>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((i8_tile_kernel<MODE, WM, WN, FM, FN, NB, true>), grid, block, 0, st, p);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_pair(const I8TileArgs &p, hipStream_t st)
{
    switch (i8_tile_choice(2 * (int64_t)p.M, p.K, p.N, true, device_cus())) {
    case 64: return launch_tiles<MODE, 2, 2, 2, 1, 3>(p, st);
    case 128: return launch_tiles<MODE, 2, 2, 2, 2, 3>(p, st);
    default: return launch_tiles<MODE, 2, 4, 4, 2, 2>(p, st);
    }
}

} // namespace

hipError_t launch_i8_tiles(I8Mat w, I8Mat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                           hipStream_t st)
{
    I8TileArgs p{};
    p.w = w;
    p.x = x;
    p.y = y;
    p.ldy = M;
    p.type = type;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    switch (i8_tile_choice(M, K, N, false, device_cus())) {
    case 64: return launch_tiles<kPlain, 2, 2, 1, 1, 4>(p, st);
    case 128: return launch_tiles<kPlain, 2, 2, 2, 2, 3>(p, st);
    default: return launch_tiles<kPlain, 2, 4, 4, 2, 2>(p, st);
    }
}

hipError_t launch_gated_tiles(I8Mat gate, I8Mat up, I8Mat x, void *h, int type, int act, int64_t I,
                              int64_t H, int64_t N, hipStream_t st)
{
    I8TileArgs p{};
    p.w = gate;
    p.w2 = up;
    p.x = x;
    p.y = h;
    p.ldy = I;
    p.type = type;
    p.act = act;
    p.M = (int)I;
    p.K = (int)H;
    p.N = (int)N;
    return launch_pair<kGated>(p, st);
}

hipError_t launch_gated_grads_i8(I8Mat gate, I8Mat up, I8Mat x, const uint16_t *dh, uint16_t *d,
                                 int64_t ldd, int type, int act, int64_t I, int64_t H, int64_t N,
                                 hipStream_t st)
{
    I8TileArgs p{};
    p.w = gate;
    p.w2 = up;
    p.x = x;
    p.y = d;
    p.dh = dh;
    p.e = grad_exponents(d, N, ldd);
    p.ldy = 2 * ldd;
    p.part = ldd;
    p.type = type;
    p.act = act;
    p.M = (int)I;
    p.K = (int)H;
    p.N = (int)N;
    if (type == kBF16)
        hipLaunchKernelGGL(grad_exponents_kernel<kBF16>, dim3((unsigned)N), dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(grad_exponents_kernel<kF16>, dim3((unsigned)N), dim3(256), 0, st, p);
    const hipError_t err = hipGetLastError();
    return err != hipSuccess ? err : launch_pair<kGrads>(p, st);
}

} // namespace gq
