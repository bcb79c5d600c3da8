// mxfp4_tiles.hip -- products of two MXFP4 matrices on workgroup tiles.
//
// Y[n][r] = sum_k w[r][k] x[n][k].  A workgroup of WM x WN waves owns 32 FM WM
// weight rows by 32 FN WN activation rows; a wave holds FM x FN accumulators of the
// scaled 32x32x64 product, whose operand is one block (16 bytes, one scale) per lane
// as it lies in memory.  Codes go global -> LDS by direct copies, 256 columns (128
// bytes of a row: whole cache lines) per stage, NB stages in turn; the scales go
// along, 16 bytes of a row (512 columns) every second stage, since a line fetched per
// row and stage for four or eight bytes of scales would cost as much as the codes.
//
// What bounds it, on 256 x 256 tiles at 4096 x 14336 by 4096 rows: the matrix cores
// under the power limit.  The kernel takes 111 us (4.3 PFLOP/s; 117 with the weights from
// HBM); the same products on unchanging registers, without copies and LDS reads, take
// 94 us.  Steps that got there (same shape): stages of 128 columns with the scales by
// dwords 152 us (bound by requests to the L2), 128-byte rows and 16-byte scales 130,
// operands read a step ahead with the products pinned between the reads 117, copies spread
// between the products 113, results stored through LDS 109 (111 in the last trace).
//
// LDS rows are 128 bytes (eight blocks); block c of row r sits in slot
// c ^ ((r >> 1) & 7): the 16 lanes of a read phase touch 16 rows and 16 distinct
// 16-byte bank groups.
//
// Workgroups are numbered so that each XCD (blockIdx mod 8) receives a contiguous
// run of tiles, in groups of eight tile rows, columns one after another: the 32 tiles
// an XCD runs at once are about 8 x 4 and share their rows in its L2.
#include <algorithm>
#include <type_traits>

#include "gq_internal.h"
#include "gq_lds_dma.h"
#include "mxfp4_device.h"
#include "mxfp4_tile.h"

namespace gq {

namespace {

struct TileArgs {
    MxMat w;
    const void *x;     // activations: codes
    const uint8_t *xs; // and scales
    void *y;
    int ytype;
    int M, K, N;
    int tiles_m, tiles_total, tiles_whole;
};

template <int OA, int OB>
__device__ __forceinline__ float16_t mx_mfma32_fp4(uint4 a, uint32_t sa, uint4 b, uint32_t sb,
                                                   float16_t c)
{
    const i8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, OA, (int)sa, OB,
                                                           (int)sb);
}

// SL: the scales go through LDS as well (K % 512 == 0, so that sixteen scales of a
// row, two stages', are one aligned copy); otherwise registers.
template <int WM, int WN, int FM, int FN, int NB, bool SL>
constexpr int mx_lds_bytes()
{
    constexpr int BR = 32 * FM * WM + 32 * FN * WN;
    return std::max(NB * BR * 128 + (SL ? (NB / 2 + 1) * BR * 16 : 0), WM * WN * store_scratch(4 * FM, 4));
}

// The tile of weight rows m0 .. and activation rows n0 ..: NB stages in LDS, of which
// NB - 1 are in flight when a stage begins.
template <int WM, int WN, int FM, int FN, int NB, bool SL>
__device__ __forceinline__ void mx_tile(const TileArgs &p, int m0, int n0, uint8_t *lds)
{
    constexpr int NW = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN, BR = BM + BN;
    constexpr int NC = BR / 8 / NW;                      // 1 KB copies per wave and stage
    constexpr int NS = SL ? (BR / 64 + NW - 1) / NW : 0; // 64-row scale copies
    constexpr int kScales = NB * BR * 128;               // byte offset of the scales
    constexpr int NSB = NB / 2 + 1;                      // and their 512-column places
    // one wave a SIMD: the compiler keeps the accumulators in the other register file
    constexpr bool AGPR = NW <= 4 && mx_lds_bytes<WM, WN, FM, FN, NB, SL>() > (80 << 10);
    static_assert(NC * 8 * NW == BR && BM % 64 == 0 && BN % 64 == 0, "whole copies");
    const int M = p.M, K = p.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 31, h = lane >> 5;
    const int mv = min(M - m0, BM), nv = min(p.N - n0, BN); // valid rows
    const int nblk = K >> 5, nst = (nblk + 7) >> 3;
    const uint8_t *aq = p.w.q + (int64_t)m0 * (K >> 1);
    const uint8_t *bq = reinterpret_cast<const uint8_t *>(p.x) + (int64_t)n0 * (K >> 1);
    const uint8_t *as = p.w.s + (int64_t)m0 * nblk;
    const uint8_t *bs = p.xs + (int64_t)n0 * nblk;

    // copy i of this wave: tile rows 8 (NC wave + i) + lane / 8 (weight rows first),
    // slot lane % 8; the 8 rows are all weights or all activations
    uint32_t off[NC], chk[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int row = 8 * (NC * wave + i) + (lane >> 3);
        const int rr = row < BM ? min(row, mv - 1) : min(row - BM, nv - 1);
        off[i] = (uint32_t)rr * (uint32_t)(K >> 1);
        chk[i] = (lane & 7) ^ swz8(row);
    }
    uint32_t soff[NS + 1];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int row = min(64 * (NS * wave + i), BR - 64) + lane;
        soff[i] = (uint32_t)(row < BM ? min(row, mv - 1) : min(row - BM, nv - 1)) * (uint32_t)nblk;
    }
    const uint32_t base = lds_addr(lds);
    // copy i of stage st, i >= NC: scales, every second stage.  Past the last stage
    // the copies repeat it into the buffer whose turn it is, which no one reads.
    auto copy1 = [&](int st, int i) {
        const int src = min(st, nst - 1);
        if (i < NC) {
            const uint32_t last = (uint32_t)(nblk - 1 - 8 * src); // blocks past it repeat it
            const int row0 = 8 * (NC * wave + i);
            load_lds16((row0 < BM ? aq : bq) + (int64_t)src * 128,
                       off[i] + 16u * (SL ? chk[i] : min(chk[i], last)),
                       __builtin_amdgcn_readfirstlane(base + (st % NB * BR + row0) * 128));
        } else if (i < NC + NS && (st & 1) == 0) {
            const int row0 = min(64 * (NS * wave + i - NC), BR - 64);
            load_lds16((row0 < BM ? as : bs) + (int64_t)(src >> 1) * 16, soff[i - NC],
                       __builtin_amdgcn_readfirstlane(base + kScales +
                                                      ((st >> 1) % NSB * BR + row0) * 16));
        }
    };

    float16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = float16_t{};

    // one step's operands; the scales of a stage, of which bytes 0 and 2 of word
    // t / 2, after a shift by the lane's half, are the lane's of steps t, t + 1
    struct Frag {
        uint4 a[FM], b[FN];
    };
    struct Scale {
        uint2 a[FM], b[FN];
    };
    auto load_scale = [&](const uint8_t *row, int st) -> uint2 {
        uint2 v;
        if (8 * st + 8 <= nblk) {
            __builtin_memcpy(&v, row + 8 * st, 8);
        } else { // blocks past the last get scale 1
            uint32_t t[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[i >> 2] |= (8 * st + i < nblk ? (uint32_t)row[8 * st + i] : 127u)
                             << (8 * (i & 3));
            v = make_uint2(t[0], t[1]);
        }
        return v;
    };
    auto scales = [&](int st, Scale &s) {
        const uint8_t *S = lds + kScales + (st >> 1) % NSB * BR * 16 + 8 * (st & 1);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int row = 32 * (FM * wm + i) + r;
            if constexpr (SL)
                s.a[i] = *reinterpret_cast<const uint2 *>(S + (32 * FM * wm + r) * 16 + 512 * i);
            else
                s.a[i] = load_scale(as + (int64_t)min(row, mv - 1) * nblk, st);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int row = 32 * (FN * wn + j) + r;
            if constexpr (SL)
                s.b[j] = *reinterpret_cast<const uint2 *>(S + (BM + 32 * FN * wn + r) * 16 + 512 * j);
            else
                s.b[j] = load_scale(bs + (int64_t)min(row, nv - 1) * nblk, st);
        }
    };
    auto shift = [&](Scale &s) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
            s.a[i].x >>= 8 * h, s.a[i].y >>= 8 * h;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            s.b[j].x >>= 8 * h, s.b[j].y >>= 8 * h;
    };
    // operand addresses: the swizzle of row 32 i + r is that of r
    uint32_t rof[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        rof[t] = r * 128 + 16 * ((2 * t + h) ^ swz8(r));
    const int arow = 32 * FM * wm * 128, brow = (BM + 32 * FN * wn) * 128;
    auto read = [&](int st, int t, Frag &f) {
        const uint8_t *S = lds + st % NB * BR * 128 + rof[t];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            f.a[i] = ld16(S + arow + 32 * i * 128);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            f.b[j] = ld16(S + brow + 32 * j * 128);
        __builtin_amdgcn_sched_barrier(0);
    };
    // the products of step t of stage st; copies c0 .. c0 + 3 of stage stc (uniform)
    // are issued between them
    auto multiply = [&](int st, auto tc, Frag &f, const Scale &s, int stc, int c0) {
        constexpr int t = decltype(tc)::value;
        if constexpr (!SL) { // blocks past the last are zero
            const bool none = 8 * st + 2 * t + h >= nblk;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                f.a[i].x = none ? 0 : f.a[i].x;
                f.a[i].y = none ? 0 : f.a[i].y;
                f.a[i].z = none ? 0 : f.a[i].z;
                f.a[i].w = none ? 0 : f.a[i].w;
            }
        }
        constexpr int CP = (NC + NS + 1) / 2, EV = FM * FN / CP > 0 ? FM * FN / CP : 1;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = mx_mfma32_fp4<2 * (t & 1), 2 * (t & 1)>(
                    f.a[i], t < 2 ? s.a[i].x : s.a[i].y, f.b[j], t < 2 ? s.b[j].x : s.b[j].y,
                    acc[i][j]);
                // the products stay where they are written, between reads and copies
                if constexpr (AGPR)
                    asm volatile("" : "+a"(acc[i][j]));
                else
                    asm volatile("" : "+v"(acc[i][j]));
                const int u = i * FN + j;
                if (c0 >= 0 && u % EV == EV - 1 && u / EV < CP && c0 + u / EV < NC + NS)
                    copy1(stc, c0 + u / EV);
            }
        if (c0 >= 0)
#pragma unroll
            for (int u = FM * FN / EV; u < CP; ++u)
                if (c0 + u < NC + NS)
                    copy1(stc, c0 + u);
    };

    // Operands are read one step ahead of their products, so that the LDS works while
    // the matrix cores do.
    constexpr int CP = (NC + NS + 1) / 2;
#pragma unroll
    for (int g = 0; g < NB - 1; ++g)
#pragma unroll
        for (int i = 0; i < NC + NS; ++i)
            copy1(g, i);
    wait_copies<(NB - 2) * NC>(); // (scale copies among the newer ones: a wait for more)
    Frag f0, f1;
    Scale s0, s1;
    scales(0, s0);
    read(0, 0, f0);
#pragma unroll
    for (int i = 0; i < CP; ++i)
        copy1(NB - 1, i);
    for (int st = 0; st < nst; ++st) {
        shift(s0);
        read(st, 1, f1);
        multiply(st, std::integral_constant<int, 0>{}, f0, s0, st + NB - 1, CP);
        read(st, 2, f0);
        multiply(st, std::integral_constant<int, 1>{}, f1, s0, 0, -1);
        read(st, 3, f1);
        multiply(st, std::integral_constant<int, 2>{}, f0, s0, 0, -1);
        // the next stage's copies have landed and every wave has read this stage,
        // whose place the one after takes
        wait_copies<(NB - 2) * NC>();
        scales(st + 1, s1); // (after the last stage: read and not used)
        read(st + 1, 0, f0);
        multiply(st, std::integral_constant<int, 3>{}, f1, s0, st + NB, 0);
        s0 = s1;
    }
    wait_copies<0>();

    // element v of an accumulator: weight row 8 (v / 4) + 4 h + v % 4, activation row r
    const int64_t m = m0 + 32 * FM * wm;
    if (m >= M)
        return;
    uint8_t *scr = lds + wave * store_scratch(4 * FM, 4);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = 32 * (FN * wn + j);
        if (n >= nv)
            break;
        float4_t v[4 * FM];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                v[4 * i + v4] = float4_t{acc[i][j][4 * v4], acc[i][j][4 * v4 + 1],
                                         acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]};
        if (p.ytype == kF32)
            store_rows<kF32>(scr, p.y, n0 + n, nv - n, m, M, v);
        else if (p.ytype == kF16)
            store_rows<kF16>(scr, p.y, n0 + n, nv - n, m, M, v);
        else
            store_rows<kBF16>(scr, p.y, n0 + n, nv - n, m, M, v);
    }
}

// Whether a launch of these tiles may cut its last ones: the 256-row ones (14336 x 4096 by
// 4096 rows, 3.5 rounds, 133 -> 130 us; smaller tiles won nothing).
constexpr bool cuts(int FM) { return FM == 4; }

template <int WM, int WN, int FM, int FN, int NB, bool SL>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx_tile_kernel(TileArgs p)
{
    constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    __shared__ __attribute__((aligned(16))) uint8_t lds[std::max(
        mx_lds_bytes<WM, WN, FM, FN, NB, SL>(),
        cuts(FM) ? mx_lds_bytes<WM, WN, FM, FN / 2, NB + 1, SL>() : 0)]; // (halves: one stage more)
    const TileWork work = tile_work(p.tiles_total, p.tiles_whole);
    if (work.tile < 0)
        return;
    int tm, tn;
    tile_pos(work.tile, p.tiles_m, p.tiles_total / p.tiles_m, tm, tn);
    if constexpr (cuts(FM)) {
        if (work.half >= 0) {
            const int n0 = tn * BN + work.half * (BN / 2);
            if (n0 < p.N)
                mx_tile<WM, WN, FM, FN / 2, NB + 1, SL>(p, tm * BM, n0, lds);
            return;
        }
    }
    mx_tile<WM, WN, FM, FN, NB, SL>(p, tm * BM, tn * BN, lds);
}

template <int WM, int WN, int FM, int FN, int NB>
hipError_t launch_mx(TileArgs p, hipStream_t st)
{
    constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_total = p.tiles_m * ((p.N + BN - 1) / BN);
    p.tiles_whole = cuts(FM) ? tiles_whole(p.tiles_total, device_cus()) : p.tiles_total;
    const dim3 grid(tile_grid(p.tiles_total, p.tiles_whole)), block(64 * WM * WN);
    if (p.K % 512 == 0)
        hipLaunchKernelGGL((mx_tile_kernel<WM, WN, FM, FN, NB, true>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((mx_tile_kernel<WM, WN, FM, FN, NB, false>), grid, block, 0, st, p);
    return hipGetLastError();
}

} // namespace

// The tile for a shape, from an estimate of the time of a stage (256 columns): full rounds
// of tiles on the device, and a last one by how many CUs it has.  The smaller tiles keep
// two or three stages of copies in flight: with one, a stage of a lone tile takes the
// length of a read from memory.  Measured with the weights coming from HBM, us for K 14336
// (56 stages): 64 x 64 tiles 22 up to one per CU (one stage in flight 44), 41 at two, 71 at
// four; 128 x 128 35 alone, 45 at one per CU (one stage in flight 53, 58), 79 at two;
// 256 x 256 59-70 for a round in halves, 85 alone, 110-120 a full round.  So 4096 x 14336
// takes by 130 rows 24 us on the first (42, 60 on the others), by 1024 rows 46 on the second
// (78, 67), by 2048 rows 73 on the third (148, 88).
static int mx_tile_choice(int64_t M, int64_t N)
{
    const int64_t cus = device_cus();
    auto tiles = [&](int64_t b) { return (M + b - 1) / b * ((N + b - 1) / b); };
    auto last = [&](int64_t rest, double lone, double full) {
        return rest ? lone + (full - lone) * (double)rest / (double)cus : 0;
    };
    const int64_t t1 = tiles(64), t2 = tiles(128), t3 = tiles(256), whole = tiles_whole(t3, cus);
    const double t64 = 0.39 + 0.36 * std::max(0.0, (double)t1 / (double)cus - 1.0);
    const double t128 = 0.75 * (double)(t2 / cus) + last(t2 % cus, 0.63, 0.78);
    const double t256 = 2.1 * (double)(t3 / cus) +
                        (whole < t3 ? last(2 * (t3 - whole), 1.02, 1.22) : last(t3 % cus, 1.5, 2.1));
    return t64 <= t128 && t64 <= t256 ? 64 : t128 <= t256 ? 128 : 256;
}

hipError_t launch_mx_tiles(MxMat w, MxMat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                           hipStream_t st)
{
    TileArgs p{};
    p.w = w;
    p.x = x.q;
    p.xs = x.s;
    p.y = y;
    p.ytype = type;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    switch (mx_tile_choice(M, N)) {
    case 64: return launch_mx<2, 2, 1, 1, 4>(p, st);
    case 128: return launch_mx<2, 2, 2, 2, 3>(p, st);
    default: return launch_mx<2, 4, 4, 2, 2>(p, st);
    }
}

} // namespace gq
