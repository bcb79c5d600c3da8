// mxfp4_tiles16.hip -- MXFP4 weights times 16-bit activations on workgroup tiles, and
// the expert products of the mixture-of-experts layer on the same tiles.
//
// A workgroup of WM x WN waves owns 32 FM WM weight rows by 32 FN WN activation rows;
// a wave holds FM x FN accumulators of the 32x32x16 product.  Activations go global ->
// LDS by direct copies, 64 columns (128 bytes of a row) per stage, NB stages in turn.
// Codes go the same way, 256 columns (128 bytes) per chunk, two or three in turn, a
// quarter of a chunk's rows per stage; scales 512 columns (16 bytes) at a time.
//
// Lane (r, h) of a stage takes block h of weight row r: one 16-byte LDS read and one
// scale; the four products of a stage take eight of its columns each (columns
// 32 h + 8 s + 0..7 in product s), converted with the scale just before, two values an
// instruction.  The activations are read in the same order (16-byte chunk 4 h + s).
// Conversions and LDS reads are one product ahead of the matrix instructions.
//
// Gate/up: fragment 0 of a wave holds rows of the gate matrix, fragment 1 the same
// rows of the up matrix, so h = silu(g) u is formed in registers.  It is stored in the
// activations' 16-bit type, the operand of the down product (the layer's formula; the Q4_K
// and Q8_0 layers round it alike): a second 16-bit part would double that product's matrix
// instructions, a third more for the layer, and the traffic of h.  The error of the layer is
// 1.4 times that with h in binary32 (64 experts, top-8, hidden 2048, intermediate 1024, mean
// over the outputs: bfloat16 2.3e-3 and 1.7e-3, binary16 2.9e-4 and 2.1e-4).
//
// Binary16 weights are rounded where binary16 does not hold them (scales below 104 and above
// 140; layers have 110 to 130): the matrix instructions take both operands in one type, and
// bfloat16 parts of binary16 activations would be two products for one.
#include <algorithm>
#include <type_traits>

#include "gq_internal.h"
#include "gq_lds_dma.h"
#include "mxfp4_device.h"
#include "mxfp4_tile.h"

namespace gq {

namespace {

enum { kDense = 0, kGateUp = 1, kDown = 2 };

struct Tile16Args {
    MxMat w, w2; // gate/up: gate, up
    const uint16_t *x;
    void *y;
    int M, K, N;
    int tiles_m, tiles_total, tiles_whole;
    // grouped experts: token tiles of sorted positions, one expert each
    const int32_t *sorted, *tiles, *offsets;
    int max_tiles, topk, E;
    int64_t eq, es; // code and scale bytes per expert
    const float *wts;
    int weight_input;
};

template <bool BF16>
__device__ __forceinline__ float16_t mfma32(uint4 a, uint4 b, float16_t c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, a),
                                                       __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                                      __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// Code chunks in LDS at NB activation stages.
constexpr int code_chunks(int NB) { return NB > 2 ? 3 : 2; }
constexpr int lds_bytes(int BM, int BN, int NB, int SM)
{
    return NB * BN * 128 + code_chunks(NB) * BM * 128 + (SM ? 2 * BM * 16 : 0);
}

// One tile: weight rows from m0 (gate/up: BM / 2 rows of each matrix) of expert e
// against activation rows n0 .. n0 + nv - 1.
template <bool BF16, int MODE, int WM, int WN, int KG, int FM, int FN, int NB, int SM>
__device__ __forceinline__ void tile16(const Tile16Args &p, int m0, int n0, int nv, int e,
                                       uint8_t *lds)
{
    constexpr int NW = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN;
    constexpr int CX = BN / 8 / NW;  // activation copies per wave and stage
    constexpr int CW = BM / 32 / NW; // code copies per wave and stage
    constexpr int NC = code_chunks(NB);
    // few accumulators: registers for a whole stage's operands (read a product ahead, a
    // wave of few products waits for the LDS in each of them)
    constexpr bool WIDE = FM * FN <= 4;
    // one wave a SIMD: the compiler keeps the accumulators in the other register file
    constexpr bool AGPR = NW * KG <= 4 && KG * lds_bytes(BM, BN, NB, SM) > (80 << 10);
    // the waits count copies: every wave issues as many
    static_assert(CX * 8 * NW == BN && CW * 32 * NW == BM && NB <= 6, "copies per wave");
    constexpr int CS = SM ? (BM / 64 + NW - 1) / NW : 0; // scale copies per wave and 8 stages
    constexpr int kW = NB * BN * 128, kS = kW + NC * BM * 128; // byte offsets in LDS
    static_assert(MODE != kGateUp || (FM == 2 && BM % 128 == 0), "gate and up fragments in pairs");
    const int M = p.M, K = p.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wall = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wall / NW, wave = wall % NW; // K group, wave in it
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 31, h = lane >> 5;
    // this group's run of K: whole chunks of 256 (512) columns, at least one; the
    // groups step alike, as often as the longest
    const KRun run = k_run<KG>(K >> 5, SM, kg);
    const int nblk = run.blocks, nst = (nblk + 1) >> 1, nch = (nblk + 7) >> 3;
    const int steps = KG == 1 ? nst : (run.longest + 1) >> 1;
    lds += kg * lds_bytes(BM, BN, NB, SM);
    // weight rows of the tile: BW of each matrix
    constexpr int BW = MODE == kGateUp ? BM / 2 : BM;
    const int mv = min(M - m0, BW);
    const int64_t qo = e * p.eq + (int64_t)m0 * (K >> 1) + 16 * run.first;
    const int64_t so = e * p.es + (int64_t)m0 * (K >> 5) + run.first;
    const uint8_t *wq0 = p.w.q + qo, *ws0 = p.w.s + so;
    const uint8_t *wq1 = MODE == kGateUp ? p.w2.q + qo : wq0, *ws1 = MODE == kGateUp ? p.w2.s + so : ws0;
    const uint16_t *xb = (MODE == kGateUp ? p.x : p.x + (int64_t)n0 * K) + 32 * run.first;

    // activation copy i: rows 8 (CX wave + i) + lane / 8, slot lane % 8
    uint32_t xoff[CX], xchk[CX];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const int row = 8 * (CX * wave + i) + (lane >> 3);
        const int rr = min(row, nv - 1);
        const uint32_t src = MODE == kGateUp ? (uint32_t)(p.sorted[n0 + rr] / p.topk) : (uint32_t)rr;
        xoff[i] = src * (uint32_t)K * 2u;
        xchk[i] = (lane & 7) ^ swz8(row);
    }
    // code copy i of quarter j: rows 8 (BM / 32 j + CW wave + i) + lane / 8
    const uint32_t base = lds_addr(lds);
    auto copy_x1 = [&](int st, int i) {
        const int idx = CX * wave + i;
        const int src = min(st, nst - 1);
        const uint32_t last = (uint32_t)(4 * (nblk - 2 * src) - 1); // chunks past it repeat it
        load_lds16(xb + (int64_t)src * 64, xoff[i] + 16u * (SM == kScale1 ? min(xchk[i], last) : xchk[i]),
                   __builtin_amdgcn_readfirstlane(base + st % NB * (BN * 128) + 1024u * idx));
    };
    auto copy_w1 = [&](int q, int i) { // quarter q & 3 of chunk q >> 2
        const int idx = CW * wave + i;
        const int ch = q >> 2, src = min(ch, nch - 1);
        const uint32_t last = (uint32_t)(nblk - 1 - 8 * src);
        const int row0 = 8 * (BM / 32 * (q & 3) + idx), row = row0 + (lane >> 3);
        const bool second = MODE == kGateUp && row0 >= BW;
        const int rr = min(second ? row - BW : row, mv - 1);
        const uint32_t chk = (uint32_t)((lane & 7) ^ swz8(row));
        load_lds16((second ? wq1 : wq0) + (int64_t)src * 128,
                   (uint32_t)rr * (uint32_t)(K >> 1) + 16u * (SM == kScale16 ? chk : min(chk, last)),
                   __builtin_amdgcn_readfirstlane(base + kW + ch % NC * (BM * 128) + 128u * row0));
    };
    auto copy_s = [&](int c) { // 512-column chunk c
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            const int idx = CS * wave + i;
            if (BM / 64 % NW != 0 && idx >= BM / 64)
                return;
            const int row0 = 64 * idx, row = row0 + lane;
            const bool second = MODE == kGateUp && row0 >= BW;
            const uint8_t *src = (second ? ws1 : ws0) + (int64_t)c * 16;
            const uint32_t off = (uint32_t)min(second ? row - BW : row, mv - 1) * (uint32_t)(K >> 5);
            const uint32_t dst = base + kS + (c & 1) * (BM * 16);
            if constexpr (SM == kScale16) {
                load_lds16(src, off, __builtin_amdgcn_readfirstlane(dst + 16u * row0));
            } else { // [4][BM] dwords; past the row the last again
                const int last = (nblk >> 2) - 1 - 4 * c;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load_lds4(src + 4 * min(j, last), off,
                              __builtin_amdgcn_readfirstlane(dst + 4u * (j * BM + row0)));
            }
        }
    };

    // this lane's weight row of fragment i, in the tile
    auto wrow = [&](int i) {
        return MODE == kGateUp ? i * BW + 32 * wm + r : 32 * (FM * wm + i) + r;
    };
    const uint32_t rof = 16 * (h ^ swz8(r)); // the swizzle of row 32 i + r is that of r
    uint32_t xof[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        xof[s] = (32 * FN * wn + r) * 128 + 16 * ((4 * h + s) ^ swz8(r));

    struct Codes {
        uint4 q[FM];
        uint32_t s[FM];
    };
    auto read_codes = [&](int st, Codes &c) {
        const uint8_t *W = lds + kW + (st >> 2) % NC * (BM * 128);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            c.q[i] = ld16(W + wrow(i) * 128 + (rof ^ (32 * (st & 3))));
            const uint8_t *S = lds + kS + ((st >> 3) & 1) * (BM * 16);
            if constexpr (SM == kScale16) {
                c.s[i] = S[wrow(i) * 16 + 2 * (st & 7) + h];
            } else if constexpr (SM == kScale4) {
                c.s[i] = S[(((st & 7) >> 1) * BM + wrow(i)) * 4 + 2 * (st & 1) + h];
            } else {
                const int row = wrow(i), rr = min(MODE == kGateUp ? row - i * BW : row, mv - 1);
                const int blk = 2 * st + h;
                c.s[i] = blk < nblk ? (MODE == kGateUp && i ? ws1 : ws0)[(int64_t)rr * (K >> 5) + blk] : 127u;
                if (blk >= nblk) // past the last block: zeros
                    c.q[i] = make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto read_x = [&](int st, int s, uint4 (&b)[FN]) {
        const uint8_t *X = lds + st % NB * (BN * 128) + xof[s];
#pragma unroll
        for (int j = 0; j < FN; ++j)
            b[j] = ld16(X + 32 * j * 128);
    };
    auto convert = [&](const Codes &c, auto sc, uint4 (&a)[FM]) {
        constexpr int s = decltype(sc)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint32_t d = s == 0 ? c.q[i].x : s == 1 ? c.q[i].y : s == 2 ? c.q[i].z : c.q[i].w;
            a[i] = mx_values8<BF16>(d, mx_scale(c.s[i]));
        }
    };

    float16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = float16_t{};
    auto multiply = [&](uint4 (&a)[FM], uint4 (&b)[FN], auto between) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = mfma32<BF16>(a[i], b[j], acc[i][j]);
                // the products stay where they are written, between reads and copies
                if constexpr (AGPR)
                    asm volatile("" : "+a"(acc[i][j]));
                else
                    asm volatile("" : "+v"(acc[i][j]));
                between(i * FN + j);
            }
    };
    // a short last stage (K % 64 == 32): the lanes of its second block take zeros, for
    // what was copied there may be infinite
    auto mask_x = [&](int st, uint4 (&b)[FN]) {
        if constexpr (SM == kScale1) {
            const bool none = 2 * st + h >= nblk;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                b[j].x = none ? 0 : b[j].x;
                b[j].y = none ? 0 : b[j].y;
                b[j].z = none ? 0 : b[j].z;
                b[j].w = none ? 0 : b[j].w;
            }
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;

    // Copies go in groups: group g is the activations of stage g, quarter g + 4 of the
    // codes (WIDE: g + 3) and, every eighth time, the scales stage g + 1 begins with.  After the
    // barrier that ends stage st (every wave has read stage st, and the codes of stage
    // st + 1) group st + NB takes the places that came free: activations of stage st,
    // codes of chunk (st + NB + 4) / 4 - NC, whose last stage is at most st + 1 while
    // NB <= (NC == 2 ? 2 : 6).  At that barrier the groups up to st + 1 have landed,
    // NB - 2 newer ones may be in flight.
    constexpr int QL = WIDE ? 3 : 4;
    auto group = [&](int g, int u) { // copy u of the group
        if (u < CX)
            copy_x1(g, u);
        else if (u < CX + CW)
            copy_w1(g + QL, u - CX);
        else if (SM != kScale1 && u == CX + CW && ((g + 1) & 7) == 0 && (g + 1) >> 3 < (nblk + 15) >> 4)
            copy_s((g + 1) >> 3);
    };
#pragma unroll
    for (int i = 0; i < CX; ++i)
        copy_x1(0, i);
#pragma unroll
    for (int q = 0; q < QL + 1; ++q)
#pragma unroll
        for (int i = 0; i < CW; ++i)
            copy_w1(q, i);
    if constexpr (SM != kScale1)
        copy_s(0);
#pragma unroll
    for (int g = 1; g < NB; ++g)
#pragma unroll
        for (int u = 0; u < CX + CW; ++u)
            group(g, u);
    wait_copies<(NB - 1) * (CX + CW)>();
    auto nothing = [](int) {};
    if constexpr (WIDE) {
        // a whole stage's operands in registers, read one stage ahead
        struct Ops {
            uint4 b[4][FN];
            Codes c;
        };
        auto load = [&](int st, Ops &o) {
            read_codes(st, o.c);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                read_x(st, s, o.b[s]);
        };
        auto stage = [&](int st, Ops &cur, Ops &nxt) {
            // the next stage's copies have landed, every wave has read this one's
            wait_copies<(NB - 2) * (CX + CW)>();
            load(st + 1, nxt); // (after the last stage: read and not used)
            uint4 a0[FM], a1[FM];
            // one copy after each of the first products
            constexpr int P = FM * FN;
            auto copies = [&](int s) {
                return [&, s](int u) { group(st + NB, s * P + u); };
            };
            convert(cur.c, I0{}, a0);
            convert(cur.c, I1{}, a1);
            mask_x(st, cur.b[0]);
            multiply(a0, cur.b[0], copies(0));
            convert(cur.c, I2{}, a0);
            mask_x(st, cur.b[1]);
            multiply(a1, cur.b[1], copies(1));
            convert(cur.c, I3{}, a1);
            mask_x(st, cur.b[2]);
            multiply(a0, cur.b[2], copies(2));
            mask_x(st, cur.b[3]);
            multiply(a1, cur.b[3], copies(3));
#pragma unroll
            for (int u = 4 * P; u < CX + CW + 1; ++u)
                group(st + NB, u);
        };
        Ops o0, o1;
        load(0, o0);
        for (int st = 0; st < nst; st += 2) {
            stage(st, o0, o1);
            if (st + 1 < nst)
                stage(st + 1, o1, o0);
        }
        if constexpr (KG > 1) // a shorter run keeps the others' barriers
            for (int st = nst; st < steps; ++st)
                wait_copies<0>();
    } else {
        Codes c0, c1;
        uint4 a0[FM], a1[FM], b0[FN], b1[FN];
        read_codes(0, c0);
        read_x(0, 0, b0);
        mask_x(0, b0);
        convert(c0, I0{}, a0);
        static_assert(KG == 1, "one run");
        for (int st = 0; st < nst; ++st) {
            read_x(st, 1, b1);
            read_codes(st + 1, c1); // (after the last stage: read and not used)
            convert(c0, I1{}, a1);
            multiply(a0, b0, nothing);
            read_x(st, 2, b0);
            mask_x(st, b1);
            convert(c0, I2{}, a0);
            multiply(a1, b1, nothing);
            read_x(st, 3, b1);
            mask_x(st, b0);
            convert(c0, I3{}, a1);
            multiply(a0, b0, nothing);
            // the next stage's copies have landed and every wave has read this stage,
            // whose place the one after takes
            wait_copies<(NB - 2) * (CX + CW)>();
            read_x(st + 1, 0, b0); // (after the last stage: read and not used)
            mask_x(st, b1);
            c0 = c1;
            convert(c0, I0{}, a0);
            multiply(a1, b1, [&](int u) { group(st + NB, u); });
#pragma unroll
            for (int u = FM * FN; u < CX + CW + 1; ++u)
                group(st + NB, u);
            mask_x(st + 1, b0);
        }
    }
    wait_copies<0>();

    if constexpr (KG > 1) {
        // groups 1 .. hand their sums to group 0, which adds them in group order
        float4_t *red = reinterpret_cast<float4_t *>(lds - kg * lds_bytes(BM, BN, NB, SM));
        static_assert((KG - 1) * BM * BN * 4 <= KG * lds_bytes(BM, BN, NB, SM), "sums fit");
        if (kg > 0)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4)
                        red[((((kg - 1) * NW + wave) * FM + i) * FN + j) * 256 + v4 * 64 + lane] =
                            float4_t{acc[i][j][4 * v4], acc[i][j][4 * v4 + 1],
                                     acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]};
        __syncthreads();
        if (kg > 0)
            return;
        for (int g = 0; g < KG - 1; ++g)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        const float4_t v = red[(((g * NW + wave) * FM + i) * FN + j) * 256 + v4 * 64 + lane];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc[i][j][4 * v4 + c] += v[c];
                    }
    }

    // element v of an accumulator: weight row 8 (v / 4) + 4 h + v % 4, activation row r
    constexpr int G = MODE == kGateUp ? 4 : 4 * FM, ES = MODE == kDown ? 4 : 2;
    constexpr int TYPE = MODE == kDown ? kF32 : BF16 ? kBF16 : kF16;
    constexpr int kScr = KG > 1 ? (KG - 1) * BM * BN * 4 : 0; // past the groups' sums
    static_assert(kScr + NW * store_scratch(G, ES) <= KG * lds_bytes(BM, BN, NB, SM), "scratch fits");
    const int64_t m = m0 + 8 * G * wm;
    if (m >= M)
        return;
    uint8_t *scr = lds + kScr + wave * store_scratch(G, ES);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = 32 * (FN * wn + j);
        if (n >= nv)
            break;
        float4_t v[G];
        if constexpr (MODE == kGateUp) {
            const float pw = p.weight_input ? p.wts[p.sorted[n0 + min(n + r, nv - 1)]] : 1.f;
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[v4][c] = silu(pw * acc[0][j][4 * v4 + c]) * (pw * acc[1][j][4 * v4 + c]);
        } else {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4)
                    v[4 * i + v4] = float4_t{acc[i][j][4 * v4], acc[i][j][4 * v4 + 1],
                                             acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]};
        }
        store_rows<TYPE>(scr, p.y, n0 + n, nv - n, m, M, v);
    }
}

// Whether a launch of these tiles may cut its last ones: the 256-row ones.  14336 x 4096 by
// 4096 rows (3.5 rounds) 375 -> 367 us; 128-row tiles lost 2-4 % to the second body at
// most shapes.
constexpr bool cuts(int FN) { return FN == 4; }

template <bool BF16, int WM, int WN, int KG, int FM, int FN, int NB, int SM>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void gemm_tile16_kernel(Tile16Args p)
{
    constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    // (halves have room for another stage)
    constexpr int kBytes = KG * lds_bytes(BM, BN, NB, SM), kHalf = lds_bytes(BM, BN / 2, NB + 1, SM);
    __shared__ __attribute__((aligned(16))) uint8_t lds[cuts(FN) && kHalf > kBytes ? kHalf : kBytes];
    const TileWork work = tile_work(p.tiles_total, p.tiles_whole);
    if (work.tile < 0)
        return;
    int tm, tn;
    tile_pos(work.tile, p.tiles_m, p.tiles_total / p.tiles_m, tm, tn);
    if constexpr (cuts(FN)) {
        if (work.half >= 0) {
            const int n0 = tn * BN + work.half * (BN / 2);
            if (n0 < p.N)
                tile16<BF16, kDense, WM, WN, KG, FM, FN / 2, NB + 1, SM>(p, tm * BM, n0,
                                                                         min(p.N - n0, BN / 2), 0, lds);
            return;
        }
    }
    tile16<BF16, kDense, WM, WN, KG, FM, FN, NB, SM>(p, tm * BM, tn * BN, min(p.N - tn * BN, BN), 0, lds);
}

// Expert products: blockIdx.x runs over row tiles, blockIdx.y over token tiles (up to 32
// FN WN sorted positions of one expert).  The hardware deals consecutive workgroups to
// the 8 XCDs in turn; XCD x takes token tiles x, x + 8, .. each with all its row tiles, so
// that a tile's activations are read into one L2 (gridDim.y is a multiple of 8).
// A token tile of at most 64 tokens (an expert's remainder) takes FR < FN fragments.
template <bool BF16, int MODE, int WM, int WN, int KG, int FM, int FN, int FR, int NB, int SM>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void moe_tile16_kernel(Tile16Args p)
{
    constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN, BW = MODE == kGateUp ? BM / 2 : BM;
    __shared__ __attribute__((aligned(16))) uint8_t lds[KG * lds_bytes(BM, BN, NB, SM)];
    const int rt = (int)gridDim.x;
    const int b = (int)blockIdx.x + rt * (int)blockIdx.y;
    const int k = b >> 3, t = 8 * (k / rt) + (b & 7);
    if (t >= p.offsets[p.E + 1])
        return;
    const int e = p.tiles[t], n0 = p.tiles[p.max_tiles + t];
    const int nv = min(p.offsets[e + 1] - n0, BN);
    const int m0 = k % rt * BW;
    if (FR < FN && nv <= 32 * FR * WN)
        tile16<BF16, MODE, WM, WN, KG, FM, FR, NB, SM>(p, m0, n0, nv, e, lds);
    else
        tile16<BF16, MODE, WM, WN, KG, FM, FN, NB, SM>(p, m0, n0, nv, e, lds);
}

template <bool BF16, int MODE, int WM, int WN, int KG, int FM, int FN, int FR, int NB>
hipError_t launch_moe_one(const Tile16Args &p, hipStream_t st)
{
    constexpr int BM = 32 * FM * WM, BW = MODE == kGateUp ? BM / 2 : BM;
    const dim3 grid((unsigned)((p.M + BW - 1) / BW), (unsigned)((p.max_tiles + 7) / 8 * 8)),
        block(64 * WM * WN * KG);
    switch (scale_mode<KG>(p.K)) {
    case kScale16:
        hipLaunchKernelGGL((moe_tile16_kernel<BF16, MODE, WM, WN, KG, FM, FN, FR, NB, kScale16>), grid, block, 0, st, p);
        break;
    case kScale4:
        hipLaunchKernelGGL((moe_tile16_kernel<BF16, MODE, WM, WN, KG, FM, FN, FR, NB, kScale4>), grid, block, 0, st, p);
        break;
    case kScale1:
        hipLaunchKernelGGL((moe_tile16_kernel<BF16, MODE, WM, WN, KG, FM, FN, FR, NB, kScale1>), grid, block, 0, st, p);
        break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <bool BF16, int WM, int WN, int KG, int FM, int FN, int FR, int NB>
hipError_t launch_moe_pair(const MxMoeArgs &a, int max_tiles, hipStream_t st)
{
    Tile16Args p{};
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
    p.M = (int)a.I;
    p.K = (int)a.H;
    hipError_t err = launch_moe_one<BF16, kGateUp, WM, WN, KG, FM, FN, FR, NB>(p, st);
    if (err != hipSuccess)
        return err;
    p.w = a.down;
    p.x = reinterpret_cast<const uint16_t *>(a.ws + a.off[4]);
    p.y = a.ws + a.off[5];
    p.M = (int)a.H;
    p.K = (int)a.I;
    return launch_moe_one<BF16, kDown, WM, WN, KG, FM, FN, FR, NB>(p, st);
}

// The tile for a shape, from an estimate of its time in us per 1024 columns: full rounds of
// tiles on the device at `full`, a last one between `lone` and `full` by how many CUs it
// has.  All but the 256 x 256 tiles, whose LDS holds no more, keep two or more stages of
// copies in flight: one stage in flight leaves every stage the length of a read from
// memory.  Measured with the weights coming from HBM, one workgroup a CU, us for K 14336
// alone and full: 256 x 256 214, 350; 256 x 128 169, 188; 128 x 128 106, 115 (one stage in
// flight 165, and 197 for two a CU); 128 x 64 with K in two runs 61, 68 (72); 64 x 64 in two
// runs 40, 44 (one stage, four runs 53, 57); 64 x 32 in four runs 30, 28.  So 4096 x 14336
// takes by 64 rows 32 us on 64 x 32 tiles (45, 65 on the next), by 130 rows 45 on 64 x 64
// (55, 64), by 512 rows 69 on 128 x 64 (88, 112), by 1024 rows 117 on 128 x 128 (130, 171),
// by 2048 rows 190 on 256 x 128 (196, 227); 14336 x 4096 by 1024 rows 92 on 256 x 256 (112).
int tile16_choice(int64_t M, int64_t K, int64_t N)
{
    const int64_t cus = device_cus(), chunks = (K + 255) / 256;
    auto time = [&](int64_t bm, int64_t bn, double lone, double full) {
        const int64_t tiles = (M + bm - 1) / bm * ((N + bn - 1) / bn), rest = tiles % cus;
        return (double)(tiles / cus) * full + (rest ? lone + (full - lone) * rest / cus : 0);
    };
    // 256 x 256: a last round cut in halves costs about what one of 256 x 128 does
    const int64_t big = (M + 255) / 256 * ((N + 255) / 256), whole = tiles_whole(big, cus);
    const double cut = whole < big ? 12.6 + 1.8 * 2 * (double)(big - whole) / cus : 0;
    const double t[6] = {whole < big ? 24.0 * (double)(whole / cus) + cut : time(256, 256, 15.3, 24.0),
                         time(256, 128, 12.1, 13.5),
                         time(128, 128, 7.6, 8.3),
                         chunks >= 2 ? time(128, 64, 4.35, 4.9) : 1e30,
                         chunks >= 2 ? time(64, 64, 2.9, 3.1) : 1e30,
                         chunks >= 4 ? time(64, 32, 2.15, 2.0) : 1e30};
    return (int)(std::min_element(t, t + 6) - t);
}

template <bool BF16, int WM, int WN, int KG, int FM, int FN, int NB>
hipError_t launch_dense(Tile16Args p, hipStream_t st)
{
    constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_total = p.tiles_m * ((p.N + BN - 1) / BN);
    p.tiles_whole = cuts(FN) ? tiles_whole(p.tiles_total, device_cus()) : p.tiles_total;
    const dim3 grid(tile_grid(p.tiles_total, p.tiles_whole)), block(64 * WM * WN * KG);
    switch (scale_mode<KG>(p.K)) {
    case kScale16:
        hipLaunchKernelGGL((gemm_tile16_kernel<BF16, WM, WN, KG, FM, FN, NB, kScale16>), grid, block, 0, st, p);
        break;
    case kScale4:
        hipLaunchKernelGGL((gemm_tile16_kernel<BF16, WM, WN, KG, FM, FN, NB, kScale4>), grid, block, 0, st, p);
        break;
    case kScale1:
        hipLaunchKernelGGL((gemm_tile16_kernel<BF16, WM, WN, KG, FM, FN, NB, kScale1>), grid, block, 0, st, p);
        break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dense_choice(const Tile16Args &p, hipStream_t st)
{
    switch (tile16_choice(p.M, p.K, p.N)) {
    case 0: return launch_dense<BF16, 4, 2, 1, 2, 4, 2>(p, st);
    case 1: return launch_dense<BF16, 2, 2, 1, 4, 2, 2>(p, st);
    case 2: return launch_dense<BF16, 2, 2, 1, 2, 2, 3>(p, st);
    case 3: return launch_dense<BF16, 2, 1, 2, 2, 2, 3>(p, st);
    case 4: return launch_dense<BF16, 2, 1, 2, 1, 2, 4>(p, st);
    default: return launch_dense<BF16, 2, 1, 4, 1, 1, 3>(p, st);
    }
}

} // namespace

hipError_t launch_gemm_tiles16(MxMat w, const uint16_t *x, uint16_t *y, int type, int64_t M,
                               int64_t K, int64_t N, hipStream_t st)
{
    Tile16Args p{};
    p.w = w;
    p.x = x;
    p.y = y;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    return type == kBF16 ? launch_dense_choice<true>(p, st) : launch_dense_choice<false>(p, st);
}

// Tokens of a tile of the expert products (0: the weight-streaming kernel), by the mean
// number of tokens an expert has.  Measured, us for the whole layer at 64 experts, top-8,
// hidden 2048, intermediate 1024, binary16, weights from HBM: 64 tokens (mean 8) 75 on the
// weight-streaming kernel, 91 on 64-token tiles; 128 tokens 101 and 90; 256 tokens 158, 95
// and 102 on 128-token tiles; 512 tokens (mean 64) 133 and 120; 1024 tokens 192 on 128-token
// and 197 on 256-token tiles, 2048 tokens 312 and 284.
int moe_tile16_tokens(int64_t T, int64_t E, int64_t topk)
{
    const int64_t mean = T * topk / E;
    return mean < 12 ? 0 : mean <= 40 ? 64 : mean < 160 ? 128 : 256;
}

hipError_t launch_moe_tiles16(const MxMoeArgs &a, int tokens, int max_tiles, hipStream_t st)
{
    const bool bf = a.type == kBF16;
    switch (tokens) {
    case 64:
        return bf ? launch_moe_pair<true, 2, 2, 1, 2, 1, 1, 3>(a, max_tiles, st)
                  : launch_moe_pair<false, 2, 2, 1, 2, 1, 1, 3>(a, max_tiles, st);
    case 128:
        return bf ? launch_moe_pair<true, 2, 2, 1, 2, 2, 1, 2>(a, max_tiles, st)
                  : launch_moe_pair<false, 2, 2, 1, 2, 2, 1, 2>(a, max_tiles, st);
    default:
        return bf ? launch_moe_pair<true, 4, 2, 1, 2, 4, 1, 2>(a, max_tiles, st)
                  : launch_moe_pair<false, 4, 2, 1, 2, 4, 1, 2>(a, max_tiles, st);
    }
}

} // namespace gq
