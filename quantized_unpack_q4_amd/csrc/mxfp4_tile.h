// mxfp4_tile.h -- what the workgroup-tile kernels of the MXFP4 products share.
#pragma once

#include "gq_lds_dma.h"
#include "mxfp4_device.h"
#include "mxfp4_krun.h"

namespace gq {

// LDS rows are 128 bytes (eight 16-byte chunks); chunk c of row r sits in slot
// c ^ swz8(r): the 16 lanes of a read phase touch 16 rows and 16 distinct 16-byte
// bank groups.
__device__ __forceinline__ int swz8(int row) { return (row >> 1) & 7; }

__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return (uint32_t)(size_t)(const __attribute__((address_space(3))) void *)p;
}

// The work of this workgroup.  Workgroups are dealt to the 8 XCDs in turn; each XCD gets a
// contiguous run of tiles.  Where the last round of tiles would leave at least half the CUs
// idle, its tiles are cut in two along the activation rows: `whole` tiles come first, the
// rest as halves (14336 x 4096 by 4096 rows is 3.5 rounds of 256 x 256 tiles on 256 CUs).
struct TileWork {
    int tile, half; // half: -1 whole, else 0 or 1; tile -1: nothing
};
__device__ __forceinline__ TileWork tile_work(int total, int whole)
{
    int b = blockIdx.x;
    const bool cut = b >= (whole + 7) / 8 * 8;
    const int n = cut ? 2 * (total - whole) : whole;
    if (cut)
        b -= (whole + 7) / 8 * 8;
    const int t = (b % 8) * ((n + 7) / 8) + b / 8;
    if (t >= n)
        return {-1, -1};
    return cut ? TileWork{whole + t / 2, t & 1} : TileWork{t, -1};
}
// How many of the tiles are not cut, and the workgroups of the launch.
inline int tiles_whole(int64_t total, int64_t cus)
{
    const int64_t rest = total % cus;
    return (int)(rest > 0 && 2 * rest <= cus ? total - rest : total);
}
inline unsigned tile_grid(int64_t total, int64_t whole)
{
    return (unsigned)((whole + 7) / 8 * 8 + (2 * (total - whole) + 7) / 8 * 8);
}

// Tile (tm, tn) number t: in groups of eight tile rows, columns one after another.
__device__ __forceinline__ void tile_pos(int t, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int g = t / (8 * tiles_n), rows = min(8, tiles_m - 8 * g);
    const int i = t - g * 8 * tiles_n;
    tm = 8 * g + i % rows;
    tn = i / rows;
}

// Waits until at most VM of this wave's copies are in flight and its LDS reads are
// done, then for the workgroup.
template <int VM>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// Bytes of a wave's scratch for store_rows.
constexpr int store_scratch(int G, int esize) { return 32 * (8 * G * esize + 16); }

// Stores 32 activation rows by 8 G weight rows of a wave's accumulators: lane (r, h)
// holds v[g] = weight rows 8 g + 4 h + 0..3 of activation row r.  The values go through
// LDS (rows padded by 16 bytes), so that a row leaves as whole runs of 16 G (32 G)
// bytes instead of 16-byte pieces of 32 rows; on 256 x 256 tiles of 4096 columns that
// takes a tenth off the whole product.  y at (activation row n, weight row m), nv
// activation rows and mleft weight rows exist.
template <int TYPE, int G>
__device__ __forceinline__ void store_rows(uint8_t *scr, void *y, int64_t n, int nv, int64_t m,
                                           int64_t M, const float4_t (&v)[G])
{
    constexpr int ES = TYPE == kF32 ? 4 : 2, ST = 8 * G * ES + 16, CE = 16 / ES;
    constexpr int CPR = 8 * G / CE; // 16-byte chunks of a row
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        uint8_t *d = scr + r * ST + (8 * g + 4 * h) * ES;
        if constexpr (TYPE == kF32)
            *reinterpret_cast<float4_t *>(d) = v[g];
        else
            *reinterpret_cast<uint2 *>(d) = make_uint2(mx_pack2<TYPE == kBF16>(v[g][0], v[g][1]),
                                                       mx_pack2<TYPE == kBF16>(v[g][2], v[g][3]));
    }
    lds_wave_order();
    const bool vec = M % CE == 0; // rows start 16-byte aligned
    const int64_t mleft = M - m;
#pragma unroll
    for (int k = 0; k < 32 * CPR / 64; ++k) {
        const int c = lane + 64 * k, row = c / CPR, col = c % CPR * CE;
        if (row >= nv || col >= mleft)
            continue;
        const uint8_t *s = scr + row * ST + col * ES;
        uint8_t *d = reinterpret_cast<uint8_t *>(y) + ((n + row) * M + m + col) * ES;
        if (vec) { // whole chunks exist: mleft is a multiple of CE too
            *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(s);
        } else {
#pragma unroll
            for (int i = 0; i < CE; ++i)
                if (col + i < mleft) {
                    if constexpr (ES == 4)
                        reinterpret_cast<float *>(d)[i] = reinterpret_cast<const float *>(s)[i];
                    else
                        reinterpret_cast<uint16_t *>(d)[i] = reinterpret_cast<const uint16_t *>(s)[i];
                }
        }
    }
    lds_wave_order();
}

} // namespace gq
