// mxfp4_krun.h -- how groups of waves share out the columns of an MXFP4 product with 16-bit
// activations, and how its scales are read.  Host and device.
#pragma once

#include <hip/hip_runtime.h>

namespace gq {

// How a row's scales reach the lanes: 16 bytes (512 columns) at a time through LDS where
// K % 512 == 0, by dwords through LDS where K % 128 == 0, else byte by byte.
enum { kScale1 = 0, kScale4 = 1, kScale16 = 2 };

// Whether KG groups of waves have a run of K each (else -1), and how its scales are read then.
template <int KG>
__host__ __device__ inline int scale_mode(int K)
{
    const int chunks = (K + 255) / 256;
    return chunks < KG ? -1 : K % 512 == 0 && chunks >= 2 * KG ? kScale16 : K % 128 == 0 ? kScale4 : kScale1;
}

// The run of K of one of KG groups of waves, in blocks of 32 columns: of the whole chunks
// of 256 columns (512 with kScale16; the last may be short) group g takes every KG-th part, at
// least one chunk each.
struct KRun {
    int first, blocks, longest;
};
template <int KG>
__host__ __device__ inline KRun k_run(int nblk, int mode, int g)
{
    if (KG == 1)
        return {0, nblk, nblk};
    const int unit = mode == kScale16 ? 16 : 8;
    const int units = (nblk + unit - 1) / unit;
    const int a = units * g / KG * unit, b = units * (g + 1) / KG * unit;
    return {a, (b < nblk ? b : nblk) - a, (units + KG - 1) / KG * unit};
}

} // namespace gq
