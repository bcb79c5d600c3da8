// moe.hip -- grouping and combine steps of the mixture-of-experts layer.
//
// The pages' engines run mixture-of-experts checkpoints with their own expert
// routing (page "Frink Inference: the Rust alternative to llama.cpp", opening
// paragraph; page "Building a Rust Inference Engine That Matches
// Llama.cpp", section "Utility": OLMoE-1B-7B).  Given each token's top-k
// expert ids and weights, the layer here is four launches on one stream:
//   1. group    one workgroup counts assignments per expert, scans the counts,
//               lists the token tiles of every expert and gives each
//               (token, slot) assignment a stable position in expert order
//               (ties keep assignment order, so the result is deterministic);
//   2. gate/up  grouped matrix product with the SwiGLU epilogue (gemm.hip;
//               moe_skinny.hip when the experts average 48 tokens or fewer,
//               the 256 x 256 tiles of gemm_big.hip from 160 on);
//   3. down     grouped matrix product into binary32 rows (likewise);
//   4. combine  out[t] = sum over slots, in slot order, of weight * row.
// The layer over MXFP4 stacks (mxfp4_skinny.hip, mxfp4_tiles16.hip) shares 1 and 4.
// No atomics touch the outputs and nothing waits on the host.
#include "gq_device.h"
#include "gq_internal.h"
#include "mxfp4_device.h"

namespace gq {

constexpr int kMaxExperts = 256;
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / 64;
constexpr int kGroupBatch = 16;

hipError_t launch_moe_gemms(const MoeArgs &a, int bn, int max_tiles, hipStream_t s);

int moe_token_tile(int64_t assignments, int64_t experts)
{
    const int64_t mean = assignments / (experts > 0 ? experts : 1);
    return mean <= 48 ? 32 : mean <= 96 ? 64 : 128;
}

// Lanes of this wave whose valid expert id equals this lane's (8 ballots over
// the id bits, E <= 256).
__device__ __forceinline__ uint64_t same_expert_lanes(bool valid, int e)
{
    uint64_t peers = __ballot(valid);
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
        const bool set = valid && ((e >> bit) & 1);
        const uint64_t b = __ballot(set);
        peers &= set ? b : ~b;
    }
    return peers;
}

// Exclusive prefix sum of v over threads 0 .. 64*nw - 1 (nw <= 4 waves);
// every thread of the workgroup must call it.  Returns the exclusive prefix
// and sets *total.
__device__ __forceinline__ int block_exclusive_scan(int v, int nw, int *scratch, int *total)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(inc, off, 64);
        if (lane >= off)
            inc += u;
    }
    if (wave < nw && lane == 63)
        scratch[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        before += w < wave ? scratch[w] : 0;
        all += scratch[w];
    }
    __syncthreads();
    *total = all;
    return before + inc - v;
}

// offsets[0..E-1]: first sorted position of each expert; offsets[E]: number of
// valid assignments; offsets[E+1]: number of token tiles; offsets[E+2]:
// assignments dropped because their id lies outside [0, E).
//
// Wave w owns the contiguous slice [w*S, (w+1)*S) of the assignments: it
// counts its slice per expert (LDS adds into its own counters), one scan
// across waves and experts turns the counts into starting positions, and a
// second walk of the slice hands out positions in assignment order (ballot
// ranking among the lanes of a chunk with the same expert), so the order is
// stable by (expert, assignment index) and no atomic touches a position.  Both walks load the ids of up to
// kGroupBatch 64-id chunks at once before processing them in order, so a
// walk waits for one load latency per batch rather than one per chunk.
__global__ __launch_bounds__(kGroupThreads) void moe_group_kernel(
    const int32_t *__restrict__ ids, int A, int E, int BN, int max_tiles,
    int32_t *__restrict__ offsets, int32_t *__restrict__ sorted, int32_t *__restrict__ pos_of,
    int32_t *__restrict__ tiles)
{
    __shared__ int wstart[kGroupWaves][kMaxExperts]; // per wave: count, then first position
    __shared__ int wdrop[kGroupWaves];
    __shared__ int scratch[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int S = (A + kGroupWaves - 1) / kGroupWaves;
    const int a_begin = wave * S, a_end = min(A, a_begin + S);
    const uint64_t below = (lane == 0) ? 0ull : (~0ull >> (64 - lane));

    for (int i = tid; i < kGroupWaves * kMaxExperts; i += kGroupThreads)
        wstart[i / kMaxExperts][i % kMaxExperts] = 0;
    __syncthreads();

    // ids of chunks c0, c0 + 64, ... (kGroupBatch of them), -1 past the slice
    auto load_batch = [&](int c0, int (&ev)[kGroupBatch]) {
#pragma unroll
        for (int u = 0; u < kGroupBatch; ++u) {
            const int a = c0 + 64 * u + lane;
            ev[u] = a < a_end ? ids[a] : -1;
        }
    };

    // 1. per-wave counts
    int drop = 0;
    for (int c0 = a_begin; c0 < a_end; c0 += 64 * kGroupBatch) {
        int ev[kGroupBatch];
        load_batch(c0, ev);
#pragma unroll
        for (int u = 0; u < kGroupBatch; ++u) {
            const int a = c0 + 64 * u + lane;
            if (c0 + 64 * u >= a_end)
                break; // wave-uniform
            const int e = ev[u];
            const bool valid = e >= 0 && e < E;
            // counts only: one LDS add per assignment (a sum, so the order
            // of the adds does not matter)
            if (valid)
                atomicAdd(&wstart[wave][e], 1);
            drop += __popcll(__ballot(a < a_end && !valid));
        }
    }
    if (lane == 0)
        wdrop[wave] = drop;
    __syncthreads();

    // 2. per expert: total count, then expert bases and token tiles (scans
    // over experts, E <= 256 = 4 waves of threads)
    const int nw = (E + 63) / 64;
    int cnt = 0;
    if (tid < E) {
        for (int w = 0; w < kGroupWaves; ++w)
            cnt += wstart[w][tid];
    }
    int total_valid = 0, total_big = 0, total_small = 0;
    const int base = block_exclusive_scan(tid < E ? cnt : 0, nw, scratch, &total_valid);
    const int ntile = tid < E ? (cnt + BN - 1) / BN : 0;
    // tiles of 64 tokens or fewer (an expert's remainder when BN > 64) are
    // the cheapest: they go after every other tile, so that they fill the
    // last round of workgroups instead of leaving large tiles for it
    const int rem = tid < E ? cnt % BN : 0;
    const int nsmall = BN > 64 && rem > 0 && rem <= 64 ? 1 : 0;
    const int nbig = ntile - nsmall;
    const int tbase = block_exclusive_scan(nbig, nw, scratch, &total_big);
    const int sbase = block_exclusive_scan(nsmall, nw, scratch, &total_small);
    const int total_tiles = total_big + total_small;
    if (tid < E) {
        offsets[tid] = base;
        int run = base;
        for (int w = 0; w < kGroupWaves; ++w) {
            const int t = wstart[w][tid];
            wstart[w][tid] = run;
            run += t;
        }
        for (int i = 0; i < nbig; ++i) {
            tiles[tbase + i] = tid;
            tiles[max_tiles + tbase + i] = base + i * BN;
        }
        if (nsmall) {
            tiles[total_big + sbase] = tid;
            tiles[max_tiles + total_big + sbase] = base + nbig * BN;
        }
    }
    if (tid == 0) {
        int nd = 0;
        for (int w = 0; w < kGroupWaves; ++w)
            nd += wdrop[w];
        offsets[E] = total_valid;
        offsets[E + 1] = total_tiles;
        offsets[E + 2] = nd;
    }
    __syncthreads();

    // 3. positions, in assignment order within each wave's slice
    for (int c0 = a_begin; c0 < a_end; c0 += 64 * kGroupBatch) {
        int ev[kGroupBatch];
        load_batch(c0, ev);
#pragma unroll
        for (int u = 0; u < kGroupBatch; ++u) {
            const int a = c0 + 64 * u + lane;
            if (c0 + 64 * u >= a_end)
                break; // wave-uniform
            const int e = ev[u];
            const bool valid = e >= 0 && e < E;
            const uint64_t peers = same_expert_lanes(valid, e);
            const int rank = __popcll(peers & below);
            const int pos = valid ? wstart[wave][e] + rank : -1;
            if (valid && rank == 0)
                wstart[wave][e] += __popcll(peers);
            if (valid)
                sorted[pos] = a;
            if (a < a_end)
                pos_of[a] = pos;
        }
    }
}

// Adds the rows of N slots of a token from slot s0 on, in slot order; the rows are loaded
// at once.  Past the last slot that one is loaded again and not added.
template <int N>
__device__ __forceinline__ void combine_slots(const float *__restrict__ D,
                                              const int32_t *__restrict__ pos_of,
                                              const float *__restrict__ wts, int64_t first, int s0,
                                              int topk, int H, int c, bool unit, float4_t &a)
{
    int pos[N];
    float wgt[N];
    float4 d[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int64_t i = first + min(s0 + u, topk - 1);
        pos[u] = pos_of[i];
        wgt[u] = wts[i];
    }
#pragma unroll
    for (int u = 0; u < N; ++u) // (a dropped slot: any row, not added)
        d[u] = ldf4(D + (int64_t)max(pos[u], 0) * H + c);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (s0 + u >= topk || pos[u] < 0)
            continue;
        const float w = unit ? 1.f : wgt[u];
        a[0] = fmaf(w, d[u].x, a[0]);
        a[1] = fmaf(w, d[u].y, a[1]);
        a[2] = fmaf(w, d[u].z, a[2]);
        a[3] = fmaf(w, d[u].w, a[3]);
    }
}

// One thread per 4 output columns of one token; BF16: a bfloat16 output instead of binary16.
// The slots go N at a time (8: the rest as four, two or one).
template <bool BF16, int N>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float *__restrict__ D,
                                                          const int32_t *__restrict__ pos_of,
                                                          const float *__restrict__ wts,
                                                          uint16_t *__restrict__ out, int H,
                                                          int topk, int col_blocks, int unit)
{
    const int t = blockIdx.x / col_blocks;
    const int c = ((blockIdx.x % col_blocks) * 256 + threadIdx.x) * 4;
    if (c >= H)
        return;
    const int64_t first = (int64_t)t * topk;
    float4_t a = {0.f, 0.f, 0.f, 0.f};
    int s = 0;
    for (; topk - s > (N == 8 ? 4 : 0); s += N)
        combine_slots<N>(D, pos_of, wts, first, s, topk, H, c, unit, a);
    if constexpr (N == 8) {
        if (topk - s > 2)
            combine_slots<4>(D, pos_of, wts, first, s, topk, H, c, unit, a);
        else if (topk - s == 2)
            combine_slots<2>(D, pos_of, wts, first, s, topk, H, c, unit, a);
        else if (topk - s == 1)
            combine_slots<1>(D, pos_of, wts, first, s, topk, H, c, unit, a);
    }
    *reinterpret_cast<uint2 *>(out + (int64_t)t * H + c) =
        make_uint2(mx_pack2<BF16>(a[0], a[1]), mx_pack2<BF16>(a[2], a[3]));
}

hipError_t launch_moe_group(const int32_t *ids, uint8_t *ws, const size_t *off, int64_t A,
                            int64_t E, int bn, int max_tiles, hipStream_t s)
{
    hipLaunchKernelGGL(moe_group_kernel, dim3(1), dim3(kGroupThreads), 0, s, ids, (int)A, (int)E,
                       bn, max_tiles, reinterpret_cast<int32_t *>(ws + off[0]),
                       reinterpret_cast<int32_t *>(ws + off[1]),
                       reinterpret_cast<int32_t *>(ws + off[2]),
                       reinterpret_cast<int32_t *>(ws + off[3]));
    return hipGetLastError();
}

// Slots at a time: one where the device is full of workgroups (then the loads of others
// hide a load's latency), else all up to four, rounded up to a power of two, or eight.
// Measured, us for 1, 2, 4 and 8 at a time, hidden 2048: 4 tokens top-8 4.6, 3.9, 3.4, 3.0;
// 256 tokens top-8 5.4, 4.7, 4.3, 4.4; 2048 tokens top-8 20.8, 21.2, 21.2, 21.2 (inside
// the layer 21.4 and 22.6 for one and eight), top-2 7.6, 7.4, 7.5, 9.6, top-1 5.4, 5.8, 7.1, 9.4.
static int combine_slots_at_once(int64_t blocks, int64_t topk)
{
    return topk == 1 || blocks > 8 * device_cus() ? 1 : topk == 2 ? 2 : topk <= 4 ? 4 : 8;
}

template <bool BF16>
static void combine(const float *d, const int32_t *pos_of, const float *wts, uint16_t *out,
                    int64_t T, int H, int topk, int unit, hipStream_t s)
{
    const int col_blocks = (H / 4 + 255) / 256;
    const dim3 grid((unsigned)(T * col_blocks)), block(256);
    switch (combine_slots_at_once(T * col_blocks, topk)) {
    case 1:
        hipLaunchKernelGGL((moe_combine_kernel<BF16, 1>), grid, block, 0, s, d, pos_of, wts, out, H,
                           topk, col_blocks, unit);
        break;
    case 2:
        hipLaunchKernelGGL((moe_combine_kernel<BF16, 2>), grid, block, 0, s, d, pos_of, wts, out, H,
                           topk, col_blocks, unit);
        break;
    case 4:
        hipLaunchKernelGGL((moe_combine_kernel<BF16, 4>), grid, block, 0, s, d, pos_of, wts, out, H,
                           topk, col_blocks, unit);
        break;
    default:
        hipLaunchKernelGGL((moe_combine_kernel<BF16, 8>), grid, block, 0, s, d, pos_of, wts, out, H,
                           topk, col_blocks, unit);
    }
}

hipError_t launch_moe_combine(const float *d, const int32_t *pos_of, const float *wts,
                              uint16_t *out, bool bf16, int64_t T, int64_t H, int64_t topk,
                              bool unit, hipStream_t s)
{
    if (bf16)
        combine<true>(d, pos_of, wts, out, T, (int)H, (int)topk, (int)unit, s);
    else
        combine<false>(d, pos_of, wts, out, T, (int)H, (int)topk, (int)unit, s);
    return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs &a, hipStream_t s)
{
    const int64_t A = a.T * a.topk;
    // the 256 x 256 tiles take whole runs of 256 weights: Q8_0 stacks whose
    // H or I is not a multiple of 256 use the 128-row tile kernel instead
    const bool big = moe_big_applies(A, a.E, a.H, a.I) && (!a.q8_0 || a.I % 256 == 0);
    const int bn = big ? moe_big_token_tile() : moe_token_tile(A, a.E);
    const int max_tiles = (int)((A + bn - 1) / bn + a.E);
    hipError_t err = launch_moe_group(a.ids, a.ws, a.off, A, a.E, bn, max_tiles, s);
    if (err != hipSuccess)
        return err;
    err = big ? launch_moe_big(a, max_tiles, s)
              : moe_skinny_applies(A, a.E) ? launch_moe_skinny(a, s)
                                           : launch_moe_gemms(a, bn, max_tiles, s);
    if (err != hipSuccess)
        return err;
    return launch_moe_combine(reinterpret_cast<const float *>(a.ws + a.off[5]),
                              reinterpret_cast<const int32_t *>(a.ws + a.off[2]), a.wts, a.out,
                              false, a.T, a.H, a.topk, a.weight_input != 0, s);
}

} // namespace gq
