// i8_internal.h -- launchers of the 8-bit integer (int8) operators.  Arguments are already
// validated by i8_api.cpp when these are called: sizes positive, reduction lengths of integer
// sums at most 131071 (their 8-bit products then sum up in 32 bits), rows of codes a multiple
// of 16 bytes apart, at most 2^22 (256 rows' byte offsets fit 32 bits), pointers non-null and
// 16-byte aligned.
#pragma once

#include "mxfp4_internal.h" // element types

namespace gq {

// Codes [rows][ld], of which K of every row count, and a scale per row.  Every row has the
// bytes up to the next multiple of 16 behind it; what they hold is not used.
struct I8Mat {
    const int8_t *q;
    int64_t ld;
    const float *s;
};

// act(z) = z sigmoid(p(z)): p = z, or the tanh form of GELU.
constexpr int kSilu = 0, kGelu = 1;

hipError_t launch_quantize_i8(const void *x, int type, int64_t ldx, int8_t *q, int64_t ldq,
                              float *s, int64_t N, int64_t K, hipStream_t st);
hipError_t launch_dequant_i8(I8Mat w, void *out, int type, int64_t M, int64_t K, hipStream_t st);

// Whether B rows of K floats are quantised by the workgroups that multiply them; the next two
// take no others.
bool i8_fused(int64_t K, int64_t B);
// y[b][r] = sum_k w[r][k] x[b][k] with x quantised per row, 1 <= B <= 16, x and y of `type`.
hipError_t launch_gemv_i8(I8Mat w, const void *x, void *y, int type, int64_t M, int64_t K, int B,
                          hipStream_t st);
// Y[n][r] = sum_k w[r][k] x[n][k].
hipError_t launch_gemm_i8(I8Mat w, I8Mat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                          hipStream_t st);

// h[n][i] = act(g) u, g and u the products with gate and up; h dense [N][I] of `type`.
hipError_t launch_gated_i8(I8Mat gate, I8Mat up, I8Mat x, void *h, int type, int act, int64_t I,
                           int64_t H, int64_t N, hipStream_t st);
// The same from 1 to 16 float rows x [N][H], x and h of `type`.
hipError_t launch_gated_gemv_i8(I8Mat gate, I8Mat up, const void *x, void *h, int type, int act,
                                int64_t I, int64_t H, int N, hipStream_t st);
// The gradients of g and u for a gradient dh [N][I] of h (of `type`, 16 bits), each times its
// weight row's scale and 2^-e, e a whole number for each of the N rows: d [N][2][ldd] in binary16,
// zeros from I to the next multiple of 8, and e at grad_exponents(d, N, ldd).
hipError_t launch_gated_grads_i8(I8Mat gate, I8Mat up, I8Mat x, const uint16_t *dh, uint16_t *d,
                                 int64_t ldd, int type, int act, int64_t I, int64_t H, int64_t N,
                                 hipStream_t st);
// Behind d, 256-byte aligned as seen from it.
constexpr int64_t grad_exponent_bytes(int64_t N) { return (N * 4 + 255) / 256 * 256; }
inline int *grad_exponents(uint16_t *d, int64_t N, int64_t ldd)
{
    return reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(d) + (N * 2 * ldd * 2 + 255) / 256 * 256);
}

// dx[n][k] = sum over the parts p and rows m < M of d_p[n][m] w16_p[m][k], w16 each weight
// rounded to the 16-bit type of d and dx; rows of d are ldd elements apart, a multiple of 8, with
// zeros from M to the next multiple of 8.  scaled: d is launch_gated_grads_i8's, the weights are
// the codes, and sums are multiplied by 2^e.
struct I8GradPart {
    I8Mat w;
    const uint16_t *d;
};
// The workspace `partial`, this many bytes: for two parts (scaled) it begins with the e's,
// grad_exponent_bytes(N); the sum may be cut into runs, whose sums then go through the rest.
size_t grad_partial_bytes(int nparts, int64_t M, int64_t K, int64_t N);
hipError_t launch_grad_i8(const I8GradPart *parts, int nparts, bool scaled, int64_t ldd,
                          uint16_t *dx, int type, int64_t M, int64_t K, int64_t N, void *partial,
                          hipStream_t st);

// Rows of M 16-bit values, ldd apart, to rows ldo apart (a multiple of 8), zeros behind them.
hipError_t launch_align_rows(const uint16_t *d, int64_t ldd, uint16_t *out, int64_t ldo, int64_t M,
                             int64_t N, hipStream_t st);

// The workgroup-tile forms of the products, for more rows than the streaming kernels take.
hipError_t launch_i8_tiles(I8Mat w, I8Mat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                           hipStream_t st);
hipError_t launch_gated_tiles(I8Mat gate, I8Mat up, I8Mat x, void *h, int type, int act, int64_t I,
                              int64_t H, int64_t N, hipStream_t st);

// The feed-forward block; workspace regions off[]: codes of x, their scales, h, its codes,
// their scales, total.
struct I8FfnArgs {
    I8Mat gate, up, down;
    const uint16_t *x;
    uint16_t *out;
    int type, act;
    int64_t T, H, I;
    uint8_t *ws;
    size_t off[6];
};
hipError_t launch_ffn_i8(const I8FfnArgs &a, hipStream_t st);

} // namespace gq
