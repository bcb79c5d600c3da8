// mxfp4_internal.h -- launchers of the microscaled 4-bit (MXFP4) operators.
// Arguments are already validated by mxfp4_api.cpp (sizes positive, K a
// multiple of 32 up to 2^22, which keeps the byte offsets of 256 rows of 16-bit values
// in 32 bits, pointers non-null and 16-byte aligned) when these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gq {

// Element types, the values of gq_dtype.
constexpr int kF32 = 0, kF16 = 1, kBF16 = 2;

// An MXFP4 matrix: codes [rows][K/2] and scales [rows][K/32].
struct MxMat {
    const uint8_t *q, *s;
};

hipError_t launch_quantize_mxfp4(const void *x, int type, int64_t ldx, uint8_t *q, uint8_t *s,
                                 int64_t N, int64_t K, hipStream_t st);
hipError_t launch_dequant_mxfp4(MxMat w, void *out, int type, int64_t M, int64_t K,
                                hipStream_t st);

// y[b][r] = sum_k w[r][k] x[b][k], binary32 activations, 1 <= B <= 16.
hipError_t launch_gemv_mxfp4(MxMat w, const float *x, float *y, int64_t M, int64_t K, int B,
                             hipStream_t st);
// Y[n][r] = sum_k w[r][k] X[n][k], X and Y of one 16-bit type.
hipError_t launch_gemm_mxfp4(MxMat w, const uint16_t *x, uint16_t *y, int type, int64_t M,
                             int64_t K, int64_t N, hipStream_t st);
// The same with MXFP4 activations; Y of any of the three types.
hipError_t launch_gemm_mxfp4_mxfp4(MxMat w, MxMat x, void *y, int type, int64_t M, int64_t K,
                                   int64_t N, hipStream_t st);

// Their workgroup-tile forms, for more than 16 activation rows.
hipError_t launch_gemm_tiles16(MxMat w, const uint16_t *x, uint16_t *y, int type, int64_t M,
                               int64_t K, int64_t N, hipStream_t st);
hipError_t launch_mx_tiles(MxMat w, MxMat x, void *y, int type, int64_t M, int64_t K, int64_t N,
                           hipStream_t st);

// The mixture-of-experts layer (workspace regions as in MoeArgs).
struct MxMoeArgs {
    MxMat gate, up, down; // E stacked matrices each
    const uint16_t *x;
    const int32_t *ids;
    const float *wts;
    uint16_t *out;
    int type; // kF16 or kBF16: x, h, out
    int64_t T, H, I, E, topk;
    uint8_t *ws;
    size_t off[7];
    int weight_input;
};
// Its expert products on tiles of so many tokens (0: use the weight-streaming kernel).
int moe_tile16_tokens(int64_t T, int64_t E, int64_t topk);
hipError_t launch_moe_tiles16(const MxMoeArgs &a, int tokens, int max_tiles, hipStream_t st);
hipError_t launch_moe_mxfp4(const MxMoeArgs &a, hipStream_t st);

// The grouping and combine launches of the mixture-of-experts layer (moe.hip):
// token tiles of bn sorted positions.
hipError_t launch_moe_group(const int32_t *ids, uint8_t *ws, const size_t *off, int64_t A,
                            int64_t E, int bn, int max_tiles, hipStream_t st);
hipError_t launch_moe_combine(const float *d, const int32_t *pos_of, const float *wts,
                              uint16_t *out, bool bf16, int64_t T, int64_t H, int64_t topk,
                              bool unit, hipStream_t st);

} // namespace gq
