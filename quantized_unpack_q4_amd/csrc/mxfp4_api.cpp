// mxfp4_api.cpp -- the C ABI of the microscaled 4-bit (MXFP4) operators: argument
// checks and launches, by the rules of gq_api.cpp.
#include "gq.h"

#include <hip/hip_runtime.h>
#include <string.h>

#include "gq_checks.h"
#include "mxfp4_internal.h"

namespace {

using namespace gq::checks;

// Largest sizes: a launch has fewer than 2^32 threads in a grid dimension, and the tile
// kernels reach 256 rows of K 16-bit values (the grouped one: all T rows of x) by 32-bit
// byte offsets.
constexpr int64_t kMaxK = (int64_t)1 << 22;
constexpr int64_t kMaxRows = (int64_t)1 << 26;
constexpr int64_t kMaxTokens = (int64_t)1 << 21;
constexpr int64_t kMaxOutputs = (int64_t)1 << 37;
constexpr int64_t kMaxValues = (int64_t)1 << 34;

gq_status check_type(const char *fn, const char *name, int type, bool f32)
{
    if (type == GQ_F16 || type == GQ_BF16 || (f32 && type == GQ_F32))
        return GQ_OK;
    return fail(GQ_EINVAL, "%s: %s = %d must be %sGQ_F16 or GQ_BF16", fn, name, type,
                f32 ? "GQ_F32, " : "");
}

gq_status check_most(const char *fn, const char *name, int64_t v, int64_t most)
{
    if (v > most)
        return fail(GQ_ESHAPE, "%s: %s = %lld exceeds the supported maximum %lld", fn, name,
                    (long long)v, (long long)most);
    return GQ_OK;
}

gq_status check_values(const char *fn, const char *names, int64_t rows, int64_t K)
{
    if (rows > kMaxValues / K)
        return fail(GQ_ESHAPE, "%s: %s = %lld * %lld exceeds 2^34 values", fn, names,
                    (long long)rows, (long long)K);
    return GQ_OK;
}

// The checks the three products share, without the activation pointers.
gq_status product_checks(const char *fn, int64_t M, int64_t K, int64_t N)
{
    GQ_TRY(check_dim(fn, "M", M, true));
    GQ_TRY(check_most(fn, "M", M, kMaxRows));
    GQ_TRY(check_k(fn, "K", K, 32));
    GQ_TRY(check_most(fn, "K", K, kMaxK));
    GQ_TRY(check_dim(fn, "N", N, true));
    GQ_TRY(check_most(fn, "N", N, kMaxTokens));
    return check_most(fn, "M*N", M * N, kMaxOutputs);
}

// The sizes the expert layer takes, and its workspace's regions.
gq_status moe_shape(const char *fn, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk,
                    size_t off[7])
{
    GQ_TRY(moe_layout(fn, T, H, I, E, topk, 32, off));
    GQ_TRY(check_most(fn, "H", H, kMaxK));
    GQ_TRY(check_most(fn, "I", I, kMaxK));
    return check_most(fn, "T*H", T * H, ((int64_t)1 << 31) - 1);
}

} // namespace

extern "C" {

gq_status gq_quantize_mxfp4(const void *x, int x_type, int64_t ldx, uint8_t *q, uint8_t *s,
                            int64_t N, int64_t K, void *stream)
{
    static const char fn[] = "gq_quantize_mxfp4";
    GQ_TRY(check_type(fn, "x_type", x_type, true));
    GQ_TRY(check_dim(fn, "N", N, true));
    GQ_TRY(check_k(fn, "K", K, 32));
    GQ_TRY(check_values(fn, "N*K", N, K));
    if (N == 0)
        return GQ_OK;
    if (ldx < K && N > 1)
        return fail(GQ_ESHAPE, "%s: ldx = %lld is below K = %lld", fn, (long long)ldx,
                    (long long)K);
    if (N > 1 && ldx > ((int64_t)1 << 40))
        return fail(GQ_ESHAPE, "%s: ldx = %lld exceeds 2^40", fn, (long long)ldx);
    if (N > 1 && ldx % (x_type == GQ_F32 ? 4 : 8) != 0)
        return fail(GQ_EALIGN, "%s: rows %lld elements apart do not all start 16-byte aligned", fn,
                    (long long)ldx);
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "q", q));
    GQ_TRY(check_ptr(fn, "s", s));
    return launched(fn, gq::launch_quantize_mxfp4(x, x_type, N > 1 ? ldx : K, q, s, N, K,
                                                  (hipStream_t)stream));
}

gq_status gq_dequant_mxfp4(const uint8_t *q, const uint8_t *s, void *out, int out_type, int64_t M,
                           int64_t K, void *stream)
{
    static const char fn[] = "gq_dequant_mxfp4";
    GQ_TRY(check_type(fn, "out_type", out_type, true));
    GQ_TRY(check_dim(fn, "M", M, true));
    GQ_TRY(check_k(fn, "K", K, 32));
    GQ_TRY(check_values(fn, "M*K", M, K));
    if (M == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "q", q));
    GQ_TRY(check_ptr(fn, "s", s));
    GQ_TRY(check_ptr(fn, "out", out));
    return launched(fn, gq::launch_dequant_mxfp4({q, s}, out, out_type, M, K, (hipStream_t)stream));
}

gq_status gq_gemv_mxfp4(const uint8_t *wq, const uint8_t *ws, const float *x, float *y, int64_t M,
                        int64_t K, int64_t B, void *stream)
{
    static const char fn[] = "gq_gemv_mxfp4";
    if (B < 0 || B > GQ_GEMV_MAX_BATCH)
        return fail(GQ_EINVAL, "%s: B = %lld is outside [0, %d]", fn, (long long)B,
                    GQ_GEMV_MAX_BATCH);
    GQ_TRY(product_checks(fn, M, K, B));
    if (M == 0 || B == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "wq", wq));
    GQ_TRY(check_ptr(fn, "ws", ws));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "y", y));
    return launched(fn, gq::launch_gemv_mxfp4({wq, ws}, x, y, M, K, (int)B, (hipStream_t)stream));
}

gq_status gq_gemm_mxfp4(const uint8_t *wq, const uint8_t *ws, const uint16_t *x, uint16_t *y,
                        int type, int64_t M, int64_t K, int64_t N, void *stream)
{
    static const char fn[] = "gq_gemm_mxfp4";
    GQ_TRY(check_type(fn, "type", type, false));
    GQ_TRY(product_checks(fn, M, K, N));
    if (M == 0 || N == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "wq", wq));
    GQ_TRY(check_ptr(fn, "ws", ws));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "y", y));
    return launched(fn, gq::launch_gemm_mxfp4({wq, ws}, x, y, type, M, K, N, (hipStream_t)stream));
}

gq_status gq_gemm_mxfp4_mxfp4(const uint8_t *wq, const uint8_t *ws, const uint8_t *xq,
                              const uint8_t *xs, void *y, int y_type, int64_t M, int64_t K,
                              int64_t N, void *stream)
{
    static const char fn[] = "gq_gemm_mxfp4_mxfp4";
    GQ_TRY(check_type(fn, "y_type", y_type, true));
    GQ_TRY(product_checks(fn, M, K, N));
    if (M == 0 || N == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "wq", wq));
    GQ_TRY(check_ptr(fn, "ws", ws));
    GQ_TRY(check_ptr(fn, "xq", xq));
    GQ_TRY(check_ptr(fn, "xs", xs));
    GQ_TRY(check_ptr(fn, "y", y));
    return launched(fn, gq::launch_gemm_mxfp4_mxfp4({wq, ws}, {xq, xs}, y, y_type, M, K, N,
                                                    (hipStream_t)stream));
}

size_t gq_moe_mxfp4_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk)
{
    size_t off[7];
    char saved[sizeof g_err];
    memcpy(saved, g_err, sizeof g_err);
    if (moe_shape("gq_moe_mxfp4_workspace_bytes", T, H, I, E, topk, off) != GQ_OK)
        return 0;
    memcpy(g_err, saved, sizeof g_err);
    return off[6];
}

gq_status gq_moe_mxfp4_workspace_offsets(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk,
                                         size_t off[7])
{
    static const char fn[] = "gq_moe_mxfp4_workspace_offsets";
    if (!off)
        return fail(GQ_EINVAL, "%s: off is NULL", fn);
    return moe_shape(fn, T, H, I, E, topk, off);
}

gq_status gq_moe_gemm_mxfp4(const uint8_t *wq_gate, const uint8_t *ws_gate, const uint8_t *wq_up,
                            const uint8_t *ws_up, const uint8_t *wq_down, const uint8_t *ws_down,
                            const uint16_t *x, const int32_t *topk_ids, const float *topk_w,
                            uint16_t *out, int type, int64_t T, int64_t H, int64_t I, int64_t E,
                            int64_t topk, int64_t input_weighted, void *ws, size_t ws_bytes,
                            void *stream)
{
    static const char fn[] = "gq_moe_gemm_mxfp4";
    gq::MxMoeArgs a{};
    GQ_TRY(check_type(fn, "type", type, false));
    GQ_TRY(moe_shape(fn, T, H, I, E, topk, a.off));
    if (T == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "wq_gate", wq_gate));
    GQ_TRY(check_ptr(fn, "ws_gate", ws_gate));
    GQ_TRY(check_ptr(fn, "wq_up", wq_up));
    GQ_TRY(check_ptr(fn, "ws_up", ws_up));
    GQ_TRY(check_ptr(fn, "wq_down", wq_down));
    GQ_TRY(check_ptr(fn, "ws_down", ws_down));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "topk_ids", topk_ids));
    GQ_TRY(check_ptr(fn, "topk_w", topk_w));
    GQ_TRY(check_ptr(fn, "out", out));
    if (!ws)
        return fail(GQ_EWORKSPACE, "%s: ws is NULL (needs %zu bytes)", fn, a.off[6]);
    if (!aligned16(ws))
        return fail(GQ_EALIGN, "%s: ws (%p) is not 16-byte aligned", fn, ws);
    if (ws_bytes < a.off[6])
        return fail(GQ_EWORKSPACE, "%s: ws_bytes = %zu is below the required %zu", fn, ws_bytes,
                    a.off[6]);
    a.gate = {wq_gate, ws_gate};
    a.up = {wq_up, ws_up};
    a.down = {wq_down, ws_down};
    a.x = x;
    a.ids = topk_ids;
    a.wts = topk_w;
    a.out = out;
    a.type = type;
    a.T = T;
    a.H = H;
    a.I = I;
    a.E = E;
    a.topk = topk;
    a.ws = (uint8_t *)ws;
    a.weight_input = input_weighted != 0;
    return launched(fn, gq::launch_moe_mxfp4(a, (hipStream_t)stream));
}

} // extern "C"
