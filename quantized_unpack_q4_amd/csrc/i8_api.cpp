// i8_api.cpp -- the C ABI of the 8-bit integer (int8) operators: argument checks and
// launches, by the rules of gq_api.cpp.
#include "gq.h"

#include <hip/hip_runtime.h>
#include <string.h>

#include "gq_checks.h"
#include "i8_internal.h"

namespace {

using namespace gq::checks;

// Largest sizes: sums of 131071 products of codes (each at most 2^14) fit 32 bits; the tile
// kernels reach 256 rows of codes (16-bit gradients) by 32-bit byte offsets; a launch has
// fewer than 2^32 threads in a grid dimension.
constexpr int64_t kMaxK = 131071;
constexpr int64_t kMaxLd = (int64_t)1 << 22;
constexpr int64_t kMaxGradRows = (int64_t)1 << 22;
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

gq_status check_act(const char *fn, int act)
{
    if (act == GQ_SILU || act == GQ_GELU)
        return GQ_OK;
    return fail(GQ_EINVAL, "%s: act = %d must be GQ_SILU or GQ_GELU", fn, act);
}

gq_status check_most(const char *fn, const char *name, int64_t v, int64_t most)
{
    if (v > most)
        return fail(GQ_ESHAPE, "%s: %s = %lld exceeds the supported maximum %lld", fn, name,
                    (long long)v, (long long)most);
    return GQ_OK;
}

gq_status check_size(const char *fn, const char *name, int64_t v, int64_t most, bool allow_zero)
{
    GQ_TRY(check_dim(fn, name, v, allow_zero));
    return check_most(fn, name, v, most);
}

// The distance of rows of K codes.
gq_status check_ld(const char *fn, const char *name, int64_t ld, int64_t K, int64_t most)
{
    if (ld < K)
        return fail(GQ_ESHAPE, "%s: %s = %lld is below the %lld codes of a row", fn, name,
                    (long long)ld, (long long)K);
    if (ld % 16 != 0)
        return fail(GQ_EALIGN, "%s: rows of codes %s = %lld bytes apart do not all start 16-byte aligned",
                    fn, name, (long long)ld);
    return check_most(fn, name, ld, most);
}

gq_status check_values(const char *fn, const char *names, int64_t rows, int64_t K)
{
    if (rows > kMaxValues / K)
        return fail(GQ_ESHAPE, "%s: %s = %lld * %lld exceeds 2^34 values", fn, names,
                    (long long)rows, (long long)K);
    return GQ_OK;
}

gq_status product_sizes(const char *fn, const char *m, int64_t M, const char *k, int64_t K,
                        const char *n, int64_t N)
{
    GQ_TRY(check_size(fn, m, M, kMaxRows, true));
    GQ_TRY(check_size(fn, k, K, kMaxK, false));
    GQ_TRY(check_size(fn, n, N, kMaxTokens, true));
    return check_most(fn, "the number of outputs", M * N, kMaxOutputs);
}

gq_status check_ws(const char *fn, const char *name, const void *ws, size_t have, size_t need)
{
    if (!ws)
        return fail(GQ_EWORKSPACE, "%s: %s is NULL (needs %zu bytes)", fn, name, need);
    if (!aligned16(ws))
        return fail(GQ_EALIGN, "%s: %s (%p) is not 16-byte aligned", fn, name, ws);
    if (have < need)
        return fail(GQ_EWORKSPACE, "%s: ws_bytes = %zu is below the required %zu", fn, have, need);
    return GQ_OK;
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// The workspace of the matrix-vector product: codes, scales, total (zero where it takes none).
void gemv_layout(int64_t K, int64_t B, size_t off[3])
{
    const bool fused = B == 0 || gq::i8_fused(K, B);
    off[0] = 0;
    off[1] = fused ? 0 : up((size_t)(B * up16(K)));
    off[2] = fused ? 0 : up(off[1] + (size_t)B * 4);
}

// The sizes the feed-forward block takes, and its workspace's regions.
gq_status ffn_shape(const char *fn, int64_t T, int64_t H, int64_t I, size_t off[6])
{
    GQ_TRY(check_size(fn, "T", T, kMaxTokens, true));
    GQ_TRY(check_size(fn, "H", H, kMaxK, false));
    GQ_TRY(check_size(fn, "I", I, kMaxK, false));
    GQ_TRY(check_values(fn, "T*H", T, H));
    GQ_TRY(check_values(fn, "T*I", T, I));
    size_t o = 0;
    off[0] = o;
    o = up(o + (size_t)(T * up16(H)));
    off[1] = o;
    o = up(o + (size_t)T * 4);
    off[2] = o;
    o = up(o + (size_t)T * I * 2);
    off[3] = o;
    o = up(o + (size_t)(T * up16(I)));
    off[4] = o;
    o = up(o + (size_t)T * 4);
    off[5] = o;
    return GQ_OK;
}

// Gradients of the product: the sizes taken, and the workspace: dy's rows where they do not all
// start 16-byte aligned and hold a multiple of 8 values, the sums of its runs, total.
int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
gq_status gemm_backward_shape(const char *fn, int64_t M, int64_t K, int64_t N, int64_t ldd,
                              size_t off[3])
{
    GQ_TRY(check_size(fn, "M", M, kMaxGradRows, false));
    GQ_TRY(check_size(fn, "K", K, kMaxK, false));
    GQ_TRY(check_size(fn, "N", N, kMaxTokens, true));
    GQ_TRY(check_most(fn, "the number of outputs", N * K, kMaxOutputs));
    if (N > 1 && ldd < M)
        return fail(GQ_ESHAPE, "%s: ldd = %lld is below M = %lld", fn, (long long)ldd,
                    (long long)M);
    if (N > 1)
        GQ_TRY(check_most(fn, "ldd", ldd, kMaxGradRows));
    const bool align = N > 0 && (M % 8 != 0 || (N > 1 && ldd % 8 != 0));
    off[0] = 0;
    off[1] = align ? up((size_t)N * up8(M) * 2) : 0;
    off[2] = N > 0 ? off[1] + gq::grad_partial_bytes(1, M, K, N) : 0;
    return GQ_OK;
}

// The gated half's: the gradients of g and u, rows of each so many elements apart; their
// exponents (grad_exponents) and the sums of the runs; total.
int64_t grad_ld(int64_t I) { return (I + 63) / 64 * 64; }
gq_status gated_backward_shape(const char *fn, int64_t N, int64_t H, int64_t I, size_t off[3])
{
    GQ_TRY(product_sizes(fn, "I", I, "H", H, "N", N));
    GQ_TRY(check_most(fn, "I", I, kMaxGradRows / 2));
    GQ_TRY(check_most(fn, "N*H", N * H, kMaxOutputs));
    off[0] = 0;
    off[1] = up((size_t)N * 2 * grad_ld(I) * 2);
    off[2] = off[1] + (N > 0 && I > 0 ? gq::grad_partial_bytes(2, I, H, N) : 0);
    return GQ_OK;
}

template <class F>
size_t quietly(F shape, size_t *bytes)
{
    char saved[sizeof g_err];
    memcpy(saved, g_err, sizeof g_err);
    if (shape() != GQ_OK)
        return 0;
    memcpy(g_err, saved, sizeof g_err);
    return *bytes;
}

gq_status check_matrix(const char *fn, const char *q, const void *qp, const char *s, const void *sp)
{
    GQ_TRY(check_ptr(fn, q, qp));
    return check_ptr(fn, s, sp);
}

} // namespace

extern "C" {

gq_status gq_quantize_i8(const void *x, int x_type, int64_t ldx, int8_t *q, int64_t ldq, float *s,
                         int64_t N, int64_t K, void *stream)
{
    static const char fn[] = "gq_quantize_i8";
    GQ_TRY(check_type(fn, "x_type", x_type, true));
    GQ_TRY(check_dim(fn, "N", N, true));
    GQ_TRY(check_dim(fn, "K", K, false));
    GQ_TRY(check_values(fn, "N*K", N, K));
    GQ_TRY(check_ld(fn, "ldq", ldq, K, (int64_t)1 << 40));
    if (N == 0)
        return GQ_OK;
    if (ldx < K && N > 1)
        return fail(GQ_ESHAPE, "%s: ldx = %lld is below K = %lld", fn, (long long)ldx,
                    (long long)K);
    if (N > 1)
        GQ_TRY(check_most(fn, "ldx", ldx, (int64_t)1 << 40));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "q", q));
    GQ_TRY(check_ptr(fn, "s", s));
    return launched(fn, gq::launch_quantize_i8(x, x_type, N > 1 ? ldx : K, q, ldq, s, N, K,
                                               (hipStream_t)stream));
}

gq_status gq_dequant_i8(const int8_t *q, int64_t ldq, const float *s, void *out, int out_type,
                        int64_t M, int64_t K, void *stream)
{
    static const char fn[] = "gq_dequant_i8";
    GQ_TRY(check_type(fn, "out_type", out_type, true));
    GQ_TRY(check_dim(fn, "M", M, true));
    GQ_TRY(check_dim(fn, "K", K, false));
    GQ_TRY(check_values(fn, "M*K", M, K));
    GQ_TRY(check_ld(fn, "ldq", ldq, K, (int64_t)1 << 40));
    if (M == 0)
        return GQ_OK;
    GQ_TRY(check_ptr(fn, "q", q));
    GQ_TRY(check_ptr(fn, "s", s));
    GQ_TRY(check_ptr(fn, "out", out));
    return launched(fn, gq::launch_dequant_i8({q, ldq, s}, out, out_type, M, K, (hipStream_t)stream));
}

gq_status gq_gemv_i8(const int8_t *wq, int64_t ldw, const float *ws, const void *x, void *y,
                     int type, int64_t M, int64_t K, int64_t B, void *wsp, size_t ws_bytes,
                     void *stream)
{
    static const char fn[] = "gq_gemv_i8";
    GQ_TRY(check_type(fn, "type", type, true));
    if (B < 0 || B > GQ_GEMV_MAX_BATCH)
        return fail(GQ_EINVAL, "%s: B = %lld is outside [0, %d]", fn, (long long)B,
                    GQ_GEMV_MAX_BATCH);
    GQ_TRY(product_sizes(fn, "M", M, "K", K, "B", B));
    GQ_TRY(check_ld(fn, "ldw", ldw, K, kMaxLd));
    if (M == 0 || B == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq", wq, "ws", ws));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "y", y));
    size_t off[3];
    gemv_layout(K, B, off);
    if (off[2] == 0)
        return launched(fn, gq::launch_gemv_i8({wq, ldw, ws}, x, y, type, M, K, (int)B,
                                               (hipStream_t)stream));
    GQ_TRY(check_ws(fn, "wsp", wsp, ws_bytes, off[2]));
    int8_t *xq = (int8_t *)wsp;
    float *xs = (float *)((char *)wsp + off[1]);
    GQ_TRY(launched(fn, gq::launch_quantize_i8(x, type, K, xq, up16(K), xs, B, K,
                                               (hipStream_t)stream)));
    return launched(fn, gq::launch_gemm_i8({wq, ldw, ws}, {xq, up16(K), xs}, y, type, M, K, B,
                                           (hipStream_t)stream));
}

size_t gq_gemv_i8_workspace_bytes(int64_t K, int64_t B)
{
    static const char fn[] = "gq_gemv_i8_workspace_bytes";
    size_t off[3] = {};
    auto shape = [&] {
        if (B < 0 || B > GQ_GEMV_MAX_BATCH)
            return fail(GQ_EINVAL, "%s: B = %lld is outside [0, %d]", fn, (long long)B,
                        GQ_GEMV_MAX_BATCH);
        GQ_TRY(check_size(fn, "K", K, kMaxK, false));
        gemv_layout(K, B, off);
        return GQ_OK;
    };
    return quietly(shape, &off[2]);
}

gq_status gq_gemm_i8(const int8_t *wq, int64_t ldw, const float *ws, const int8_t *xq, int64_t ldx,
                     const float *xs, void *y, int y_type, int64_t M, int64_t K, int64_t N,
                     void *stream)
{
    static const char fn[] = "gq_gemm_i8";
    GQ_TRY(check_type(fn, "y_type", y_type, true));
    GQ_TRY(product_sizes(fn, "M", M, "K", K, "N", N));
    GQ_TRY(check_ld(fn, "ldw", ldw, K, kMaxLd));
    GQ_TRY(check_ld(fn, "ldx", ldx, K, kMaxLd));
    if (M == 0 || N == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq", wq, "ws", ws));
    GQ_TRY(check_matrix(fn, "xq", xq, "xs", xs));
    GQ_TRY(check_ptr(fn, "y", y));
    return launched(fn, gq::launch_gemm_i8({wq, ldw, ws}, {xq, ldx, xs}, y, y_type, M, K, N,
                                           (hipStream_t)stream));
}

gq_status gq_gemm_i8_backward(const int8_t *wq, int64_t ldw, const float *ws, const uint16_t *dy,
                              int64_t ldd, uint16_t *dx, int type, int64_t M, int64_t K, int64_t N,
                              void *wsp, size_t ws_bytes, void *stream)
{
    static const char fn[] = "gq_gemm_i8_backward";
    size_t off[3];
    GQ_TRY(check_type(fn, "type", type, false));
    GQ_TRY(gemm_backward_shape(fn, M, K, N, ldd, off));
    GQ_TRY(check_ld(fn, "ldw", ldw, K, kMaxLd));
    if (N == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq", wq, "ws", ws));
    GQ_TRY(check_ptr(fn, "dy", dy));
    GQ_TRY(check_ptr(fn, "dx", dx));
    if (off[2])
        GQ_TRY(check_ws(fn, "wsp", wsp, ws_bytes, off[2]));
    if (N == 1)
        ldd = up8(M);
    if (off[1]) {
        GQ_TRY(launched(fn, gq::launch_align_rows(dy, ldd, (uint16_t *)wsp, up8(M), M, N,
                                                  (hipStream_t)stream)));
        dy = (const uint16_t *)wsp;
        ldd = up8(M);
    }
    const gq::I8GradPart part{{wq, ldw, ws}, dy};
    return launched(fn, gq::launch_grad_i8(&part, 1, false, ldd, dx, type, M, K, N,
                                           (char *)wsp + off[1], (hipStream_t)stream));
}

size_t gq_gemm_i8_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t ldd)
{
    size_t off[3] = {};
    return quietly([&] { return gemm_backward_shape("gq_gemm_i8_backward_workspace_bytes", M, K, N, ldd, off); },
                   &off[2]);
}

gq_status gq_gated_i8(const int8_t *wq_gate, int64_t ld_gate, const float *ws_gate,
                      const int8_t *wq_up, int64_t ld_up, const float *ws_up, const int8_t *xq,
                      int64_t ldx, const float *xs, void *h, int h_type, int act, int64_t I,
                      int64_t H, int64_t N, void *stream)
{
    static const char fn[] = "gq_gated_i8";
    GQ_TRY(check_type(fn, "h_type", h_type, true));
    GQ_TRY(check_act(fn, act));
    GQ_TRY(product_sizes(fn, "I", I, "H", H, "N", N));
    GQ_TRY(check_ld(fn, "ld_gate", ld_gate, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ld_up", ld_up, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ldx", ldx, H, kMaxLd));
    if (I == 0 || N == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq_gate", wq_gate, "ws_gate", ws_gate));
    GQ_TRY(check_matrix(fn, "wq_up", wq_up, "ws_up", ws_up));
    GQ_TRY(check_matrix(fn, "xq", xq, "xs", xs));
    GQ_TRY(check_ptr(fn, "h", h));
    return launched(fn, gq::launch_gated_i8({wq_gate, ld_gate, ws_gate}, {wq_up, ld_up, ws_up},
                                            {xq, ldx, xs}, h, h_type, act, I, H, N,
                                            (hipStream_t)stream));
}

size_t gq_gated_i8_backward_workspace_bytes(int64_t N, int64_t H, int64_t I)
{
    size_t off[3] = {};
    return quietly([&] { return gated_backward_shape("gq_gated_i8_backward_workspace_bytes", N, H, I, off); },
                   &off[2]);
}

gq_status gq_gated_i8_backward(const int8_t *wq_gate, int64_t ld_gate, const float *ws_gate,
                               const int8_t *wq_up, int64_t ld_up, const float *ws_up,
                               const int8_t *xq, int64_t ldx, const float *xs, const uint16_t *dh,
                               uint16_t *dx, int type, int act, int64_t I, int64_t H, int64_t N,
                               void *ws, size_t ws_bytes, void *stream)
{
    static const char fn[] = "gq_gated_i8_backward";
    size_t off[3];
    GQ_TRY(check_type(fn, "type", type, false));
    GQ_TRY(check_act(fn, act));
    GQ_TRY(gated_backward_shape(fn, N, H, I, off));
    if (I == 0)
        return fail(GQ_EINVAL, "%s: I = 0 must be positive", fn);
    GQ_TRY(check_ld(fn, "ld_gate", ld_gate, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ld_up", ld_up, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ldx", ldx, H, kMaxLd));
    if (N == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq_gate", wq_gate, "ws_gate", ws_gate));
    GQ_TRY(check_matrix(fn, "wq_up", wq_up, "ws_up", ws_up));
    GQ_TRY(check_matrix(fn, "xq", xq, "xs", xs));
    GQ_TRY(check_ptr(fn, "dh", dh));
    GQ_TRY(check_ptr(fn, "dx", dx));
    GQ_TRY(check_ws(fn, "ws", ws, ws_bytes, off[2]));
    uint16_t *d = (uint16_t *)ws; // [N][2][ldd]: of g, of u
    const int64_t ldd = grad_ld(I);
    const gq::I8Mat gate{wq_gate, ld_gate, ws_gate}, upm{wq_up, ld_up, ws_up};
    GQ_TRY(launched(fn, gq::launch_gated_grads_i8(gate, upm, {xq, ldx, xs}, dh, d, ldd, type, act, I,
                                                  H, N, (hipStream_t)stream)));
    const gq::I8GradPart parts[2] = {{gate, d}, {upm, d + ldd}};
    return launched(fn, gq::launch_grad_i8(parts, 2, true, 2 * ldd, dx, type, I, H, N,
                                           (char *)ws + off[1], (hipStream_t)stream));
}

size_t gq_ffn_i8_workspace_bytes(int64_t T, int64_t H, int64_t I)
{
    size_t off[6] = {};
    return quietly([&] { return ffn_shape("gq_ffn_i8_workspace_bytes", T, H, I, off); }, &off[5]);
}

gq_status gq_ffn_i8(const int8_t *wq_gate, int64_t ld_gate, const float *ws_gate,
                    const int8_t *wq_up, int64_t ld_up, const float *ws_up, const int8_t *wq_down,
                    int64_t ld_down, const float *ws_down, const uint16_t *x, uint16_t *out,
                    int type, int act, int64_t T, int64_t H, int64_t I, void *ws, size_t ws_bytes,
                    void *stream)
{
    static const char fn[] = "gq_ffn_i8";
    gq::I8FfnArgs a{};
    GQ_TRY(check_type(fn, "type", type, false));
    GQ_TRY(check_act(fn, act));
    GQ_TRY(ffn_shape(fn, T, H, I, a.off));
    GQ_TRY(check_ld(fn, "ld_gate", ld_gate, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ld_up", ld_up, H, kMaxLd));
    GQ_TRY(check_ld(fn, "ld_down", ld_down, I, kMaxLd));
    if (T == 0)
        return GQ_OK;
    GQ_TRY(check_matrix(fn, "wq_gate", wq_gate, "ws_gate", ws_gate));
    GQ_TRY(check_matrix(fn, "wq_up", wq_up, "ws_up", ws_up));
    GQ_TRY(check_matrix(fn, "wq_down", wq_down, "ws_down", ws_down));
    GQ_TRY(check_ptr(fn, "x", x));
    GQ_TRY(check_ptr(fn, "out", out));
    GQ_TRY(check_ws(fn, "ws", ws, ws_bytes, a.off[5]));
    a.gate = {wq_gate, ld_gate, ws_gate};
    a.up = {wq_up, ld_up, ws_up};
    a.down = {wq_down, ld_down, ws_down};
    a.x = x;
    a.out = out;
    a.type = type;
    a.act = act;
    a.T = T;
    a.H = H;
    a.I = I;
    a.ws = (uint8_t *)ws;
    return launched(fn, gq::launch_ffn_i8(a, (hipStream_t)stream));
}

} // extern "C"
