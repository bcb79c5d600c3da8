// Drives the C entry points of csrc/i8_api.cpp with counting stand-ins for its device
// launchers: refusals, the largest accepted sizes, workspaces, and the calls that do no work.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "gq.h"
#include "i8_internal.h"

static int g_launches = 0, g_failing = 0; // the g_failing-th launch fails
static hipError_t launch() { return ++g_launches == g_failing ? hipErrorInvalidValue : hipSuccess; }
namespace gq {
bool i8_fused(int64_t K, int64_t B) { return B * K <= 4096; }
size_t grad_partial_bytes(int parts, int64_t M, int64_t K, int64_t N)
{
    return M > 64 ? (size_t)(parts * N * K * 4) : 0;
}
hipError_t launch_quantize_i8(const void *, int, int64_t, int8_t *, int64_t, float *, int64_t, int64_t, hipStream_t)
{
    return launch();
}
hipError_t launch_dequant_i8(I8Mat, void *, int, int64_t, int64_t, hipStream_t) { return launch(); }
hipError_t launch_gemv_i8(I8Mat, const void *, void *, int, int64_t, int64_t, int, hipStream_t) { return launch(); }
hipError_t launch_gemm_i8(I8Mat, I8Mat, void *, int, int64_t, int64_t, int64_t, hipStream_t) { return launch(); }
hipError_t launch_gated_i8(I8Mat, I8Mat, I8Mat, void *, int, int, int64_t, int64_t, int64_t, hipStream_t)
{
    return launch();
}
hipError_t launch_gated_grads_i8(I8Mat, I8Mat, I8Mat, const uint16_t *, uint16_t *, int64_t, int, int, int64_t,
                                 int64_t, int64_t, hipStream_t)
{
    return launch();
}
hipError_t launch_grad_i8(const I8GradPart *, int, bool, int64_t, uint16_t *, int, int64_t, int64_t, int64_t, void *,
                          hipStream_t)
{
    return launch();
}
hipError_t launch_align_rows(const uint16_t *, int64_t, uint16_t *, int64_t, int64_t, int64_t, hipStream_t)
{
    return launch();
}
hipError_t launch_ffn_i8(const I8FfnArgs &, hipStream_t) { return launch(); }
} // namespace gq

static void expect(int line, gq_status got, gq_status want, int launches)
{
    if (got != want || g_launches != launches) {
        fprintf(stderr, "line %d: status %d, wanted %d; %d launches, wanted %d\n", line, (int)got,
                (int)want, g_launches, launches);
        exit(1);
    }
    g_launches = g_failing = 0;
}
static void require(int line, bool ok)
{
    if (!ok) {
        fprintf(stderr, "line %d\n", line);
        exit(1);
    }
}
#define REFUSED(want, call) expect(__LINE__, call, want, 0)
#define RUNS(n, call) expect(__LINE__, call, GQ_OK, n)
#define NOTHING(call) expect(__LINE__, call, GQ_OK, 0)
#define CHECK(cond) require(__LINE__, cond)

int main()
{
    alignas(16) static uint8_t mem[64];
    int8_t *q = (int8_t *)mem, *odd = (int8_t *)mem + 1;
    float *f = (float *)mem;
    uint16_t *h = (uint16_t *)mem;
    const int64_t big = INT64_MAX, n21 = (int64_t)1 << 21, m26 = (int64_t)1 << 26, ld22 = (int64_t)1 << 22;
    const size_t all = SIZE_MAX;

    for (int64_t bad : {(int64_t)-1, INT64_MIN, (int64_t)0, big}) {
        const gq_status st = bad <= 0 ? GQ_EINVAL : GQ_ESHAPE;
        REFUSED(st, gq_quantize_i8(q, GQ_F32, 64, q, 64, f, 2, bad, nullptr));
        REFUSED(st, gq_dequant_i8(q, 64, f, q, GQ_F32, 2, bad, nullptr));
        REFUSED(st, gq_gemv_i8(q, 64, f, q, q, GQ_F32, 2, bad, 1, nullptr, 0, nullptr));
        REFUSED(st, gq_gemm_i8(q, 64, f, q, 64, f, q, GQ_F32, 2, bad, 2, nullptr));
        REFUSED(st, gq_gemm_i8_backward(q, 64, f, h, 8, h, GQ_F16, 8, bad, 2, nullptr, 0, nullptr));
        REFUSED(st, gq_gemm_i8_backward(q, 64, f, h, 8, h, GQ_F16, bad, 64, 2, nullptr, 0, nullptr));
        REFUSED(st, gq_gated_i8(q, 64, f, q, 64, f, q, 64, f, q, GQ_F32, 0, 2, bad, 2, nullptr));
        REFUSED(st, gq_gated_i8_backward(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 0, 2, bad, 2, mem, all, nullptr));
        REFUSED(st, gq_gated_i8_backward(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 0, bad, 64, 2, mem, all, nullptr));
        REFUSED(st, gq_ffn_i8(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 0, 2, bad, 64, mem, all, nullptr));
        REFUSED(st, gq_ffn_i8(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 0, 2, 64, bad, mem, all, nullptr));
        CHECK(gq_gemv_i8_workspace_bytes(bad, 1) == 0);
        CHECK(gq_gemm_i8_backward_workspace_bytes(bad, 64, 2, 64) == 0);
        CHECK(gq_gated_i8_backward_workspace_bytes(2, bad, 64) == 0);
        CHECK(gq_ffn_i8_workspace_bytes(2, bad, 64) == 0 && gq_ffn_i8_workspace_bytes(2, 64, bad) == 0);
        if (bad) {
            REFUSED(st, gq_quantize_i8(q, GQ_F32, 64, q, 64, f, bad, 64, nullptr));
            REFUSED(st, gq_gemm_i8(q, 64, f, q, 64, f, q, GQ_F32, bad, 64, 2, nullptr));
            REFUSED(st, gq_gemm_i8(q, 64, f, q, 64, f, q, GQ_F32, 2, 64, bad, nullptr));
            REFUSED(st, gq_gemm_i8_backward(q, 64, f, h, 8, h, GQ_F16, 8, 64, bad, nullptr, 0, nullptr));
            REFUSED(st, gq_ffn_i8(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 0, bad, 64, 64, mem, all, nullptr));
            REFUSED(bad < 0 ? GQ_ESHAPE : GQ_EALIGN, gq_gemm_i8(q, bad, f, q, 64, f, q, GQ_F32, 2, 64, 2, nullptr));
            REFUSED(GQ_ESHAPE, gq_quantize_i8(q, GQ_F32, bad, q, 64, f, 2, 64, nullptr));
            REFUSED(GQ_ESHAPE, gq_gemm_i8_backward(q, 64, f, h, bad, h, GQ_F16, 8, 64, 2, nullptr, 0, nullptr));
        }
    }
    REFUSED(GQ_ESHAPE, gq_gemm_i8(q, big - 15, f, q, 64, f, q, GQ_F32, 2, 64, 2, nullptr));
    REFUSED(GQ_EALIGN, gq_quantize_i8(odd, GQ_F32, 64, q, 64, f, 2, 64, nullptr));
    REFUSED(GQ_EALIGN, gq_gemv_i8(odd, 64, f, q, q, GQ_F32, 2, 64, 1, nullptr, 0, nullptr));
    REFUSED(GQ_EINVAL, gq_gated_i8(q, 64, f, q, 64, nullptr, q, 64, f, q, GQ_F32, 0, 2, 64, 2, nullptr));

    // the largest sizes
    RUNS(1, gq_quantize_i8(q, GQ_BF16, (int64_t)1 << 40, q, (int64_t)1 << 40, f, (int64_t)1 << 4, (int64_t)1 << 30, nullptr));
    RUNS(1, gq_dequant_i8(q, 16, f, q, GQ_F16, (int64_t)1 << 30, 16, nullptr));
    RUNS(1, gq_gemm_i8(q, ld22, f, q, ld22, f, q, GQ_F32, m26, 131071, (int64_t)1 << 11, nullptr));
    RUNS(1, gq_gemm_i8(q, 131072, f, q, 131072, f, q, GQ_F32, (int64_t)1 << 16, 131071, n21, nullptr));
    REFUSED(GQ_ESHAPE, gq_gemm_i8(q, ld22 + 16, f, q, 64, f, q, GQ_F32, 2, 64, 2, nullptr));
    {
        const size_t need = gq_gemm_i8_backward_workspace_bytes(ld22, 16, n21, ld22);
        CHECK(need == (size_t)n21 * 16 * 4);
        RUNS(1, gq_gemm_i8_backward(q, 16, f, h, ld22, h, GQ_F16, ld22, 16, n21, mem, need, nullptr));
        REFUSED(GQ_EWORKSPACE, gq_gemm_i8_backward(q, 16, f, h, ld22, h, GQ_F16, ld22, 16, n21, mem, need - 1, nullptr));
        CHECK(gq_gated_i8_backward_workspace_bytes((int64_t)1 << 16, 16, n21) >= (size_t)n21 << 18);
        CHECK(gq_gated_i8_backward_workspace_bytes(n21, 16, n21) == 0); // more outputs than are taken
        CHECK(gq_gated_i8_backward_workspace_bytes(2, 16, n21 + 1) == 0);
        CHECK(gq_ffn_i8_workspace_bytes((int64_t)1 << 17, 131071, 131071) > (size_t)1 << 35);
        CHECK(gq_ffn_i8_workspace_bytes(((int64_t)1 << 17) + 2, 131071, 131071) == 0);
    }

    // one launch or two, with a workspace or without; the first may fail
    RUNS(1, gq_gemv_i8(q, 64, f, q, q, GQ_F32, 2, 64, 16, nullptr, 0, nullptr));
    {
        const size_t need = gq_gemv_i8_workspace_bytes(4097, 2);
        CHECK(need >= 2 * (4112 + 4));
        RUNS(2, gq_gemv_i8(q, 4112, f, q, q, GQ_F32, 2, 4097, 2, mem, need, nullptr));
        g_failing = 1;
        expect(__LINE__, gq_gemv_i8(q, 4112, f, q, q, GQ_F32, 2, 4097, 2, mem, need, nullptr), GQ_EHIP, 1);
        REFUSED(GQ_EWORKSPACE, gq_gemv_i8(q, 4112, f, q, q, GQ_F32, 2, 4097, 2, nullptr, need, nullptr));
    }
    RUNS(1, gq_gemm_i8_backward(q, 64, f, h, 8, h, GQ_BF16, 8, 64, 2, nullptr, 0, nullptr));
    RUNS(1, gq_gemm_i8_backward(q, 64, f, h, -5, h, GQ_BF16, 8, 64, 1, nullptr, 0, nullptr));
    RUNS(2, gq_gemm_i8_backward(q, 64, f, h, 9, h, GQ_BF16, 8, 64, 2, mem, 256, nullptr));
    RUNS(2, gq_gemm_i8_backward(q, 64, f, h, 0, h, GQ_BF16, 7, 64, 1, mem, 256, nullptr));
    g_failing = 1;
    expect(__LINE__, gq_gemm_i8_backward(q, 64, f, h, 9, h, GQ_BF16, 8, 64, 2, mem, 256, nullptr), GQ_EHIP, 1);
    {
        const size_t need = gq_gated_i8_backward_workspace_bytes(2, 64, 100);
        CHECK(need == 2 * 2 * 128 * 2 + 2 * 2 * 64 * 4);
        RUNS(2, gq_gated_i8_backward(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 1, 100, 64, 2, mem, need, nullptr));
        g_failing = 2;
        expect(__LINE__, gq_gated_i8_backward(q, 64, f, q, 64, f, q, 64, f, h, h, GQ_F16, 1, 100, 64, 2, mem, need, nullptr),
               GQ_EHIP, 2);
    }
    RUNS(1, gq_ffn_i8(q, 64, f, q, 64, f, q, 112, f, h, h, GQ_F16, 1, 2, 64, 100, mem,
                      gq_ffn_i8_workspace_bytes(2, 64, 100), nullptr));

    NOTHING(gq_quantize_i8(nullptr, GQ_F32, -1, nullptr, 64, nullptr, 0, 64, nullptr));
    NOTHING(gq_dequant_i8(nullptr, 64, nullptr, nullptr, GQ_F32, 0, 64, nullptr));
    NOTHING(gq_gemv_i8(nullptr, 4112, nullptr, nullptr, nullptr, GQ_F32, 0, 4097, 16, nullptr, 0, nullptr));
    NOTHING(gq_gemm_i8(nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, GQ_F32, 5, 64, 0, nullptr));
    NOTHING(gq_gemm_i8_backward(nullptr, 64, nullptr, nullptr, 0, nullptr, GQ_F16, 9, 64, 0, nullptr, 0, nullptr));
    NOTHING(gq_gated_i8(nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, GQ_F32, 0, 0, 64, 5, nullptr));
    NOTHING(gq_gated_i8_backward(nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, nullptr, GQ_F16,
                                 0, 8, 64, 0, nullptr, 0, nullptr));
    NOTHING(gq_ffn_i8(nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, 64, nullptr, nullptr, nullptr, GQ_F16, 0, 0, 64,
                      64, nullptr, 0, nullptr));
    printf("all checks passed\n");
    return 0;
}
