// Drives the C entry points of csrc/mxfp4_api.cpp with counting stand-ins for its device
// launchers: every refusal, the largest accepted sizes, and the calls that do no work.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "gq.h"
#include "mxfp4_internal.h"

static int g_launches = 0;
namespace gq {
hipError_t launch_quantize_mxfp4(const void *, int, int64_t, uint8_t *, uint8_t *, int64_t, int64_t, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_dequant_mxfp4(MxMat, void *, int, int64_t, int64_t, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_gemv_mxfp4(MxMat, const float *, float *, int64_t, int64_t, int, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_gemm_mxfp4(MxMat, const uint16_t *, uint16_t *, int, int64_t, int64_t, int64_t, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_gemm_mxfp4_mxfp4(MxMat, MxMat, void *, int, int64_t, int64_t, int64_t, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_moe_mxfp4(const MxMoeArgs &, hipStream_t)
{
    return ++g_launches, hipErrorInvalidValue;
}
} // namespace gq

static void expect(int line, gq_status got, gq_status want, int launches)
{
    if (got != want || g_launches != launches) {
        fprintf(stderr, "line %d: status %d, wanted %d; %d launches, wanted %d\n", line, (int)got,
                (int)want, g_launches, launches);
        exit(1);
    }
    g_launches = 0;
}
#define REFUSED(want, call) expect(__LINE__, call, want, 0)
#define RUNS(call) expect(__LINE__, call, GQ_OK, 1)
#define NOTHING(call) expect(__LINE__, call, GQ_OK, 0)

int main()
{
    alignas(16) static uint8_t mem[64];
    uint8_t *b = mem, *odd = mem + 1;
    float *f = (float *)mem;
    uint16_t *h = (uint16_t *)mem;
    const int64_t big = INT64_MAX, k22 = (int64_t)1 << 22, m26 = (int64_t)1 << 26, n21 = (int64_t)1 << 21;

    for (int64_t bad : {(int64_t)-1, INT64_MIN, (int64_t)0, big, (int64_t)33}) {
        const gq_status st = bad <= 0 ? GQ_EINVAL : GQ_ESHAPE;
        REFUSED(st, gq_quantize_mxfp4(f, GQ_F32, 32, b, b, 1, bad, nullptr));
        REFUSED(st, gq_dequant_mxfp4(b, b, f, GQ_F32, 1, bad, nullptr));
        REFUSED(st, gq_gemv_mxfp4(b, b, f, f, 16, bad, 1, nullptr));
        REFUSED(st, gq_gemm_mxfp4(b, b, h, h, GQ_F16, 16, bad, 1, nullptr));
        REFUSED(st, gq_gemm_mxfp4_mxfp4(b, b, b, b, f, GQ_F32, 16, bad, 1, nullptr));
    }
    for (int64_t bad : {(int64_t)-1, INT64_MIN, big}) {
        const gq_status st = bad <= 0 ? GQ_EINVAL : GQ_ESHAPE;
        REFUSED(st, gq_quantize_mxfp4(f, GQ_F32, 32, b, b, bad, 32, nullptr));
        REFUSED(st, gq_dequant_mxfp4(b, b, f, GQ_F32, bad, 32, nullptr));
        REFUSED(st, gq_gemv_mxfp4(b, b, f, f, bad, 32, 1, nullptr));
        REFUSED(GQ_EINVAL, gq_gemv_mxfp4(b, b, f, f, 16, 32, bad, nullptr));
        REFUSED(st, gq_gemm_mxfp4(b, b, h, h, GQ_F16, 16, 32, bad, nullptr));
        REFUSED(st, gq_gemm_mxfp4_mxfp4(b, b, b, b, f, GQ_F32, bad, 32, 1, nullptr));
    }
    for (int bad : {-1, 3, 1000}) {
        REFUSED(GQ_EINVAL, gq_quantize_mxfp4(f, bad, 32, b, b, 1, 32, nullptr));
        REFUSED(GQ_EINVAL, gq_dequant_mxfp4(b, b, f, bad, 1, 32, nullptr));
        REFUSED(GQ_EINVAL, gq_gemm_mxfp4(b, b, h, h, bad, 16, 32, 1, nullptr));
        REFUSED(GQ_EINVAL, gq_gemm_mxfp4_mxfp4(b, b, b, b, f, bad, 16, 32, 1, nullptr));
    }
    REFUSED(GQ_EINVAL, gq_gemm_mxfp4(b, b, h, h, GQ_F32, 16, 32, 1, nullptr));
    // strides
    REFUSED(GQ_ESHAPE, gq_quantize_mxfp4(f, GQ_F32, 31, b, b, 2, 32, nullptr));
    REFUSED(GQ_ESHAPE, gq_quantize_mxfp4(f, GQ_F32, big, b, b, 2, 32, nullptr));
    REFUSED(GQ_EALIGN, gq_quantize_mxfp4(f, GQ_F32, 34, b, b, 2, 32, nullptr));
    REFUSED(GQ_EALIGN, gq_quantize_mxfp4(f, GQ_F16, 36, b, b, 2, 32, nullptr));
    RUNS(gq_quantize_mxfp4(f, GQ_F32, 36, b, b, 2, 32, nullptr));
    RUNS(gq_quantize_mxfp4(f, GQ_F32, -5, b, b, 1, 32, nullptr));
    // the largest sizes, and one more
    RUNS(gq_gemv_mxfp4(b, b, f, f, m26, k22, 16, nullptr));
    REFUSED(GQ_ESHAPE, gq_gemv_mxfp4(b, b, f, f, m26 + 1, k22, 16, nullptr));
    REFUSED(GQ_ESHAPE, gq_gemv_mxfp4(b, b, f, f, 16, k22 + 32, 16, nullptr));
    REFUSED(GQ_EINVAL, gq_gemv_mxfp4(b, b, f, f, 16, 32, 17, nullptr));
    RUNS(gq_gemm_mxfp4(b, b, h, h, GQ_BF16, ((int64_t)1 << 16), k22, n21, nullptr));
    REFUSED(GQ_ESHAPE, gq_gemm_mxfp4(b, b, h, h, GQ_BF16, m26, 32, n21, nullptr));
    REFUSED(GQ_ESHAPE, gq_gemm_mxfp4(b, b, h, h, GQ_BF16, 1, 32, n21 + 1, nullptr));
    RUNS(gq_dequant_mxfp4(b, b, f, GQ_F32, (int64_t)1 << 29, 32, nullptr));
    REFUSED(GQ_ESHAPE, gq_dequant_mxfp4(b, b, f, GQ_F32, ((int64_t)1 << 29) + 1, 32, nullptr));
    // pointers
    REFUSED(GQ_EINVAL, gq_gemv_mxfp4(nullptr, b, f, f, 16, 32, 1, nullptr));
    REFUSED(GQ_EALIGN, gq_gemv_mxfp4(odd, b, f, f, 16, 32, 1, nullptr));
    REFUSED(GQ_EALIGN, gq_gemm_mxfp4_mxfp4(b, b, b, odd, f, GQ_F32, 16, 32, 1, nullptr));
    // no rows: no work, no pointers looked at
    NOTHING(gq_quantize_mxfp4(nullptr, GQ_F32, 0, nullptr, nullptr, 0, 32, nullptr));
    NOTHING(gq_gemv_mxfp4(nullptr, nullptr, nullptr, nullptr, 0, 32, 1, nullptr));
    NOTHING(gq_gemm_mxfp4(nullptr, nullptr, nullptr, nullptr, GQ_F16, 16, 32, 0, nullptr));
    NOTHING(gq_gemm_mxfp4_mxfp4(nullptr, nullptr, nullptr, nullptr, nullptr, GQ_F32, 0, 32, 1, nullptr));
    // the expert layer
    const size_t need = gq_moe_mxfp4_workspace_bytes(4, 64, 32, 8, 2);
    auto moe = [&](int type, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, void *ws, size_t bytes) {
        return gq_moe_gemm_mxfp4(b, b, b, b, b, b, h, (const int32_t *)mem, f, h, type, T, H, I, E, topk, 0,
                                 ws, bytes, nullptr);
    };
    if (!need || gq_moe_mxfp4_workspace_bytes(4, 33, 32, 8, 2) || gq_moe_mxfp4_workspace_bytes(big, 32, 32, 8, 2))
        return fprintf(stderr, "workspace bytes\n"), 1;
    expect(__LINE__, moe(GQ_F16, 4, 64, 32, 8, 2, b, need), GQ_EHIP, 1); // (the stand-in fails)
    REFUSED(GQ_EWORKSPACE, moe(GQ_F16, 4, 64, 32, 8, 2, b, need - 1));
    REFUSED(GQ_EWORKSPACE, moe(GQ_F16, 4, 64, 32, 8, 2, nullptr, need));
    REFUSED(GQ_EALIGN, moe(GQ_F16, 4, 64, 32, 8, 2, odd, need));
    REFUSED(GQ_EINVAL, moe(GQ_F32, 4, 64, 32, 8, 2, b, need));
    REFUSED(GQ_ESHAPE, moe(GQ_BF16, 4, 48, 32, 8, 2, b, need));
    REFUSED(GQ_ESHAPE, moe(GQ_BF16, 4, 64, 32, 257, 2, b, need));
    REFUSED(GQ_EINVAL, moe(GQ_BF16, 4, 64, 32, 8, 9, b, need));
    REFUSED(GQ_ESHAPE, moe(GQ_BF16, n21, 64, 32, 8, 1, b, SIZE_MAX));
    REFUSED(GQ_ESHAPE, moe(GQ_BF16, 1 << 20, 2048, 32, 8, 1, b, SIZE_MAX));
    REFUSED(GQ_ESHAPE, moe(GQ_BF16, 4, k22 + 32, 32, 8, 1, b, SIZE_MAX));
    NOTHING(moe(GQ_BF16, 0, 64, 32, 8, 2, nullptr, 0));
    puts("all checks passed");
    return 0;
}
