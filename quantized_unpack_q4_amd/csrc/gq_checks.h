// gq_checks.h -- argument checks and the per-thread error message shared by the
// files of the C ABI.  Host only.
#pragma once

#include "gq.h"

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>

namespace gq {
namespace checks {

inline thread_local char g_err[512] = "";

inline gq_status fail(gq_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline gq_status check_ptr(const char *fn, const char *name, const void *p)
{
    if (!p)
        return fail(GQ_EINVAL, "%s: %s is NULL", fn, name);
    if (!aligned16(p))
        return fail(GQ_EALIGN, "%s: %s (%p) is not 16-byte aligned", fn, name, p);
    return GQ_OK;
}

// Sizes the kernels index with 32-bit row/column counts.
constexpr int64_t kMaxDim = (int64_t)1 << 30;

inline gq_status check_dim(const char *fn, const char *name, int64_t v, bool allow_zero)
{
    if (v < 0 || (!allow_zero && v == 0))
        return fail(GQ_EINVAL, "%s: %s = %lld must be %s", fn, name, (long long)v,
                    allow_zero ? "non-negative" : "positive");
    if (v > kMaxDim)
        return fail(GQ_ESHAPE, "%s: %s = %lld exceeds the supported maximum %lld", fn, name,
                    (long long)v, (long long)kMaxDim);
    return GQ_OK;
}

inline gq_status check_k(const char *fn, const char *name, int64_t K, int64_t block)
{
    gq_status st = check_dim(fn, name, K, false);
    if (st != GQ_OK)
        return st;
    if (K % block != 0)
        return fail(GQ_ESHAPE, "%s: %s = %lld is not a multiple of the %lld-weight block", fn,
                    name, (long long)K, (long long)block);
    return GQ_OK;
}

inline gq_status launched(const char *fn, hipError_t e)
{
    if (e != hipSuccess)
        return fail(GQ_EHIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return GQ_OK;
}

#define GQ_TRY(expr)                                                                           \
    do {                                                                                       \
        gq_status st_ = (expr);                                                                \
        if (st_ != GQ_OK)                                                                      \
            return st_;                                                                        \
    } while (0)

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Regions of the mixture-of-experts workspace (gq_moe_workspace_offsets); H and
// I are multiples of `block`.
inline gq_status moe_layout(const char *fn, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk,
                            int64_t block, size_t off[7])
{
    GQ_TRY(check_dim(fn, "T", T, true));
    GQ_TRY(check_k(fn, "H", H, block));
    GQ_TRY(check_k(fn, "I", I, block));
    if (E < 1 || E > 256)
        return fail(GQ_ESHAPE, "%s: E = %lld is outside the supported range [1, 256]", fn,
                    (long long)E);
    if (topk < 1 || topk > E)
        return fail(GQ_EINVAL, "%s: topk = %lld is outside [1, E = %lld]", fn, (long long)topk,
                    (long long)E);
    const int64_t A = T * topk;
    if (A > ((int64_t)1 << 20))
        return fail(GQ_ESHAPE, "%s: T*topk = %lld exceeds the supported maximum %lld", fn,
                    (long long)A, (long long)1 << 20);
    size_t o = 0;
    off[0] = o;
    o = up(o + (size_t)(E + 3) * 4);
    off[1] = o;
    o = up(o + (size_t)A * 4);
    off[2] = o;
    o = up(o + (size_t)A * 4);
    off[3] = o;
    o = up(o + (size_t)2 * (A + E) * 4);
    off[4] = o;
    o = up(o + (size_t)A * I * 2);
    off[5] = o;
    o = up(o + (size_t)A * H * 4);
    off[6] = o;
    return GQ_OK;
}

} // namespace checks
} // namespace gq
