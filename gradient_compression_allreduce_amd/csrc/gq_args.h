// gq_args.h -- argument checks of the C-ABI files (gq_mx4.cpp,
// gq_ortho.cpp, gq_tensors.cpp, gq_embed.cpp): each returns GQ_OK or sets the calling thread's error text.
// Not part of the ABI.
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

// Error reporting shared with gq_abi.cpp (GQ_OK clears the text).
extern "C" __attribute__((visibility("hidden"))) gq_status
gq_set_error_internal(gq_status code, const char *op, const char *what);

namespace gq {
namespace {

constexpr int64_t kMaxElems = int64_t{1} << 40;

__attribute__((format(printf, 3, 4))) gq_status arg_fail(gq_status code, const char *op,
                                                         const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return gq_set_error_internal(code, op, buf);
}

inline gq_status arg_ok() { return gq_set_error_internal(GQ_OK, "", ""); }

inline gq_status arg_ptr(const char *op, const char *name, const void *p, uintptr_t align) {
    if (!p) return arg_fail(GQ_ERR_INVALID, op, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return arg_fail(GQ_ERR_ALIGN, op, "%s = %p is not %d-byte aligned", name, p,
                        static_cast<int>(align));
    return GQ_OK;
}

template <typename P>
gq_status arg_ptrs(const char *op, const char *name, P const *arr, int32_t W, uintptr_t align) {
    if (!arr) return arg_fail(GQ_ERR_INVALID, op, "%s is NULL", name);
    for (int32_t w = 0; w < W; ++w) {
        if (!arr[w]) return arg_fail(GQ_ERR_INVALID, op, "%s[%d] is NULL", name, w);
        if (reinterpret_cast<uintptr_t>(arr[w]) % align)
            return arg_fail(GQ_ERR_ALIGN, op, "%s[%d] = %p is not %d-byte aligned", name, w,
                            static_cast<const void *>(arr[w]), static_cast<int>(align));
    }
    return GQ_OK;
}

inline gq_status arg_ranks(const char *op, int32_t W) {
    if (W < 1 || W > GQ_MAX_RANKS)
        return arg_fail(GQ_ERR_INVALID, op, "W = %d outside [1, %d]", W, GQ_MAX_RANKS);
    return GQ_OK;
}

inline gq_status arg_dtype(const char *op, const char *name, gq_dtype dt) {
    if (dt != GQ_F32 && dt != GQ_F16 && dt != GQ_BF16)
        return arg_fail(GQ_ERR_INVALID, op, "unknown %s %d", name, static_cast<int>(dt));
    return GQ_OK;
}

inline gq_status arg_mul(const char *op, float in_mul) {
    if (!std::isfinite(in_mul) || !(in_mul > 0.0f))
        return arg_fail(GQ_ERR_INVALID, op, "in_mul = %g must be finite and > 0",
                        static_cast<double>(in_mul));
    return GQ_OK;
}

// A matrix of rows x cols elements whose rows lie ld apart.
inline gq_status arg_matrix(const char *op, int64_t rows, int64_t cols, int64_t ld) {
    if (rows < 1 || cols < 1 || rows > kMaxElems || cols > kMaxElems)
        return arg_fail(GQ_ERR_INVALID, op, "rows = %lld, cols = %lld outside [1, 2^40]",
                        static_cast<long long>(rows), static_cast<long long>(cols));
    if (ld < cols || rows > kMaxElems / ld)
        return arg_fail(GQ_ERR_INVALID, op, "ld = %lld below cols, or rows * ld above 2^40",
                        static_cast<long long>(ld));
    return GQ_OK;
}

inline gq_status arg_launch(const char *op, hipError_t e) {
    if (e != hipSuccess)
        return arg_fail(GQ_ERR_HIP, op, "launch failed: %s", hipGetErrorString(e));
    return arg_ok();
}

inline size_t elem_bytes(gq_dtype dt) { return dt == GQ_F32 ? 4 : 2; }

#define GQ_ARG(expr)                      \
    do {                                  \
        const gq_status st_ = (expr);     \
        if (st_ != GQ_OK) return st_;     \
    } while (0)

}  // namespace
}  // namespace gq
