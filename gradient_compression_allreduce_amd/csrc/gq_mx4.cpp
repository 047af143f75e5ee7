// gq_mx4.cpp -- the C-ABI entry points of the microscaled 4-bit format:
// argument checks and dispatch.  Contracts: include/gq.h.
#include <cstring>

#include "gq_args.h"
#include "gq_mx4.h"
#include "gq_mx4_product.h"

using namespace gq;

namespace {

int64_t blocks(int64_t cols) { return (cols + MX_BLOCK - 1) / MX_BLOCK; }

// Short last blocks make the codes longer than the matrix: bounded apart.
gq_status check_blocks(const char *op, int64_t rows, int64_t cols) {
    if (rows > kMaxElems / (blocks(cols) * MX_BLOCK))
        return arg_fail(GQ_ERR_INVALID, op, "%lld rows of %lld blocks: above 2^40 codes",
                        static_cast<long long>(rows), static_cast<long long>(blocks(cols)));
    return GQ_OK;
}

gq_status check_product(const char *op, int64_t m, int64_t n, int64_t k) {
    if (m < 1 || n < 1 || m > (1 << 28) || n > (1 << 28) || m > (int64_t{1} << 36) / n)
        return arg_fail(GQ_ERR_INVALID, op,
                        "m = %lld, n = %lld outside [1, 2^28], or m * n above 2^36",
                        static_cast<long long>(m), static_cast<long long>(n));
    if (k < 1 || k > (1 << 24))
        return arg_fail(GQ_ERR_INVALID, op, "k = %lld outside [1, 2^24]",
                        static_cast<long long>(k));
    return GQ_OK;
}

int64_t product_workspace(int64_t m, int64_t n, int64_t k) {
    const MxPlan p = mx4_product_plan(m, n, k, true);
    return p.splits > 1 ? int64_t{4} * p.splits * m * n : 0;
}

gq_status fill_reduce(const char *op, const uint8_t *const *q, const uint8_t *const *scale,
                      int32_t W, int64_t rows, int64_t cols, MxRArgs &a) {
    GQ_ARG(arg_ranks(op, W));
    GQ_ARG(arg_matrix(op, rows, cols, cols));
    GQ_ARG(check_blocks(op, rows, cols));
    GQ_ARG(arg_ptrs(op, "q", q, W, 16));
    GQ_ARG(arg_ptrs(op, "scale", scale, W, 1));
    std::memset(&a, 0, sizeof a);
    for (int32_t w = 0; w < W; ++w) {
        a.q[w] = q[w];
        a.scale[w] = scale[w];
    }
    a.rows = rows;
    a.cols = cols;
    a.nb = blocks(cols);
    a.W = W;
    return GQ_OK;
}

}  // namespace

extern "C" {

gq_status gq_mx4_sizes(int64_t rows, int64_t cols, int64_t *n_scales, int64_t *code_bytes) {
    const char *op = "gq_mx4_sizes";
    GQ_ARG(arg_matrix(op, rows, cols, cols));
    GQ_ARG(check_blocks(op, rows, cols));
    if (n_scales) *n_scales = rows * blocks(cols);
    if (code_bytes) *code_bytes = rows * blocks(cols) * MX_BYTES;
    return arg_ok();
}

gq_status gq_mx4_quantize(const void *const *x, int32_t W, gq_dtype dt, float in_mul, int64_t rows,
                          int64_t cols, int64_t ld, int32_t transpose, uint8_t *const *scale_out,
                          uint8_t *const *q_out, gq_stream stream) {
    const char *op = "gq_mx4_quantize";
    GQ_ARG(arg_ranks(op, W));
    GQ_ARG(arg_dtype(op, "dtype", dt));
    GQ_ARG(arg_mul(op, in_mul));
    if (rows == 1) ld = cols;
    GQ_ARG(arg_matrix(op, rows, cols, ld));
    if (transpose) GQ_ARG(check_blocks(op, cols, rows));
    else GQ_ARG(check_blocks(op, rows, cols));
    GQ_ARG(arg_ptrs(op, "x", x, W, 16));
    GQ_ARG(arg_ptrs(op, "scale_out", scale_out, W, 1));
    GQ_ARG(arg_ptrs(op, "q_out", q_out, W, 16));
    MxQArgs a;
    std::memset(&a, 0, sizeof a);
    for (int32_t w = 0; w < W; ++w) {
        a.x[w] = x[w];
        a.scale[w] = scale_out[w];
        a.q[w] = q_out[w];
    }
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.in_mul = in_mul;
    a.W = W;
    return arg_launch(op, launch_mx4_quantize(a, dt, transpose != 0,
                                              static_cast<hipStream_t>(stream)));
}

gq_status gq_mx4_reduce_dequant(const uint8_t *const *q, const uint8_t *const *scale, int32_t W,
                                int64_t rows, int64_t cols, float *r_out, gq_stream stream) {
    const char *op = "gq_mx4_reduce_dequant";
    MxRArgs a;
    GQ_ARG(fill_reduce(op, q, scale, W, rows, cols, a));
    GQ_ARG(arg_ptr(op, "r_out", r_out, 16));
    a.r = r_out;
    return arg_launch(op, launch_mx4_reduce(a, static_cast<hipStream_t>(stream)));
}

gq_status gq_mx4_reduce_requantize(const uint8_t *const *q, const uint8_t *const *scale, int32_t W,
                                   int64_t rows, int64_t cols, float *r_out, uint8_t *scale_out,
                                   uint8_t *q_out, gq_stream stream) {
    const char *op = "gq_mx4_reduce_requantize";
    MxRArgs a;
    GQ_ARG(fill_reduce(op, q, scale, W, rows, cols, a));
    if (r_out) GQ_ARG(arg_ptr(op, "r_out", r_out, 16));
    GQ_ARG(arg_ptr(op, "scale_out", scale_out, 1));
    GQ_ARG(arg_ptr(op, "q_out", q_out, 16));
    a.r = r_out;
    a.scale_out = scale_out;
    a.q_out = q_out;
    return arg_launch(op, launch_mx4_reduce(a, static_cast<hipStream_t>(stream)));
}

gq_status gq_mx4_product_workspace(int64_t m, int64_t n, int64_t k, int64_t *bytes) {
    const char *op = "gq_mx4_product_workspace";
    GQ_ARG(check_product(op, m, n, k));
    if (!bytes) return arg_fail(GQ_ERR_INVALID, op, "bytes is NULL");
    *bytes = product_workspace(m, n, k);
    return arg_ok();
}

gq_status gq_mx4_product(const uint8_t *a, const uint8_t *a_scale, const uint8_t *b,
                         const uint8_t *b_scale, int64_t m, int64_t n, int64_t k, gq_dtype dt,
                         int32_t accumulate, void *c, int64_t ldc, void *workspace,
                         int64_t workspace_bytes, gq_stream stream) {
    const char *op = "gq_mx4_product";
    GQ_ARG(check_product(op, m, n, k));
    GQ_ARG(arg_dtype(op, "dtype", dt));
    if (accumulate && dt != GQ_F32)
        return arg_fail(GQ_ERR_INVALID, op, "accumulate needs a GQ_F32 result");
    if (m == 1) ldc = n;
    GQ_ARG(arg_matrix(op, m, n, ldc));
    GQ_ARG(arg_ptr(op, "a", a, 16));
    GQ_ARG(arg_ptr(op, "a_scale", a_scale, 1));
    GQ_ARG(arg_ptr(op, "b", b, 16));
    GQ_ARG(arg_ptr(op, "b_scale", b_scale, 1));
    GQ_ARG(arg_ptr(op, "c", c, elem_bytes(dt)));
    if (workspace) {
        GQ_ARG(arg_ptr(op, "workspace", workspace, 16));
        const int64_t need = product_workspace(m, n, k);
        if (workspace_bytes < need)
            return arg_fail(GQ_ERR_CAPACITY, op, "workspace of %lld bytes, needs %lld",
                            static_cast<long long>(workspace_bytes),
                            static_cast<long long>(need));
    }
    MxPArgs p;
    std::memset(&p, 0, sizeof p);
    p.a = a;
    p.sa = a_scale;
    p.b = b;
    p.sb = b_scale;
    p.c = c;
    p.part = static_cast<float *>(workspace);
    p.m = m;
    p.n = n;
    p.nb = blocks(k);
    p.ldc = ldc;
    const size_t quad = 4 * elem_bytes(dt);
    p.vec = ldc % 4 == 0 && reinterpret_cast<uintptr_t>(c) % quad == 0;
    p.add = accumulate != 0;
    return arg_launch(op, launch_mx4_product(p, k, dt, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
