// gq_embed.cpp -- the C-ABI entry points of the embedding's lookup and
// gradient: argument checks, workspace and dispatch.  Contracts: include/gq.h.
#include <algorithm>
#include <cmath>

#include "gq_args.h"
#include "gq_embed.h"

using namespace gq;

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxCols = int64_t{1} << 24;

gq_status check_sizes(const char *op, int64_t tokens, int64_t rows, int64_t cols) {
    if (tokens < 0 || tokens > kMaxTokens || rows < 1 || rows > kMaxRows || cols < 1 ||
        cols > kMaxCols)
        return arg_fail(GQ_ERR_INVALID, op,
                        "tokens = %lld outside [0, 2^30], rows = %lld outside [1, 2^30], or "
                        "cols = %lld outside [1, 2^24]", static_cast<long long>(tokens),
                        static_cast<long long>(rows), static_cast<long long>(cols));
    return GQ_OK;
}

gq_status check_index(const char *op, const void *idx, int32_t idx_bytes, int64_t tokens) {
    if (idx_bytes != 4 && idx_bytes != 8)
        return arg_fail(GQ_ERR_INVALID, op, "idx_bytes = %d must be 4 or 8", idx_bytes);
    return tokens ? arg_ptr(op, "idx", idx, static_cast<uintptr_t>(idx_bytes)) : GQ_OK;
}

// `rows` rows of cols elements, ld apart (ld counts from two rows on).
gq_status check_rows(const char *op, const char *name, const void *p, gq_dtype dt, int64_t rows,
                     int64_t cols, int64_t &ld) {
    if (rows <= 1) ld = cols;
    if (ld < cols || (rows && ld > kMaxElems / rows))
        return arg_fail(GQ_ERR_INVALID, op,
                        "%s: row stride %lld below cols, or rows * stride above 2^40", name,
                        static_cast<long long>(ld));
    return rows ? arg_ptr(op, name, p, elem_bytes(dt)) : GQ_OK;
}

gq_status check_mul(const char *op, float mul) {
    if (!std::isfinite(mul))
        return arg_fail(GQ_ERR_INVALID, op, "mul = %g must be finite", static_cast<double>(mul));
    return GQ_OK;
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Whether one launch takes the gradient, in which the work group that has the most
// frequent token's row sums that row alone: up to EG_SMALL tokens, and 2^21 elements of dy,
// or 2^22 where the table is long and tokens are likely to be spread over more rows.  One
// launch costs by the most frequent token's elements, which the host does not know, and
// three by rows x columns of the table, so a bound on dy's elements is right for
// neither; it bounds what one launch can lose.  One launch / three, bf16 into fp32, the
// r-th most frequent token 1/r as often as the first:
//   added, 30522 rows: 2048 tokens of 2048 25 / 28 us, of 2049 32 / 33, 1024 of 4096
//   25 / 35, of 4100 38 / 38, 512 of 8192 25 / 51, and above the limit 512 of 8200 35 / 54,
//   512 of 12288 44 / 71, 64 of 66000 51 / 304;
//   the whole gradient: 512 of 8200 into 30522 228 / 214, 512 of 9000 into 16384 160 / 138,
//   1024 of 2048 into 200 17 / 22, 256 of 8192 into 100 22 / 19, of 8200 27 / 19,
//   2000 of 1100 into 173 29 / 23;
//   added, 2000 of 2048 into 30522 with 25, 50 and 100% of one token: 67 / 27, 126 / 27 and
//   244 / 23, 512 of 12288 124 / 71, 248 / 70 and 481 / 66.
bool is_small(int64_t tokens, int64_t rows, int64_t cols) {
    return tokens <= EG_SMALL && tokens * cols <= (rows >= 8192 ? 1 << 22 : 1 << 21);
}

// The parts of a gradient's workspace, and its bytes (at least 16).
struct Workspace {
    int64_t order = 0, piece_row = 0, keys = 0, part = 0, bytes = 16;
    int64_t pieces = 0;
};

Workspace grad_workspace(int64_t tokens, int64_t rows, int64_t cols) {
    Workspace w;
    if (is_small(tokens, rows, cols)) return w;
    w.pieces = (tokens + EG_PIECE - 1) / EG_PIECE;
    w.order = round16(4 * (rows + 1));
    w.piece_row = w.order + round16(4 * tokens);
    w.keys = w.piece_row + round16(4 * w.pieces);
    w.part = w.keys;
    if (tokens > EG_BLOCK * EG_HELD)
        w.part += 4 * ((tokens + EG_KEYS - 1) / EG_KEYS * EG_KEYS);
    w.bytes = w.part + w.pieces * 2 * 4 * ((cols + 511) / 512 * 512);
    return w;
}

}  // namespace

extern "C" {

gq_status gq_embed(const void *idx, int32_t idx_bytes, int64_t tokens, const void *table,
                   gq_dtype dt, int64_t rows, int64_t cols, int64_t ld, float mul,
                   gq_dtype out_dt, void *out, int64_t ldo, gq_stream stream) {
    const char *op = "gq_embed";
    GQ_ARG(check_sizes(op, tokens, rows, cols));
    GQ_ARG(arg_dtype(op, "dtype", dt));
    GQ_ARG(arg_dtype(op, "out's dtype", out_dt));
    GQ_ARG(check_mul(op, mul));
    GQ_ARG(check_index(op, idx, idx_bytes, tokens));
    GQ_ARG(check_rows(op, "table", table, dt, rows, cols, ld));
    GQ_ARG(check_rows(op, "out", out, out_dt, tokens, cols, ldo));
    if (!tokens) return arg_ok();
    const EmArgs a = {idx, table, out, tokens, rows, cols, ld, ldo, mul, idx_bytes == 8};
    return arg_launch(op, launch_embed(a, dt, out_dt, static_cast<hipStream_t>(stream)));
}

gq_status gq_embed_grad_workspace(int64_t tokens, int64_t rows, int64_t cols, int64_t *bytes) {
    const char *op = "gq_embed_grad_workspace";
    if (!bytes) return arg_fail(GQ_ERR_INVALID, op, "bytes is NULL");
    GQ_ARG(check_sizes(op, tokens, rows, cols));
    *bytes = grad_workspace(tokens, rows, cols).bytes;
    return arg_ok();
}

gq_status gq_embed_grad(const void *idx, int32_t idx_bytes, int64_t tokens, const void *dy,
                        gq_dtype dt, int64_t ldy, float mul, int64_t skip, int64_t rows,
                        int64_t cols, gq_dtype out_dt, int32_t accumulate, void *grad,
                        int64_t ldg, void *workspace, int64_t workspace_bytes,
                        gq_stream stream) {
    const char *op = "gq_embed_grad";
    GQ_ARG(check_sizes(op, tokens, rows, cols));
    GQ_ARG(arg_dtype(op, "dtype", dt));
    GQ_ARG(arg_dtype(op, "grad's dtype", out_dt));
    if (accumulate && out_dt != GQ_F32)
        return arg_fail(GQ_ERR_INVALID, op, "accumulate needs a GQ_F32 gradient");
    GQ_ARG(check_mul(op, mul));
    GQ_ARG(check_index(op, idx, idx_bytes, tokens));
    GQ_ARG(check_rows(op, "dy", dy, dt, tokens, cols, ldy));
    GQ_ARG(check_rows(op, "grad", grad, out_dt, rows, cols, ldg));
    GQ_ARG(arg_ptr(op, "workspace", workspace, 16));
    const Workspace w = grad_workspace(tokens, rows, cols);
    if (workspace_bytes < w.bytes)
        return arg_fail(GQ_ERR_CAPACITY, op, "workspace of %lld bytes, needs %lld",
                        static_cast<long long>(workspace_bytes), static_cast<long long>(w.bytes));
    if (!tokens && accumulate) return arg_ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool wide = idx_bytes == 8, add = accumulate != 0;
    if (is_small(tokens, rows, cols)) {
        // two work groups per compute unit
        const int64_t per = std::min<int64_t>(EG_SMALL_ROWS, (rows + 511) / 512);
        const EgSmallArgs a = {idx, dy,  grad, tokens, rows, cols, ldy, ldg, skip,
                               static_cast<int32_t>(per), mul, wide, add};
        return arg_launch(op, launch_embed_grad_small(a, dt, out_dt, st));
    }
    char *ws = static_cast<char *>(workspace);
    EgSortArgs sa = {};
    sa.idx = idx;
    sa.T = tokens;
    sa.rows = rows;
    sa.skip = skip;
    sa.keys = w.part > w.keys ? reinterpret_cast<uint32_t *>(ws + w.keys) : nullptr;
    sa.start = reinterpret_cast<int32_t *>(ws);
    sa.order = reinterpret_cast<int32_t *>(ws + w.order);
    sa.piece_row = reinterpret_cast<int32_t *>(ws + w.piece_row);
    // Rows without a token are cleared by the sort or, where they are nearly all and
    // long, beside the sums, by more waves (with as many reads as writes the two together
    // are slower).  fp32, by the sort / beside the sums: 4000 tokens into 262144
    // rows of 900 columns 257 / 202 us, 30000 of 300 123 / 112, 16384 into 30522 of
    // 1024 53 / 54, 131072 into 100003 of 2048 299 / 327.  (Eight rows are one wave's: of
    // few and very long rows the waves are few, and 3 tokens of 2^20 into 100 take 1230 us.)
    const bool apart = !add && rows / 4 >= tokens &&
                       cols * static_cast<int64_t>(elem_bytes(out_dt)) >= 1024;
    sa.grad = add || apart ? nullptr : static_cast<char *>(grad);
    sa.cols = cols;
    sa.ldg = ldg;
    sa.elem = static_cast<int32_t>(elem_bytes(out_dt));
    sa.rows_per = static_cast<int32_t>(std::min<int64_t>(EG_SORT_ROWS, (rows + 255) / 256));
    sa.wide = wide;
    const EgSumArgs ga = {dy, grad, sa.start, sa.order, sa.piece_row,
                          reinterpret_cast<float *>(ws + w.part),
                          rows, cols, ldy, ldg, w.pieces, 0, 0, mul, add, apart};
    hipError_t e = launch_embed_sort(sa, st);
    if (e == hipSuccess) e = launch_embed_sum(ga, dt, out_dt, st);
    if (e == hipSuccess) e = launch_embed_join(ga, dt, out_dt, st);
    return arg_launch(op, e);
}

}  // extern "C"
