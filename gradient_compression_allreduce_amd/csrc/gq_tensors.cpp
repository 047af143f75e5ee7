// gq_tensors.cpp -- the C-ABI entry points of tensor lists: the list (its
// tensors cut into tiles, and the norm's scratch memory), the norm and the
// clip.  Contracts: include/gq.h.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <vector>

#include "gq_args.h"
#include "gq_tensors.h"

using namespace gq;

namespace {

// The bytes of one tensor.
struct Span {
    uintptr_t begin, end;
};

}  // namespace

struct gq_tensors {
    int device = -1;
    int64_t n = 0, count = 0, n_tiles = 0, n_longs = 0, bytes = 0;
    int64_t data_bytes = 0;             // of the tensors
    std::vector<int64_t> numel;
    std::vector<Span> spans;            // of the tensors that are not empty, in order
    char *d_mem = nullptr;              // one allocation, parted as below
    TnTile *d_tiles = nullptr;
    TnLong *d_longs = nullptr;
    double *d_parts = nullptr, *d_sums = nullptr;
    uint32_t *d_ticket = nullptr;
};

namespace {

constexpr int64_t kMaxCount = 1 << 20;
constexpr int64_t kMaxTotal = int64_t{1} << 36;     // at most 2^24 + 2^20 tiles

bool span_before(const Span &a, const Span &b) { return a.begin < b.begin; }

// Whether a tensor of one list shares memory with one of another.
bool overlap(const std::vector<Span> &a, const std::vector<Span> &b) {
    size_t i = 0, j = 0;
    if (a.empty() || b.empty() || a.back().end <= b.front().begin ||
        b.back().end <= a.front().begin)
        return false;
    while (i < a.size() && j < b.size()) {
        if (a[i].end <= b[j].begin) ++i;
        else if (b[j].end <= a[i].begin) ++j;
        else return true;
    }
    return false;
}

// Whether `bytes` bytes from p on share memory with a tensor of a list.
bool touches(const std::vector<Span> &spans, const void *p, int64_t bytes) {
    const Span at = {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes};
    // the first tensor that ends behind p (they lie in order and apart)
    const auto first = std::partition_point(spans.begin(), spans.end(),
                                            [&](const Span &s) { return s.end <= at.begin; });
    return first != spans.end() && first->begin < at.end;
}

gq_status tensors_create(const char *op, void *const *x, const int64_t *numel, const gq_dtype *dt,
                         int64_t count, gq_tensors **out) {
    std::vector<Span> spans;
    std::vector<TnTile> tiles;
    std::vector<TnLong> longs;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        GQ_ARG(arg_dtype(op, "dtype", dt[i]));
        if (numel[i] < 0 || numel[i] > kMaxTotal - total)
            return arg_fail(GQ_ERR_INVALID, op,
                            "tensor %lld of %lld elements: a length below 0, or more than 2^36 "
                            "elements together", static_cast<long long>(i),
                            static_cast<long long>(numel[i]));
        total += numel[i];
        if (!numel[i]) continue;
        GQ_ARG(arg_ptr(op, "a tensor", x[i], elem_bytes(dt[i])));
        const uintptr_t p = reinterpret_cast<uintptr_t>(x[i]);
        spans.push_back({p, p + numel[i] * elem_bytes(dt[i])});
    }
    std::sort(spans.begin(), spans.end(), span_before);
    for (size_t i = 1; i < spans.size(); ++i)
        if (spans[i].begin < spans[i - 1].end)
            return arg_fail(GQ_ERR_INVALID, op, "two tensors of the list share memory at %p",
                            reinterpret_cast<void *>(spans[i].begin));
    for (int64_t i = 0; i < count; ++i) {
        const int64_t at = static_cast<int64_t>(tiles.size());
        const bool one = numel[i] <= TN_TILE;
        for (int64_t e = 0; e < numel[i]; e += TN_TILE)
            tiles.push_back({static_cast<char *>(x[i]) + e * elem_bytes(dt[i]),
                             static_cast<uint32_t>(std::min<int64_t>(TN_TILE, numel[i] - e)) |
                                 static_cast<uint32_t>(dt[i]) << 16,
                             one ? static_cast<int32_t>(i) : -1});
        // (an empty tensor's norm is the sum over no tiles)
        if (!one || !numel[i]) longs.push_back({at, static_cast<int64_t>(tiles.size()), i});
    }

    std::unique_ptr<gq_tensors> T(new gq_tensors);
    T->n = total;
    T->count = count;
    T->n_tiles = static_cast<int64_t>(tiles.size());
    T->numel.assign(numel, numel + count);
    for (const Span &s : spans) T->data_bytes += static_cast<int64_t>(s.end - s.begin);
    T->spans = std::move(spans);
    hipError_t e = hipGetDevice(&T->device);
    T->n_longs = static_cast<int64_t>(longs.size());
    const size_t at_longs = tiles.size() * sizeof(TnTile);
    const size_t at_sums = at_longs + longs.size() * sizeof(TnLong);
    const size_t at_parts = at_sums + tiles.size() * sizeof(double);
    const size_t at_ticket = at_parts + TN_MAX_GRID * sizeof(double);
    T->bytes = static_cast<int64_t>(at_ticket + sizeof(uint64_t));
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void **>(&T->d_mem), T->bytes);
    if (e == hipSuccess) {
        T->d_tiles = reinterpret_cast<TnTile *>(T->d_mem);
        T->d_longs = reinterpret_cast<TnLong *>(T->d_mem + at_longs);
        T->d_sums = reinterpret_cast<double *>(T->d_mem + at_sums);
        T->d_parts = reinterpret_cast<double *>(T->d_mem + at_parts);
        T->d_ticket = reinterpret_cast<uint32_t *>(T->d_mem + at_ticket);
        if (!tiles.empty())
            e = hipMemcpy(T->d_tiles, tiles.data(), at_longs, hipMemcpyHostToDevice);
    }
    if (e == hipSuccess && !longs.empty())
        e = hipMemcpy(T->d_longs, longs.data(), longs.size() * sizeof(TnLong),
                      hipMemcpyHostToDevice);
    const uint64_t zero = 0;
    if (e == hipSuccess) e = hipMemcpy(T->d_ticket, &zero, sizeof zero, hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        const long long size = T->bytes;
        if (T->d_mem) (void)hipFree(T->d_mem);
        (void)hipGetLastError();        // (or the thread's next launch would report it)
        return arg_fail(GQ_ERR_HIP, op, "making a list of %lld bytes failed: %s", size,
                        hipGetErrorString(e));
    }
    *out = T.release();
    return arg_ok();
}

gq_status check_list(const char *op, const char *name, const gq_tensors *t) {
    if (!t) return arg_fail(GQ_ERR_INVALID, op, "%s is NULL", name);
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return arg_fail(GQ_ERR_HIP, op, "hipGetDevice failed");
    if (dev != t->device)
        return arg_fail(GQ_ERR_DEVICE, op, "current device %d, %s lives on device %d", dev, name,
                        t->device);
    return GQ_OK;
}

}  // namespace

extern "C" {

gq_status gq_tensors_create(void *const *x, const int64_t *numel, const gq_dtype *dt,
                            int64_t count, gq_tensors **out) {
    const char *op = "gq_tensors_create";
    if (!out) return arg_fail(GQ_ERR_INVALID, op, "out is NULL");
    *out = nullptr;
    if (!x || !numel || !dt) return arg_fail(GQ_ERR_INVALID, op, "x, numel or dt is NULL");
    if (count < 1 || count > kMaxCount)
        return arg_fail(GQ_ERR_INVALID, op, "count = %lld outside [1, 2^20]",
                        static_cast<long long>(count));
    try {
        return tensors_create(op, x, numel, dt, count, out);
    } catch (const std::bad_alloc &) {
        return arg_fail(GQ_ERR_INVALID, op, "out of host memory");
    }
}

gq_status gq_tensors_destroy(gq_tensors *t) {
    if (!t) return arg_ok();
    if (t->d_mem) (void)hipFree(t->d_mem);
    delete t;
    return arg_ok();
}

gq_status gq_tensors_info(const gq_tensors *t, int64_t *n, int64_t *count, int64_t *bytes) {
    if (!t) return arg_fail(GQ_ERR_INVALID, "gq_tensors_info", "list is NULL");
    if (n) *n = t->n;
    if (count) *count = t->count;
    if (bytes) *bytes = t->bytes;
    return arg_ok();
}

gq_status gq_tensors_norm(gq_tensors *t, float in_mul, float *norm, float *norms,
                          gq_stream stream) {
    const char *op = "gq_tensors_norm";
    GQ_ARG(arg_mul(op, in_mul));
    GQ_ARG(arg_ptr(op, "norm", norm, 4));
    if (norms) GQ_ARG(arg_ptr(op, "norms", norms, 4));
    GQ_ARG(check_list(op, "the list", t));
    const int64_t norms_bytes = norms ? 4 * t->count : 0;
    if (touches(t->spans, norm, 4) || touches(t->spans, norms, norms_bytes))
        return arg_fail(GQ_ERR_INVALID, op, "norm or norms lies in a tensor of the list");
    if (norm >= norms && norm < norms + norms_bytes / 4)
        return arg_fail(GQ_ERR_INVALID, op, "norm is one of norms");
    hipStream_t st = static_cast<hipStream_t>(stream);
    const TnNormArgs a = {t->d_tiles, t->n_tiles, t->d_parts, t->d_sums, t->d_ticket, norm, norms,
                          in_mul, t->data_bytes > TN_CACHED};
    hipError_t e = launch_tensors_norm(a, st);
    if (e == hipSuccess && norms && t->n_longs)
        e = launch_tensors_each({t->d_longs, t->d_sums, norms, t->n_longs, in_mul}, st);
    return arg_launch(op, e);
}

gq_status gq_tensors_clip(const gq_tensors *t, const float *norm, float max_norm, float eps,
                          float in_mul, const gq_tensors *out, gq_stream stream) {
    const char *op = "gq_tensors_clip";
    GQ_ARG(arg_mul(op, in_mul));
    if (!(max_norm >= 0.0f))
        return arg_fail(GQ_ERR_INVALID, op, "max_norm = %g must be >= 0",
                        static_cast<double>(max_norm));
    if (!std::isfinite(eps) || !(eps >= 0.0f))
        return arg_fail(GQ_ERR_INVALID, op, "eps = %g must be finite and >= 0",
                        static_cast<double>(eps));
    GQ_ARG(arg_ptr(op, "norm", norm, 4));
    GQ_ARG(check_list(op, "the list", t));
    if (out == t) out = nullptr;
    if (out) {
        GQ_ARG(check_list(op, "out", out));
        if (out->numel != t->numel)
            return arg_fail(GQ_ERR_INVALID, op, "out's tensors have other lengths than the list's");
        if (overlap(t->spans, out->spans))
            return arg_fail(GQ_ERR_INVALID, op, "out shares memory with the list");
    }
    // (one wave would write it while others read it)
    if (touches((out ? out : t)->spans, norm, 4))
        return arg_fail(GQ_ERR_INVALID, op, "norm lies in a tensor that the call writes");
    const int64_t bytes = t->data_bytes + (out ? out->data_bytes : 0);
    const TnClipArgs a = {t->d_tiles, out ? out->d_tiles : t->d_tiles, t->n_tiles, norm, max_norm,
                          eps, in_mul, bytes > TN_CACHED};
    return arg_launch(op, launch_tensors_clip(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
