// gq_ortho.cpp -- the C-ABI entry points of the orthogonalised update: plans
// (the matrices of a model, their workspace and the launches' tile tables)
// and the step.  Contracts: include/gq.h.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "gq_args.h"
#include "gq_ortho.h"

using namespace gq;

struct gq_ortho {
    int device = -1;
    int64_t n = 0;                 // elements of the flat buffers
    int64_t n_mats = 0;
    int32_t steps = 0;
    int32_t tile_g = 0, tile_x = 0;   // of G and Q, and of X
    float eps = 0.0f;
    OrSteps coef = {};
    bool small = false;            // every matrix fits one work group
    int64_t ws_bytes = 0;
    char *d_mem = nullptr;         // one allocation: workspace, partials, tables
    _Float16 *d_ws = nullptr;
    double *d_part = nullptr;
    float *d_sums = nullptr;       // partial sums of G where its K is split
    float *d_diag = nullptr;
    uint8_t *d_low = nullptr;
    OrMat *d_mats = nullptr;
    OrTile *d_tiles[OR_TABLES] = {};
    int64_t n_tiles[OR_TABLES] = {};
};

namespace {

constexpr int64_t kMaxSide = 1 << 22;       // longer side (buffer bounds are 32 bits)
constexpr int64_t kMaxShort = 1 << 15;      // shorter side
constexpr int64_t kMaxMats = 1 << 20;
// Elements of a plan, sides rounded up to its tile: 2^22 tiles of 64 x 64, whose
// tables the host builds (24 bytes a tile).
constexpr int64_t kMaxPadded = int64_t{1} << 34;
constexpr int64_t kCus = 256;

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// A run of one matrix's tiles that should share an XCD's L2 cache.
struct Run {
    int64_t first, count;
    int64_t cost;
};

// Work group i runs on XCD i % 8.  The tiles' runs are dealt out to the eight
// XCDs, the costliest first, each to the XCD with the least work so far;
// an XCD that runs out earlier gets empty entries.
std::vector<OrTile> deal(const std::vector<OrTile> &tiles, std::vector<Run> runs) {
    std::stable_sort(runs.begin(), runs.end(),
                     [](const Run &p, const Run &q) { return p.cost > q.cost; });
    std::vector<OrTile> queue[8];
    int64_t load[8] = {};
    for (const Run &r : runs) {
        const int x = static_cast<int>(std::min_element(load, load + 8) - load);
        queue[x].insert(queue[x].end(), tiles.begin() + r.first,
                        tiles.begin() + r.first + r.count);
        load[x] += r.cost * r.count;
    }
    size_t longest = 0;
    for (const auto &v : queue) longest = std::max(longest, v.size());
    std::vector<OrTile> out(8 * longest, OrTile{-1, 0, 0, -1, 0, 0});
    for (int x = 0; x < 8; ++x)
        for (size_t i = 0; i < queue[x].size(); ++i) out[8 * i + x] = queue[x][i];
    while (!out.empty() && out.back().mat < 0) out.pop_back();
    return out;
}

// Adds the runs of 32 among the tiles from `first` on, of `cost` each.
void add_runs(std::vector<Run> &runs, int64_t first, int64_t end, int64_t cost) {
    for (int64_t f = first; f < end; f += 32)
        runs.push_back({f, std::min<int64_t>(32, end - f), cost});
}

// Tiles of all matrices' s x l outputs.
std::vector<OrTile> x_tiles(const std::vector<OrMat> &mats, int tile) {
    std::vector<OrTile> tiles;
    std::vector<Run> runs;
    for (size_t m = 0; m < mats.size(); ++m) {
        const int ts = mats[m].sp / tile, tl = mats[m].lp / tile;
        const int64_t first = static_cast<int64_t>(tiles.size());
        for (int i0 = 0; i0 < ts; i0 += 8)
            for (int j = 0; j < tl; ++j)
                for (int i = i0; i < std::min(ts, i0 + 8); ++i)
                    tiles.push_back({static_cast<int32_t>(m), i, j, -1, 0, 0});
        add_runs(runs, first, static_cast<int64_t>(tiles.size()), mats[m].sp);
    }
    return deal(tiles, runs);
}

// Tiles of the upper halves of all matrices' s x s outputs: for G, with K split
// where it is long and there are few tiles, for the joins of what was split,
// and for Q.  Returns the number of partial sums.  K goes into parts of 1024
// columns or more, as many as give two work groups per compute unit (128 x 30522,
// fp32, momentum, five steps: 738 us with K whole, 191 in parts).
int64_t g_tiles(const std::vector<OrMat> &mats, int tile, std::vector<OrTile> &gram,
                std::vector<OrTile> &join, std::vector<OrTile> &poly) {
    int64_t total = 0, parts = 0;
    for (const OrMat &m : mats) total += static_cast<int64_t>(m.sp / tile) * (m.sp / tile + 1) / 2;
    const int64_t want = tile == 64 ? 2 * kCus / total : 1;
    std::vector<OrTile> g, q;
    std::vector<Run> gr, qr;
    for (size_t m = 0; m < mats.size(); ++m) {
        const int ts = mats[m].sp / tile;
        const int64_t groups = (mats[m].lp + 127) / 128;
        const int64_t splits = std::max<int64_t>(1, std::min(want, groups / 8));
        // (an even number of groups a part: the loop's rounds are of two)
        const int64_t per = splits == 1 ? groups : round_up((groups + splits - 1) / splits, 2);
        const int64_t count = (groups + per - 1) / per;
        const int64_t g0 = static_cast<int64_t>(g.size()), q0 = static_cast<int64_t>(q.size());
        for (int i = 0; i < ts; ++i) {
            for (int j = i; j < ts; ++j) {
                OrTile t = {static_cast<int32_t>(m), i, j, -1, 0, static_cast<int32_t>(groups)};
                q.push_back(t);
                if (count == 1) {
                    g.push_back(t);
                    continue;
                }
                t.part = static_cast<int32_t>(parts);
                t.count = static_cast<int32_t>(count);
                join.push_back(t);
                for (int64_t k = 0; k < count; ++k) {
                    t.part = static_cast<int32_t>(parts++);
                    t.first = static_cast<int32_t>(k * per);
                    t.count = static_cast<int32_t>(std::min(per, groups - k * per));
                    g.push_back(t);
                }
            }
        }
        add_runs(gr, g0, static_cast<int64_t>(g.size()), per);
        add_runs(qr, q0, static_cast<int64_t>(q.size()), mats[m].sp);
    }
    gram = deal(g, gr);
    poly = deal(q, qr);
    return parts;
}

// Tiles of the products: `g` of the s x s G and Q (their upper halves), `x` of
// the s x l X.  Sides are rounded up to the larger.  A size must give the
// device enough tiles: one work group per compute unit with tiles of 256, nearly
// two with tiles of 128 (64: any number).  Of the pairs that do, the one that
// takes least time by what a tile costs a compute unit: its start (filling the
// buffers, writing it out) and 64 of K a step, in us, fitted to times of the pairs.
// Measured, us a call of five steps on fp32 gradients with momentum, all pairs of a
// row in turn, medians, g / x (* the choice; 24 of 768 x 768 on 128/256 have 216
// tiles of X, too few by the rule, and 8 percent less time):
//                       64/64  64/128  64/256 128/128 128/256 256/256
//   one 2048 x 2048       422*    437     612     499     670    1027
//   4 of 1024 x 4096      663     602     551*    668     615    1011
//   16 of 1024 x 1024     826     755     706     717     670*    696
//   one 4096 x 4096      2487    2205    2029    1989    1821*   1982
//   one 8192 x 8192     21010   18972   17506   13623   12198   11710*
//   24 of 768 x 768       576     552     513     502*    463     580
//   36 of 256 x 2304      393     388*    400     462     476     681
//   60 of 200 x 1000      292     281*    267     311     296     428
//   300 of 64 x 512       186*    272     652     303     648     786
//   ResNet-152's 156     1337    1220*   1250    1291    1319    1600
//   BERT-Large's 145    13091   11308   10465    9760    8950    8769*
struct Tiles {
    int g, x;
};

Tiles choose_tiles(const int64_t *rows, const int64_t *cols, int64_t n) {
    const int size[3] = {64, 128, 256};
    const double start[3] = {0.5, 2.5, 15.0}, step[3] = {0.2, 0.65, 1.9};
    const int64_t enough[3] = {1, 15 * kCus / 8, kCus};
    Tiles best = {64, 64};
    double least = 0.0;
    for (int kg = 0; kg < 3; ++kg) {
        for (int kx = 0; kx < 3; ++kx) {
            const int64_t g = size[kg], x = size[kx], pad = std::max(g, x);
            int64_t n_g = 0, n_x = 0;
            double time = 0.0;
            for (int64_t i = 0; i < n; ++i) {
                const int64_t s = round_up(std::min(rows[i], cols[i]), pad);
                const int64_t l = round_up(std::max(rows[i], cols[i]), pad);
                const int64_t upper = s / g * (s / g + 1) / 2, all = s / x * (l / x);
                n_g += upper;
                n_x += all;
                // G over l, Q and X over s
                const double steps = static_cast<double>(l + s) / 64.0;
                time += static_cast<double>(upper) * (2.0 * start[kg] + steps * step[kg]);
                time += static_cast<double>(all) *
                        (start[kx] + static_cast<double>(s) / 64.0 * step[kx]);
            }
            if (n_g < enough[kg] || n_x < enough[kx]) continue;
            if (least == 0.0 || time < least) {
                least = time;
                best = {static_cast<int>(g), static_cast<int>(x)};
            }
        }
    }
    return best;
}

// Whether every matrix fits one work group.  64 x 147 (fp32, momentum, five
// steps): 23 us in one launch, 64 us in 17 of tiles, which the host takes 53 us
// to issue.  (64 x 1024 would take 141 us in one work group's LDS: tiles.)
bool fits_small(const int64_t *rows, const int64_t *cols, int64_t n) {
    for (int64_t i = 0; i < n; ++i)
        if (std::min(rows[i], cols[i]) > OR_SMALL_S || std::max(rows[i], cols[i]) > OR_SMALL_L)
            return false;
    return true;
}

gq_status ortho_create(const char *op, const int64_t *h_off, const int64_t *h_rows,
                       const int64_t *h_cols, int64_t n_mats, int32_t steps, const float *coef,
                       float eps, const float *out_mul, gq_ortho **out) {
    std::vector<OrMat> mats(static_cast<size_t>(n_mats));
    const bool small = fits_small(h_rows, h_cols, n_mats);
    const Tiles chosen = small ? Tiles{64, 64} : choose_tiles(h_rows, h_cols, n_mats);
    const int tile_g = chosen.g, tile_x = chosen.x;
    const int tile = std::max(tile_g, tile_x);      // what the sides are rounded up to
    // (before any table is built: theirs are the sizes that this bounds)
    int64_t padded = 0;
    for (int64_t i = 0; i < n_mats && !small; ++i) {
        padded += round_up(h_rows[i], tile) * round_up(h_cols[i], tile);
        if (padded >= kMaxPadded)
            return arg_fail(GQ_ERR_INVALID, op,
                            "2^34 elements or more with sides rounded up to %d (matrix %lld)", tile,
                            static_cast<long long>(i));
    }
    std::vector<OrTile> tab[OR_TABLES];
    int64_t at = 0, parts = 0, diags = 0, lows = 0;
    for (int64_t i = 0; i < n_mats; ++i) {
        OrMat &m = mats[static_cast<size_t>(i)];
        std::memset(&m, 0, sizeof m);
        m.off = h_off[i];
        m.rows = static_cast<int32_t>(h_rows[i]);
        m.cols = static_cast<int32_t>(h_cols[i]);
        m.tr = m.rows > m.cols;
        m.s = std::min(m.rows, m.cols);
        m.l = std::max(m.rows, m.cols);
        m.sp = static_cast<int32_t>(round_up(m.s, tile));
        m.lp = static_cast<int32_t>(round_up(m.l, tile));
        m.scale = std::exp2(std::round(0.5f * std::log2(static_cast<float>(m.l))));
        m.out_mul = out_mul ? out_mul[i] : 1.0f;
        m.align = (m.off | m.cols) % 8 == 0 ? 8 : (m.off | m.cols) % 4 == 0 ? 4 : 1;
        if (small) continue;    // neither workspace nor tables
        const int64_t xl = static_cast<int64_t>(m.sp) * m.lp, al = static_cast<int64_t>(m.sp) * m.sp;
        for (int k = 0; k < 2; ++k) {
            m.x[k] = at;
            at += xl;
        }
        m.a = at;
        at += al;
        m.b = at;
        at += al;
        m.low = lows;
        if (steps >= OR_LOW_STEPS) lows += xl;
        m.diag = diags;
        diags += 2 * static_cast<int64_t>(m.sp);
        // at most 1024 partial sums a matrix, of at least 8192 elements
        const int64_t elems = (m.off & 3) + static_cast<int64_t>(m.rows) * m.cols;
        m.chunk = std::max<int64_t>(8192, round_up((elems + 1023) / 1024, 4));
        m.part = static_cast<int32_t>(parts);
        m.parts = static_cast<int32_t>((elems + m.chunk - 1) / m.chunk);
        parts += m.parts;
        for (int32_t p = 0; p < m.parts; ++p)
            tab[OR_NORM].push_back({static_cast<int32_t>(i), p, 0, -1, 0, 0});
        const int rp = m.tr ? m.lp : m.sp, cp = m.tr ? m.sp : m.lp;
        for (int r = 0; r < rp / OR_CAST_TILE; ++r)
            for (int c = 0; c < cp / OR_CAST_TILE; ++c)
                tab[OR_CAST].push_back({static_cast<int32_t>(i), r, c, -1, 0, 0});
    }
    int64_t sums = 0;
    if (!small) {
        sums = g_tiles(mats, tile_g, tab[OR_GRAM], tab[OR_JOIN], tab[OR_POLY]);
        tab[OR_X] = x_tiles(mats, tile_x);
    }
    gq_ortho *P = new gq_ortho;
    P->steps = steps;
    P->tile_g = tile_g;
    P->tile_x = tile_x;
    P->eps = eps;
    static const float quintic[3] = {3.4445f, -4.7750f, 2.0315f};
    P->coef.steps = steps;
    for (int32_t k = 0; k < 3 * steps; ++k) P->coef.coef[k] = coef ? coef[k] : quintic[k % 3];
    P->small = small;
    P->n_mats = n_mats;
    P->n = h_off[n_mats - 1] + h_rows[n_mats - 1] * h_cols[n_mats - 1];
    hipError_t e = hipGetDevice(&P->device);
    // one allocation, every part at a multiple of 256 bytes
    int64_t size = round_up(at * 2, 256);
    const int64_t part_at = size;
    size += round_up(parts * 8, 256);
    const int64_t sums_at = size;
    size += sums * tile_g * tile_g * 4;
    const int64_t diag_at = size;
    size += round_up(diags * 4, 256);
    const int64_t low_at = size;
    size += round_up(lows, 256);
    const int64_t mats_at = size;
    size += round_up(static_cast<int64_t>(mats.size() * sizeof(OrMat)), 256);
    int64_t tab_at[OR_TABLES];
    for (int k = 0; k < OR_TABLES; ++k) {
        tab_at[k] = size;
        size += round_up(static_cast<int64_t>(tab[k].size() * sizeof(OrTile)), 256);
    }
    P->ws_bytes = size;
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&P->d_mem), static_cast<size_t>(size));
    if (e == hipSuccess) {
        P->d_ws = reinterpret_cast<_Float16 *>(P->d_mem);
        P->d_part = reinterpret_cast<double *>(P->d_mem + part_at);
        P->d_sums = reinterpret_cast<float *>(P->d_mem + sums_at);
        P->d_diag = reinterpret_cast<float *>(P->d_mem + diag_at);
        P->d_low = reinterpret_cast<uint8_t *>(P->d_mem + low_at);
        P->d_mats = reinterpret_cast<OrMat *>(P->d_mem + mats_at);
        e = hipMemcpy(P->d_mats, mats.data(), mats.size() * sizeof(OrMat), hipMemcpyHostToDevice);
    }
    for (int k = 0; k < OR_TABLES && e == hipSuccess; ++k) {
        P->d_tiles[k] = reinterpret_cast<OrTile *>(P->d_mem + tab_at[k]);
        P->n_tiles[k] = static_cast<int64_t>(tab[k].size());
        e = hipMemcpy(P->d_tiles[k], tab[k].data(), tab[k].size() * sizeof(OrTile),
                      hipMemcpyHostToDevice);
    }
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        (void)hipGetLastError();
        if (P->d_mem) (void)hipFree(P->d_mem);
        delete P;
        return arg_fail(GQ_ERR_HIP, op, "allocating %lld bytes failed: %s",
                        static_cast<long long>(size), hipGetErrorString(e));
    }
    *out = P;
    return arg_ok();
}

}  // namespace

extern "C" {

gq_status gq_ortho_create(const int64_t *h_off, const int64_t *h_rows, const int64_t *h_cols,
                          int64_t n_mats, int32_t steps, const float *coef, float eps,
                          const float *out_mul, gq_ortho **out) {
    const char *op = "gq_ortho_create";
    if (!out) return arg_fail(GQ_ERR_INVALID, op, "out is NULL");
    *out = nullptr;
    if (!h_off || !h_rows || !h_cols)
        return arg_fail(GQ_ERR_INVALID, op, "h_off, h_rows or h_cols is NULL");
    if (n_mats < 1 || n_mats > kMaxMats)
        return arg_fail(GQ_ERR_INVALID, op, "n_mats = %lld outside [1, %lld]",
                        static_cast<long long>(n_mats), static_cast<long long>(kMaxMats));
    if (steps < 1 || steps > GQ_ORTHO_MAX_STEPS)
        return arg_fail(GQ_ERR_INVALID, op, "steps = %d outside [1, %d]", steps,
                        GQ_ORTHO_MAX_STEPS);
    if (!std::isfinite(eps) || !(eps >= 0.0f))
        return arg_fail(GQ_ERR_INVALID, op, "eps = %g must be finite and >= 0",
                        static_cast<double>(eps));
    for (int32_t k = 0; coef && k < 3 * steps; ++k)
        if (!std::isfinite(coef[k]))
            return arg_fail(GQ_ERR_INVALID, op, "coef[%d] is not finite", k);
    int64_t end = 0;
    for (int64_t i = 0; i < n_mats; ++i) {
        const int64_t r = h_rows[i], c = h_cols[i];
        if (r < 1 || c < 1 || std::max(r, c) > kMaxSide || std::min(r, c) > kMaxShort)
            return arg_fail(GQ_ERR_INVALID, op,
                            "matrix %lld of %lld x %lld: sides must be 1 .. %lld, the shorter one "
                            "at most %lld", static_cast<long long>(i), static_cast<long long>(r),
                            static_cast<long long>(c), static_cast<long long>(kMaxSide),
                            static_cast<long long>(kMaxShort));
        if (h_off[i] < end || h_off[i] > kMaxElems - r * c)
            return arg_fail(GQ_ERR_INVALID, op,
                            "matrix %lld at %lld overlaps the one before, or ends above 2^40",
                            static_cast<long long>(i), static_cast<long long>(h_off[i]));
        end = h_off[i] + r * c;
        if (out_mul && !std::isfinite(out_mul[i]))
            return arg_fail(GQ_ERR_INVALID, op, "out_mul[%lld] is not finite",
                            static_cast<long long>(i));
    }
    try {
        return ortho_create(op, h_off, h_rows, h_cols, n_mats, steps, coef, eps, out_mul, out);
    } catch (const std::bad_alloc &) {
        return arg_fail(GQ_ERR_INVALID, op, "out of host memory");
    }
}

gq_status gq_ortho_destroy(gq_ortho *p) {
    if (!p) return arg_ok();
    if (p->d_mem) (void)hipFree(p->d_mem);
    delete p;
    return arg_ok();
}

gq_status gq_ortho_info(const gq_ortho *p, int64_t *n, int64_t *n_mats, int64_t *bytes,
                        int32_t *tile) {
    if (!p) return arg_fail(GQ_ERR_INVALID, "gq_ortho_info", "plan is NULL");
    if (n) *n = p->n;
    if (n_mats) *n_mats = p->n_mats;
    if (bytes) *bytes = p->ws_bytes;
    if (tile) *tile = p->tile_x;
    return arg_ok();
}

gq_status gq_ortho_tiles(const gq_ortho *p, int32_t *tile_g, int32_t *tile_x) {
    if (!p) return arg_fail(GQ_ERR_INVALID, "gq_ortho_tiles", "plan is NULL");
    if (tile_g) *tile_g = p->small ? 0 : p->tile_g;
    if (tile_x) *tile_x = p->small ? 0 : p->tile_x;
    return arg_ok();
}

gq_status gq_ortho_step(gq_ortho *p, const void *g, gq_dtype dt, float in_mul, float *momentum,
                        float mu, int32_t nesterov, gq_dtype out_dt, void *out, gq_stream stream) {
    const char *op = "gq_ortho_step";
    GQ_ARG(arg_dtype(op, "dtype", dt));
    GQ_ARG(arg_mul(op, in_mul));
    if (out_dt != GQ_F16 && out_dt != GQ_BF16)
        return arg_fail(GQ_ERR_INVALID, op, "out must be GQ_F16 or GQ_BF16, got %d",
                        static_cast<int>(out_dt));
    GQ_ARG(arg_ptr(op, "g", g, 16));
    GQ_ARG(arg_ptr(op, "out", out, 16));
    if (momentum) {
        GQ_ARG(arg_ptr(op, "momentum", momentum, 16));
        if (!std::isfinite(mu) || !(mu >= 0.0f))
            return arg_fail(GQ_ERR_INVALID, op, "mu = %g must be finite and >= 0",
                            static_cast<double>(mu));
    }
    if (!p) return arg_fail(GQ_ERR_INVALID, op, "plan is NULL");
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return arg_fail(GQ_ERR_HIP, op, "hipGetDevice failed");
    if (dev != p->device)
        return arg_fail(GQ_ERR_DEVICE, op, "current device %d, plan lives on device %d", dev,
                        p->device);
    hipStream_t st = static_cast<hipStream_t>(stream);
    OrArgs a;
    std::memset(&a, 0, sizeof a);
    a.mats = p->d_mats;
    a.ws = p->d_ws;
    a.part = p->d_part;
    a.sums = p->d_sums;
    a.diag = p->d_diag;
    a.low = p->d_low;
    a.tile_x = p->tile_x;
    a.low_out = p->steps >= OR_LOW_STEPS;
    a.g = g;
    a.m = momentum;
    a.out = out;
    a.in_mul = in_mul;
    a.mu = mu;
    a.eps = p->eps;
    a.nesterov = nesterov != 0;
    if (p->small)
        return arg_launch(op, launch_ortho_small(a, p->coef, p->n_mats, dt, out_dt, st));
    a.tiles = p->d_tiles[OR_NORM];
    hipError_t e = launch_ortho_norm(a, p->n_tiles[OR_NORM], dt, st);
    a.tiles = p->d_tiles[OR_CAST];
    if (e == hipSuccess) e = launch_ortho_cast(a, p->n_tiles[OR_CAST], dt, st);
    for (int32_t k = 0; k < p->steps && e == hipSuccess; ++k) {
        a.a = p->coef.coef[3 * k];
        a.b = p->coef.coef[3 * k + 1];
        a.c = p->coef.coef[3 * k + 2];
        a.cur = k & 1;
        a.low_in = p->steps - k >= OR_LOW_STEPS;
        a.low_out = p->steps - k - 1 >= OR_LOW_STEPS;
        a.tiles = p->d_tiles[OR_GRAM];
        e = launch_ortho_mm(a, p->n_tiles[OR_GRAM], p->tile_g, OR_MM_GRAM, out_dt, st);
        a.tiles = p->d_tiles[OR_JOIN];
        if (e == hipSuccess && p->n_tiles[OR_JOIN] > 0)
            e = launch_ortho_mm(a, p->n_tiles[OR_JOIN], p->tile_g, OR_MM_JOIN, out_dt, st);
        a.tiles = p->d_tiles[OR_POLY];
        if (e == hipSuccess)
            e = launch_ortho_mm(a, p->n_tiles[OR_POLY], p->tile_g, OR_MM_POLY, out_dt, st);
        a.tiles = p->d_tiles[OR_X];
        if (e == hipSuccess)
            e = launch_ortho_mm(a, p->n_tiles[OR_X], p->tile_x,
                                k + 1 < p->steps ? OR_MM_STEP : OR_MM_LAST, out_dt, st);
    }
    return arg_launch(op, e);
}

}  // extern "C"
