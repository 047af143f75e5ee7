// gq_ortho.hip -- gfx950 kernels of the orthogonalised update: momentum, then
// T steps of the quintic Newton-Schulz iteration on every matrix of a plan,
//   X <- u / (|u|_F + eps);  G = X X^T;  Q = b G + c G G;  X <- a X + Q X.
//   k_ortho_norm  momentum, and each matrix's sum of squares in binary64;
//   k_ortho_cast  X in fp16 from u and the sum of squares;
//   k_ortho_small the whole update of a matrix that fits one work group's LDS;
//   k_ortho_mm    the three products of a step over the tiles of all
//                 matrices together (gq_mm.h: the tile loop), the polynomial
//                 and the update in its epilogue.
// The iterates are held in fp16, not bf16: all singular values stay below
// about 1.3, so the exponent range of bf16 is not needed and the three more
// bits are, since the iteration multiplies a rounding in a small singular
// direction by up to a each step.  X is stored times a power of two near
// sqrt(l), which keeps the entries of a matrix with many columns out of the
// subnormal range.  Products are summed in binary32, and the polynomial and
// the update are computed in binary32 from those sums and rounded once.
// G and Q are symmetric: only tiles on and above the diagonal are computed,
// and each is written to both places.
#include <hip/hip_fp16.h>

#include "gq_mm.h"
#include "gq_ortho.h"

namespace gq {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int OR_BLOCK = 256;
// Launches of up to this many tiles of 64 run on a ring of four buffers, two
// work groups per compute unit, longer ones on two buffers and five work
// groups.  One 1024 x 1024 matrix (136 and 256 tiles, five steps): 162 us on
// the ring, 196 on two buffers; one 2048 x 2048 (528 and 1024): 484 and 419.
constexpr int64_t OR_FEW = 512;

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v.bits) << 16);
}

// Elements e .. e + 3 of x (e a multiple of 4), those in [lo, hi); the
// others 0.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T *x, int64_t e, int64_t lo, int64_t hi) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (e >= lo && e + 4 <= hi) {
        if constexpr (sizeof(T) == 4) {
            v = *reinterpret_cast<const f32x4 *>(x + e);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(x + e);
            const uint32_t h[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                T t;
                const uint16_t b = static_cast<uint16_t>(h[k]);
                __builtin_memcpy(&t, &b, 2);
                v[k] = to_f32(t);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k >= lo && e + k < hi) v[k] = to_f32(x[e + k]);
    }
    return v;
}

__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = sh[0];
#pragma unroll
    for (int i = 1; i < OR_BLOCK / 64; ++i) r += sh[i];
    return r;
}

// What takes u to X as it is stored, in binary64: the norm's reciprocal may lie
// outside the range of binary32.  (A zero matrix stays zero without an eps, too.)
__device__ __forceinline__ double or_mul(float scale, double sum, float eps) {
    const double norm = __dsqrt_rn(sum) + static_cast<double>(eps);
    return norm == 0.0 ? 0.0 : static_cast<double>(scale) / norm;
}

// ---- momentum and sums of squares ---------------------------------------------
// A work group takes one chunk of a matrix, cut at multiples of four elements
// of the flat buffers (whose starts are 16-byte aligned).  Bound by HBM: 335M
// fp16 gradients with momentum 575 us, 5.8 TB/s.
template <typename T, bool MOM>
__global__ __launch_bounds__(OR_BLOCK) void k_ortho_norm(const OrArgs a) {
    __shared__ double sh[OR_BLOCK / 64];
    const OrTile t = a.tiles[blockIdx.x];
    const OrMat &mt = a.mats[t.mat];
    const int64_t lo = mt.off, hi = lo + static_cast<int64_t>(mt.rows) * mt.cols;
    const int64_t e0 = (lo & ~int64_t{3}) + t.i * mt.chunk;
    const int64_t e1 = e0 + mt.chunk < hi ? e0 + mt.chunk : hi;
    const T *g = static_cast<const T *>(a.g);
    double sum = 0.0;
    for (int64_t e = e0 + 4 * threadIdx.x; e < e1; e += 4 * OR_BLOCK) {
        f32x4 u = load4(g, e, lo, hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = __fmul_rn(u[k], a.in_mul);
        if (MOM) {
            const f32x4 old = load4(a.m, e, lo, hi);
            f32x4 m;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = __fadd_rn(__fmul_rn(a.mu, old[k]), u[k]);
                u[k] = a.nesterov ? __fadd_rn(u[k], __fmul_rn(a.mu, m[k])) : m[k];
            }
            if (e >= lo && e + 4 <= hi) {
                *reinterpret_cast<f32x4 *>(a.m + e) = m;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (e + k >= lo && e + k < hi) a.m[e + k] = m[k];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += static_cast<double>(u[k]) * static_cast<double>(u[k]);
    }
    sum = block_sum(sum, sh);
    if (threadIdx.x == 0) a.part[mt.part + t.i] = sum;
}

// ---- X --------------------------------------------------------------------------
// A work group takes a 64 x 64 tile of the padded matrix as it lies in the
// gradient, and writes it to X, turned in LDS where X is the transpose.  Each
// work group adds up its matrix's partial sums itself, always in the same
// order.  Bound by HBM: 335M elements from the momentum 455 us, 4.4 TB/s.
template <typename T, bool MOM>
__global__ __launch_bounds__(OR_BLOCK) void k_ortho_cast(const OrArgs a) {
    __shared__ double sh[OR_BLOCK / 64];
    __shared__ _Float16 turn[OR_CAST_TILE][OR_CAST_TILE + 4];
    const OrTile t = a.tiles[blockIdx.x];
    const OrMat &mt = a.mats[t.mat];
    double sum = 0.0;
    for (int i = threadIdx.x; i < mt.parts; i += OR_BLOCK) sum += a.part[mt.part + i];
    sum = block_sum(sum, sh);
    const double mul = or_mul(mt.scale, sum, a.eps);
    const T *g = static_cast<const T *>(a.g);
    const int c = (threadIdx.x & 15) * 4;
    _Float16 *x = a.ws + mt.x[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        const int row = t.i * OR_CAST_TILE + r, col = t.j * OR_CAST_TILE + c;
        f32x4 u = {0.f, 0.f, 0.f, 0.f};
        if (row < mt.rows) {
            const int64_t e = mt.off + static_cast<int64_t>(row) * mt.cols + col;
            const int n = mt.cols - col;    // elements of the row from col on
            f32x4 gv = u, mv = u;
            const bool need_g = !MOM || a.nesterov;
            if (mt.align > 1 && n >= 4) {
                if (need_g) gv = load4(g, e, e, e + 4);
                if (MOM) mv = *reinterpret_cast<const f32x4 *>(a.m + e);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= n) continue;
                    if (need_g) gv[k] = to_f32(g[e + k]);
                    if (MOM) mv[k] = a.m[e + k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float gk = __fmul_rn(gv[k], a.in_mul);
                u[k] = !MOM ? gk : a.nesterov ? __fadd_rn(gk, __fmul_rn(a.mu, mv[k])) : mv[k];
                // nothing where there is no element, whatever the norm
                u[k] = k < n ? static_cast<float>(u[k] * mul) : 0.0f;
            }
        }
        f16x4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = static_cast<_Float16>(u[k]);
        if (mt.tr) {
#pragma unroll
            for (int k = 0; k < 4; ++k) turn[c + k][r] = h[k];
        } else {
            *reinterpret_cast<f16x4 *>(x + static_cast<int64_t>(row) * mt.lp + col) = h;
        }
    }
    if (!mt.tr) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        *reinterpret_cast<f16x4 *>(x + static_cast<int64_t>(t.j * OR_CAST_TILE + r) * mt.lp +
                                   t.i * OR_CAST_TILE + c) =
            *reinterpret_cast<const f16x4 *>(&turn[r][c]);
    }
}

// ---- the products -----------------------------------------------------------------

__device__ __forceinline__ uint16_t out_bits(float v, bool bf16) {
    if (!bf16) return __half_as_ushort(__float2half_rn(v));
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
    return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));

// A wave's part of the tile, TM x TN 16-bit values, on its way out through
// LDS, so that its stores fill whole lines: 16-byte chunk c of row r lies at
// chunk c ^ (r & 7) (TN = 64) or c ^ (r >> 1 & 3) (TN = 32).
template <int TN>
__device__ __forceinline__ int out_at(int r, int chunk) {
    const int turn = TN == 64 ? r & 7 : (r >> 1) & 3;
    return r * TN * 2 + ((chunk ^ turn) << 4);
}

// Eight values from row r, column 8 * chunk on.
template <int TN>
__device__ __forceinline__ u16x8 out_row(const char *lds, int r, int chunk) {
    return *reinterpret_cast<const u16x8 *>(lds + out_at<TN>(r, chunk));
}

// Eight values down column c16 + lane % 16, from row r32 + 8 * (lane / 16) on.
template <int TN>
__device__ __forceinline__ u16x8 out_col(const char *lds, int r32, int c16) {
    const int lane = threadIdx.x & 63, q = lane & 15;
    u16x8 v;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r = r32 + 8 * (lane >> 4) + 4 * t + (q >> 2);
        const char *p = lds + out_at<TN>(r, (c16 >> 3) + ((q >> 1) & 1)) + (q & 1) * 8;
        const mm_i16x4 h = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4 *)p);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * t + k] = static_cast<unsigned short>(h[k]);
    }
    return v;
}

// The first n of eight values; al: how many elements o is a multiple of.
__device__ __forceinline__ void store8(uint16_t *o, u16x8 v, int n, int al) {
    if (n >= 8 && al == 8) {
        *reinterpret_cast<u16x8 *>(o) = v;
    } else if (n >= 8 && al == 4) {
        *reinterpret_cast<u16x4 *>(o) = u16x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<u16x4 *>(o + 4) = u16x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) o[k] = v[k];
    }
}

// a X of the wave's part of the tile, added while those rows of X pass through
// LDS as rows of K: X is then read once.
struct AddX {
    float a;
    int i0;     // the tile's first row
    template <typename S>
    __device__ __forceinline__ void operator()(MmAcc<S> &acc, const char *q, int step, int b) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int lane = mm_tid() & 63;
        constexpr int BN = S::QUAD ? 128 : S::T;      // columns of q
        constexpr int RUN = S::QUAD ? 4 : S::FM;      // instruction rows that lie together
#pragma unroll
        for (int i0r = 0; i0r < S::FM; i0r += RUN) {
            const int row = i0 + S::part_row(wave, i0r) - 64 * step;
            if (row < 0 || row >= 64) continue;
#pragma unroll
            for (int i = i0r; i < i0r + RUN; ++i) {
#pragma unroll
                for (int j = 0; j < S::FN; ++j) {
                    const int col = (S::part_col(wave, 0) + 16 * j + (lane >> 4) * 4);
                    const f16x4 x = *reinterpret_cast<const f16x4 *>(
                        q + mm_cols_at<BN>(row + 16 * (i - i0r) + (lane & 15), col));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc.c[b][i][j][k] =
                            __fmaf_rn(a, static_cast<float>(x[k]), acc.c[b][i][j][k]);
                }
                __builtin_amdgcn_sched_barrier(0);   // few registers at a time
            }
        }
    }
};

// MODE OR_MM_GRAM: G = X X^T          (K: columns of X)
//      OR_MM_POLY: Q = b G + c G G    (G = G^T)
//      OR_MM_STEP: X <- a X + Q X     (K: rows of X)
//      OR_MM_LAST, OR_MM_LAST_BF16: the same into the caller's output
//      OR_MM_JOIN: G from the partial sums that OR_MM_GRAM left of tiles whose
//                  K it split, added in the order of K
// 97 matrices of 1024 x 1024 and 48 of 1024 x 4096, tiles of 256, us a launch: G
// 379 (0.81 PFLOP/s of the upper half), Q 258 (0.60), X 743 (0.83), the last X 751.
// With K = 1024 a tile's loop is 16 steps, and filling the buffers and writing the
// tile out are a third of its time (X without its loop 220, of that 150 the
// stores); one work group per compute unit leaves nobody to cover them.
template <typename S, int MODE>
__global__ __launch_bounds__(S::THREADS) void k_ortho_mm(const OrArgs a) {
    MM_LDS(S);
    constexpr bool LAST = MODE == OR_MM_LAST || MODE == OR_MM_LAST_BF16;
    constexpr bool TO_G = MODE == OR_MM_GRAM || MODE == OR_MM_JOIN;
    const OrTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const OrMat &mt = a.mats[t.mat];
    const int sp = mt.sp, lp = mt.lp;
    const int i0 = t.i * S::T, j0 = t.j * S::T;
    const _Float16 *x = a.ws + mt.x[a.cur];
    const _Float16 *pm = MODE == OR_MM_GRAM ? x : a.ws + (MODE == OR_MM_POLY ? mt.a : mt.b);
    const int kdim = MODE == OR_MM_GRAM ? lp : sp;
    MmAcc<S> acc = {};
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    constexpr int SUMS = S::PARTS * S::FM * S::FN;      // groups of four sums per lane
    auto at = [&](int part, int k) {                    // a lane's k-th four of a partial sum
        return reinterpret_cast<mm_f32x4 *>(a.sums + static_cast<int64_t>(part) * (S::T * S::T)) +
               (wave * SUMS + k) * 64 + lane;
    };
    mm_f32x4 *flat = &acc.c[0][0][0];
    if constexpr (MODE == OR_MM_JOIN) {
        for (int p = 0; p < t.count; ++p)
#pragma unroll
            for (int k = 0; k < SUMS; ++k) flat[k] += *at(t.part + p, k);
    } else {
        const MmRows p = mm_rows(pm, kdim * 2, i0, sp, S::T);
        const int groups = (kdim + 127) / 128;
        if constexpr (MODE == OR_MM_GRAM) {
            const MmRows q = mm_rows(pm, kdim * 2, j0, sp, S::T);
            mm_loop<S, false>(p, q, MmScale{}, t.first, t.count, mm_lds, nullptr, MmNoExtra{}, acc);
            if (t.part >= 0) {
#pragma unroll
                for (int k = 0; k < SUMS; ++k) *at(t.part, k) = flat[k];
                return;
            }
        } else if constexpr (MODE == OR_MM_POLY) {
            const MmRows q = mm_rows(pm, kdim * 2, j0, sp, S::T);
            mm_loop<S, false>(p, q, MmScale{}, 0, groups, mm_lds, nullptr, MmNoExtra{}, acc);
        } else {
            const MmCols q = {reinterpret_cast<const char *>(x + j0), static_cast<uint32_t>(lp) * 2u,
                              static_cast<uint32_t>(j0) * 2u, sp};
            mm_loop<S, false>(p, q, MmScale{}, 0, groups, mm_lds, nullptr, AddX{a.a, i0}, acc);
        }
    }
    constexpr int TM = 16 * S::FM, TN = 16 * S::FN, PART = TM * TN * 2;
    static_assert(PART * S::PARTS * S::WM * S::WN <= S::UNIT * S::BUFFERS,
                  "a wave's part of the tile fits its part of the buffers");
    char *lds = mm_lds.own<S>(wave);
#pragma unroll
    for (int b = 0; b < S::PARTS; ++b) {
#pragma unroll
        for (int i = 0; i < S::FM; ++i) {
            const int rl = 16 * i + (lane & 15);
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                const int cl = 16 * j + (lane >> 4) * 4;
                const mm_f32x4 v = acc.c[b][i][j];
                u16x4 h;
                if constexpr (MODE == OR_MM_POLY) {
                    const int64_t r = i0 + S::part_row(wave, i) + (lane & 15);
                    const int64_t c = j0 + S::part_col(wave, b) + cl;
                    const f16x4 gm = *reinterpret_cast<const f16x4 *>(pm + r * sp + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = out_bits(__fmaf_rn(a.c, v[k], a.b * static_cast<float>(gm[k])),
                                        false);
                } else {
                    // (both factors are powers of two but for out_mul)
                    const float mul = TO_G ? 1.0f / (mt.scale * mt.scale)
                                      : LAST ? mt.out_mul / mt.scale : 1.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = out_bits(v[k] * mul, MODE == OR_MM_LAST_BF16);
                }
                *reinterpret_cast<u16x4 *>(lds + b * PART + out_at<TN>(rl, cl >> 3) +
                                           (cl & 4) * 2) = h;
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // by rows, and for what is symmetric (off the diagonal) or turned by columns
    uint16_t *d;
    int ld, ldt, rows = 0x7fffffff, cols = 0x7fffffff, al = 8;
    bool by_rows = true, by_cols = false;
    if constexpr (TO_G || MODE == OR_MM_POLY) {
        d = reinterpret_cast<uint16_t *>(a.ws + (TO_G ? mt.a : mt.b));
        ld = ldt = sp;
        by_cols = t.i != t.j;
    } else if constexpr (!LAST) {
        d = reinterpret_cast<uint16_t *>(a.ws + mt.x[a.cur ^ 1]);
        ld = ldt = lp;
    } else {
        d = static_cast<uint16_t *>(a.out) + mt.off;
        ld = mt.l;
        ldt = mt.s;
        rows = mt.s;
        cols = mt.l;
        al = mt.align;
        by_rows = !mt.tr;
        by_cols = !by_rows;
    }
#pragma unroll
    for (int b = 0; b < S::PARTS; ++b) {
        const char *part = lds + b * PART;
        const int c0 = j0 + S::part_col(wave, b);
        if (by_rows) {
            constexpr int CH = TN / 8, RI = 64 / CH;    // chunks per row, rows per pass
#pragma unroll
            for (int k = 0; k < TM / RI; ++k) {
                const int rl = k * RI + lane / CH, chunk = lane % CH;
                const u16x8 v = out_row<TN>(part, rl, chunk);
                const int r = i0 + S::part_row(wave, rl >> 4) + (rl & 15), c = c0 + 8 * chunk;
                if (r < rows && c < cols)
                    store8(d + static_cast<int64_t>(r) * ld + c, v, cols - c, al);
            }
        }
        if (by_cols) {
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
#pragma unroll
                for (int k = 0; k < TM / 32; ++k) {
                    const u16x8 v = out_col<TN>(part, 32 * k, 16 * j);
                    const int c = c0 + 16 * j + (lane & 15);
                    const int r = i0 + S::part_row(wave, 2 * k) + 8 * (lane >> 4);
                    if (r < rows && c < cols)
                        store8(d + static_cast<int64_t>(c) * ldt + r, v, rows - r, al);
                }
            }
        }
    }
}

// ---- small matrices ----------------------------------------------------------------
// All steps of a matrix with s <= 64 and l <= LP in one work group of eight
// waves, X, G and Q in LDS: one launch instead of 2 + 3 T, which for such
// sizes are all latency (64 x 147, five steps: see the figures at the rule in
// gq_ortho.cpp).  The arithmetic is that of the tiled kernels.
//   G and Q: each wave takes two of the sixteen 16 x 16 blocks;
//   X: each wave takes every eighth block of 16 columns, and as a block of
//   a X + Q X needs those columns alone, writes it in place.
// In LDS the 16-byte chunks of row r lie at chunk ^ (r & 7).
__device__ __forceinline__ int sm_at(int r, int col, int pitch) {
    return r * pitch * 2 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2;
}

// Elements k0 + 8 * (lane / 16) on of row r16 + lane % 16.
__device__ __forceinline__ mm_f16x8 sm_row(const char *m, int r16, int k0, int pitch) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const mm_f16x8 *>(
        m + sm_at(r16 + (lane & 15), k0 + 8 * (lane >> 4), pitch));
}

// Elements k0 + 8 * (lane / 16) on of column c16 + lane % 16.
__device__ __forceinline__ mm_f16x8 sm_col(const char *m, int c16, int k0, int pitch) {
    const int lane = threadIdx.x & 63, q = lane & 15;
    mm_i16x4 h[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const char *p = m + sm_at(k0 + 8 * (lane >> 4) + 4 * t + (q >> 2), c16 + 4 * (q & 3), pitch);
        h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4 *)p);
    }
    return __builtin_bit_cast(mm_f16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename T, int LP>
__global__ __launch_bounds__(512) void k_ortho_small(const OrArgs a, const OrSteps st, int bf16) {
    __shared__ __align__(128) char xs[64 * LP * 2];
    __shared__ __align__(128) char gs[64 * 64 * 2];
    __shared__ __align__(128) char qs[64 * 64 * 2];
    __shared__ double sh[8];
    const OrMat &mt = a.mats[blockIdx.x];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lp = (mt.l + 63) & ~63;           // columns in use, a multiple of 64
    const int rows = mt.rows, cols = mt.cols;
    const T *g = static_cast<const T *>(a.g) + mt.off;
    float *mom = a.m ? a.m + mt.off : nullptr;
    // momentum and the sum of squares.  The matrix as it lies, 64 x LP or LP x
    // 64, is cut into rows of 64 elements, which the waves take in turn; u
    // stays in registers.
    constexpr int PER = LP / 8;                 // elements per lane
    const int across = mt.tr ? 1 : LP / 64;     // rows of 64 elements per row
    float u[PER];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int piece = i * 8 + wave, r = piece / across, c = piece % across * 64 + lane;
        u[i] = 0.0f;
        if (r < rows && c < cols) {
            const int e = r * cols + c;
            u[i] = __fmul_rn(to_f32(g[e]), a.in_mul);
            if (mom) {
                const float m = __fadd_rn(__fmul_rn(a.mu, mom[e]), u[i]);
                mom[e] = m;
                u[i] = a.nesterov ? __fadd_rn(u[i], __fmul_rn(a.mu, m)) : m;
            }
        }
        sum += static_cast<double>(u[i]) * static_cast<double>(u[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) sh[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += sh[i];
    const double mul = or_mul(mt.scale, sum, a.eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int piece = i * 8 + wave, r = piece / across, c = piece % across * 64 + lane;
        // zeros around the matrix, whatever the norm
        const bool in = r < rows && c < cols;
        const _Float16 h = static_cast<_Float16>(in ? static_cast<float>(u[i] * mul) : 0.0f);
        const int xr = mt.tr ? c : r, xc = mt.tr ? r : c;
        if (xc < lp) *reinterpret_cast<_Float16 *>(xs + sm_at(xr, xc, lp)) = h;
    }
    __syncthreads();
    const float inv = 1.0f / (mt.scale * mt.scale);     // a power of two
    const int bi = (wave >> 1) * 16, bj = (wave & 1) * 32;   // the wave's blocks of G and Q
    for (int k = 0; k < st.steps; ++k) {
        const float ca = st.coef[3 * k], cb = st.coef[3 * k + 1], cc = st.coef[3 * k + 2];
        mm_f32x4 acc[2] = {};
        for (int k1 = 0; k1 < lp; k1 += 64) {
            mm_f16x8 p[2], q[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p[h] = sm_row(xs, bi, k1 + 32 * h, lp);
#pragma unroll
                for (int j = 0; j < 2; ++j) q[h][j] = sm_row(xs, bj + 16 * j, k1 + 32 * h, lp);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[h][j], p[h], acc[j], 0, 0, 0);
        }
        const int r = bi + (lane & 15);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = bj + 16 * j + (lane >> 4) * 4;
            f16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = static_cast<_Float16>(acc[j][i] * inv);
            *reinterpret_cast<f16x4 *>(gs + sm_at(r, c, 64)) = h;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = mm_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k0 = 0; k0 < 64; k0 += 32) {
            const mm_f16x8 p = sm_row(gs, bi, k0, 64);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(sm_row(gs, bj + 16 * j, k0, 64), p,
                                                                acc[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = bj + 16 * j + (lane >> 4) * 4;
            const f16x4 gm = *reinterpret_cast<const f16x4 *>(gs + sm_at(r, c, 64));
            f16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = static_cast<_Float16>(__fmaf_rn(cc, acc[j][i], cb * static_cast<float>(gm[i])));
            *reinterpret_cast<f16x4 *>(qs + sm_at(r, c, 64)) = h;
        }
        __syncthreads();
        const bool last = k + 1 == st.steps;
        for (int c16 = wave * 16; c16 < lp; c16 += 128) {
            mm_f32x4 x[4] = {};
#pragma unroll
            for (int k0 = 0; k0 < 64; k0 += 32) {
                const mm_f16x8 q = sm_col(xs, c16, k0, lp);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q, sm_row(qs, 16 * i, k0, 64), x[i],
                                                                  0, 0, 0);
            }
            const int c = c16 + (lane >> 4) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int xr = 16 * i + (lane & 15);
                f16x4 *px = reinterpret_cast<f16x4 *>(xs + sm_at(xr, c, lp));
                const f16x4 xv = *px;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[i][e] = __fmaf_rn(ca, static_cast<float>(xv[e]), x[i][e]);
                if (!last) {
                    f16x4 h;
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(x[i][e]);
                    *px = h;
                } else if (xr < mt.s) {
                    const float om = mt.out_mul / mt.scale;
                    uint16_t *o = static_cast<uint16_t *>(a.out) + mt.off;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < mt.l)
                            o[mt.tr ? (c + e) * mt.s + xr : xr * mt.l + c + e] =
                                out_bits(x[i][e] * om, bf16 != 0);
                }
            }
        }
        __syncthreads();
    }
}

template <typename T>
void small_typed(const OrArgs &a, const OrSteps &st, int64_t n, int bf16, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(n));
    hipLaunchKernelGGL((k_ortho_small<T, OR_SMALL_L>), grid, dim3(512), 0, s, a, st, bf16);
}

template <typename S>
void mm_shape(const OrArgs &a, int64_t n, OrMode mode, bool bf16, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(n)), blk(S::THREADS);
    switch (mode) {
    case OR_MM_GRAM: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_GRAM>), grid, blk, 0, st, a); break;
    case OR_MM_POLY: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_POLY>), grid, blk, 0, st, a); break;
    case OR_MM_STEP: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_STEP>), grid, blk, 0, st, a); break;
    default:
        if (bf16) hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_LAST_BF16>), grid, blk, 0, st, a);
        else hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_LAST>), grid, blk, 0, st, a);
    }
}

template <typename T>
void norm_typed(const OrArgs &a, int64_t n, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(n)), blk(OR_BLOCK);
    if (a.m) hipLaunchKernelGGL((k_ortho_norm<T, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_ortho_norm<T, false>), grid, blk, 0, st, a);
}

template <typename T>
void cast_typed(const OrArgs &a, int64_t n, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(n)), blk(OR_BLOCK);
    if (a.m) hipLaunchKernelGGL((k_ortho_cast<T, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_ortho_cast<T, false>), grid, blk, 0, st, a);
}

}  // namespace

hipError_t launch_ortho_norm(const OrArgs &a, int64_t n, gq_dtype dt, hipStream_t st) {
    if (dt == GQ_F32) norm_typed<float>(a, n, st);
    else if (dt == GQ_F16) norm_typed<__half>(a, n, st);
    else norm_typed<bf16_t>(a, n, st);
    return hipGetLastError();
}

hipError_t launch_ortho_cast(const OrArgs &a, int64_t n, gq_dtype dt, hipStream_t st) {
    if (dt == GQ_F32) cast_typed<float>(a, n, st);
    else if (dt == GQ_F16) cast_typed<__half>(a, n, st);
    else cast_typed<bf16_t>(a, n, st);
    return hipGetLastError();
}

hipError_t launch_ortho_small(const OrArgs &a, const OrSteps &st, int64_t n, gq_dtype dt,
                              gq_dtype out, hipStream_t s) {
    const int bf16 = out == GQ_BF16;
    if (dt == GQ_F32) small_typed<float>(a, st, n, bf16, s);
    else if (dt == GQ_F16) small_typed<__half>(a, st, n, bf16, s);
    else small_typed<bf16_t>(a, st, n, bf16, s);
    return hipGetLastError();
}

hipError_t launch_ortho_mm(const OrArgs &a, int64_t n, int tile, OrMode mode, gq_dtype out,
                           hipStream_t st) {
    if (mode == OR_MM_JOIN) {   // tiles of 64 (the sums lie alike for both of their shapes)
        hipLaunchKernelGGL((k_ortho_mm<MmSmall, OR_MM_JOIN>), dim3(static_cast<unsigned>(n)),
                           dim3(MmSmall::THREADS), 0, st, a);
        return hipGetLastError();
    }
    const bool bf16 = out == GQ_BF16;
    if (tile == 256) mm_shape<MmBig>(a, n, mode, bf16, st);
    else if (tile == 128) mm_shape<MmMid>(a, n, mode, bf16, st);
    else if (n > OR_FEW) mm_shape<MmSmall>(a, n, mode, bf16, st);
    else mm_shape<MmFew>(a, n, mode, bf16, st);
    return hipGetLastError();
}

}  // namespace gq
