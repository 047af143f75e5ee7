// gq_ortho.hip -- gfx950 kernels of the orthogonalised update: momentum, then
// T steps of the quintic Newton-Schulz iteration on every matrix of a plan,
//   X <- u / (|u|_F + eps);  G = X X^T;  Q = b G + c G G;  X <- a X + Q X.
// As it is computed, with D and E the diagonals of G and Q, in fp32, G0 and Q0
// the rest, in fp16, and X = x + y, x in fp16 and y of 8 bits:
//   D + G0 = x x^T
//   E + Q0 = b (D + G0) + c (D D + D G0 + G0 D + G0 G0)
//   X <- (a + E) (x + y) + Q0 x
//   k_ortho_norm  momentum, and each matrix's sum of squares in binary64;
//   k_ortho_cast  X from u and the sum of squares;
//   k_ortho_small the whole update of a matrix that fits one work group's LDS;
//   k_ortho_mm    the three products of a step over the tiles of all
//                 matrices together (gq_mm.h: the tile loop), the polynomial
//                 and the update in its epilogue.
// The iteration multiplies an error in a small singular direction by up to a
// each step, and a rounding of X puts noise of all of X's size into all
// directions: with x alone the result was 1 to 4 percent off where a few
// directions hold nearly all of a gradient.  So X has y while three steps or more
// are to come (a^2 = 12 times half a step of x is what a rounding grows to
// without).  The products take x alone: their rounding reaches a direction only
// through Q, which is small in the steps that still have errors to grow.  In the
// last steps, where Q is not small, G and Q are nearly multiples of the identity,
// and with their diagonals exact only what is left of them is rounded or meets a
// rounded x.  Errors in the Frobenius norm, with x alone and whole G and Q / so:
// 300 x 310, two directions over noise of 1/64 of their norm 1.4e-2 / 7.0e-4, of
// 1/256 4.5e-2 / 2.0e-3; sixteen directions as strong as the noise 1.4e-3 / 7.5e-4;
// for 5 to 10 percent more time.  (Products of both halves of X, G and Q in the
// last two steps would come to 1e-4 in the last of these, for 1.8 times the
// operations; y in 16 bits to half the error in the second, for 13 to 23 percent.)
// x is fp16, not bf16: all singular values stay below about 1.3, so bf16's
// exponents are not needed and the three more bits are.  X is stored times a power
// of two near sqrt(l), which keeps the entries of a matrix with many columns out
// of the subnormal range.
// Products are summed in binary32, and the polynomial and the update are
// computed in binary32 from those sums and rounded once.
// G and Q are symmetric: only tiles on and above the diagonal are computed,
// and each is written to both places.
#include <hip/hip_fp16.h>

#include "gq_mm.h"
#include "gq_ortho.h"

namespace gq {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

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

// y: what fp16 leaves of a value, times OR_LOW, in the 8-bit format of 4 exponent
// and 3 fraction bits (up to 448, whole steps of 2^-9 below 2^-6), so X is held to
// 2^-16 of a value between 2^-7 and 2^5.  The entries of X lie there: their mean
// square, times the power of two that X is stored with, grows from about 1 / s to
// about 1.
constexpr float OR_LOW = 16384.0f;

// Four values' y; h: the values in fp16.
__device__ __forceinline__ uint32_t or_low4(f32x4 v, f16x4 h) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        y[k] = __builtin_amdgcn_fmed3f((v[k] - static_cast<float>(h[k])) * OR_LOW, -448.0f, 448.0f);
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true));
}

// Where the four elements (r, c) .. (r, c + 3) of a tile of X lie among those
// that k_ortho_mm's lanes hold: wave, instruction (block, row, column), lane.  A
// wave's instruction then reads and writes 256 bytes of y in a row.
template <typename S>
__device__ __forceinline__ int or_quad(uint32_t r, uint32_t c) {
    constexpr uint32_t TM = S::QUAD ? 64 : S::T / S::WM, TN = S::QUAD ? 32 : S::T / S::WN;
    constexpr uint32_t half = S::QUAD ? 128 : S::T;
    const uint32_t wave = r % half / TM * S::WN + c % half / TN;
    const uint32_t i = r / half * 4 + r % TM / 16, j = c % TN / 16, b = c / half;
    return (wave * (S::PARTS * S::FM * S::FN) + (b * S::FM + i) * S::FN + j) * 64 +
           (c >> 2 & 3) * 16 + (r & 15);
}

// Where y of the 16 x 16 elements from (row, col) on begins: 256 bytes in a row.
template <typename S>
__device__ __forceinline__ int64_t or_block(uint32_t lp, uint32_t row, uint32_t col) {
    const int64_t t = static_cast<int64_t>(row / S::T) * (lp / S::T) + col / S::T;
    return t * (S::T * S::T) + 4 * or_quad<S>(row % S::T, col % S::T);
}

// ---- momentum and sums of squares ---------------------------------------------
// A work group takes one chunk of a matrix, cut at multiples of four elements
// of the flat buffers (whose starts are 16-byte aligned).  Bound by HBM, with
// momentum: 303M fp16 gradients 582 us, 5.2 TB/s; 60M of fp32 123 us, 5.9 TB/s.
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
// order.  303M elements from their momentum 547 us, 3.9 TB/s; 60M from fp32
// gradients and momentum 160 us, 4.1 TB/s: its loads start when the norm is known.
template <typename T, bool MOM>
__global__ __launch_bounds__(OR_BLOCK) void k_ortho_cast(const OrArgs a) {
    __shared__ double sh[OR_BLOCK / 64];
    __shared__ _Float16 turn[OR_CAST_TILE][OR_CAST_TILE + 4];
    __shared__ __align__(16) uint8_t ys[OR_CAST_TILE * OR_CAST_TILE];
    const OrTile t = a.tiles[blockIdx.x];
    const OrMat &mt = a.mats[t.mat];
    double sum = 0.0;
    for (int i = threadIdx.x; i < mt.parts; i += OR_BLOCK) sum += a.part[mt.part + i];
    sum = block_sum(sum, sh);
    const double mul = or_mul(mt.scale, sum, a.eps);
    const T *g = static_cast<const T *>(a.g);
    const int c = (threadIdx.x & 15) * 4;
    _Float16 *x = a.ws + mt.x[0];
    // where y of X's element (r, c) of the tile waits: by blocks of 16 x 16
    auto slot = [](int r, int c) {
        return ((r >> 4) * 4 + (c >> 4)) * 256 + (c >> 2 & 3) * 64 + (r & 15) * 4 + (c & 3);
    };
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
        const uint32_t y = or_low4(u, h);
        if (mt.tr) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                turn[c + k][r] = h[k];
                ys[slot(c + k, r)] = static_cast<uint8_t>(y >> (8 * k));
            }
        } else {
            *reinterpret_cast<f16x4 *>(x + static_cast<int64_t>(row) * mt.lp + col) = h;
            *reinterpret_cast<uint32_t *>(ys + slot(r, c)) = y;
        }
    }
    __syncthreads();
    const int row0 = (mt.tr ? t.j : t.i) * OR_CAST_TILE, col0 = (mt.tr ? t.i : t.j) * OR_CAST_TILE;
    if (a.low_out) {
        const int block = threadIdx.x >> 4, at = (threadIdx.x & 15) * 16;
        const uint32_t row = row0 + (block >> 2) * 16, col = col0 + (block & 3) * 16;
        const int64_t to = a.tile_x == 256 ? or_block<MmBig>(mt.lp, row, col)
                           : a.tile_x == 128 ? or_block<MmMid>(mt.lp, row, col)
                                             : or_block<MmSmall>(mt.lp, row, col);
        *reinterpret_cast<uint4 *>(a.low + mt.low + to + at) =
            *reinterpret_cast<const uint4 *>(ys + block * 256 + at);
    }
    if (!mt.tr) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        *reinterpret_cast<f16x4 *>(x + static_cast<int64_t>(row0 + r) * mt.lp + col0 + c) =
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

// (a + E) x of the wave's part of the tile, added while those rows of x pass
// through LDS as rows of K: x is then read once.
template <typename S>
struct AddX {
    float (&f)[S::FM];      // a + E of the lane's row of each instruction row
    int i0;                 // the tile's first row
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
                            __fmaf_rn(f[i], static_cast<float>(x[k]), acc.c[b][i][j][k]);
                }
                __builtin_amdgcn_sched_barrier(0);   // few registers at a time
            }
        }
    }
};

// MODE OR_MM_GRAM: D and G0                   (K: columns of x)
//      OR_MM_POLY: E and Q0                   (G0 = G0^T)
//      OR_MM_STEP: x, y <- (a + E) X + Q0 x   (K: rows of x)
//      OR_MM_LAST, OR_MM_LAST_BF16: the same into the caller's output
//      OR_MM_JOIN: D and G0 from the partial sums that OR_MM_GRAM left of tiles
//                  whose K it split, added in the order of K
// 97 matrices of 1024 x 1024 and 48 of 1024 x 4096, tiles of 256, us a launch
// (medians of a kernel trace): G 389 (0.80 PFLOP/s of the upper half), Q 271 (0.57),
// X 788 (0.79; the first two read and write y), the last X 748 (0.83).  With
// K = 1024 a tile's loop is 16 steps, and filling the buffers and writing the tile
// out are a third of its time (X without its loop 220, of that 150 the stores);
// one work group per compute unit leaves nobody to cover them.
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
    float *const diag = a.diag + mt.diag;               // D, then E
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
            float f[S::FM];
#pragma unroll
            for (int i = 0; i < S::FM; ++i)
                f[i] = a.a + diag[sp + i0 + S::part_row(wave, i) + (lane & 15)];
            mm_loop<S, false>(p, q, MmScale{}, 0, groups, mm_lds, nullptr, AddX<S>{f, i0}, acc);
            if constexpr (!LAST) {
                // the same of y, and the new one's, in the order of the lanes
                uint32_t *const low = reinterpret_cast<uint32_t *>(
                    a.low + mt.low + (static_cast<int64_t>(t.i) * (lp / S::T) + t.j) *
                                         (S::T * S::T)) + wave * SUMS * 64 + lane;
                if (a.low_in) {
#pragma unroll
                    for (int k = 0; k < SUMS; ++k) {
                        const uint32_t w = low[k * 64];
                        const float by = f[k / S::FN % S::FM] * (1.0f / OR_LOW);
                        const f32x2 y0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
                        const f32x2 y1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
                        flat[k][0] = __fmaf_rn(by, y0.x, flat[k][0]);
                        flat[k][1] = __fmaf_rn(by, y0.y, flat[k][1]);
                        flat[k][2] = __fmaf_rn(by, y1.x, flat[k][2]);
                        flat[k][3] = __fmaf_rn(by, y1.y, flat[k][3]);
                        if (k % 16 == 15) __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if (a.low_out) {
#pragma unroll
                    for (int k = 0; k < SUMS; ++k) {
                        f16x4 h;
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(flat[k][e]);
                        low[k * 64] = or_low4(flat[k], h);
                        if (k % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    }
                    // (or all of h would be kept for below, in registers that
                    // the sums leave no room for)
                    mm_pin(flat, std::integral_constant<int, SUMS>{});
                }
            }
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
                // (the diagonals' elements, and 0 in their places)
                const int r = i0 + S::part_row(wave, i) + (lane & 15);
                const int c = j0 + S::part_col(wave, b) + cl;
                if constexpr (MODE == OR_MM_POLY) {
                    const f16x4 gm =
                        *reinterpret_cast<const f16x4 *>(pm + static_cast<int64_t>(r) * sp + c);
                    const mm_f32x4 dc = *reinterpret_cast<const mm_f32x4 *>(diag + c);
                    const float dr = diag[r];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = __fmaf_rn(a.c, dr + dc[k], a.b);
                        h[k] = out_bits(__fmaf_rn(a.c, v[k], f * static_cast<float>(gm[k])), false);
                        if (r == c + k) {
                            diag[sp + r] = __fmaf_rn(a.c, v[k], __fmaf_rn(a.c, dr, a.b) * dr);
                            h[k] = 0;
                        }
                    }
                } else {
                    // (both factors are powers of two but for out_mul)
                    const float mul = TO_G ? 1.0f / (mt.scale * mt.scale)
                                      : LAST ? mt.out_mul / mt.scale : 1.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[k] = out_bits(v[k] * mul, MODE == OR_MM_LAST_BF16);
                        if (TO_G && r == c + k) {
                            diag[r] = v[k] * mul;
                            h[k] = 0;
                        }
                    }
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
// waves, x, G0 and Q0 in LDS: one launch instead of 2 + 3 T, which for such
// sizes are all latency (64 x 147, five steps: see the figures at the rule in
// gq_ortho.cpp).  The arithmetic is that of the tiled kernels, but that X itself
// is held in binary32.
//   G and Q: each wave takes two of the sixteen 16 x 16 blocks;
//   X: each wave takes every eighth block of 16 columns, holds them in
//   registers, and as a block of (a + E) X + Q0 x needs those columns alone,
//   writes its x in place.
// In LDS the 16-byte chunks of row r lie at chunk ^ (r & 7).
__device__ __forceinline__ int sm_at(int r, int col, int pitch) {
    return r * pitch * 2 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2;
}

// Elements k0 + 8 * (lane / 16) on of row r16 + lane % 16.
__device__ __forceinline__ mm_f16x8 sm_row(const char *m, int r16, int k0, int pitch, int lane) {
    return *reinterpret_cast<const mm_f16x8 *>(
        m + sm_at(r16 + (lane & 15), k0 + 8 * (lane >> 4), pitch));
}

// Elements k0 + 8 * (lane / 16) on of column c16 + lane % 16.
__device__ __forceinline__ mm_f16x8 sm_col(const char *m, int c16, int k0, int pitch, int lane) {
    const int q = lane & 15;
    mm_i16x4 h[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const char *p = m + sm_at(k0 + 8 * (lane >> 4) + 4 * t + (q >> 2), c16 + 4 * (q & 3), pitch);
        h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4 *)p);
    }
    return __builtin_bit_cast(mm_f16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename T, int LP>
__global__ __launch_bounds__(512, 4) void k_ortho_small(const OrArgs a, const OrSteps st, int bf16) {
    // u in fp32 at first, in rows of lp + 4 (so that a column falls into sixteen
    // banks), then x, G0 and Q0
    __shared__ __align__(128) char mem[64 * (LP + 4) * 4];
    char *const xs = mem, *const gs = mem + 64 * LP * 2, *const qs = gs + 64 * 64 * 2;
    static_assert(64 * (LP + 4) * 4 >= 64 * LP * 2 + 2 * 64 * 64 * 2, "x, G0 and Q0 fit");
    __shared__ __align__(16) float ds[64], es[64];      // the diagonals of G and Q
    __shared__ double sh[8];
    const OrMat &mt = a.mats[blockIdx.x];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rows = mt.rows, cols = mt.cols, s = mt.s, l = mt.l;
    const bool tr = mt.tr != 0;
    const int lp = (l + 63) & ~63;              // columns in use, a multiple of 64
    const int64_t off = mt.off;
    const float om = mt.out_mul / mt.scale;
    const T *g = static_cast<const T *>(a.g) + off;
    float *mom = a.m ? a.m + off : nullptr;
    // momentum and the sum of squares: the matrix as it lies, in pieces of 64
    // elements of a row.  A wave takes every eighth row, with the loads of BATCH
    // pieces under way together.
    constexpr int BATCH = 16;
    const int lacross = cols > 128 ? 2 : cols > 64 ? 1 : 0;
    float *const us = reinterpret_cast<float *>(mem);
    const int pitch = lp + 4;
    double sum = 0.0;
    for (int k0 = 0; wave + 8 * (k0 >> lacross) < rows; k0 += BATCH) {
        float u[BATCH], old[BATCH];
        auto place = [&](int i, int &r, int &c) {
            r = wave + 8 * ((k0 + i) >> lacross);
            c = ((k0 + i) & ((1 << lacross) - 1)) * 64 + lane;
            return r < rows && c < cols;
        };
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            int r, c;
            u[i] = old[i] = 0.0f;
            if (place(i, r, c)) {
                u[i] = to_f32(g[r * cols + c]);
                if (mom) old[i] = mom[r * cols + c];
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            int r, c;
            if (!place(i, r, c)) continue;
            u[i] = __fmul_rn(u[i], a.in_mul);
            if (mom) {
                const float m = __fadd_rn(__fmul_rn(a.mu, old[i]), u[i]);
                mom[r * cols + c] = m;
                u[i] = a.nesterov ? __fadd_rn(u[i], __fmul_rn(a.mu, m)) : m;
            }
            us[tr ? c * pitch + r : r * pitch + c] = u[i];
            sum += static_cast<double>(u[i]) * static_cast<double>(u[i]);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) sh[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += sh[i];
    const double mul = or_mul(mt.scale, sum, a.eps);
    // the wave's blocks of X, and zeros around the matrix, whatever the norm
    constexpr int MINE = LP / 128;
    f32x4 mine[MINE][4] = {};
#pragma unroll
    for (int t = 0; t < MINE; ++t) {
        const int c = wave * 16 + t * 128 + (lane >> 4) * 4;
        if (wave * 16 + t * 128 >= lp) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * i + (lane & 15);
            const f32x4 v = *reinterpret_cast<const f32x4 *>(us + r * pitch + c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mine[t][i][k] = r < s && c + k < l ? static_cast<float>(v[k] * mul) : 0.0f;
        }
    }
    __syncthreads();
    auto put = [&](int t, int ln) {         // x of block t
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f16x4 h;
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = static_cast<_Float16>(mine[t][i][k]);
            *reinterpret_cast<f16x4 *>(
                xs + sm_at(16 * i + (ln & 15), wave * 16 + t * 128 + (ln >> 4) * 4, lp)) = h;
        }
    };
#pragma unroll
    for (int t = 0; t < MINE; ++t)
        if (wave * 16 + t * 128 < lp) put(t, lane);
    __syncthreads();
    const float inv = 1.0f / (mt.scale * mt.scale);     // a power of two
    const int bi = (wave >> 1) * 16, bj = (wave & 1) * 32;   // the wave's blocks of G and Q
    for (int k = 0; k < st.steps; ++k) {
        const int ln = mm_tid() & 63;
        const float ca = st.coef[3 * k], cb = st.coef[3 * k + 1], cc = st.coef[3 * k + 2];
        mm_f32x4 acc[2] = {};
        for (int k1 = 0; k1 < lp; k1 += 64) {
            mm_f16x8 p[2], q[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p[h] = sm_row(xs, bi, k1 + 32 * h, lp, ln);
#pragma unroll
                for (int j = 0; j < 2; ++j) q[h][j] = sm_row(xs, bj + 16 * j, k1 + 32 * h, lp, ln);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[h][j], p[h], acc[j], 0, 0, 0);
        }
        const int r = bi + (ln & 15);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = bj + 16 * j + (ln >> 4) * 4;
            f16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = static_cast<_Float16>(acc[j][i] * inv);
                if (r == c + i) {
                    ds[r] = acc[j][i] * inv;
                    h[i] = static_cast<_Float16>(0.0f);
                }
            }
            *reinterpret_cast<f16x4 *>(gs + sm_at(r, c, 64)) = h;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = mm_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k0 = 0; k0 < 64; k0 += 32) {
            const mm_f16x8 p = sm_row(gs, bi, k0, 64, ln);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(sm_row(gs, bj + 16 * j, k0, 64, ln), p,
                                                                acc[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = bj + 16 * j + (ln >> 4) * 4;
            const f16x4 gm = *reinterpret_cast<const f16x4 *>(gs + sm_at(r, c, 64));
            const f32x4 dc = *reinterpret_cast<const f32x4 *>(ds + c);
            const float dr = ds[r];
            f16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = __fmaf_rn(cc, dr + dc[i], cb);
                h[i] = static_cast<_Float16>(__fmaf_rn(cc, acc[j][i], f * static_cast<float>(gm[i])));
                if (r == c + i) {
                    es[r] = __fmaf_rn(cc, acc[j][i], __fmaf_rn(cc, dr, cb) * dr);
                    h[i] = static_cast<_Float16>(0.0f);
                }
            }
            *reinterpret_cast<f16x4 *>(qs + sm_at(r, c, 64)) = h;
        }
        __syncthreads();
        const bool last = k + 1 == st.steps;
#pragma unroll
        for (int t = 0; t < MINE; ++t) {
            const int c16 = wave * 16 + t * 128;
            if (c16 >= lp) continue;
            mm_f32x4 x[4] = {};
#pragma unroll
            for (int k0 = 0; k0 < 64; k0 += 32) {
                const mm_f16x8 q = sm_col(xs, c16, k0, lp, ln);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q, sm_row(qs, 16 * i, k0, 64, ln), x[i],
                                                                  0, 0, 0);
            }
            const int c = c16 + (ln >> 4) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int xr = 16 * i + (ln & 15);
                const float f = ca + es[xr];
                f32x4 &v = mine[t][i];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __fmaf_rn(f, v[e], x[i][e]);
                if (last && xr < s) {
                    uint16_t *o = static_cast<uint16_t *>(a.out) + off;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < l)
                            o[tr ? (c + e) * s + xr : xr * l + c + e] =
                                out_bits(v[e] * om, bf16 != 0);
                }
            }
            if (!last) put(t, ln);
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
