// gq_ortho.hip -- gfx950 kernels of the orthogonalised update: momentum, then
// T steps of the quintic Newton-Schulz iteration on every matrix of a plan,
//   X <- u / (|u|_F + eps);  G = X X^T;  Q = b G + c G G;  X <- a X + Q X.
//   k_ortho_norm  momentum, and each matrix's sum of squares in binary64;
//   k_ortho_cast  X in fp16 from u and the sum of squares;
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

// ---- momentum and sums of squares ---------------------------------------------
// A work group takes one chunk of a matrix, cut at multiples of four elements
// of the flat buffers (whose starts are 16-byte aligned).
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
// order.
template <typename T, bool MOM>
__global__ __launch_bounds__(OR_BLOCK) void k_ortho_cast(const OrArgs a) {
    __shared__ double sh[OR_BLOCK / 64];
    __shared__ _Float16 turn[OR_CAST_TILE][OR_CAST_TILE + 4];
    const OrTile t = a.tiles[blockIdx.x];
    const OrMat &mt = a.mats[t.mat];
    double sum = 0.0;
    for (int i = threadIdx.x; i < mt.parts; i += OR_BLOCK) sum += a.part[mt.part + i];
    sum = block_sum(sum, sh);
    // in binary64: the norm's reciprocal may lie outside the range of binary32
    const double mul = static_cast<double>(mt.scale) /
                       (__dsqrt_rn(sum) + static_cast<double>(a.eps));
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
//      OR_MM_LAST: the same into the caller's output
template <typename S, int MODE>
__global__ __launch_bounds__(S::THREADS) void k_ortho_mm(const OrArgs a, int bf16) {
    MM_LDS(S);
    const OrTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const OrMat &mt = a.mats[t.mat];
    const int sp = mt.sp, lp = mt.lp;
    const int i0 = t.i * S::T, j0 = t.j * S::T;
    const _Float16 *x = a.ws + mt.x[a.cur];
    const _Float16 *pm = MODE == OR_MM_GRAM ? x : a.ws + (MODE == OR_MM_POLY ? mt.a : mt.b);
    const int kdim = MODE == OR_MM_GRAM ? lp : sp;
    const MmRows p = mm_rows(pm, kdim * 2, i0, sp, S::T);
    MmAcc<S> acc = {};
    const int groups = (kdim + 127) / 128;
    if constexpr (MODE == OR_MM_GRAM || MODE == OR_MM_POLY) {
        const MmRows q = mm_rows(pm, kdim * 2, j0, sp, S::T);
        mm_loop<S, false>(p, q, MmScale{}, 0, groups, mm_lds, nullptr, MmNoExtra{}, acc);
    } else {
        const MmCols q = {reinterpret_cast<const char *>(x + j0), static_cast<uint32_t>(lp) * 2u,
                          static_cast<uint32_t>(j0) * 2u, sp};
        mm_loop<S, false>(p, q, MmScale{}, 0, groups, mm_lds, nullptr, AddX{a.a, i0}, acc);
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    constexpr int TM = 16 * S::FM, TN = 16 * S::FN, PART = TM * TN * 2;
    static_assert(PART * S::PARTS * S::WM * S::WN <= 2 * S::UNIT * (S::QUAD ? 4 : 1),
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
                    const float mul = MODE == OR_MM_GRAM ? 1.0f / (mt.scale * mt.scale)
                                      : MODE == OR_MM_LAST ? mt.out_mul / mt.scale : 1.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = out_bits(v[k] * mul, MODE == OR_MM_LAST && bf16);
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
    if constexpr (MODE == OR_MM_GRAM || MODE == OR_MM_POLY) {
        d = reinterpret_cast<uint16_t *>(a.ws + (MODE == OR_MM_GRAM ? mt.a : mt.b));
        ld = ldt = sp;
        by_cols = t.i != t.j;
    } else if constexpr (MODE == OR_MM_STEP) {
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

template <typename S>
void mm_shape(const OrArgs &a, int64_t n, OrMode mode, int bf16, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(n)), blk(S::THREADS);
    switch (mode) {
    case OR_MM_GRAM: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_GRAM>), grid, blk, 0, st, a, bf16); break;
    case OR_MM_POLY: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_POLY>), grid, blk, 0, st, a, bf16); break;
    case OR_MM_STEP: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_STEP>), grid, blk, 0, st, a, bf16); break;
    case OR_MM_LAST: hipLaunchKernelGGL((k_ortho_mm<S, OR_MM_LAST>), grid, blk, 0, st, a, bf16); break;
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

hipError_t launch_ortho_mm(const OrArgs &a, int64_t n, int tile, OrMode mode, gq_dtype out,
                           hipStream_t st) {
    const int bf16 = out == GQ_BF16;
    if (tile == 256) mm_shape<MmBig>(a, n, mode, bf16, st);
    else if (tile == 128) mm_shape<MmMid>(a, n, mode, bf16, st);
    else mm_shape<MmSmall>(a, n, mode, bf16, st);
    return hipGetLastError();
}

}  // namespace gq
