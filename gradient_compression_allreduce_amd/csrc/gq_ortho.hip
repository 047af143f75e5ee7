// gq_ortho.hip -- gfx950 kernels of the orthogonalised update: momentum, then
// T steps of the quintic Newton-Schulz iteration on every matrix of a plan,
//   X <- u / (|u|_F + eps);  G = X X^T;  Q = b G + c G G;  X <- a X + Q X.
//   k_ortho_norm  momentum, and each matrix's sum of squares in binary64;
//   k_ortho_cast  X and X^T in fp16 from u and the sum of squares;
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

// ---- X and X^T ------------------------------------------------------------------
// A work group takes a 64 x 64 tile of the padded matrix as it lies in the
// gradient, and writes it to X and, turned in LDS, to X^T (or the other way
// round where X is the transpose).  Each work group adds up its matrix's
// partial sums itself, always in the same order.
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
    const int rp = mt.tr ? mt.lp : mt.sp, cp = mt.tr ? mt.sp : mt.lp;
    _Float16 *direct = a.ws + (mt.tr ? mt.xt[0] : mt.x[0]);
    _Float16 *turned = a.ws + (mt.tr ? mt.x[0] : mt.xt[0]);
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
            if (mt.vec && n >= 4) {
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
        for (int k = 0; k < 4; ++k) {
            h[k] = static_cast<_Float16>(u[k]);
            turn[c + k][r] = h[k];
        }
        *reinterpret_cast<f16x4 *>(direct + static_cast<int64_t>(row) * cp + col) = h;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        const f16x4 h = *reinterpret_cast<const f16x4 *>(&turn[r][c]);
        *reinterpret_cast<f16x4 *>(turned + static_cast<int64_t>(t.j * OR_CAST_TILE + r) * rp +
                                   t.i * OR_CAST_TILE + c) = h;
    }
}

// ---- the products -----------------------------------------------------------------

__device__ __forceinline__ uint16_t out_bits(float v, bool bf16) {
    if (!bf16) return __half_as_ushort(__float2half_rn(v));
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
    return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

// MODE OR_MM_GRAM: G = X X^T          (K: columns of X)
//      OR_MM_POLY: Q = b G + c G G    (G = G^T)
//      OR_MM_STEP: X <- a X + Q X     (both X and X^T written)
//      OR_MM_LAST: the same into the caller's output
template <typename S, int MODE>
__global__ __launch_bounds__(S::THREADS) void k_ortho_mm(const OrArgs a, int bf16) {
    __shared__ __align__(128) char s0[S::STAGE];
    __shared__ __align__(128) char s1[S::STAGE];
    const OrTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const OrMat &mt = a.mats[t.mat];
    const int sp = mt.sp, lp = mt.lp;
    const int i0 = t.i * S::BM, j0 = t.j * S::BN;
    const _Float16 *x = a.ws + mt.x[a.cur], *xt = a.ws + mt.xt[a.cur];
    const _Float16 *pm = MODE == OR_MM_GRAM ? x : a.ws + (MODE == OR_MM_POLY ? mt.a : mt.b);
    const _Float16 *qm = MODE == OR_MM_GRAM ? x : MODE == OR_MM_POLY ? pm : xt;
    const int kdim = MODE == OR_MM_GRAM ? lp : sp;
    const int qrows = MODE >= OR_MM_STEP ? lp : sp;
    const MmRows p = mm_rows(pm, kdim * 2, i0, sp, S::BM);
    const MmRows q = mm_rows(qm, kdim * 2, j0, qrows, S::BN);
    mm_f32x4 acc[S::FM][S::FN] = {};
    mm_loop<S, false>(p, q, MmScale{}, 0, (kdim / 64 + 1) / 2, s0, s1, acc);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r0 = i0 + wave / S::WN * (S::BM / S::WM) + (lane & 15);
    const int c0 = j0 + wave % S::WN * (S::BN / S::WN) + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const int64_t r = r0 + 16 * i;
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
            const int64_t c = c0 + 16 * j;
            mm_f32x4 v = acc[i][j];
            f16x4 h;
            if constexpr (MODE == OR_MM_GRAM || MODE == OR_MM_POLY) {
                _Float16 *d = a.ws + (MODE == OR_MM_GRAM ? mt.a : mt.b);
                if constexpr (MODE == OR_MM_GRAM) {
                    const float inv = 1.0f / (mt.scale * mt.scale);   // a power of two
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = static_cast<_Float16>(v[k] * inv);
                } else {
                    const f16x4 gm = *reinterpret_cast<const f16x4 *>(pm + r * sp + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = static_cast<_Float16>(
                            __fmaf_rn(a.c, v[k], a.b * static_cast<float>(gm[k])));
                }
                *reinterpret_cast<f16x4 *>(d + r * sp + c) = h;
                if (t.i != t.j) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) d[(c + k) * sp + r] = h[k];
                }
            } else {
                const f16x4 xv = *reinterpret_cast<const f16x4 *>(x + r * lp + c);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = __fmaf_rn(a.a, static_cast<float>(xv[k]), v[k]);
                if constexpr (MODE == OR_MM_STEP) {
                    _Float16 *dx = a.ws + mt.x[a.cur ^ 1], *dt = a.ws + mt.xt[a.cur ^ 1];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[k] = static_cast<_Float16>(v[k]);
                        dt[(c + k) * sp + r] = h[k];
                    }
                    *reinterpret_cast<f16x4 *>(dx + r * lp + c) = h;
                } else {
                    const float mul = mt.out_mul / mt.scale;
                    uint16_t *o = static_cast<uint16_t *>(a.out) + mt.off;
                    if (r >= mt.s) continue;
                    uint16_t ob[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) ob[k] = out_bits(v[k] * mul, bf16 != 0);
                    if (!mt.tr && mt.vec && c + 4 <= mt.l) {
                        *reinterpret_cast<uint2 *>(o + r * mt.l + c) =
                            make_uint2(ob[0] | (static_cast<uint32_t>(ob[1]) << 16),
                                       ob[2] | (static_cast<uint32_t>(ob[3]) << 16));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (c + k < mt.l) o[mt.tr ? (c + k) * mt.s + r : r * mt.l + c + k] = ob[k];
                    }
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
    if (tile == 256) mm_shape<MmShape<256, 256, 2, 4>>(a, n, mode, bf16, st);
    else if (tile == 128) mm_shape<MmShape<128, 128, 2, 2>>(a, n, mode, bf16, st);
    else mm_shape<MmShape<64, 64, 2, 2>>(a, n, mode, bf16, st);
    return hipGetLastError();
}

}  // namespace gq
