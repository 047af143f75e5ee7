// gq_mx4_product.hip -- C = A B^T, or C += A B^T, of two MX4 matrices on the
// scaled 4-bit matrix instructions of gfx950 (gq_mm.h: the tile loop; the
// product of two blocks takes their two scale bytes as operands, so nothing
// is decoded).  Sums are binary32.
//   k_mx4_product  a tile of C; or, where C has too few tiles to fill the
//                  device, the tile's share of K into a partial C of its own;
//   k_mx4_join     adds the partial sums in the order of K.
// Measured, medians of 200 launches in a kernel trace: 8192^3 294 us, 3.7 PFLOP/s
// (events over calls in a row 297 - 309, with inputs that are not in the cache 317;
// the first launches after a pause up to 390); 4096 x 1024 x 16384 50 us in four
// parts and 15 to join them, 2.1 PFLOP/s; 1024 x 1024 x 512 added to fp32 6.4 us;
// 7 x 30522 x 1024 9.7 us.  8192 x 8192 with K = 1024 takes 85 us and each further
// 256 of K 7.8, 4.4 PFLOP/s: the loop runs near the instructions' rate, and 54 us do
// not depend on K, four rounds of filling the buffers and storing C with one work
// group per compute unit.
#include <hip/hip_fp16.h>

#include "gq_mm.h"
#include "gq_mx4.h"
#include "gq_mx4_product.h"

namespace gq {
namespace {

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > kInfBits) return static_cast<uint16_t>((u >> 16) | 0x40u);
    return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ uint16_t f16_bits(float v) {
    return __half_as_ushort(__float2half_rn(v));
}

// Four consecutive columns of a row of C, `n` of them inside.
template <gq_dtype DT>
__device__ __forceinline__ void store4(void *c, int64_t at, mm_f32x4 v, int n, bool vec,
                                       bool add) {
    if constexpr (DT == GQ_F32) {
        float *p = static_cast<float *>(c) + at;
        if (n >= 4 && vec) {
            mm_f32x4 *q = reinterpret_cast<mm_f32x4 *>(p);
            if (add) {
                const mm_f32x4 o = *q;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = __fadd_rn(o[k], v[k]);
            }
            *q = v;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) p[k] = add ? __fadd_rn(p[k], v[k]) : v[k];
        }
    } else {
        uint16_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = DT == GQ_F16 ? f16_bits(v[k]) : bf16_bits(v[k]);
        uint16_t *p = static_cast<uint16_t *>(c) + at;
        if (n >= 4 && vec) {
            *reinterpret_cast<uint2 *>(p) =
                make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                           h[2] | (static_cast<uint32_t>(h[3]) << 16));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) p[k] = h[k];
        }
    }
}

template <typename S, gq_dtype DT>
__global__ __launch_bounds__(S::THREADS) void k_mx4_product(const MxPArgs a) {
    MM_LDS(S);
    __shared__ __align__(128) char mm_scale[S::SCALE_LDS];
    const int tm = static_cast<int>((a.m + S::T - 1) / S::T);
    const int tn = static_cast<int>((a.n + S::T - 1) / S::T);
    int t = mm_xcd(blockIdx.x, gridDim.x);
    const int split = t / (tm * tn);
    int ti, tj;
    mm_tile(t - split * tm * tn, tm, tn, ti, tj);
    const int64_t i0 = static_cast<int64_t>(ti) * S::T, j0 = static_cast<int64_t>(tj) * S::T;
    const uint32_t bytes = static_cast<uint32_t>(a.nb) * MX_BYTES;
    const MmRows p = mm_rows(a.a, bytes, i0, a.m, S::T);
    const MmRows q = mm_rows(a.b, bytes, j0, a.n, S::T);
    const MmScale sc = mm_scale_of<S>(a.sa, a.sb, i0, j0, a.m, a.n, a.nb, a.a);
    MmAcc<S> acc = {};
    const int all = static_cast<int>((a.nb + 15) / 16);
    const int k0 = split * a.groups;
    mm_loop<S, true>(p, q, sc, k0, all - k0 < a.groups ? all - k0 : a.groups, mm_lds, mm_scale,
                     MmNoExtra{}, acc);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    void *c = a.c;
    int64_t ldc = a.ldc;
    bool vec = a.vec != 0, add = a.add != 0;
    if (a.splits > 1) {
        c = a.part + split * a.m * a.n;
        ldc = a.n;
        vec = a.n % 4 == 0;
        add = false;
    }
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
        const int64_t r = i0 + S::part_row(wave, i) + (lane & 15);
        if (r >= a.m) continue;
#pragma unroll
        for (int b = 0; b < S::PARTS; ++b) {
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                const int64_t col = j0 + S::part_col(wave, b) + 16 * j + (lane >> 4) * 4;
                const int left = a.n - col < 4 ? static_cast<int>(a.n - col) : 4;
                if (left <= 0) continue;
                if (DT != GQ_F32 && a.splits > 1)
                    store4<GQ_F32>(c, r * ldc + col, acc.c[b][i][j], left, vec, false);
                else
                    store4<DT>(c, r * ldc + col, acc.c[b][i][j], left, vec, add);
            }
        }
    }
}

template <gq_dtype DT>
__global__ __launch_bounds__(256) void k_mx4_join(const MxPArgs a) {
    const int64_t total = a.m * a.n;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
         e += static_cast<int64_t>(gridDim.x) * 256) {
        float v = a.part[e];
        for (int s = 1; s < a.splits; ++s) v = __fadd_rn(v, a.part[s * total + e]);
        const int64_t row = e / a.n, at = row * a.ldc + (e - row * a.n);
        if constexpr (DT == GQ_F32) {
            float *c = static_cast<float *>(a.c) + at;
            *c = a.add ? __fadd_rn(*c, v) : v;
        } else {
            static_cast<uint16_t *>(a.c)[at] = DT == GQ_F16 ? f16_bits(v) : bf16_bits(v);
        }
    }
}

int64_t tiles(const MxPArgs &a, int t) { return (a.m + t - 1) / t * ((a.n + t - 1) / t); }

template <typename S>
hipError_t product_shape(const MxPArgs &a, gq_dtype dt, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(tiles(a, S::T) * a.splits));
    const dim3 blk(S::THREADS);
    if (dt == GQ_F32) hipLaunchKernelGGL((k_mx4_product<S, GQ_F32>), grid, blk, 0, st, a);
    else if (dt == GQ_F16) hipLaunchKernelGGL((k_mx4_product<S, GQ_F16>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_mx4_product<S, GQ_BF16>), grid, blk, 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t want = (a.m * a.n + 255) / 256;
    const dim3 jg(static_cast<unsigned>(want < 4096 ? want : 4096));
    if (dt == GQ_F32) hipLaunchKernelGGL(k_mx4_join<GQ_F32>, jg, dim3(256), 0, st, a);
    else if (dt == GQ_F16) hipLaunchKernelGGL(k_mx4_join<GQ_F16>, jg, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_mx4_join<GQ_BF16>, jg, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

// The tile and the number of parts of K for an m x n x k product: of tiles of
// 256, 128 and 64, with K whole or in as many parts (of 1024 elements or more)
// as fill the compute units, the one that takes least time by
//   start + work groups per compute unit * steps * step  (+ what the join moves),
// start and step (256 elements of K) in us as they were measured alone.  Measured,
// us, tile / parts (* the choice):
//   1024 x 3000 x 1024      64/1  16.2   128/1  11.5*  256/1  17.2
//   1000 x 2048 x 8192      64/1  36.4   128/1  34.2   128/2  29.5*  256/1  63
//   1024 x 1024 x 16384     64/1  38.7   128/1  60.7   128/4  30.1*  256/1 115
//   4096 x 1024 x 4096      64/1  39.4   128/1  22.8*  256/1  39.1   256/4  39.1
//   4096 x 1024 x 16384     64/1 129     128/1  74.4   256/1 118     256/4  64.6*
//   3500 x 4096 x 8192      64/1 205     128/1 108     256/1  74.1*  256/2 111
//   7 x 30522 x 8192        64/1  36.3*  128/1  40.9   256/1  58.7   256/2  40.6
//   512 x 512 x 8192        64/1  20.1    64/4  13.7*  128/1  33.2   256/1  63
MxPlan mx4_product_plan(int64_t m, int64_t n, int64_t k, bool split) {
    static const struct { int tile; double start, step; } kinds[3] = {
        {256, 11.0, 1.85}, {128, 8.5, 1.0}, {64, 6.5, 0.52}};
    constexpr double kJoin = 3.0, kBytes = 7e6;     // us a launch, bytes a us
    MxPArgs a{};
    a.m = m;
    a.n = n;
    const int64_t groups = ((k + MX_BLOCK - 1) / MX_BLOCK + 15) / 16;
    MxPlan best{};
    double least = 0.0;
    for (const auto &kind : kinds) {
        const int64_t t = tiles(a, kind.tile);
        int64_t parts = split && t < MX_CUS ? MX_CUS / t : 1;
        if (parts > groups / 2) parts = groups / 2;
        for (const int64_t want : {int64_t{1}, parts}) {
            if (want < 1) continue;
            // (an even number of groups a part: the ring's rounds are of two)
            const int64_t per = want == 1 ? groups : ((groups + want - 1) / want + 1) / 2 * 2;
            const int64_t splits = (groups + per - 1) / per;
            const double rounds = static_cast<double>((t * splits + MX_CUS - 1) / MX_CUS);
            double us = kind.start + rounds * 2.0 * static_cast<double>(per) * kind.step;
            if (splits > 1)
                us += kJoin + static_cast<double>(2 * splits + 1) * 4.0 * static_cast<double>(m) *
                                  static_cast<double>(n) / kBytes;
            if (least == 0.0 || us < least) {
                least = us;
                best = {kind.tile, static_cast<int32_t>(splits), static_cast<int32_t>(per)};
            }
        }
    }
    return best;
}

hipError_t launch_mx4_product(const MxPArgs &in, int64_t k, gq_dtype dt, hipStream_t st) {
    MxPArgs a = in;
    const MxPlan p = mx4_product_plan(a.m, a.n, k, a.part != nullptr);
    a.splits = p.splits;
    a.groups = p.groups;
    if (p.tile == 256) return product_shape<MmBig>(a, dt, st);
    if (p.tile == 128) return product_shape<MmMid>(a, dt, st);
    // Up to two tiles of 64 per compute unit: a ring of four buffers.  16 x 4096 x
    // 16384 21.0 -> 16.0 us, 1024 x 1024 x 16384 53 -> 36 us; but its rounds are
    // of two groups: 1024 x 1024 x 512 5.6 us, 6.3 on the ring.
    const bool even = a.groups % 2 == 0 || a.groups > 4;
    if (even && tiles(a, 64) * a.splits <= 2 * MX_CUS) return product_shape<MmFew>(a, dt, st);
    return product_shape<MmSmall>(a, dt, st);
}

}  // namespace gq
