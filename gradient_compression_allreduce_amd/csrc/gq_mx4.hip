// gq_mx4.hip -- gfx950 kernels of the microscaled 4-bit gradient exchange:
//   k_mx4_quantize       codes and scales of W ranks' gradients, blocks along
//                        contiguous 16-byte aligned rows;
//   k_mx4_quantize_any   the same for rows of any alignment;
//   k_mx4_quantize_cols  blocks down the columns (the transposed matrix's
//                        codes), as a product over the rows reads them;
//   k_mx4_reduce         the rank-order fp32 sum of W ranks' codes and, fused
//                        with it, that sum's codes.
// The format and its arithmetic: gq_mx4.h.  All of it is bound by HBM: a
// block's maximum needs the block alone, so every input is read once and
// every output written once, with no exchange between waves.
#include <hip/hip_fp16.h>

#include "gq_mx4.h"

namespace gq {
namespace {

constexpr int MXQ_BLOCK = 256;
constexpr int MXQ_SLOTS = 4;      // 16-byte slots per lane in flight
constexpr int MXT_WAVES = 8;      // transposed: 8 x 16 bytes = one line per column
constexpr int MXR_BLOCK = 256;
constexpr int MXR_RG = 8;         // ranks loaded together
constexpr uint32_t kAbs = 0x7fffffffu;
constexpr int64_t MX_MAX_GRID = 1 << 20;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v.bits) << 16);
}

template <typename T>
__device__ __forceinline__ float slot_f32(const u32x4 &r, int k);
template <>
__device__ __forceinline__ float slot_f32<float>(const u32x4 &r, int k) {
    return __uint_as_float(r[k]);
}
template <>
__device__ __forceinline__ float slot_f32<__half>(const u32x4 &r, int k) {
    const uint32_t w = r[k >> 1];
    return __half2float(__ushort_as_half(static_cast<unsigned short>((k & 1) ? w >> 16 : w)));
}
template <>
__device__ __forceinline__ float slot_f32<bf16_t>(const u32x4 &r, int k) {
    const uint32_t w = r[k >> 1];
    return __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// Max over aligned groups of 4, 8 or 32 lanes (every lane gets it): within
// quads by quad permutes, then by mirrors of half rows and rows, whose other
// half holds one value already.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
    m = umax(m, dpp<0xB1>(m));                      // lanes 1 0 3 2
    m = umax(m, dpp<0x4E>(m));                      // lanes 2 3 0 1
    if (L >= 8) m = umax(m, dpp<0x141>(m));         // half row mirrored
    if (L >= 16) m = umax(m, dpp<0x140>(m));        // row mirrored
    if (L >= 32) m = umax(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
    return m;
}

// ---- quantize, rows ---------------------------------------------------------
// Lane l of a work group takes the 16-byte slots l, l + 256, ... of its 16 KiB
// of input; the 8 (fp32) or 4 (16-bit) lanes that hold a block combine their
// maxima by lane permutes and write 2 or 4 bytes of codes each.  A row's
// slots are counted up to whole blocks; those past its end read as zeros.
template <typename T, bool MUL, bool ROWS>
__global__ __launch_bounds__(MXQ_BLOCK) void k_mx4_quantize(const MxQArgs a) {
    constexpr int V = 16 / sizeof(T);
    constexpr int L = MX_BLOCK / V;
    const int w = blockIdx.y;
    const T *x = static_cast<const T *>(a.x[w]);
    uint8_t *q = a.q[w], *sc = a.scale[w];
    const int64_t spr = a.nb * L, total = a.rows * spr;
    const int64_t chunk = MXQ_BLOCK * MXQ_SLOTS;
    for (int64_t c0 = blockIdx.x * chunk; c0 < total; c0 += gridDim.x * chunk) {
        u32x4 raw[MXQ_SLOTS];
#pragma unroll
        for (int s = 0; s < MXQ_SLOTS; ++s) {
            const int64_t j = c0 + s * MXQ_BLOCK + threadIdx.x;
            int64_t row = 0, col = j * V;
            if (ROWS) {   // total < 2^32 here
                const uint32_t r32 = static_cast<uint32_t>(j) / static_cast<uint32_t>(spr);
                row = r32;
                col = static_cast<int64_t>(static_cast<uint32_t>(j) -
                                           r32 * static_cast<uint32_t>(spr)) * V;
            }
            const T *p = x + row * a.ld + col;
            raw[s] = u32x4{0, 0, 0, 0};
            if (j < total) {
                if (col + V <= a.cols) {
                    raw[s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        if (col + k >= a.cols) continue;
                        if constexpr (V == 4)
                            raw[s][k] = reinterpret_cast<const uint32_t *>(p)[k];
                        else
                            raw[s][k >> 1] |= static_cast<uint32_t>(
                                reinterpret_cast<const uint16_t *>(p)[k]) << (16 * (k & 1));
                    }
                }
            }
        }
#pragma unroll
        for (int s = 0; s < MXQ_SLOTS; ++s) {
            const int64_t j = c0 + s * MXQ_BLOCK + threadIdx.x;
            float g[V];
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                g[k] = slot_f32<T>(raw[s], k);
                if (MUL) g[k] = __fmul_rn(g[k], a.in_mul);
                m = umax(m, __float_as_uint(g[k]) & kAbs);
            }
            const uint32_t b = mx_byte(group_max<L>(m));
            const float mul = mx_mult(b);
            uint32_t code = mx_code2<0>(0u, g[0] * mul, g[1] * mul);
            code = mx_code2<1>(code, g[2] * mul, g[3] * mul);
            if constexpr (V == 8) {
                code = mx_code2<2>(code, g[4] * mul, g[5] * mul);
                code = mx_code2<3>(code, g[6] * mul, g[7] * mul);
            }
            if (b == 255u) code = 0u;
            if (j < total) {
                if constexpr (V == 4)
                    reinterpret_cast<uint16_t *>(q)[j] = static_cast<uint16_t>(code);
                else
                    reinterpret_cast<uint32_t *>(q)[j] = code;
                if ((threadIdx.x & (L - 1)) == 0) sc[j / L] = static_cast<uint8_t>(b);
            }
        }
    }
}

// Rows of any start and length: half a wave takes a block, one element per
// lane (coalesced loads of the element's size, no alignment needed).
template <typename T, bool MUL>
__global__ __launch_bounds__(MXQ_BLOCK) void k_mx4_quantize_any(const MxQArgs a) {
    constexpr int UB = 4;   // blocks in flight per half wave
    const int w = blockIdx.y;
    const T *x = static_cast<const T *>(a.x[w]);
    const int e = threadIdx.x & 31;
    const int64_t total = a.rows * a.nb;
    const int64_t half = static_cast<int64_t>(blockIdx.x) * (MXQ_BLOCK / 32) + (threadIdx.x >> 5);
    const int64_t halves = static_cast<int64_t>(gridDim.x) * (MXQ_BLOCK / 32);
    for (int64_t i0 = half * UB; i0 < total; i0 += halves * UB) {
        float g[UB];
        int64_t row = i0 / a.nb, b = i0 - row * a.nb;
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int64_t col = b * MX_BLOCK + e;
            g[u] = 0.0f;
            if (i0 + u < total && col < a.cols) g[u] = to_f32(x[row * a.ld + col]);
            if (++b == a.nb) {
                b = 0;
                ++row;
            }
        }
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            if (MUL) g[u] = __fmul_rn(g[u], a.in_mul);
            const uint32_t s = mx_byte(group_max<32>(__float_as_uint(g[u]) & kAbs));
            const float v = g[u] * mx_mult(s);
            const float next = __uint_as_float(dpp<0xB1>(__float_as_uint(v)));
            uint32_t code = mx_code2<0>(0u, v, next) & 0xffu;
            if (s == 255u) code = 0u;
            if (i0 + u < total) {
                if ((e & 1) == 0)
                    a.q[w][(i0 + u) * MX_BYTES + (e >> 1)] = static_cast<uint8_t>(code);
                if (e == 0) a.scale[w][i0 + u] = static_cast<uint8_t>(s);
            }
        }
    }
}

// ---- quantize, columns ------------------------------------------------------
// A wave takes 32 rows of 64 * F columns: every lane holds F whole blocks in
// registers, so no lane needs another's maximum.  The eight waves of a work
// group take consecutive blocks of the same columns, so the 16-byte stores of
// a column fill a 128-byte line in the L2 cache.  F elements are one 16-byte
// load where every row is aligned for it, otherwise F = 1.
template <typename T, bool MUL, int F>
__device__ __forceinline__ void quantize_cols(const MxQArgs &a, int64_t b, int64_t col) {
    const int w = blockIdx.y;
    const T *x = static_cast<const T *>(a.x[w]);
    const int64_t r0 = b * MX_BLOCK;
    const T *p = x + r0 * a.ld + col;
    const bool whole = r0 + MX_BLOCK <= a.rows && col + F <= a.cols;
    u32x4 raw[F > 1 ? MX_BLOCK : 1];
    float one[F > 1 ? 1 : MX_BLOCK];
#pragma unroll
    for (int i = 0; i < MX_BLOCK; ++i) {
        if constexpr (F > 1) {
            raw[i] = u32x4{0, 0, 0, 0};
            if (whole) {
                raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + i * a.ld));
            } else if (r0 + i < a.rows) {
#pragma unroll
                for (int k = 0; k < F; ++k) {
                    if (col + k >= a.cols) continue;
                    const T *e = p + i * a.ld + k;
                    if constexpr (F == 4)
                        raw[i][k] = *reinterpret_cast<const uint32_t *>(e);
                    else
                        raw[i][k >> 1] |= static_cast<uint32_t>(
                            *reinterpret_cast<const uint16_t *>(e)) << (16 * (k & 1));
                }
            }
        } else {
            one[i] = r0 + i < a.rows ? to_f32(p[i * a.ld]) : 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < F; ++k) {
        if (col + k >= a.cols) break;
        auto get = [&](int i) {
            float g;
            if constexpr (F > 1) g = slot_f32<T>(raw[i], k);
            else g = one[i];
            return MUL ? __fmul_rn(g, a.in_mul) : g;
        };
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < MX_BLOCK; ++i) m = umax(m, __float_as_uint(get(i)) & kAbs);
        const uint32_t s = mx_byte(m);
        const float mul = mx_mult(s);
        u32x4 code;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c = mx_code2<0>(0u, get(8 * i) * mul, get(8 * i + 1) * mul);
            c = mx_code2<1>(c, get(8 * i + 2) * mul, get(8 * i + 3) * mul);
            c = mx_code2<2>(c, get(8 * i + 4) * mul, get(8 * i + 5) * mul);
            c = mx_code2<3>(c, get(8 * i + 6) * mul, get(8 * i + 7) * mul);
            code[i] = s == 255u ? 0u : c;
        }
        const int64_t o = (col + k) * a.nb + b;
        *reinterpret_cast<u32x4 *>(a.q[w] + o * MX_BYTES) = code;
        a.scale[w][o] = static_cast<uint8_t>(s);
    }
}

template <typename T, bool MUL, int F>
__global__ __launch_bounds__(64 * MXT_WAVES) void k_mx4_quantize_cols(const MxQArgs a,
                                                                      int64_t col_groups,
                                                                      int64_t n_groups) {
    for (int64_t i = blockIdx.x; i < n_groups; i += gridDim.x) {
        const int64_t b = i / col_groups * MXT_WAVES + (threadIdx.x >> 6);
        const int64_t col = (i % col_groups * 64 + (threadIdx.x & 63)) * F;
        if (b < a.nb && col < a.cols) quantize_cols<T, MUL, F>(a, b, col);
    }
}

// ---- reduce -----------------------------------------------------------------
// A lane sums a whole block: 16 bytes of codes and a scale byte per rank, 32
// sums in registers, ranks in order.  A value times its scale is exact, so
// one fused multiply-add per element rounds the sum alone.  The sum's codes
// need the lane's own maximum only.  The sums leave through the wave's 8 KiB
// of LDS, so that the wave's stores of 16 bytes per lane are contiguous.
// FLAT: rows == 1 or whole blocks, so the sums are one 16-byte aligned array.
template <bool SUM, bool CODES, bool FLAT>
__global__ __launch_bounds__(MXR_BLOCK) void k_mx4_reduce(const MxRArgs a) {
    __shared__ f32x4 lds[SUM ? MXR_BLOCK * 8 : 1];
    const int lane = threadIdx.x & 63;
    const int64_t total = a.rows * a.nb;
    const int64_t step = static_cast<int64_t>(gridDim.x) * MXR_BLOCK;
    for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * MXR_BLOCK + (threadIdx.x & ~63);
         w0 < total; w0 += step) {
        const int64_t j = w0 + lane;
        const bool in = j < total;
        float acc[MX_BLOCK];
#pragma unroll
        for (int i = 0; i < MX_BLOCK; ++i) acc[i] = 0.0f;
        for (int r0 = 0; r0 < a.W; r0 += MXR_RG) {
            u32x4 raw[MXR_RG];
            uint32_t sb[MXR_RG];
#pragma unroll
            for (int r = 0; r < MXR_RG; ++r) {
                if (r0 + r >= a.W) break;
                raw[r] = u32x4{0, 0, 0, 0};
                sb[r] = 0;
                if (in) {
                    raw[r] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(a.q[r0 + r]) + j);
                    sb[r] = a.scale[r0 + r][j];
                }
            }
#pragma unroll
            for (int r = 0; r < MXR_RG; ++r) {
                if (r0 + r >= a.W) break;
                const float two = mx_two(sb[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t c = raw[r][i];
                    const f32x2_t v0 = mx_value2<0>(c), v1 = mx_value2<1>(c);
                    const f32x2_t v2 = mx_value2<2>(c), v3 = mx_value2<3>(c);
                    float *p = acc + 8 * i;
                    p[0] = __fmaf_rn(v0.x, two, p[0]);
                    p[1] = __fmaf_rn(v0.y, two, p[1]);
                    p[2] = __fmaf_rn(v1.x, two, p[2]);
                    p[3] = __fmaf_rn(v1.y, two, p[3]);
                    p[4] = __fmaf_rn(v2.x, two, p[4]);
                    p[5] = __fmaf_rn(v2.y, two, p[5]);
                    p[6] = __fmaf_rn(v3.x, two, p[6]);
                    p[7] = __fmaf_rn(v3.y, two, p[7]);
                }
            }
        }
        int64_t row = 0, b = j;
        if (!FLAT) {
            row = j / a.nb;
            b = j - row * a.nb;
        }
        if (CODES) {
            const int64_t left = a.cols - b * MX_BLOCK;   // elements from the block's first on
            uint32_t m = 0;
            float g[MX_BLOCK];
#pragma unroll
            for (int i = 0; i < MX_BLOCK; ++i) {
                g[i] = i < left ? acc[i] : 0.0f;
                m = umax(m, __float_as_uint(g[i]) & kAbs);
            }
            const uint32_t s = mx_byte(m);
            const float mul = mx_mult(s);
            u32x4 code;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *p = g + 8 * i;
                uint32_t c = mx_code2<0>(0u, p[0] * mul, p[1] * mul);
                c = mx_code2<1>(c, p[2] * mul, p[3] * mul);
                c = mx_code2<2>(c, p[4] * mul, p[5] * mul);
                c = mx_code2<3>(c, p[6] * mul, p[7] * mul);
                code[i] = s == 255u ? 0u : c;
            }
            if (in) {
                reinterpret_cast<u32x4 *>(a.q_out)[j] = code;
                a.scale_out[j] = static_cast<uint8_t>(s);
            }
        }
        if (SUM) {
            // 16-byte piece p of lane l's block at slot 8 l + (p ^ (l & 7)):
            // the eight lanes of a line's pieces fall into different banks
            f32x4 *my = lds + (threadIdx.x & ~63) * 8;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                my[8 * lane + (p ^ (lane & 7))] =
                    f32x4{acc[4 * p], acc[4 * p + 1], acc[4 * p + 2], acc[4 * p + 3]};
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (FLAT) {
                const int64_t n = a.rows * a.cols;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = i * 64 + lane, blk = t >> 3, p = t & 7;
                    const f32x4 v = my[8 * blk + (p ^ (blk & 7))];
                    const int64_t e = (w0 + blk) * MX_BLOCK + 4 * p;
                    if (e + 4 <= n) {
                        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(a.r + e));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (e + k < n) a.r[e + k] = v[k];
                    }
                }
            } else {
                for (int i = 0; i < 32; ++i) {
                    const int blk = 2 * i + (lane >> 5), k = lane & 31;
                    const int64_t jj = w0 + blk;
                    if (jj >= total) break;
                    const float v = my[8 * blk + ((k >> 2) ^ (blk & 7))][k & 3];
                    const int64_t rr = jj / a.nb, cc = (jj - rr * a.nb) * MX_BLOCK + k;
                    if (cc < a.cols) a.r[rr * a.cols + cc] = v;
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    }
}

int64_t groups(int64_t work, int64_t per) {
    const int64_t g = (work + per - 1) / per;
    return g < MX_MAX_GRID ? g : MX_MAX_GRID;
}

template <typename T, bool MUL>
hipError_t quantize_typed(const MxQArgs &in, bool transpose, hipStream_t st) {
    MxQArgs a = in;
    constexpr int V = 16 / sizeof(T);
    constexpr int64_t L = MX_BLOCK / V;
    const bool wide = a.ld % V == 0;    // every row starts 16-byte aligned
    const unsigned W = static_cast<unsigned>(a.W);
    if (transpose) {
        a.nb = (a.rows + MX_BLOCK - 1) / MX_BLOCK;
        const int64_t per = 64 * (wide ? V : 1);
        const int64_t cg = (a.cols + per - 1) / per;
        const int64_t n = cg * ((a.nb + MXT_WAVES - 1) / MXT_WAVES);
        const dim3 grid(static_cast<unsigned>(groups(n, 1)), W);
        if (wide)
            hipLaunchKernelGGL((k_mx4_quantize_cols<T, MUL, V>), grid, dim3(64 * MXT_WAVES), 0, st,
                               a, cg, n);
        else
            hipLaunchKernelGGL((k_mx4_quantize_cols<T, MUL, 1>), grid, dim3(64 * MXT_WAVES), 0, st,
                               a, cg, n);
        return hipGetLastError();
    }
    a.nb = (a.cols + MX_BLOCK - 1) / MX_BLOCK;
    if (a.ld == a.cols && a.cols % MX_BLOCK == 0) {   // whole blocks: one long row
        a.cols *= a.rows;
        a.nb *= a.rows;
        a.rows = 1;
    }
    const int64_t slots = a.rows * a.nb * L;
    if (a.rows == 1) {
        const dim3 grid(static_cast<unsigned>(groups(slots, MXQ_BLOCK * MXQ_SLOTS)), W);
        hipLaunchKernelGGL((k_mx4_quantize<T, MUL, false>), grid, dim3(MXQ_BLOCK), 0, st, a);
    } else if (wide && slots < (int64_t{1} << 32) - MXQ_BLOCK * MXQ_SLOTS) {
        const dim3 grid(static_cast<unsigned>(groups(slots, MXQ_BLOCK * MXQ_SLOTS)), W);
        hipLaunchKernelGGL((k_mx4_quantize<T, MUL, true>), grid, dim3(MXQ_BLOCK), 0, st, a);
    } else {
        const dim3 grid(static_cast<unsigned>(groups(a.rows * a.nb, MXQ_BLOCK / 32 * 4)), W);
        hipLaunchKernelGGL((k_mx4_quantize_any<T, MUL>), grid, dim3(MXQ_BLOCK), 0, st, a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t quantize_mul(const MxQArgs &a, bool transpose, hipStream_t st) {
    return a.in_mul != 1.0f ? quantize_typed<T, true>(a, transpose, st)
                            : quantize_typed<T, false>(a, transpose, st);
}

template <bool SUM, bool CODES>
void reduce_flat(const MxRArgs &in, hipStream_t st) {
    MxRArgs a = in;
    if (a.cols % MX_BLOCK == 0) {   // whole blocks: one long row
        a.cols *= a.rows;
        a.nb *= a.rows;
        a.rows = 1;
    }
    const dim3 grid(static_cast<unsigned>(groups(a.rows * a.nb, MXR_BLOCK)));
    if (a.rows == 1)
        hipLaunchKernelGGL((k_mx4_reduce<SUM, CODES, true>), grid, dim3(MXR_BLOCK), 0, st, a);
    else
        hipLaunchKernelGGL((k_mx4_reduce<SUM, CODES, false>), grid, dim3(MXR_BLOCK), 0, st, a);
}

}  // namespace

hipError_t launch_mx4_quantize(const MxQArgs &a, gq_dtype dt, bool transpose, hipStream_t st) {
    if (dt == GQ_F32) return quantize_mul<float>(a, transpose, st);
    if (dt == GQ_F16) return quantize_mul<__half>(a, transpose, st);
    return quantize_mul<bf16_t>(a, transpose, st);
}

hipError_t launch_mx4_reduce(const MxRArgs &a, hipStream_t st) {
    if (a.r && a.q_out) reduce_flat<true, true>(a, st);
    else if (a.r) reduce_flat<true, false>(a, st);
    else reduce_flat<false, true>(a, st);
    return hipGetLastError();
}

}  // namespace gq
