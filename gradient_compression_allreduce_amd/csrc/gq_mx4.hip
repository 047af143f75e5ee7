// gq_mx4.hip -- gfx950 kernels of the microscaled 4-bit gradient exchange:
//   k_mx4_quantize       codes and scales of W ranks' gradients, blocks along
//                        the rows;
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
constexpr int MXT_BLOCKS = 8;     // transposed: 8 x 16 bytes = one line per column
constexpr int MXR_BLOCK = 256;
constexpr int MXR_RG = 8;         // ranks loaded together
constexpr uint32_t kAbs = 0x7fffffffu;
constexpr int64_t MX_MAX_GRID = 1 << 20;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

struct bf16_t { uint16_t bits; };

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

template <typename T>
__device__ __forceinline__ uint32_t load_bits(const T *p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t *>(p);
    else return *reinterpret_cast<const uint16_t *>(p);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// Max over aligned groups of 4 or 8 lanes (every lane gets it): within quads by
// quad permutes, then by the mirror of half a row, whose other half holds one
// value already.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
    static_assert(L == 4 || L == 8, "the lanes that hold a block");
    m = umax(m, dpp<0xB1>(m));                      // lanes 1 0 3 2
    m = umax(m, dpp<0x4E>(m));                      // lanes 2 3 0 1
    if (L == 8) m = umax(m, dpp<0x141>(m));         // half row mirrored
    return m;
}

// ---- quantize, rows ---------------------------------------------------------
// Lane l of a work group takes the 16-byte slots l, l + 256, ... of its 16 KiB
// of input; the 8 (fp32) or 4 (16-bit) lanes that hold a block combine their
// maxima by lane permutes and write 2 or 4 bytes of codes each.  A row's
// slots are counted up to whole blocks; those past its end read as zeros.
// Rows may start at any element: a slot is one load of 16 bytes either way, and
// the last, short one of a row is the 16 bytes that end with the row, shifted.
// 8 ranks of 60.2M fp32: 352 us, 6.2 TB/s (fp16, 8 of 335M: 1.17 ms, 5.8 TB/s); rows
// of 4100 bf16, 8191 of them: 16 us, 5.2 TB/s (an element per lane: 52 us).

// The bytes of v from byte n on (0 < n < 16), zeros behind them.
__device__ __forceinline__ u32x4 drop_bytes(const u32x4 &v, int n) {
    const uint64_t lo = (static_cast<uint64_t>(v[1]) << 32) | v[0];
    const uint64_t hi = (static_cast<uint64_t>(v[3]) << 32) | v[2];
    const int s = 8 * (n & 7);
    const uint64_t l = s ? lo >> s | hi << (64 - s) : lo, h = hi >> s;
    const uint64_t x = n >= 8 ? h : l, y = n >= 8 ? 0 : h;
    return u32x4{static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32),
                 static_cast<uint32_t>(y), static_cast<uint32_t>(y >> 32)};
}

typedef u32x4 __attribute__((aligned(2))) u32x4_any;     // at any element

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
        int over[MXQ_SLOTS];            // elements past the row's end
        auto place = [&](int s, int64_t &col) {
            const int64_t j = c0 + s * MXQ_BLOCK + threadIdx.x;
            int64_t row = 0;
            col = j * V;
            if (ROWS) {   // total < 2^32 here
                const uint32_t r32 = static_cast<uint32_t>(j) / static_cast<uint32_t>(spr);
                row = r32;
                col = static_cast<int64_t>(static_cast<uint32_t>(j) -
                                           r32 * static_cast<uint32_t>(spr)) * V;
            }
            raw[s] = u32x4{0, 0, 0, 0};
            over[s] = 0;
            return j < total && col < a.cols ? x + row * a.ld + col : nullptr;
        };
        if (a.cols >= V) {
#pragma unroll
            for (int s = 0; s < MXQ_SLOTS; ++s) {
                int64_t col;
                const T *p = place(s, col);
                if (p) {
                    if (col + V > a.cols) over[s] = static_cast<int>(col + V - a.cols);
                    raw[s] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4_any *>(p - over[s]));
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < MXQ_SLOTS; ++s) {
                int64_t col;
                const T *p = place(s, col);
#pragma unroll
                for (int k = 0; k < V - 1; ++k) {
                    if (!p || k >= a.cols) continue;
                    if constexpr (V == 4)
                        raw[s][k] = load_bits(p + k);
                    else
                        raw[s][k >> 1] |= load_bits(p + k) << (16 * (k & 1));
                }
            }
        }
#pragma unroll
        for (int s = 0; s < MXQ_SLOTS; ++s) {
            const int64_t j = c0 + s * MXQ_BLOCK + threadIdx.x;
            if (over[s] > 0) raw[s] = drop_bytes(raw[s], over[s] * static_cast<int>(sizeof(T)));
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

// ---- quantize, columns ------------------------------------------------------
// A wave takes a block of 64 * F columns: a lane loads one word (F elements)
// of each of its 32 rows, and holds F whole blocks in registers, so no lane
// needs another's maximum.  A work group's eight waves take eight blocks of the
// same columns or, where there are no more than 4, 2 or 1 blocks (BW), as many of
// 2, 4 or 8 times the columns (7 x 10^6 fp32: 11 us; with seven of eight waves
// idle 41).  Their codes and scales leave through LDS, a column's (up to 128
// bytes of codes) together.  8192 x 4096: fp32 24 us, 6.3 TB/s, bf16 16 us, 5.2 TB/s;
// with 16-byte loads, four times the registers and every lane writing its
// columns' codes itself 45 and 26 us.
typedef uint32_t __attribute__((aligned(2))) u32_any;
typedef uint64_t __attribute__((aligned(1))) u64_any;

template <typename T, bool MUL>
__global__ __launch_bounds__(64 * MXT_BLOCKS) void k_mx4_quantize_cols(const MxQArgs a,
                                                                       int64_t col_groups,
                                                                       int64_t n_groups, int lbw) {
    constexpr int F = 4 / sizeof(T);
    // piece (column * BW + block) at piece ^ (piece / 8 / F % 8)
    __shared__ u32x4 codes[64 * F * MXT_BLOCKS];
    __shared__ uint64_t scales[64 * F * MXT_BLOCKS / 8];
    const int bw = 1 << lbw;
    auto slot = [](int piece) { return piece ^ (piece >> (F == 2 ? 4 : 3) & 7); };
    const int w = blockIdx.y;
    const T *x = static_cast<const T *>(a.x[w]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    for (int64_t i = blockIdx.x; i < n_groups; i += gridDim.x) {
        const int64_t b0 = i / col_groups * bw;
        const int64_t c0 = i % col_groups * (64 * F * MXT_BLOCKS >> lbw);
        const int cw = (wave >> lbw) * 64 * F + lane * F, bk = wave & (bw - 1);
        const int64_t r0 = (b0 + bk) * MX_BLOCK, col = c0 + cw;
        // columns past the last one take its word, and are not stored
        const int64_t cc = col + F <= a.cols ? col : a.cols - F;
        const int valid = a.rows - r0 < MX_BLOCK ? static_cast<int>(a.rows - r0) : MX_BLOCK;
        uint32_t raw[MX_BLOCK];
        if (valid == MX_BLOCK && cc >= 0) {
            const T *p = x + r0 * a.ld + cc;
#pragma unroll
            for (int k = 0; k < MX_BLOCK; ++k)
                raw[k] = *reinterpret_cast<const u32_any *>(p + k * a.ld);
        } else {
#pragma unroll
            for (int k = 0; k < MX_BLOCK; ++k) {
                raw[k] = 0;
                if (k >= valid) continue;
                const T *p = x + (r0 + k) * a.ld;
                if (cc >= 0) raw[k] = *reinterpret_cast<const u32_any *>(p + cc);
                else raw[k] = static_cast<uint32_t>(load_bits(p)) << 16;    // one column
            }
        }
        if (F == 2 && cc < col) {       // the last of an odd number
#pragma unroll
            for (int k = 0; k < MX_BLOCK; ++k) raw[k] >>= 16;
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            auto get = [&](int k) {
                const float g = slot_f32<T>(u32x4{raw[k], 0, 0, 0}, f);
                return MUL ? __fmul_rn(g, a.in_mul) : g;
            };
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < MX_BLOCK; ++k) m = umax(m, __float_as_uint(get(k)) & kAbs);
            const uint32_t s = mx_byte(m);
            const float mul = mx_mult(s);
            u32x4 code;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t c = mx_code2<0>(0u, get(8 * k) * mul, get(8 * k + 1) * mul);
                c = mx_code2<1>(c, get(8 * k + 2) * mul, get(8 * k + 3) * mul);
                c = mx_code2<2>(c, get(8 * k + 4) * mul, get(8 * k + 5) * mul);
                c = mx_code2<3>(c, get(8 * k + 6) * mul, get(8 * k + 7) * mul);
                code[k] = s == 255u ? 0u : c;
            }
            const int piece = ((cw + f) << lbw) + bk;
            codes[slot(piece)] = code;
            reinterpret_cast<uint8_t *>(scales)[piece] = static_cast<uint8_t>(s);
        }
        __syncthreads();
        const bool whole = b0 + MXT_BLOCKS <= a.nb;     // eight scales of a column together
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int piece = f * 64 * MXT_BLOCKS + threadIdx.x;
            const int64_t c = c0 + (piece >> lbw), k = b0 + (piece & (bw - 1));
            if (c >= a.cols || k >= a.nb) continue;
            reinterpret_cast<u32x4 *>(a.q[w])[c * a.nb + k] = codes[slot(piece)];
            if (!whole)
                a.scale[w][c * a.nb + k] = reinterpret_cast<const uint8_t *>(scales)[piece];
        }
        if (whole && threadIdx.x < 64 * F && c0 + threadIdx.x < a.cols)
            *reinterpret_cast<u64_any *>(a.scale[w] + (c0 + threadIdx.x) * a.nb + b0) =
                scales[threadIdx.x];
        __syncthreads();
    }
}

// ---- reduce -----------------------------------------------------------------
// A lane sums a whole block: 16 bytes of codes and a scale byte per rank, 32
// sums in registers, ranks in order.  A value times its scale is exact, so
// one fused multiply-add per element rounds the sum alone.  The sum's codes
// need the lane's own maximum only.  The sums leave through the wave's 8 KiB
// of LDS, so that the wave's stores of 16 bytes per lane are contiguous.
// FLAT: rows == 1 or whole blocks, so the sums are one 16-byte aligned array.
// Bound by HBM: 8 ranks of 60.2M with sum and codes 78 us, 6.8 TB/s; one rank's
// sum alone (decoding) 47 us, 5.7 TB/s; decoding 8191 rows of 4100 29 us, 5.2 TB/s
// (with 4-byte stores, a division each, 52 us).
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
            row = total <= 0xffffffffu
                      ? static_cast<uint32_t>(j) / static_cast<uint32_t>(a.nb)
                      : j / a.nb;
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
                // a block's place and length, from the lane that summed it;
                // rows start at any element
                const int64_t first = row * a.cols + b * MX_BLOCK;
                const int64_t left = in ? a.cols - b * MX_BLOCK : 0;
                const int len = static_cast<int>(left < MX_BLOCK ? left : MX_BLOCK);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int blk = i * 8 + (lane >> 3), p = lane & 7;
                    const f32x4 v = my[8 * blk + (p ^ (blk & 7))];
                    const int64_t e = __shfl(first, blk, 64) + 4 * p;
                    const int n = __shfl(len, blk, 64) - 4 * p;
                    if (n >= 4) {
                        __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any *>(a.r + e));
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            if (k < n) a.r[e + k] = v[k];
                    }
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
    constexpr int64_t L = MX_BLOCK * sizeof(T) / 16;     // slots per block
    const unsigned W = static_cast<unsigned>(a.W);
    if (transpose) {
        a.nb = (a.rows + MX_BLOCK - 1) / MX_BLOCK;
        const int lbw = a.nb > 4 ? 3 : a.nb > 2 ? 2 : a.nb > 1 ? 1 : 0;
        const int64_t C = 64 * 4 / sizeof(T) * MXT_BLOCKS >> lbw, bw = 1 << lbw;
        const int64_t cg = (a.cols + C - 1) / C, n = cg * ((a.nb + bw - 1) / bw);
        hipLaunchKernelGGL((k_mx4_quantize_cols<T, MUL>), dim3(static_cast<unsigned>(groups(n, 1)), W),
                           dim3(64 * MXT_BLOCKS), 0, st, a, cg, n, lbw);
        return hipGetLastError();
    }
    a.nb = (a.cols + MX_BLOCK - 1) / MX_BLOCK;
    if (a.ld == a.cols && a.cols % MX_BLOCK == 0) {   // whole blocks: one long row
        a.cols *= a.rows;
        a.nb *= a.rows;
        a.rows = 1;
    }
    // the rows of a launch hold less than 2^32 slots, or it is of one row
    int64_t left = a.rows, most = ((int64_t{1} << 32) - MXQ_BLOCK * MXQ_SLOTS - 1) / (a.nb * L);
    if (most < 1) most = 1;
    while (left > 0) {
        a.rows = left < most ? left : most;
        const dim3 grid(static_cast<unsigned>(groups(a.rows * a.nb * L, MXQ_BLOCK * MXQ_SLOTS)), W);
        if (a.rows == 1)
            hipLaunchKernelGGL((k_mx4_quantize<T, MUL, false>), grid, dim3(MXQ_BLOCK), 0, st, a);
        else
            hipLaunchKernelGGL((k_mx4_quantize<T, MUL, true>), grid, dim3(MXQ_BLOCK), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        left -= a.rows;
        for (unsigned w = 0; w < W && left > 0; ++w) {
            a.x[w] = static_cast<const T *>(a.x[w]) + a.rows * a.ld;
            a.q[w] += a.rows * a.nb * MX_BYTES;
            a.scale[w] += a.rows * a.nb;
        }
    }
    return hipSuccess;
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
