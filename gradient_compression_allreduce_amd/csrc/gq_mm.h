// gq_mm.h -- the matrix-core tile loop of the products C = P Q^T on gfx950,
// shared by the MX4 product and the fp16 products of the orthogonalisation.
// Not part of the ABI.
//
// Both operands are rows of contiguous K.  A K step is 128 bytes of every
// row (64 fp16 elements, 256 4-bit codes); a lane's operand of one 16 x 16
// matrix instruction is 16 bytes of a row in either type, so the loop, its
// LDS layout and its loads do not depend on the type.
//   * Loads go from global memory to LDS with no register in between
//     (16 bytes per lane), one step ahead of the arithmetic, into the other of
//     two buffers; rows and chunks outside the matrix read as zeros by the
//     buffer descriptor's bound.
//   * In LDS a row's eight 16-byte chunks are stored at (chunk ^ (row & 7)),
//     so the 16 rows that a matrix instruction reads at one chunk index fall
//     into different banks.  A wave's load writes consecutive LDS addresses, so
//     the exchange is made on the global side, in which chunk a lane asks for.
//   * The instruction's first operand is Q and its second P: a lane then
//     holds four consecutive columns of one row of C.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {
namespace {

typedef float mm_f32x4 __attribute__((ext_vector_type(4)));
typedef int mm_i32x4 __attribute__((ext_vector_type(4)));
typedef int mm_i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 mm_f16x8 __attribute__((ext_vector_type(8)));

constexpr int MM_STEP = 128;     // bytes of K per step and row

// A matrix operand's rows [row0, ...) as a buffer: `bytes` per row, `rows`
// valid rows from row0 on (at most 256 of them are read).
struct MmRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t bytes;
};

__device__ __forceinline__ MmRows mm_rows(const void *base, uint32_t bytes, int64_t row0,
                                          int64_t rows, int tile) {
    const int64_t left = rows - row0;
    const uint32_t valid = static_cast<uint32_t>(left < tile ? left : tile);
    const char *p = static_cast<const char *>(base) + row0 * bytes;
    return {__builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0,
                                              static_cast<int>(valid * bytes), 0x00027000),
            bytes};
}

// Starts the loads of R rows' K step kt into `lds` (R * 128 bytes).
template <int R, int THREADS>
__device__ __forceinline__ void mm_load(const MmRows &m, char *lds, int kt) {
    const int tid = threadIdx.x;
    const uint32_t row = tid >> 3;
    const uint32_t at = static_cast<uint32_t>(kt) * MM_STEP + (((tid & 7) ^ (row & 7)) << 4);
    // a chunk past the row's end must not read the next row
    const uint32_t off = at < m.bytes ? row * m.bytes + at : 0xfffffff0u;
    char *dst = lds + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
#pragma unroll
    for (int i = 0; i < R * 8 / THREADS; ++i) {
        const uint32_t o = off + (at < m.bytes ? i * (THREADS / 8) * m.bytes : 0u);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            m.rsrc, (__attribute__((address_space(3))) void *)(dst + i * THREADS * 16), 16,
            static_cast<int>(o), 0, 0, 0);
    }
}

// The 16 bytes of row r16 (a multiple of 16) + lane % 16 that the lane
// contributes to the matrix instruction of half kk of the step.
__device__ __forceinline__ mm_i32x4 mm_frag(const char *lds, int r16, int kk) {
    const int lane = threadIdx.x & 63;
    const int chunk = (kk * 4 + (lane >> 4)) ^ (lane & 7);
    return *reinterpret_cast<const mm_i32x4 *>(lds + (r16 + (lane & 15)) * MM_STEP + chunk * 16);
}

// Scale bytes of the MX4 rows of a tile: thread t looks after row t of the
// P rows followed by the Q rows, eight bytes per K step.
struct MmScale {
    const uint8_t *p;    // the row's scales; NULL for a row outside
    int64_t nb;
};

__device__ __forceinline__ uint64_t mm_scale8(const MmScale &s, int kt) {
    const int64_t b = static_cast<int64_t>(kt) * 8;
    uint64_t v = 0;
    if (s.p && b + 8 <= s.nb) {
        __builtin_memcpy(&v, s.p + b, 8);
    } else if (s.p) {
        for (int i = 0; i < 8; ++i)
            if (b + i < s.nb) v |= static_cast<uint64_t>(s.p[b + i]) << (8 * i);
    }
    return v;
}

// Tile shapes: BM x BN of C by WM x WN waves, FM x FN matrix instructions
// per wave and half step.
template <int BM_, int BN_, int WM_, int WN_>
struct MmShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int THREADS = 64 * WM * WN;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int STAGE = (BM + BN) * MM_STEP;            // bytes of one buffer
    static constexpr int STAGE_MX = STAGE + (BM + BN) * 8;       // with scales behind
};

// acc += the K steps [kt0, kt0 + 2 * pairs) of the tile's product.  s0 and
// s1 are two LDS arrays of a stage each (two arrays, so that the compiler
// sees that the loads under way do not touch what is being read).  Steps
// past the rows' ends add zeros.  Every load has landed on return, and all
// waves have passed their last read.
template <typename S, bool MX>
__device__ __forceinline__ void mm_loop(const MmRows &p, const MmRows &q, const MmScale &sc,
                                        int kt0, int pairs, char *s0, char *s1,
                                        mm_f32x4 (&acc)[S::FM][S::FN]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    auto load = [&](char *s, int kt) {
        mm_load<S::BM, S::THREADS>(p, s, kt);
        mm_load<S::BN, S::THREADS>(q, s + S::BM * MM_STEP, kt);
    };
    auto put_scale = [&](char *s, uint64_t v) {
        if (S::BM + S::BN == S::THREADS || static_cast<int>(threadIdx.x) < S::BM + S::BN)
            *reinterpret_cast<uint64_t *>(s + S::STAGE + threadIdx.x * 8) = v;
    };
    auto landed = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    auto compute = [&](const char *s) {
        uint2 sp[S::FM], sq[S::FN];
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < S::FM; ++i)
                sp[i] = *reinterpret_cast<const uint2 *>(s + S::STAGE +
                                                         (rm + 16 * i + (lane & 15)) * 8);
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                sq[j] = *reinterpret_cast<const uint2 *>(
                    s + S::STAGE + (S::BM + rn + 16 * j + (lane & 15)) * 8);
        }
        const int sh = (lane >> 4) * 8;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            mm_i32x4 fp[S::FM], fq[S::FN];
#pragma unroll
            for (int i = 0; i < S::FM; ++i) fp[i] = mm_frag(s, rm + 16 * i, kk);
#pragma unroll
            for (int j = 0; j < S::FN; ++j) fq[j] = mm_frag(s + S::BM * MM_STEP, rn + 16 * j, kk);
#pragma unroll
            for (int i = 0; i < S::FM; ++i) {
#pragma unroll
                for (int j = 0; j < S::FN; ++j) {
                    if constexpr (MX) {
                        const mm_i32x8 a = {fq[j].x, fq[j].y, fq[j].z, fq[j].w, 0, 0, 0, 0};
                        const mm_i32x8 b = {fp[i].x, fp[i].y, fp[i].z, fp[i].w, 0, 0, 0, 0};
                        const int sa = static_cast<int>((kk ? sq[j].y : sq[j].x) >> sh);
                        const int sb = static_cast<int>((kk ? sp[i].y : sp[i].x) >> sh);
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            a, b, acc[i][j], 4, 4, 0, sa, 0, sb);
                    } else {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(mm_f16x8, fq[j]), __builtin_bit_cast(mm_f16x8, fp[i]),
                            acc[i][j], 0, 0, 0);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    uint64_t v = 0;
    load(s0, kt0);
    if constexpr (MX) put_scale(s0, mm_scale8(sc, kt0));
    for (int k = 0; k < pairs; ++k) {
        const int kt = kt0 + 2 * k;
        landed();
        load(s1, kt + 1);
        if constexpr (MX) v = mm_scale8(sc, kt + 1);
        __builtin_amdgcn_sched_barrier(0);
        compute(s0);
        if constexpr (MX) put_scale(s1, v);
        landed();
        load(s0, kt + 2);
        if constexpr (MX) v = mm_scale8(sc, kt + 2);
        __builtin_amdgcn_sched_barrier(0);
        compute(s1);
        if constexpr (MX) put_scale(s0, v);
    }
    landed();
}

// Work group -> tile.  Consecutive work groups go to the eight XCDs in turn;
// each XCD gets a consecutive run of tiles, and within a run the tiles go
// down eight rows before the next column, so that those an XCD works on at
// one time share rows of P and Q in its L2 cache.
__device__ __forceinline__ int mm_xcd(int bid, int n) {
    const int per = n >> 3, rem = n & 7, x = bid & 7;
    return x * per + (x < rem ? x : rem) + (bid >> 3);
}

__device__ __forceinline__ void mm_tile(int t, int tm, int tn, int &ti, int &tj) {
    constexpr int G = 8;
    const int g = t / (G * tn), first = g * G;
    const int rows = tm - first < G ? tm - first : G;
    const int r = t - g * G * tn;
    ti = first + r % rows;
    tj = r / rows;
}

}  // namespace
}  // namespace gq
