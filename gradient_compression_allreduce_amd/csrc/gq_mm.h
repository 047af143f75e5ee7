// gq_mm.h -- the matrix-core tile loop of the products C = P Q^T on gfx950,
// shared by the MX4 product and the fp16 products of the orthogonalisation.
// Not part of the ABI.
//
// P is stored by rows of contiguous K; so is Q, or (fp16) Q^T is: K rows of
// contiguous columns of C.  A K step is 128 bytes of every row (64 fp16
// elements, 256 4-bit codes), a whole line of the L2 cache: with half lines
// the requests to the L2 cache bound the loop (fp16 at 8192^3: 1.02 PFLOP/s
// with steps of 64 bytes, 1.21 with 128).  A lane's operand of one 16 x 16
// matrix instruction is 16 bytes of a row in either type, so the loops,
// their LDS layout and their loads do not depend on the type.
//   * Loads go from global memory to LDS with no register in between
//     (16 bytes per lane).  Rows, columns and chunks outside the matrix read as
//     zeros by the buffer descriptor's bound; the number of steps is rounded
//     up to an even one (on a ring of four buffers to a multiple of four).
//   * In LDS the eight 16-byte chunks of row r are stored at chunk ^ (r & 7).
//     A 16-byte LDS read serves the lanes 0-3, 12-15 and 20-27 together (and
//     so on): with this order those sixteen fall into different banks.  A
//     wave's load writes consecutive LDS addresses, so the exchange is made
//     on the global side, in which chunk a lane asks for.
//   * The instruction's first operand is Q and its second P: a lane then
//     holds four consecutive columns of one row of C.
//   * mm_two (tiles of 128 and 64): two buffers of a step each; two work groups
//     per compute unit with tiles of 128, five with tiles of 64 (three in MX4,
//     whose scales take 16 KiB more) cover each other's waits.  On a ring of
//     four buffers instead (tiles of 64 where there are few of them and latency
//     counts) the loads run three steps ahead.
//   * mm_quad (tiles of 256, one work group of eight waves per compute unit):
//     each of P and Q is two halves of 128 rows with buffers of their own, and
//     the waves go through the four quadrants of C together, so a half's
//     buffer is free again after the first quadrant that reads it and its
//     next load starts then, one and a half steps ahead.  (The loop alone,
//     fp16 at 8192^3: 1.24-1.28 PFLOP/s, 1.21 with the two whole buffers, and
//     1.17-1.28 for the library's product.  The two waves of a SIMD taking
//     turns, one reading while the other multiplies, with a barrier more for
//     each quadrant: 5 percent slower in 4 bits and 3 - 7 in fp16.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace gq {
namespace {

typedef float mm_f32x4 __attribute__((ext_vector_type(4)));
typedef int mm_i32x4 __attribute__((ext_vector_type(4)));
typedef int mm_i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int mm_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mm_u32x2 __attribute__((ext_vector_type(2)));
typedef short mm_i16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 mm_f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void mm_lds_void;
typedef __attribute__((address_space(3))) mm_i16x4 mm_lds_i16x4;

constexpr int MM_STEP = 128;     // bytes of K per step and row

// The thread's number, as if it were read anew: addresses that follow from it
// are then worked out where they are used.  (The compiler would keep all of
// them in registers through the loop, which has none to spare, and reload
// some from memory in every step.)
__device__ __forceinline__ int mm_tid() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// Tile shapes: T x T of C by WM x WN waves.  A wave's part of C is PARTS
// blocks of FM x FN matrix instructions; block b, instruction row i and the
// lane's row r (0 .. 15) are at part_row / part_col of the tile.
// RING: four buffers instead of two.
template <int T_, int WM_, int WN_, bool RING_ = false>
struct MmShape {
    static constexpr int T = T_, WM = WM_, WN = WN_;
    static constexpr bool QUAD = T == 256, RING = RING_;
    static constexpr int BUFFERS = QUAD ? 8 : RING ? 4 : 2;
    static constexpr int THREADS = 64 * WM * WN;
    static constexpr int PARTS = QUAD ? 2 : 1;
    static constexpr int FM = T / WM / 16, FN = T / WN / 16 / PARTS;
    static constexpr int UNIT = QUAD ? 128 * MM_STEP : 2 * T * MM_STEP;  // bytes of one buffer
    static constexpr int PLANES = QUAD ? 4 : 2;                  // of MX4 scales
    // scale bytes of two steps: a plane for every one or two waves (with tiles
    // of 64 the planes of two waves are written and not read)
    static constexpr int SCALES = WM * WN / (T >= 128 ? 2 : 1) * 2048;
    static constexpr int SCALE_LDS = QUAD ? 4 * SCALES : 2 * SCALES;    // what is held at one time
    // first row of instruction row i, and first column of block b
    static __device__ __forceinline__ int part_row(int wave, int i) {
        if (QUAD) return (i >> 2) * 128 + wave / WN * 64 + (i & 3) * 16;
        return wave / WN * (T / WM) + 16 * i;
    }
    static __device__ __forceinline__ int part_col(int wave, int b) {
        if (QUAD) return b * 128 + wave % WN * 32;
        return wave % WN * (T / WN);
    }
};
using MmBig = MmShape<256, 2, 4>;
using MmMid = MmShape<128, 2, 2>;
using MmSmall = MmShape<64, 2, 2>;
using MmFew = MmShape<64, 2, 2, true>;

// Rows [row0, row0 + tile) of an operand, `bytes` per row, as a buffer.
struct MmRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t bytes;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_buffer(const char *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, static_cast<int>(bytes),
                                             0x00027000);
}

__device__ __forceinline__ MmRows mm_rows(const void *base, uint32_t bytes, int64_t row0,
                                          int64_t rows, int tile) {
    const int64_t left = rows - row0;
    const uint32_t valid = static_cast<uint32_t>(left < tile ? left : tile);
    return {mm_buffer(static_cast<const char *>(base) + row0 * bytes, valid * bytes), bytes};
}

__device__ __forceinline__ void mm_dma(const __amdgpu_buffer_rsrc_t &r, char *lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void *)lds, 16, static_cast<int>(off), 0, 0,
                                             0);
}

// Starts the loads of the R rows from row0 of the tile on of a step into
// `lds` (R * 128 bytes).
template <int R, int THREADS>
__device__ __forceinline__ void mm_load(const MmRows &m, char *lds, int step, int row0) {
    const int tid = mm_tid();
    const uint32_t row = tid >> 3;
    const uint32_t at = static_cast<uint32_t>(step) * MM_STEP + (((tid & 7) ^ (row & 7)) << 4);
    // a chunk past the row's end must not read the next row
    const bool in = at < m.bytes;
    const uint32_t off = in ? (row + row0) * m.bytes + at : 0xfffffff0u;
    char *dst = lds + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
#pragma unroll
    for (int i = 0; i < R * 8 / THREADS; ++i)
        mm_dma(m.rsrc, dst + i * THREADS * 16, off + (in ? i * (THREADS / 8) * m.bytes : 0u));
}

// The 16 bytes of row r16 (a multiple of 16) + lane % 16 that the lane
// contributes to a matrix instruction of half kk of the step.
__device__ __forceinline__ mm_i32x4 mm_frag(const char *lds, int r16, int kk, int lane) {
    const int chunk = (kk * 4 + (lane >> 4)) ^ (lane & 7);
    return *reinterpret_cast<const mm_i32x4 *>(lds + (r16 + (lane & 15)) * MM_STEP + chunk * 16);
}

// Q by rows of columns (fp16): `pitch` bytes between the K rows, `base` at the
// tile's first column, `skip` bytes before it in the row.
struct MmCols {
    const char *base;
    uint32_t pitch, skip;
    int rows;
};

// Where K row r of a step keeps its 32-byte pieces (16 columns): piece ^ this.
// A transposing read takes 16 columns of four rows for each 16 lanes; the
// rows that are read together fall into different banks.
template <int BN>
__device__ __forceinline__ uint32_t mm_turn(uint32_t r) {
    const uint32_t g = ((r >> 3) ^ (r >> 4)) & 1u;
    return BN >= 128 ? (r & 3u) | (g << 2) : ((r >> 1) & 1u) | (g << 1);
}

// Starts the loads of a step: 64 K rows of the BN columns from col0 of the
// tile on (BN * 128 bytes).
template <int BN, int THREADS>
__device__ __forceinline__ void mm_load(const MmCols &m, char *lds, int step, int col0) {
    const int left = m.rows - step * 64;
    const uint32_t valid = left < 0 ? 0u : left < 64 ? left : 64u;
    const __amdgpu_buffer_rsrc_t r =
        mm_buffer(m.base + static_cast<int64_t>(step) * 64 * m.pitch + col0 * 2,
                  valid ? valid * m.pitch - m.skip - col0 * 2 : 0u);
    constexpr int CH = BN / 8;           // 16-byte chunks per row
    const int tid = mm_tid();
    char *dst = lds + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
#pragma unroll
    for (int i = 0; i < BN * 8 / THREADS; ++i) {
        const uint32_t row = (i * THREADS + tid) / CH;
        const uint32_t chunk = (tid % CH) ^ (mm_turn<BN>(row) << 1);
        mm_dma(r, dst + i * THREADS * 16, row * m.pitch + chunk * 16);
    }
}

// Where element (row, col) of a step's K rows lies.
template <int BN>
__device__ __forceinline__ int mm_cols_at(uint32_t row, uint32_t col) {
    return row * (BN * 2) + (((col >> 4) ^ mm_turn<BN>(row)) << 5) + (col & 15) * 2;
}

// f[kk][j]: the lane's 8 elements of K (32 * kk + 8 * (lane / 16) on) of column
// c16 + 16 j + lane % 16, c16 a multiple of 32.  The reads and the wait for
// them are one asm block: the compiler takes the builtin for a read that may
// touch any load to LDS under way, and would wait for all of them before each.
// mm_turn does not change from a row to the 4th and the 32nd after it, so
// those are at fixed distances, and column 16 is one bit away.
template <int BN, int FN>
__device__ __forceinline__ void mm_frag_cols(const char *lds, int c16, int lane,
                                             mm_i32x4 (&f)[2][FN]) {
    const int q = lane & 15;
    constexpr int R4 = 4 * BN * 2, R32 = 32 * BN * 2;
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
        const char *p =
            lds + mm_cols_at<BN>((lane >> 4) * 8 + (q >> 2), c16 + 16 * j + (q & 3) * 4);
        const uint32_t a0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_void *)p));
        const uint32_t a1 = a0 ^ 32u;
        mm_u32x2 h[8];
        asm volatile("ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:%10\n\t"
                     "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:%10\n\t"
                     "ds_read_b64_tr_b16 %4, %8 offset:%11\n\tds_read_b64_tr_b16 %5, %8 offset:%12\n\t"
                     "ds_read_b64_tr_b16 %6, %9 offset:%11\n\tds_read_b64_tr_b16 %7, %9 offset:%12\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(h[0]), "=&v"(h[1]), "=&v"(h[2]), "=&v"(h[3]), "=&v"(h[4]),
                       "=&v"(h[5]), "=&v"(h[6]), "=&v"(h[7])
                     : "v"(a0), "v"(a1), "n"(R4), "n"(R32), "n"(R32 + R4)
                     : "memory");
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                f[kk][j + i] = __builtin_bit_cast(
                    mm_i32x4, __builtin_shufflevector(h[4 * kk + 2 * i], h[4 * kk + 2 * i + 1], 0, 1,
                                                      2, 3));
    }
}

// Scale bytes of a tile's MX4 rows, by groups of two steps (sixteen blocks).
// In LDS they lie in planes of up to 128 rows (P's, then Q's): the byte of
// block b and row 16 i + r at ((b / 4 * 16 + r) * 4 + b % 4) * 8 + i.  The
// scales of all a lane's operands of a half step are neighbours then, which
// the matrix instructions pick by number, and the lanes of a wave read 512
// bytes in a row.  A thread looks after four rows 16 apart and four blocks: it
// loads four bytes of each row and turns them, so that it writes four words.
// Rows and blocks outside take the nearest inside: their codes read as zeros.
constexpr int MM_PLANE = 2048;

struct MmScale {           // (the same for all lanes of a wave)
    const uint8_t *base;   // scales of the wave's operand, first row of the tile
    const uint8_t *ahead;  // the same; with nb < 16 any 16 bytes that can be read
    int32_t pitch;         // nb; with nb < 16: 0
    int32_t rows;          // rows inside
    int32_t nb;
    int32_t row;           // the wave's first row
    int32_t at;            // where it writes
    // a lane's rows are row + r + 16 i, its blocks of a group block .. block + 3
    static __device__ __forceinline__ int r(int tid) { return tid & 15; }
    static __device__ __forceinline__ int block(int tid) { return (tid >> 4 & 3) * 4; }
};

// For operands of m and n rows (scales sp, sq), tile (i0, j0); any: 16 bytes
// that can be read.
template <typename S>
__device__ __forceinline__ MmScale mm_scale_of(const uint8_t *sp, const uint8_t *sq, int64_t i0,
                                               int64_t j0, int64_t m, int64_t n, int64_t nb,
                                               const uint8_t *any) {
    constexpr int QUADS = S::T >= 128 ? 2 : 1;            // waves per plane
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int plane = wave / QUADS, quad = wave % QUADS;
    constexpr int HALF = S::PLANES / 2;
    const bool isp = plane < HALF;
    const int64_t first = isp ? i0 : j0, all = isp ? m : n;
    MmScale s;
    s.base = (isp ? sp : sq) + first * nb;
    s.ahead = nb < 16 ? any : s.base;
    s.pitch = nb < 16 ? 0 : static_cast<int32_t>(nb);
    s.rows = static_cast<int32_t>(all - first < S::T ? all - first : S::T);
    s.nb = static_cast<int32_t>(nb);
    s.row = plane % HALF * 128 + quad * 64;
    s.at = plane * MM_PLANE * (S::QUAD ? 4 : 1) + quad * 4;
    return s;
}

// The first group, any number of blocks: byte k of word i is row i, block k.
__device__ __forceinline__ mm_u32x4 mm_scale_any(const MmScale &s, int group) {
    const int tid = threadIdx.x;
    mm_u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int row = s.row + s.r(tid) + 16 * i;
        row = row < s.rows ? row : s.rows - 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = group * 16 + s.block(tid) + k;
            const int64_t at = static_cast<int64_t>(row) * s.nb + (b < s.nb ? b : s.nb - 1);
            v[i] |= static_cast<uint32_t>(s.base[at]) << (8 * k);
        }
    }
    return v;
}

// A later group (so nb > 16), whose loads stay in flight: words that end no
// later than the row, to be shifted down to the group's blocks when used (0
// but in the row's last group).  A group past the row's end, which the last
// group loads ahead, reads what nobody uses.
__device__ __forceinline__ mm_u32x4 mm_scale_load(const MmScale &s, int group) {
    const int tid = mm_tid();
    int b = group * 16 + s.block(tid);
    b = b < s.pitch - 4 ? b : s.pitch - 4;
    b = b < 0 ? 0 : b;
    mm_u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int row = s.row + s.r(tid) + 16 * i;
        row = row < s.rows ? row : s.rows - 1;
        uint32_t w;
        __builtin_memcpy(&w, s.ahead + static_cast<uint32_t>(row * s.pitch + b), 4);
        v[i] = w;
    }
    return v;
}

__device__ __forceinline__ mm_u32x4 mm_scale_shift(mm_u32x4 v, const MmScale &s, int group) {
    const int late = group * 16 + s.block(mm_tid()) - (s.nb - 4);
    const uint32_t by = late <= 0 ? 0u : late > 3 ? 24u : 8u * late;
    return v >> by;
}

// Tiles of 256: the scales of four groups (2048 elements of K) at once.  16
// bytes a row and group are an eighth of a line of the L2 cache each time, as
// many requests as half the codes are.  At 8192 x 8192, us with K = 1024 / 8192 /
// 32768: group by group 98 / 323 / 1130, four at once 84 / 297 / 1032 (another
// device: 85 / 302 / 1093).  A lane's
// 16 bytes of four rows are one group's, so a wave's loads are of 64 bytes a
// row.  (They are not held twice: the waves meet once more before new ones are
// written.)
struct MmScale4 {
    mm_u32x4 v[4];      // byte k of row i: block k of the group
};

typedef mm_u32x4 __attribute__((aligned(1))) mm_u32x4_any;

__device__ __forceinline__ int mm_scale4_block(int group) {
    return (group + (mm_tid() >> 4 & 3)) * 16;
}

// Four groups of a row of 16 blocks or more: bytes that end no later than the
// row, to be shifted down to the group's blocks when used.  Behind the last
// group: bytes that nobody uses.
__device__ __forceinline__ MmScale4 mm_scale4_load(const MmScale &s, int group) {
    const int tid = mm_tid();
    int b = mm_scale4_block(group);
    b = b < s.pitch - 16 ? b : s.pitch - 16;
    b = b < 0 ? 0 : b;
    MmScale4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int row = s.row + s.r(tid) + 16 * i;
        row = row < s.rows ? row : s.rows - 1;
        w.v[i] = *reinterpret_cast<const mm_u32x4_any *>(s.ahead +
                                                         static_cast<uint32_t>(row * s.pitch + b));
    }
    return w;
}

__device__ __forceinline__ void mm_scale4_shift(MmScale4 &w, const MmScale &s, int group) {
    const int late = mm_scale4_block(group) - (s.nb - 16);
    const int by = late <= 0 ? 0 : late < 16 ? late : 16;
    const int bits = 8 * (by & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t lo = (static_cast<uint64_t>(w.v[i][1]) << 32) | w.v[i][0];
        const uint64_t hi = (static_cast<uint64_t>(w.v[i][3]) << 32) | w.v[i][2];
        const uint64_t l = bits ? lo >> bits | hi << (64 - bits) : lo, h = hi >> bits;
        const uint64_t x = by >= 16 ? 0 : by >= 8 ? h : l, y = by >= 8 ? 0 : h;
        w.v[i] = mm_u32x4{static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32),
                          static_cast<uint32_t>(y), static_cast<uint32_t>(y >> 32)};
    }
}

// The bytes of rows 16 i + r for i in [first, first + F) (first a multiple of
// F): F <= 4 in w[0], otherwise in both.  (Always one read of eight bytes:
// of that one the compiler keeps what it may alias.)
template <int F>
struct MmBytes {
    uint32_t w[2];
    __device__ __forceinline__ void read(const char *row, int first) {
        pick(*reinterpret_cast<const mm_u32x2 *>(row), first);
    }
    __device__ __forceinline__ void pick(mm_u32x2 v, int first) {
        w[0] = v.x;
        w[1] = v.y;
        if (F <= 4) w[0] = (first & 4) ? v.y : v.x;
        if (F <= 2) w[0] >>= 8 * (first & 2);
    }
};

// c += the product of two MX4 operands, scale byte I of sq and J of sp.
template <int I, int J>
__device__ __forceinline__ mm_f32x4 mm_mx(mm_i32x4 q, mm_i32x4 p, mm_f32x4 c, uint32_t sq,
                                          uint32_t sp) {
    const mm_i32x8 a = {q.x, q.y, q.z, q.w, 0, 0, 0, 0}, b = {p.x, p.y, p.z, p.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, I, static_cast<int>(sq),
                                                            J, static_cast<int>(sp));
}

// f(0), f(1), ... f(N - 1), each number a constant.
template <int N, typename F>
__device__ __forceinline__ void mm_each(F &f) {
    if constexpr (N > 0) {
        mm_each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void mm_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// What the waves hand each other is in LDS, put there by loads and writes that
// have been waited for.  Buffers are loaded again behind a barrier, so a wave
// waits for its own reads here, wherever the compiler has put the matrix
// instructions that use them.  (In the loops as they are compiled all results
// have been used by then, so the wait costs nothing.)
__device__ __forceinline__ void mm_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A 4 x 4 matrix of bytes turned: pairs of rows, then pairs of pairs.
__device__ __forceinline__ mm_u32x4 mm_turn4(uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
    const uint32_t lo01 = __builtin_amdgcn_perm(v1, v0, 0x05010400u);
    const uint32_t lo23 = __builtin_amdgcn_perm(v3, v2, 0x05010400u);
    const uint32_t hi01 = __builtin_amdgcn_perm(v1, v0, 0x07030602u);
    const uint32_t hi23 = __builtin_amdgcn_perm(v3, v2, 0x07030602u);
    return mm_u32x4{__builtin_amdgcn_perm(lo23, lo01, 0x05040100u),
                    __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                    __builtin_amdgcn_perm(hi23, hi01, 0x05040100u),
                    __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
}

// Writes the thread's scale bytes of four blocks: word k of block k (PITCH bytes
// apart), byte i of row i.  (in asm: of these writes the compiler does not see
// which array they go to, and would wait for every load to LDS first.  They have
// to be waited for: mm_put_wait.)
template <int OFFSET, int PITCH>
__device__ __forceinline__ void mm_put_words(uint32_t at, mm_u32x4 w) {
    asm volatile("ds_write_b32 %0, %1 offset:%5\n\tds_write_b32 %0, %2 offset:%6\n\t"
                 "ds_write_b32 %0, %3 offset:%7\n\tds_write_b32 %0, %4 offset:%8"
                 ::"v"(at), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]), "n"(OFFSET),
                 "n"(OFFSET + PITCH), "n"(OFFSET + 2 * PITCH), "n"(OFFSET + 3 * PITCH)
                 : "memory");
}

__device__ __forceinline__ void mm_put_wait() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The thread's bytes of a group, to half `half` of the scales.
template <typename S>
__device__ __forceinline__ void mm_put_scale(const char *scale, int half, const MmScale &s,
                                             mm_u32x4 v) {
    const int tid = mm_tid();
    const char *d = scale + half * S::SCALES + s.at + ((tid >> 4 & 3) * 64 + (tid & 15) * 4) * 8;
    mm_put_words<0, 8>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_void *)d)),
                       mm_turn4(v[0], v[1], v[2], v[3]));
    mm_put_wait();
}

// The thread's bytes of four groups, each to a quarter of its plane.  Here the
// byte of block b and row 16 i + r is at ((b / 8 * 4 + b % 4) * 16 + r) * 16 +
// b / 4 % 2 * 8 + i: a lane reads both half steps' scales at once.
__device__ __forceinline__ void mm_put_scale4(const char *scale, const MmScale &s,
                                              const MmScale4 &w) {
    const int tid = mm_tid();
    const char *d = scale + s.at + (tid >> 4 & 3) * MM_PLANE + (tid & 15) * 16;
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_void *)d));
    mm_put_words<0, 256>(at, mm_turn4(w.v[0][0], w.v[1][0], w.v[2][0], w.v[3][0]));
    mm_put_words<8, 256>(at, mm_turn4(w.v[0][1], w.v[1][1], w.v[2][1], w.v[3][1]));
    mm_put_words<1024, 256>(at, mm_turn4(w.v[0][2], w.v[1][2], w.v[2][2], w.v[3][2]));
    mm_put_words<1032, 256>(at, mm_turn4(w.v[0][3], w.v[1][3], w.v[2][3], w.v[3][3]));
    mm_put_wait();
}

// The same of rows of one group, of which the thread has four blocks.
__device__ __forceinline__ void mm_put_scale4_few(const char *scale, const MmScale &s, mm_u32x4 v) {
    const int tid = mm_tid(), c = tid >> 4 & 3;
    const char *d = scale + s.at + (c >> 1) * 1024 + (tid & 15) * 16 + (c & 1) * 8;
    mm_put_words<0, 256>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_void *)d)),
                         mm_turn4(v[0], v[1], v[2], v[3]));
    mm_put_wait();
}

// c[i][j] += p[i] q[j] over one half step.
template <bool MX, int FM, int FN>
__device__ __forceinline__ void mm_block(const mm_i32x4 (&p)[FM], const mm_i32x4 (&q)[FN],
                                         const uint32_t (&sp)[2], uint32_t sq,
                                         mm_f32x4 (&c)[FM][FN]) {
    if constexpr (MX) {
        auto row = [&](auto ic) {
            constexpr int i = decltype(ic)::value;
            c[i][0] = mm_mx<0, (i & 3)>(q[0], p[i], c[i][0], sq, sp[i >> 2]);
            c[i][1] = mm_mx<1, (i & 3)>(q[1], p[i], c[i][1], sq, sp[i >> 2]);
            if constexpr (FN == 4) {
                c[i][2] = mm_mx<2, (i & 3)>(q[2], p[i], c[i][2], sq, sp[i >> 2]);
                c[i][3] = mm_mx<3, (i & 3)>(q[3], p[i], c[i][3], sq, sp[i >> 2]);
            }
        };
        mm_each<FM>(row);
    } else {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    __builtin_bit_cast(mm_f16x8, q[j]), __builtin_bit_cast(mm_f16x8, p[i]), c[i][j],
                    0, 0, 0);
    }
}

template <int N>
__device__ __forceinline__ void mm_pin(mm_f32x4 *c, std::integral_constant<int, N>) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(c[i]));
}

// The LDS of a work group.  The buffers are arrays of their own, so that the
// compiler sees that the loads under way do not touch what is being read.
// (Tiles of 256 use all, a ring the first four, the others the first two.)
#define MM_LDS(S)                                                                     \
    __shared__ __align__(128) char mm_u0[S::UNIT];                                    \
    __shared__ __align__(128) char mm_u1[S::UNIT];                                    \
    __shared__ __align__(128) char mm_u2[S::BUFFERS > 2 ? S::UNIT : 16];              \
    __shared__ __align__(128) char mm_u3[S::BUFFERS > 2 ? S::UNIT : 16];              \
    __shared__ __align__(128) char mm_u4[S::QUAD ? S::UNIT : 16];                     \
    __shared__ __align__(128) char mm_u5[S::QUAD ? S::UNIT : 16];                     \
    __shared__ __align__(128) char mm_u6[S::QUAD ? S::UNIT : 16];                     \
    __shared__ __align__(128) char mm_u7[S::QUAD ? S::UNIT : 16];                     \
    const MmLds mm_lds = {mm_u0, mm_u1, mm_u2, mm_u3, mm_u4, mm_u5, mm_u6, mm_u7}

struct MmLds {
    char *u0, *u1, *u2, *u3, *u4, *u5, *u6, *u7;
    // the wave's own 1 / (waves) of the buffers, after the loop (in asm, lest
    // the choice becomes a table of LDS addresses, which cannot be linked)
    template <typename S>
    __device__ __forceinline__ char *own(int wave) const {
        uint32_t at = 0;
        char *const u[8] = {u0, u1, u2, u3, u4, u5, u6, u7};
#pragma unroll
        for (int k = 0; k < S::BUFFERS; ++k) {
            uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_void *)u[k]));
            asm("" : "+s"(a));
            if (k == (S::BUFFERS > 2 ? wave : wave >> 1)) at = a;
        }
        if (S::BUFFERS == 2) at += (wave & 1) * (S::UNIT / 2);
        return (char *)reinterpret_cast<mm_lds_void *>(at);
    }
};

// A wave's sums: block b, instruction row i, instruction column j.
template <typename S>
struct MmAcc {
    mm_f32x4 c[S::PARTS][S::FM][S::FN];
};

// What the caller adds to the sums from a step's Q rows while they lie in LDS
// (nothing).
struct MmNoExtra {
    template <typename A>
    __device__ __forceinline__ void operator()(A &, const char *, int, int) const {}
};

// acc += the steps [2 * group0, 2 * (group0 + groups)) of the tile's product.
// MX: the operands are MX4 and `scale` is an LDS array of S::SCALE_LDS bytes.
// extra(acc, q, step, b) is called where the step's Q rows of block b lie at
// q.  Every load has landed on return, and all waves have passed their last
// read.
template <typename S, bool MX, typename Q, typename X>
__device__ __forceinline__ void mm_two(const MmRows &p, const Q &q, const MmScale &sc, int group0,
                                       int groups, const MmLds &u, char *scale, const X &extra,
                                       MmAcc<S> &acc) {
    constexpr bool ROWS = std::is_same<Q, MmRows>::value;
    constexpr int T = S::T;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int rm = S::part_row(wave, 0), rn = S::part_col(wave, 0);
    auto load = [&](char *s, int step) {
        mm_load<T, S::THREADS>(p, s, step, 0);
        mm_load<T, S::THREADS>(q, s + T * MM_STEP, step, 0);
    };
    auto compute = [&](const char *s, int half, int t, int step) {
        extra(acc, s + T * MM_STEP, step, 0);
        mm_i32x4 fq[2][S::FN];
        if constexpr (!ROWS) mm_frag_cols<T, S::FN>(s + T * MM_STEP, rn, lane, fq);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            mm_i32x4 fp[S::FM];
            MmBytes<S::FM> sp = {};
            MmBytes<S::FN> sq = {};
            if constexpr (MX) {
                const int at = half * S::SCALES + (2 * t + kk) * 512 + (lane & 15) * 32 +
                               (lane >> 4) * 8;
                sp.read(scale + at, rm / 16);
                sq.read(scale + at + MM_PLANE, rn / 16);
            }
            if constexpr (ROWS) {
#pragma unroll
                for (int j = 0; j < S::FN; ++j)
                    fq[kk][j] = mm_frag(s + T * MM_STEP, rn + 16 * j, kk, lane);
            }
#pragma unroll
            for (int i = 0; i < S::FM; ++i) fp[i] = mm_frag(s, rm + 16 * i, kk, lane);
            __builtin_amdgcn_s_setprio(1);
            mm_block<MX>(fp, fq[kk], sp.w, sq.w[0], acc.c[0]);
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (MX) mm_put_scale<S>(scale, 0, sc, mm_scale_any(sc, group0));
    mm_u32x4 v;
    if constexpr (S::RING) {
        // four steps (two groups of scales) a round; an odd last group is
        // followed by steps of zeros, so parts of K must be even
        constexpr int L = 2 * T * 8 / S::THREADS;   // a wave's loads per step
        const int first = 2 * group0;
        load(u.u0, first);
        load(u.u1, first + 1);
        load(u.u2, first + 2);
        auto one = [&](char *now, char *next, int step, int half, int t) {
            mm_wait<2 * L>();
            mm_barrier();
            if (MX && t == 0) v = mm_scale_load(sc, step / 2 + 1);
            load(next, step + 3);
            __builtin_amdgcn_sched_barrier(0);
            compute(now, half, t, step);
            // into the other half, whose last readers passed this group's
            // first barrier; written before the next barrier
            if (MX && t == 1) mm_put_scale<S>(scale, half ^ 1, sc, mm_scale_shift(v, sc, step / 2 + 1));
        };
        for (int g = 0; g < groups; g += 2) {
            const int step = first + 2 * g;
            one(u.u0, u.u3, step, 0, 0);
            one(u.u1, u.u0, step + 1, 0, 1);
            one(u.u2, u.u1, step + 2, 1, 0);
            one(u.u3, u.u2, step + 3, 1, 1);
        }
    } else {
        load(u.u0, 2 * group0);
        for (int g = 0; g < groups; ++g) {
            const int step = 2 * (group0 + g), half = g & 1;
            mm_wait<0>();
            mm_barrier();
            if constexpr (MX) v = mm_scale_load(sc, group0 + g + 1);
            load(u.u1, step + 1);
            __builtin_amdgcn_sched_barrier(0);
            compute(u.u0, half, 0, step);
            mm_wait<0>();
            mm_barrier();
            load(u.u0, step + 2);
            __builtin_amdgcn_sched_barrier(0);
            compute(u.u1, half, 1, step + 1);
            if constexpr (MX)
                mm_put_scale<S>(scale, (g + 1) & 1, sc, mm_scale_shift(v, sc, group0 + g + 1));
        }
    }
    mm_wait<0>();
    __syncthreads();
}

// The same for tiles of 256: u0 - u3 and u4 - u7 hold P0, Q0, Q1, P1 of an
// even and an odd step.
template <typename S, bool MX, typename Q, typename X>
__device__ __forceinline__ void mm_quad(const MmRows &p, const Q &q, const MmScale &sc, int group0,
                                        int groups, const MmLds &u, char *scale, const X &extra,
                                        MmAcc<S> &acc) {
    constexpr bool ROWS = std::is_same<Q, MmRows>::value;
    constexpr int L = 128 * 8 / S::THREADS;     // a wave's loads per half
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = S::part_row(wave, 0), rn = S::part_col(wave, 0);
    auto load_p = [&](char *s, int step, int h) { mm_load<128, S::THREADS>(p, s, step, 128 * h); };
    auto load_q = [&](char *s, int step, int h) { mm_load<128, S::THREADS>(q, s, step, 128 * h); };
    // one half of P (four instruction rows) and both of Q, of both half steps
    mm_i32x4 fp[2][4], fq[2][2][2];
    mm_u32x4 sp = {}, sq[2] = {};      // their scales, as read: both half steps'
    auto read_scale = [&](int plane, int quarter, int t, int lane) {
        return *reinterpret_cast<const mm_u32x4 *>(scale + (plane * 4 + quarter) * MM_PLANE +
                                                   t * 1024 + lane * 16);
    };
    auto read_p = [&](const char *s, int quarter, int t, int h) {
        const int lane = mm_tid() & 63;
        if constexpr (MX) sp = read_scale(h, quarter, t, lane);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) fp[kk][i] = mm_frag(s, rm + 16 * i, kk, lane);
        }
    };
    auto read_q = [&](const char *s, int quarter, int t, int h) {
        const int lane = mm_tid() & 63;
        if constexpr (MX) sq[h] = read_scale(2 + h, quarter, t, lane);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            if constexpr (ROWS) {
#pragma unroll
                for (int j = 0; j < 2; ++j) fq[h][kk][j] = mm_frag(s, rn + 16 * j, kk, lane);
            }
        }
        if constexpr (!ROWS) mm_frag_cols<128, 2>(s, rn, lane, fq[h]);
    };
    // quadrant (h, b): the instruction rows 4 h .. 4 h + 3 of block b.  (The
    // sums are marked as changed: matrix instructions touch no memory, and
    // across a branch the compiler would move them past the next barrier and
    // hold their operands until then.)
    auto quadrant = [&](int h, int b) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            mm_f32x4(&c)[4][2] = *reinterpret_cast<mm_f32x4(*)[4][2]>(&acc.c[b][4 * h]);
            MmBytes<4> bp;
            MmBytes<2> bq;
            bp.pick(mm_u32x2{sp[2 * kk], sp[2 * kk + 1]}, rm / 16);
            bq.pick(mm_u32x2{sq[b][2 * kk], sq[b][2 * kk + 1]}, rn / 16);
            mm_block<MX>(fp[kk], fq[b][kk], bp.w, bq.w[0], c);
        }
        if constexpr (!std::is_same<X, MmNoExtra>::value)
            mm_pin(&acc.c[b][4 * h][0], std::integral_constant<int, 8>{});
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // A step: each half is loaded again, for the step after next, once all
    // waves have read it into registers.  Loads are in the order P0 Q0 Q1 P1
    // of each step, and the waits leave those in flight that are not needed.
    auto step_of = [&](char *p0, char *q0, char *q1, char *p1, char *other_p1, int step, int quarter,
                       int t) {
        mm_wait<5 * L>();       // P0, Q0 here; Q1, P1 and three of the next step may not be
        mm_barrier();
        load_p(other_p1, step + 1, 1);
        read_p(p0, quarter, t, 0);
        read_q(q0, quarter, t, 0);
        extra(acc, q0, step, 0);
        __builtin_amdgcn_sched_barrier(0);
        quadrant(0, 0);
        mm_wait<5 * L>();       // Q1
        mm_barrier();
        load_p(p0, step + 2, 0);
        load_q(q0, step + 2, 0);
        read_q(q1, quarter, t, 1);
        extra(acc, q1, step, 1);
        __builtin_amdgcn_sched_barrier(0);
        quadrant(0, 1);
        mm_wait<6 * L>();       // P1
        mm_barrier();
        load_q(q1, step + 2, 1);
        read_p(p1, quarter, t, 1);
        __builtin_amdgcn_sched_barrier(0);
        quadrant(1, 1);
        quadrant(1, 0);
    };
    if constexpr (MX) {
        if (sc.nb < 16) {
            mm_put_scale4_few(scale, sc, mm_scale_any(sc, 0));
        } else {
            MmScale4 w = mm_scale4_load(sc, group0);
            mm_scale4_shift(w, sc, group0);
            mm_put_scale4(scale, sc, w);
        }
    }
    const int first = 2 * group0;
    load_p(u.u0, first, 0);
    load_q(u.u1, first, 0);
    load_q(u.u2, first, 1);
    load_p(u.u3, first, 1);
    load_p(u.u4, first + 1, 0);
    load_q(u.u5, first + 1, 0);
    load_q(u.u6, first + 1, 1);
    auto even = [&](int g) { step_of(u.u0, u.u1, u.u2, u.u3, u.u7, first + 2 * g, g & 3, 0); };
    auto odd = [&](int g) { step_of(u.u4, u.u5, u.u6, u.u7, u.u3, first + 2 * g + 1, g & 3, 1); };
    if constexpr (MX) {
        for (int g0 = 0; g0 < groups; g0 += 4) {
            const int last = groups - g0 < 4 ? groups - 1 : g0 + 3;
            for (int g = g0; g < last; ++g) {
                even(g);
                odd(g);
            }
            even(last);
            MmScale4 w = mm_scale4_load(sc, group0 + g0 + 4);
            odd(last);
            mm_barrier();       // all waves have read the last of the four groups
            mm_scale4_shift(w, sc, group0 + g0 + 4);
            mm_put_scale4(scale, sc, w);    // written before the next barrier
        }
    } else {
        for (int g = 0; g < groups; ++g) {
            even(g);
            odd(g);
        }
    }
    mm_wait<0>();
    __syncthreads();
}

template <typename S, bool MX, typename Q, typename X>
__device__ __forceinline__ void mm_loop(const MmRows &p, const Q &q, const MmScale &sc, int group0,
                                        int groups, const MmLds &u, char *scale, const X &extra,
                                        MmAcc<S> &acc) {
    if constexpr (S::QUAD) mm_quad<S, MX>(p, q, sc, group0, groups, u, scale, extra, acc);
    else mm_two<S, MX>(p, q, sc, group0, groups, u, scale, extra, acc);
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
