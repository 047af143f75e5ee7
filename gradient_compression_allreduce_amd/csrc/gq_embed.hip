// gq_embed.hip -- gfx950 kernels of the embedding:
//   k_embed       out[t] = mul * table[idx[t]];
//   k_embed_sort  the tokens in the order of their rows;
//   k_embed_sum   grad[v] (+)= mul * the sum of dy over row v's tokens, and the
//                 sums of the pieces of long rows;
//   k_embed_join  the long rows from their pieces' sums;
//   k_embed_grad_small  the whole gradient of few tokens.
// Bound by HBM: a lookup reads each row that it meets and writes every token's,
// a gradient reads dy and writes the table's gradient (131072 tokens of 2048 bf16 into
// 100003 rows of fp32: 1.36 GB, 298 us, 4.6 TB/s, where a copy of 4 GiB runs at
// 4.6).  Every sum has an order that idx alone gives; no two waves add to the same
// place, and none waits for another.
#include "gq_elem.h"
#include "gq_embed.h"

namespace gq {
namespace {

constexpr int EM_BLOCK = 256;
constexpr int EM_WAVES = EM_BLOCK / 64;
constexpr int EM_SLABS = 4;          // slabs of a wave in long lookups

__device__ __forceinline__ int64_t index_at(const void *idx, bool wide, int64_t t) {
    return wide ? static_cast<const int64_t *>(idx)[t] : static_cast<const int32_t *>(idx)[t];
}

// The columns of a lane: those from `lo` to `hi` of a vector of V from `col` on,
// which lies inside the row (the others are another lane's, or none's).  A row has
// V columns or more (V is 1 for short rows).
struct Cols {
    int64_t col;
    int lo, hi;
    bool any;
};

// Those of the vector from `at` on, which may start before or end behind the row.
template <int V>
__device__ __forceinline__ Cols cols_of(int64_t at, int64_t cols) {
    Cols c;
    c.any = at + V > 0 && at < cols;
    c.col = at < 0 ? 0 : at + V <= cols ? at : cols - V;
    c.lo = at < 0 ? 0 : static_cast<int>(at - c.col);
    c.hi = at < 0 ? static_cast<int>(at + V) : V;
    return c;
}

template <typename U, int V>
__device__ __forceinline__ void store_cols(U *row, const Cols &c, const float (&f)[V]) {
    if (!c.any) return;
    if (V == 1 || (c.lo == 0 && c.hi == V)) {
        store_v<true, U, V>(row + c.col, pack<U, V>(f));
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k >= c.lo && k < c.hi) store_1(row + c.col + k, f[k]);
    }
}

// Vectors of a row: 16 bytes of its wider type, or one element of few.
template <typename T, typename U>
constexpr int kWide = sizeof(T) == 4 || sizeof(U) == 4 ? 4 : 8;

// LPR lanes of a wave share a row (64, or fewer where a row has few columns), so
// a wave takes 64 / LPR slabs of LPR vectors at once, W times, one after another
// in the output, and has all of their loads in flight.  65536 tokens of 4096 bf16:
// 125 us, 512 MiB written past the caches, which keep the rows met again (one slab a
// wave 179, two 133, eight 149, stored through the caches 145).
// SHIFT: the output's rows do not all start on a line of 128 bytes, and a row's
// first slab is shortened so that the others do, as lines left to two waves cost
// more (32527 tokens of 4100 bf16 from 60 rows into fp32: 142 us as it comes, 85
// shifted, 80 for 4096 columns; of 4100 from 30522 rows into bf16 65 and 71).
template <typename T, typename U, int V, int LPR, int W, bool SHIFT>
__global__ __launch_bounds__(EM_BLOCK) void k_embed(const EmArgs a) {
    constexpr int SUB = 64 / LPR, LINE = 128 / sizeof(U);
    const int lane = threadIdx.x & 63;
    const int64_t slabs = (a.cols + (SHIFT ? LINE - 1 : 0) + LPR * V - 1) / (LPR * V);
    const int64_t n = a.T * slabs;
    const int64_t wave = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * EM_WAVES +
                         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t i0 = wave * (SUB * W) + (SUB > 1 ? lane / LPR : 0);
    const T *table = static_cast<const T *>(a.table);
    U *out = static_cast<U *>(a.out);
    int64_t t[W], v[W];
    Cols c[W];
    Raw<T, V> r[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const int64_t i = i0 + k * SUB < n ? i0 + k * SUB : n - 1;
        t[k] = SUB > 1 ? i : i / slabs;
        int64_t at = ((SUB > 1 ? 0 : i % slabs * LPR) + lane % LPR) * V;
        if (SHIFT)
            at -= reinterpret_cast<uintptr_t>(out + t[k] * a.ldo) / sizeof(U) % LINE;
        c[k] = cols_of<V>(at, a.cols);
        v[k] = index_at(a.idx, a.wide, t[k]);
        if (v[k] < 0 || v[k] >= a.rows) v[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
        if (v[k] >= 0 && c[k].any) r[k] = load_v<false, T, V>(table + v[k] * a.ld + c[k].col);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if (i0 + k * SUB >= n) break;
        float g[V];
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = v[k] >= 0 ? elem<T, V>(r[k], e) * a.mul : 0.0f;
        store_cols<U, V>(out + t[k] * a.ldo, c[k], g);
    }
}

// ---- the gradient's order of tokens -------------------------------------------
// A counting sort in which every work group has a range of rows and looks
// through all the tokens: how many name a row before its range says where in
// the order its own tokens start, so no work group needs another's counts.
// Wave w looks at the w-th sixteenth of the tokens, counts each row's and keeps
// its own tokens in a list in LDS; sums over the waves and rows before give where
// its tokens of a row go, and it puts them there.  (A wave whose list is full,
// as where one token makes up much of a batch, looks through its tokens again
// instead.)  More than 16384 tokens are first turned into row numbers of 32 bits
// (k_embed_keys), which take the fewest instructions to look through.
// Bound by instructions: up to 262144 rows T tokens are looked at by 256 work groups at
// most, 30 us for 131072 (with the tokens' places found in a second look 49), 10 for 16384;
// 7 to 15% of a gradient of 1024 columns.  Beyond, every 1024 rows are one more work group
// (of 132 KiB LDS, so a compute unit holds one) that looks at all of them, about
// 4 x 10^12 looks a second: a gradient of 8 columns, added, of 131072 tokens into 2^18, 2^20
// and 2^22 rows takes 50, 127 and 365 us, of 2^20 tokens 127, 370 and 1300; of one column,
// 2^22 tokens into 2^22 rows 4.2 ms.  Clearing the rows without a token comes on top at
// 5.5 to 6 TB/s.

// The row of token i, or ~0 where it counts for none.
__device__ __forceinline__ uint32_t row_of(const void *idx, bool wide, int64_t rows, int64_t skip,
                                           int64_t i) {
    const int64_t v = index_at(idx, wide, i);
    return v >= 0 && v < rows && v != skip ? static_cast<uint32_t>(v) : ~0u;
}

__global__ __launch_bounds__(EM_BLOCK) void k_embed_keys(const EgSortArgs a) {
    const int64_t n = (a.T + EG_KEYS - 1) / EG_KEYS * EG_KEYS;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * EM_BLOCK + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * EM_BLOCK)
        a.keys[i] = i < a.T ? row_of(a.idx, a.wide, a.rows, a.skip, i) : ~0u;
}

// Zeros into 16 bytes of a row of `bytes` from byte b on, or what is left of it.
__device__ __forceinline__ void zero_slot(char *row, int64_t b, int64_t bytes, int elem) {
    if (b + 16 <= bytes) {
        store_v<false>(reinterpret_cast<uint32_t *>(row + b), Raw<uint32_t, 4>{});
    } else {
#pragma unroll 1
        for (; b < bytes; b += elem) {
            if (elem == 4) *(elem_u32 *)(row + b) = 0;
            else *(elem_u16 *)(row + b) = 0;
        }
    }
}

// Zeros into a row, by a wave.
__device__ __forceinline__ void zero_row(char *row, int64_t bytes, int elem, int lane) {
    int64_t b = lane * 16;
    for (; b + 16 <= bytes; b += 64 * 16)
        store_v<false>(reinterpret_cast<uint32_t *>(row + b), Raw<uint32_t, 4>{});
    zero_slot(row, b, bytes, elem);
}

// Zeros into the rows of a work group's range that have no token: n_rows rows of
// cols elements of `elem` bytes from `to` on, ld elements apart, whose
// tokens are counted in `total`.  A wave takes a row, or 64 lanes as many
// slots of 16 bytes of rows that have fewer.
__device__ __forceinline__ void zero_rows(char *to, uint32_t n_rows, int64_t cols, int64_t ld,
                                          int elem, const int32_t *total, int wave, int lane) {
    const int64_t bytes = cols * elem;
    if (bytes < 64 * 16) {
        const uint32_t slots = static_cast<uint32_t>(bytes + 15) / 16;
        for (uint32_t i = wave * 64 + lane; i < n_rows * slots; i += EG_BLOCK) {
            const uint32_t r = i / slots;
            if (total[r] == 0) zero_slot(to + r * ld * elem, (i - r * slots) * 16, bytes, elem);
        }
    } else {
        for (uint32_t r = wave; r < n_rows; r += EG_WAVES)
            if (total[r] == 0) zero_row(to + r * ld * elem, bytes, elem, lane);
    }
}

// What lanes of a wave wrote to LDS is what its other lanes read from here on (LDS
// serves a wave's accesses in order: this is for the compiler).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where a wave's token of row `key` goes, and the place behind it for the wave's
// next: lanes of the same row get places in their order.  Only lanes that
// `own` a token get one.  next: the wave's own, by row.
__device__ __forceinline__ int32_t claim(uint32_t key, bool own, int32_t *next, int rows, int lane) {
    const uint64_t any = __ballot(own);
    // the lanes whose token names the same row: of a few tokens one row after
    // another, of many by the bits of their rows
    uint64_t same = any;
    if (__popcll(any) <= 8) {
        for (uint64_t left = any; left;) {
            const int first = __ffsll(static_cast<unsigned long long>(left)) - 1;
            const uint32_t k0 = __builtin_amdgcn_readlane(key, first);
            const uint64_t m = __ballot(own && key == k0);
            if (key == k0) same = m;
            left &= ~m;
        }
    } else {
        for (int b = 1; b < rows; b <<= 1) {
            const uint64_t set = __ballot((key & b) != 0);
            same &= (key & b) ? set : ~set;
        }
    }
    int32_t at = 0;
    if (own) {
        const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
        const int32_t from = next[key];
        at = from + rank;
        wave_fence();
        if (rank == 0) next[key] = from + __popcll(same);
    }
    wave_fence();
    return at;
}

// Thread r of a work group: from the waves' counts of row r's tokens
// count[wave][r], the places of the waves' first ones, and in count[EG_WAVES][r]
// how many they are; `base` tokens come before.  Returns row r's first place.
__device__ __forceinline__ int32_t places(int32_t *count, int rows, int32_t n_rows, int32_t base,
                                          int32_t *scan) {
    const int r = threadIdx.x, lane = r & 63, wave = r >> 6;
    int32_t total = 0, c[EG_WAVES];
    if (r < n_rows) {
#pragma unroll
        for (int w = 0; w < EG_WAVES; ++w) c[w] = count[w * rows + r];
#pragma unroll
        for (int w = 0; w < EG_WAVES; ++w) total += c[w];
        count[EG_WAVES * rows + r] = total;
    }
    int32_t upto = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(upto, o, 64);
        if (lane >= o) upto += u;
    }
    if (lane == 63) scan[wave] = upto;
    __syncthreads();
    int32_t at = base + upto - total;
#pragma unroll
    for (int w = 0; w < EG_WAVES; ++w) at += w < wave ? scan[w] : 0;
    if (r < n_rows) {
        int32_t next = at;
#pragma unroll
        for (int w = 0; w < EG_WAVES; ++w) {
            count[w * rows + r] = next;
            next += c[w];
        }
    }
    __syncthreads();
    return at;
}

constexpr int EG_LIST = 1024;               // tokens that a wave's list holds
constexpr int EG_LIST_BITS = 22;            // of a token's number in it, and 10 of its row

template <bool KEYS>
__global__ __launch_bounds__(EG_BLOCK) void k_embed_sort(const EgSortArgs a) {
    constexpr int NW = EG_WAVES;
    extern __shared__ int32_t count[];      // [NW + 1][rows_per], [NW][EG_LIST]
    __shared__ int32_t before[NW];
    __shared__ int32_t scan[NW];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int R = a.rows_per;
    const uint32_t row0 = blockIdx.x * static_cast<uint32_t>(R);
    const uint32_t n_rows = static_cast<uint32_t>(a.rows - row0 < R ? a.rows - row0 : R);
    const int64_t step = KEYS ? EG_KEYS : 64;
    const int64_t n = (a.T + step - 1) / step * step;
    const int64_t per = (n + NW * step - 1) / (NW * step) * step;
    const int64_t t0 = wave * per, t1 = t0 + per < n ? t0 + per : n;
    for (int i = threadIdx.x; i < NW * R; i += EG_BLOCK) count[i] = 0;
    uint32_t *list = reinterpret_cast<uint32_t *>(count + (NW + 1) * R) + wave * EG_LIST;

    // 64 * EG_HELD tokens from t on
    uint32_t row[EG_HELD];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < EG_HELD; k += KEYS ? 4 : 1) {
            if constexpr (KEYS) {
                Raw<uint32_t, 4> v = {{~0u, ~0u, ~0u, ~0u}};
                if (t + 64 * k < t1)
                    v = load_v<false, uint32_t, 4>(a.keys + t + 64 * k + 4 * lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) row[k + j] = v.w[j];
            } else {
                const int64_t i = t + 64 * k + lane;
                row[k] = ~0u;
                if (t + 64 * k < t1 && i < a.T)
                    row[k] = row_of(a.idx, a.wide, a.rows, a.skip, i);
            }
        }
    };
    // the number of row[k]'s token, where row[]'s first one has number `first`
    auto number = [&](int64_t first, int k) {
        return first + (KEYS ? 64 * (k & ~3) + 4 * lane + (k & 3) : 64 * k + lane);
    };
    if (!KEYS) load(t0);
    __syncthreads();

    int32_t *mine = count + wave * R;
    int32_t less = 0, kept = 0;
    // this wave's own tokens of row[] to the list's end, as far as it holds them;
    // row[]'s first token has number `first`
    auto keep = [&](int64_t first, bool tally) {
#pragma unroll
        for (int k = 0; k < EG_HELD; ++k) {
            if (tally) less += __popcll(__ballot(row[k] < row0));
            const uint32_t key = row[k] - row0;
            const uint64_t own = __ballot(key < n_rows);
            if (!own) continue;
            if (key < n_rows) {
                if (tally) atomicAdd(&mine[key], 1);
                const int32_t at = kept + __popcll(own & ((uint64_t{1} << lane) - 1));
                if (at < EG_LIST)
                    list[at] = key << EG_LIST_BITS | static_cast<uint32_t>(number(first, k));
            }
            kept += __popcll(own);
        }
    };
    if constexpr (KEYS) {
        for (int64_t t = t0; t < t1; t += 64 * EG_HELD) {
            load(t);
            keep(t - t0, true);
        }
    } else {
        keep(0, true);
    }
    if (lane == 0) before[wave] = less;
    __syncthreads();
    int32_t base = 0;
    for (int w = 0; w < NW; ++w) base += before[w];
    const int32_t at = places(count, R, static_cast<int32_t>(n_rows), base, scan);
    const uint32_t r = threadIdx.x;
    if (r < n_rows) {
        a.start[row0 + r] = at;
        if (row0 + r == a.rows - 1) a.start[a.rows] = at + count[NW * R + r];
    }
    // the rows that no token names (the stores go on while the rest runs)
    if (a.grad)
        zero_rows(a.grad + row0 * a.ldg * a.elem, n_rows, a.cols, a.ldg, a.elem, count + NW * R,
                  wave, lane);
    // the list's tokens to their places; their numbers count from `from`
    auto put = [&](int64_t from) {
        wave_fence();
        for (int32_t i = 0; i < kept; i += 64) {
            const bool own = i + lane < kept;
            const uint32_t e = own ? list[i + lane] : 0, key = e >> EG_LIST_BITS;
            const int32_t to = claim(key, own, mine, R, lane);
            if (!own) continue;
            a.order[to] = static_cast<int32_t>(from + (e & ((1u << EG_LIST_BITS) - 1)));
            if (to % EG_PIECE == 0) a.piece_row[to / EG_PIECE] = static_cast<int32_t>(row0 + key);
        }
    };
    if (!KEYS || (kept <= EG_LIST && per <= 1 << EG_LIST_BITS)) {
        put(t0);
    } else {
        // (a load of tokens always fits an empty list)
        static_assert(64 * EG_HELD <= EG_LIST, "");
        for (int64_t t = t0; t < t1; t += 64 * EG_HELD) {
            load(t);
            kept = 0;
            wave_fence();
            keep(0, false);
            put(t);
        }
    }
}

// ---- the sums -------------------------------------------------------------------
// A row of up to EG_PIECE tokens is summed by one wave (or, where a row has few
// columns, by LPR lanes of one).  The tokens of longer rows are summed piece by
// piece and their sums joined by k_embed_join: a row that is longer than a piece
// and lies in it starts at or before the piece's first token, or else reaches
// past its last, so a piece has at most two such rows, and two places for sums.
// 131072 tokens of 2048 bf16 into 100003 rows of fp32: 165 us, 788 MB, 4.8 TB/s (a
// wave for each row whatever its length: 6.3 ms, for the row of the most frequent
// token; pieces of 32 tokens 10 us more, of 128 9 more).  16384 of 1024 into 30522 rows,
// added: 24 us, 100 MB, 4.2 TB/s, a chain of four loads.

// What grad holds in a lane's columns, where it is added to.
template <typename U, int V, typename Args>
__device__ __forceinline__ Raw<U, V> old_of(const Args &a, int64_t row, const Cols &c) {
    Raw<U, V> r = {};
    if (a.add && c.any) r = load_v<true, U, V>(static_cast<const U *>(a.grad) + row * a.ldg + c.col);
    return r;
}

// grad's columns of a lane from their sums.
template <typename U, int V, typename Args>
__device__ __forceinline__ void finish(const Args &a, int64_t row, const Cols &c, float (&s)[V],
                                       const Raw<U, V> &old) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        // (0 is added so that a sum of zeros times a negative mul is 0 and not -0)
        s[k] = s[k] * a.mul + (a.add ? elem<U, V>(old, k) : 0.0f);
    }
    store_cols<U, V>(static_cast<U *>(a.grad) + row * a.ldg, c, s);
}

template <int V, int LPR>
struct EgShape {
    static constexpr int SUB = 64 / LPR;                // rows of a wave at once
    static constexpr int GROUP = LPR == 64 ? 4 : 1;      // rows of LPR lanes, one after another
    static constexpr int FLY = 16;                      // tokens in flight
    static __host__ __device__ int64_t slabs(int64_t cols) {
        return (cols + LPR * V - 1) / (LPR * V);
    }
};

// Value `from` (0 .. LPR - 1) of the lanes that share a row.
template <int LPR>
__device__ __forceinline__ int32_t take(int32_t v, int from) {
    if constexpr (LPR == 64) return __builtin_amdgcn_readlane(v, from);
    else return __shfl(v, from, LPR);
}

// The waves of the pieces come first (where few lanes share a row, they take a
// piece's tokens in turns and add their sums), then those of the rows.
template <typename T, typename U, int V, int LPR>
__global__ __launch_bounds__(EM_BLOCK) void k_embed_sum(const EgSumArgs a) {
    using S = EgShape<V, LPR>;
    constexpr int FLY = S::FLY, SUB = S::SUB;
    const int lane = threadIdx.x & 63, l = lane % LPR, sub = lane / LPR;
    const int64_t slabs = S::slabs(a.cols);
    int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first_block = (a.pieces * slabs + EM_WAVES - 1) / EM_WAVES;
    const bool piece = block < first_block;
    if (!piece) {
        // every so many work groups one that clears rows
        block -= first_block;
        const int64_t n = a.zero_blocks * block / a.mixed_blocks;
        if (a.zero_blocks && n != a.zero_blocks * (block + 1) / a.mixed_blocks) {
            const int64_t row0 = (n * EM_WAVES + w) * EG_ZERO;
            if (row0 >= a.rows) return;
            const int rows = static_cast<int>(a.rows - row0 < EG_ZERO ? a.rows - row0 : EG_ZERO);
            const int32_t starts = a.start[row0 + (lane < rows ? lane : rows)];
            for (int r = 0; r < rows; ++r)
                if (take<64>(starts, r) == take<64>(starts, r + 1))
                    zero_row(reinterpret_cast<char *>(static_cast<U *>(a.grad) + (row0 + r) * a.ldg),
                             a.cols * static_cast<int64_t>(sizeof(U)), sizeof(U), lane);
            return;
        }
        block -= n;
    }
    const int64_t wave = block * EM_WAVES + w;
    const int64_t g = piece ? wave : wave * SUB + (SUB > 1 ? sub : 0);
    const int64_t unit = SUB > 1 ? g : g / slabs, slab = SUB > 1 ? 0 : g % slabs;
    const Cols c = cols_of<V>((slab * LPR + l) * V, a.cols);
    const T *dy = static_cast<const T *>(a.dy);

    // the tokens of the order from `held` to held_end, LPR or fewer, one a lane
    int32_t held = 0, held_end = 0, have = 0;
    auto hold = [&](int32_t at, int32_t end) __attribute__((always_inline)) {
        held = at;
        held_end = end - at < LPR ? end : at + LPR;
        have = 0;
        if (at + l < end) have = a.order[at + l];
    };
    auto token = [&](int at) __attribute__((always_inline)) { return take<LPR>(have, at % LPR); };
    // s += the tokens first .. end - 1 of the order
    auto sum = [&](int32_t first, int32_t end, float (&s)[V]) __attribute__((always_inline)) {
        for (int32_t at = first; at < end; at += LPR) {
            const int n = end - at < LPR ? end - at : LPR;
            if (at < held || at + n > held_end) hold(at, end);
            const int skip = at - held;
            for (int j = 0; j < n; j += FLY) {
                Raw<T, V> v[FLY];
                // (tokens that come from another lane are all asked for first)
                int32_t t[FLY];
                if (SUB > 1)
#pragma unroll
                    for (int k = 0; k < FLY; ++k) t[k] = token(j + k < n ? skip + j + k : 0);
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    if (SUB == 1) t[k] = token(j + k < n ? skip + j + k : 0);
                    if (j + k < n && c.any)
                        v[k] = load_v<true, T, V>(dy + static_cast<int64_t>(t[k]) * a.ldy + c.col);
                }
#pragma unroll
                for (int k = 0; k < FLY; ++k)
                    if (j + k < n)
#pragma unroll
                        for (int e = 0; e < V; ++e) s[e] += elem<T, V>(v[k], e);
            }
        }
    };
    auto uniform = [](int32_t v) { return __builtin_amdgcn_readfirstlane(v); };

    if (piece) {
        if (unit >= a.pieces) return;
        // (what lies behind the last token's piece is of no meaning)
        const int32_t total = uniform(a.start[a.rows]);
        int32_t head = a.piece_row[unit];
        int32_t tail = a.piece_row[unit + 1 < a.pieces ? unit + 1 : unit];
        const int64_t from = unit * EG_PIECE;
        if (from >= total) return;
        const int32_t begin = static_cast<int32_t>(from);
        const int32_t stop = total - begin < EG_PIECE ? total : begin + EG_PIECE;
        head = uniform(head);
        tail = uniform(stop < total ? tail : head);
        const int32_t h0 = uniform(a.start[head]), h1 = uniform(a.start[head + 1]);
        const int32_t t0 = uniform(a.start[tail]), t1 = uniform(a.start[tail + 1]);
        if (SUB == 1) hold(begin, stop);
        float *place = a.part + (unit * 2 * slabs + slab) * (LPR * V) + l * V;
#pragma unroll 1
        for (int second = 0; second < 2; ++second) {
            const int32_t r0 = second ? t0 : h0, r1 = second ? t1 : h1;
            if (r1 - r0 <= EG_PIECE || (second && (tail == head || t0 >= stop))) continue;
            const int32_t first = second ? t0 : begin, end = r1 < stop ? r1 : stop;
            float s[V] = {};
            if constexpr (SUB == 1) {
                sum(first, end, s);
            } else {
                const int32_t each = (end - first + SUB - 1) / SUB;
                const int32_t mine = first + sub * each;
                sum(mine, mine + each < end ? mine + each : end, s);
#pragma unroll
                for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
                    for (int e = 0; e < V; ++e) s[e] += __shfl_xor(s[e], o, 64);
            }
            if (sub == 0)
                store_v<false, float, V>(place + second * slabs * (LPR * V), pack<float, V>(s));
        }
        return;
    }
    const int64_t row0 = unit * S::GROUP;
    if (row0 >= a.rows) return;
    const int rows = static_cast<int>(a.rows - row0 < S::GROUP ? a.rows - row0 : S::GROUP);
    const int32_t starts = a.start[row0 + (l < rows ? l : rows)];
    hold(take<LPR>(starts, 0), take<LPR>(starts, rows));
    for (int r = 0; r < rows; ++r) {
        const int32_t first = take<LPR>(starts, r), end = take<LPR>(starts, r + 1);
        if (end - first > EG_PIECE || first == end) continue;
        const Raw<U, V> old = old_of<U, V>(a, row0 + r, c);
        float s[V] = {};
        sum(first, end, s);
        finish<U, V>(a, row0 + r, c, s, old);
    }
}

constexpr int EG_JOIN = 512;

// Work groups of the join of each slab.
__host__ __device__ inline int64_t join_groups(int64_t pieces) {
    return pieces < 256 ? pieces : 256;
}

// The sums of a long row's pieces, added in their order: an eighth of them
// by each wave, then the waves' sums.  Work group b of a slab looks at the pieces
// b, b + grid, ..., a lane at each, for those in which a long row starts.  4.6 us where
// little is to be joined (launch and a chain of three loads), 11 us for the pieces of
// 131072 tokens of 2048.
template <typename U, int V, int LPR>
__global__ __launch_bounds__(EG_JOIN) void k_embed_join(const EgSumArgs a) {
    using S = EgShape<V, LPR>;
    constexpr int FLY = 4, NW = EG_JOIN / 64;
    __shared__ float sh[NW][V][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t slabs = S::slabs(a.cols);
    const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t grid = join_groups(a.pieces), slab = block % slabs;
    if (block >= grid * slabs) return;
    const Cols c = cols_of<V>((slab * LPR + lane) * V, lane < LPR ? a.cols : 0);
    for (int64_t p0 = block / slabs; p0 < a.pieces; p0 += grid * 64) {
        // the long row that starts in this lane's piece, if any: that of its
        // first token, or the one that the next piece starts with
        const int64_t p = p0 + grid * lane;
        const int64_t total = a.start[a.rows];
        int32_t row = -1, begin = 0, stop = 0;
        if (p * EG_PIECE < total) {
            const bool last = (p + 1) * EG_PIECE >= total;
            const int32_t r0 = a.piece_row[p], r1 = last ? r0 : a.piece_row[p + 1];
            const int32_t b0 = a.start[r0], e0 = a.start[r0 + 1];
            const int32_t b1 = a.start[r1], e1 = a.start[r1 + 1];
            if (b0 == p * EG_PIECE && e0 - b0 > EG_PIECE) {
                row = r0;
                begin = b0;
                stop = e0;
            } else if (b1 > p * EG_PIECE && b1 < (p + 1) * EG_PIECE && e1 - b1 > EG_PIECE) {
                row = r1;
                begin = b1;
                stop = e1;
            }
        }
        uint64_t found = __ballot(row >= 0);
        while (found) {
            const int from = __ffsll(static_cast<unsigned long long>(found)) - 1;
            found &= found - 1;
            const int32_t r = __builtin_amdgcn_readlane(row, from);
            const int32_t s0 = __builtin_amdgcn_readlane(begin, from);
            const int32_t s1 = __builtin_amdgcn_readlane(stop, from);
            const int32_t first = s0 / EG_PIECE, n = (s1 - 1) / EG_PIECE - first + 1;
            const int32_t lo = static_cast<int32_t>(static_cast<int64_t>(n) * w / NW);
            const int32_t hi = static_cast<int32_t>(static_cast<int64_t>(n) * (w + 1) / NW);
            Raw<U, V> old;
            if (w == 0) old = old_of<U, V>(a, r, c);
            float s[V] = {};
            if (c.any)
                for (int32_t j = lo; j < hi; j += FLY) {
                    Raw<float, V> v[FLY];
#pragma unroll
                    for (int k = 0; k < FLY; ++k)
                        if (j + k < hi) {
                            const int64_t at = first + j + k;
                            // (its first piece may start with another row)
                            const int64_t second = j + k == 0 && s0 % EG_PIECE != 0;
                            v[k] = load_v<false, float, V>(
                                a.part + ((at * 2 + second) * slabs + slab) * (LPR * V) + lane * V);
                        }
#pragma unroll
                    for (int k = 0; k < FLY; ++k)
                        if (j + k < hi)
#pragma unroll
                            for (int e = 0; e < V; ++e) s[e] += elem<float, V>(v[k], e);
                }
#pragma unroll
            for (int e = 0; e < V; ++e) sh[w][e][lane] = s[e];
            __syncthreads();
            if (w == 0) {
                for (int q = 1; q < NW; ++q)
#pragma unroll
                    for (int e = 0; e < V; ++e) s[e] += sh[q][e][lane];
                finish<U, V>(a, r, c, s, old);
            }
            __syncthreads();
        }
    }
}

// ---- a gradient of few tokens ----------------------------------------------------
// One launch: a work group of a range of rows looks through all the tokens and
// sorts those of its rows in LDS (one that has none clears its rows and ends: 7 tokens
// into 193386 rows of 10 columns 20 us with the sort, 11 without).  A wave sums a row's slab of columns; rows of more
// than EG_ALONE tokens are summed by all waves, which share out a slab's tokens, or
// several slabs', and join their sums (600 tokens into 2000 rows 9.5 us with 16, 10.2
// with 32).  512 tokens of 1024 bf16 added to 30522 rows of
// fp32: 8.7 us of launch, indexes, sort, rows, one after another (three launches 18).
constexpr int EG_ALONE = 16;

template <typename T, typename U, int V>
__global__ __launch_bounds__(EG_BLOCK) void k_embed_grad_small(const EgSmallArgs a) {
    constexpr int FLY = 8;
    constexpr int PER = EG_SMALL / EG_BLOCK;
    constexpr int R = EG_SMALL_ROWS, NW = EG_WAVES;
    __shared__ int32_t count[(NW + 1) * R];
    __shared__ int32_t order[EG_SMALL];
    __shared__ int32_t first[R];
    __shared__ int32_t scan[NW];
    __shared__ float sh[NW][V][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t row0 = block * a.rows_per;
    if (row0 >= a.rows) return;
    const uint32_t n_rows =
        static_cast<uint32_t>(a.rows - row0 < a.rows_per ? a.rows - row0 : a.rows_per);
    uint32_t key[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = k * EG_BLOCK + threadIdx.x;
        key[k] = ~0u;
        if (i < a.T) {
            const uint32_t row = row_of(a.idx, a.wide, a.rows, a.skip, i);
            if (row != ~0u) key[k] = row - static_cast<uint32_t>(row0);
        }
    }
    for (int i = threadIdx.x; i < (NW + 1) * R; i += EG_BLOCK) count[i] = 0;
    bool some = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) some = some || key[k] < n_rows;
    int32_t *mine = count + wave * R;
    const int32_t *total = count + NW * R;
    U *grad = static_cast<U *>(a.grad);
    if (!__syncthreads_or(some)) {          // (all of `total` is 0)
        if (!a.add)
            zero_rows(reinterpret_cast<char *>(grad + row0 * a.ldg), n_rows, a.cols, a.ldg,
                      sizeof(U), total, wave, lane);
        return;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (key[k] < n_rows) atomicAdd(&mine[key[k]], 1);
    __syncthreads();
    const int32_t at = places(count, R, static_cast<int32_t>(n_rows), 0, scan);
    if (threadIdx.x < R) first[threadIdx.x] = at;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const bool own = key[k] < n_rows;
        if (!__ballot(own)) continue;
        const int32_t to = claim(key[k], own, mine, R, lane);
        if (own) order[to] = k * EG_BLOCK + threadIdx.x;
    }
    __syncthreads();

    const T *dy = static_cast<const T *>(a.dy);
    const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V);
    if (!a.add)
        zero_rows(reinterpret_cast<char *>(grad + row0 * a.ldg), n_rows, a.cols, a.ldg, sizeof(U),
                  total, wave, lane);
    // s += the tokens from .. end - 1 of the order
    auto sum = [&](int32_t from, int32_t end, const Cols &c,
                   float (&s)[V]) __attribute__((always_inline)) {
        for (; from < end; from += 64) {
            const int n = end - from < 64 ? end - from : 64;
            const int32_t have = order[from + (lane < n ? lane : 0)];
            for (int j = 0; j < n; j += FLY) {
                Raw<T, V> v[FLY];
#pragma unroll
                for (int k = 0; k < FLY; ++k)
                    if (j + k < n) {
                        const int64_t t = __builtin_amdgcn_readlane(have, j + k);
                        if (c.any) v[k] = load_v<true, T, V>(dy + t * a.ldy + c.col);
                    }
#pragma unroll
                for (int k = 0; k < FLY; ++k)
                    if (j + k < n)
#pragma unroll
                        for (int e = 0; e < V; ++e) s[e] += elem<T, V>(v[k], e);
            }
        }
    };
    // this lane's rows' tokens, and the rows of few and of many as bits
    static_assert(R == 128, "two rows a lane");
    const int32_t n_of[2] = {total[lane], total[lane + 64]};
    const int32_t first_of[2] = {first[lane], first[lane + 64]};
    uint32_t items = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        for (uint64_t m = __ballot(n_of[h] > 0 && n_of[h] <= EG_ALONE); m; m &= m - 1) {
            const int bit = __ffsll(static_cast<unsigned long long>(m)) - 1;
            const int32_t n = __builtin_amdgcn_readlane(n_of[h], bit);
            const int32_t from = __builtin_amdgcn_readlane(first_of[h], bit);
            for (int64_t slab = (wave - items) % NW; slab < slabs; slab += NW) {
                const Cols c = cols_of<V>((slab * 64 + lane) * V, a.cols);
                const Raw<U, V> old = old_of<U, V>(a, row0 + 64 * h + bit, c);
                float s[V] = {};
                sum(from, from + n, c, s);
                finish<U, V>(a, row0 + 64 * h + bit, c, s, old);
            }
            items += static_cast<uint32_t>(slabs);
        }
    // `at_once` slabs at a time, each by `parts` waves
    const int at_once = slabs < NW ? static_cast<int>(slabs) : NW, parts = NW / at_once;
    const int my_slab = wave / parts, part = wave % parts;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        for (uint64_t m = __ballot(n_of[h] > EG_ALONE); m; m &= m - 1) {
            const int bit = __ffsll(static_cast<unsigned long long>(m)) - 1;
            const int64_t row = row0 + 64 * h + bit;
            const int32_t n = __builtin_amdgcn_readlane(n_of[h], bit);
            const int32_t from = __builtin_amdgcn_readlane(first_of[h], bit);
            for (int64_t s0 = 0; s0 < slabs; s0 += at_once) {
                const bool in = my_slab < at_once && s0 + my_slab < slabs;
                const Cols c = cols_of<V>(((s0 + my_slab) * 64 + lane) * V, in ? a.cols : 0);
                Raw<U, V> old;
                if (part == 0) old = old_of<U, V>(a, row, c);
                float s[V] = {};
                if (in) sum(from + n * part / parts, from + n * (part + 1) / parts, c, s);
#pragma unroll
                for (int e = 0; e < V; ++e) sh[wave][e][lane] = s[e];
                __syncthreads();
                if (part == 0 && in) {
                    for (int w = 1; w < parts; ++w)
#pragma unroll
                        for (int e = 0; e < V; ++e) s[e] += sh[wave + w][e][lane];
                    finish<U, V>(a, row, c, s, old);
                }
                __syncthreads();
            }
        }
}

// A grid of that many work groups, whose sides have less than 2^32 work-items;
// those that are too many find nothing to do.
dim3 grid_of(int64_t blocks) {
    const int64_t x = blocks < 1 << 20 ? blocks : 1 << 20;
    return dim3(static_cast<uint32_t>(x), static_cast<uint32_t>((blocks + x - 1) / x));
}

template <typename T, typename U, int V, int LPR>
hipError_t embed_as(const EmArgs &a, hipStream_t s) {
    constexpr int64_t slab = LPR * V, per = 64 / LPR * EM_WAVES, line = 128 / sizeof(U);
    const int64_t n = a.T * ((a.cols + slab - 1) / slab);
    // (slabs of several a wave where that leaves a wave for every place on the chip)
    if (n < EM_SLABS * 2048 * per) {
        k_embed<T, U, V, LPR, 1, false><<<grid_of((n + per - 1) / per), EM_BLOCK, 0, s>>>(a);
        return hipGetLastError();
    }
    constexpr int64_t all = EM_SLABS * per;
    if constexpr (LPR == 64) {
        if (reinterpret_cast<uintptr_t>(a.out) % 128 || a.ldo % line) {
            const int64_t more = a.T * ((a.cols + line - 1 + slab - 1) / slab);
            k_embed<T, U, V, LPR, EM_SLABS, true>
                <<<grid_of((more + all - 1) / all), EM_BLOCK, 0, s>>>(a);
            return hipGetLastError();
        }
    }
    k_embed<T, U, V, LPR, EM_SLABS, false><<<grid_of((n + all - 1) / all), EM_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

// Short rows by few lanes: 131072 tokens of 8 bf16 22 us with 64 lanes, 7.6 with 4;
// of 60 28 and 9.7 (16 lanes); 500000 of 30 into fp32 81 and 19.
template <typename T, typename U>
hipError_t embed_into(const EmArgs &a, hipStream_t s) {
    constexpr int V = kWide<T, U>;
    if (a.cols < V) return embed_as<T, U, 1, 8>(a, s);
    if (a.cols <= 4 * V) return embed_as<T, U, V, 4>(a, s);
    if (a.cols <= 16 * V) return embed_as<T, U, V, 16>(a, s);
    return embed_as<T, U, V, 64>(a, s);
}

template <typename T>
hipError_t embed_from(const EmArgs &a, gq_dtype out_dt, hipStream_t s) {
    if (out_dt == GQ_F32) return embed_into<T, float>(a, s);
    if (out_dt == GQ_F16) return embed_into<T, __half>(a, s);
    return embed_into<T, bf16_t>(a, s);
}

// Which launch of a gradient.
enum EgPart { EG_SUM, EG_JOINED };

template <typename T, typename U, int V, int LPR>
hipError_t sum_as(const EgSumArgs &a, EgPart part, hipStream_t s) {
    using S = EgShape<V, LPR>;
    const int64_t slabs = S::slabs(a.cols);
    if (part == EG_JOINED) {
        k_embed_join<U, V, LPR>
            <<<grid_of(join_groups(a.pieces) * slabs), EG_JOIN, 0, s>>>(a);
    } else {
        const int64_t units = (a.rows + S::GROUP - 1) / S::GROUP * slabs;
        constexpr int64_t per = S::SUB * EM_WAVES;
        EgSumArgs b = a;
        b.zero_blocks = a.zero ? (a.rows + EM_WAVES * EG_ZERO - 1) / (EM_WAVES * EG_ZERO) : 0;
        b.mixed_blocks = b.zero_blocks + (units + per - 1) / per;
        const int64_t pieces = (a.pieces * slabs + EM_WAVES - 1) / EM_WAVES;
        k_embed_sum<T, U, V, LPR><<<grid_of(pieces + b.mixed_blocks), EM_BLOCK, 0, s>>>(b);
    }
    return hipGetLastError();
}

// Lanes that share a row, and elements of each: a vector of 16 bytes by 64 lanes, and
// for short rows so that a wave has a few rows of its own.  bf16 into fp32, with 4
// lanes of vectors up to 32 columns and 16 up to 128 / as below: 131072 tokens of 8
// into 262144 rows 80 / 60 us, 16384 of 32 into 30522, added, 38 / 23, 27387 of 15 into
// 994 39 / 22; 20000 of 100 into 100, 64 lanes of 4 / as below, 36 / 27.
template <typename T, typename U>
hipError_t grad_part(const EgSumArgs &a, EgPart part, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.cols <= 16) return sum_as<T, U, 1, 16>(a, part, s);
    if (a.cols <= 64) return sum_as<T, U, 4, 16>(a, part, s);
    if (a.cols <= 16 * V) return sum_as<T, U, V, 16>(a, part, s);
    return sum_as<T, U, V, 64>(a, part, s);
}

template <typename T, typename U>
hipError_t grad_part(const EgSmallArgs &a, EgPart, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const dim3 grid = grid_of((a.rows + a.rows_per - 1) / a.rows_per);
    if (a.cols < V) k_embed_grad_small<T, U, 1><<<grid, EG_BLOCK, 0, s>>>(a);
    else k_embed_grad_small<T, U, V><<<grid, EG_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, typename Args>
hipError_t grad_from(const Args &a, gq_dtype out_dt, EgPart part, hipStream_t s) {
    if (out_dt == GQ_F32) return grad_part<T, float>(a, part, s);
    if (out_dt == GQ_F16) return grad_part<T, __half>(a, part, s);
    return grad_part<T, bf16_t>(a, part, s);
}

template <typename Args>
hipError_t grad_any(const Args &a, gq_dtype dt, gq_dtype out_dt, EgPart part, hipStream_t s) {
    if (dt == GQ_F32) return grad_from<float>(a, out_dt, part, s);
    if (dt == GQ_F16) return grad_from<__half>(a, out_dt, part, s);
    return grad_from<bf16_t>(a, out_dt, part, s);
}

}  // namespace

hipError_t launch_embed(const EmArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    if (dt == GQ_F32) return embed_from<float>(a, out_dt, s);
    if (dt == GQ_F16) return embed_from<__half>(a, out_dt, s);
    return embed_from<bf16_t>(a, out_dt, s);
}

hipError_t launch_embed_grad_small(const EgSmallArgs &a, gq_dtype dt, gq_dtype out_dt,
                                   hipStream_t s) {
    return grad_any(a, dt, out_dt, EG_SUM, s);
}

hipError_t launch_embed_sort(const EgSortArgs &a, hipStream_t s) {
    const uint32_t grid = static_cast<uint32_t>((a.rows + a.rows_per - 1) / a.rows_per);
    const size_t lds = sizeof(int32_t) * ((EG_WAVES + 1) * a.rows_per + EG_WAVES * EG_LIST);
    if (a.keys) {
        const int64_t blocks = (a.T + EM_BLOCK - 1) / EM_BLOCK;
        k_embed_keys<<<static_cast<uint32_t>(blocks < 2048 ? blocks : 2048), EM_BLOCK, 0, s>>>(a);
        k_embed_sort<true><<<grid, EG_BLOCK, lds, s>>>(a);
    } else {
        k_embed_sort<false><<<grid, EG_BLOCK, lds, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_embed_sum(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    return grad_any(a, dt, out_dt, EG_SUM, s);
}

hipError_t launch_embed_join(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    return grad_any(a, dt, out_dt, EG_JOINED, s);
}

}  // namespace gq
