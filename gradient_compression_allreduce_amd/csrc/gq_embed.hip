// gq_embed.hip -- gfx950 kernels of the embedding:
//   k_embed       out[t] = mul * table[idx[t]];
//   k_embed_sort  the tokens in the order of their rows;
//   k_embed_sum   grad[v] (+)= mul * the sum of dy over row v's tokens, and the
//                 sums of the pieces of long rows;
//   k_embed_join  the long rows from their pieces' sums.
#include "gq_elem.h"
#include "gq_embed.h"

namespace gq {
namespace {

constexpr int EM_BLOCK = 256;
constexpr int EM_WAVES = EM_BLOCK / 64;

__device__ __forceinline__ int64_t index_at(const void *idx, bool wide, int64_t t) {
    return wide ? static_cast<const int64_t *>(idx)[t] : static_cast<const int32_t *>(idx)[t];
}

// A wave takes 64 vectors of a row.
template <typename T, typename U>
__global__ __launch_bounds__(EM_BLOCK) void k_embed(const EmArgs a) {
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V);
    const T *table = static_cast<const T *>(a.table);
    U *out = static_cast<U *>(a.out);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * EM_WAVES + (threadIdx.x >> 6);
         i < a.T * slabs; i += static_cast<int64_t>(gridDim.x) * EM_WAVES) {
        const int64_t t = i / slabs, col = (i % slabs * 64 + lane) * V;
        const int64_t v = index_at(a.idx, a.wide, t);
        const bool inside = v >= 0 && v < a.rows;
        const T *x = table + (inside ? v : 0) * a.ld + col;
        U *y = out + t * a.ldo + col;
        if (col + V <= a.cols) {
            float g[V];
            const Raw<T, V> r = load_v<false, T, V>(x);
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = inside ? elem<T, V>(r, k) * a.mul : 0.0f;
            store_v<true, U, V>(y, pack<U, V>(g));
        } else {
            for (int k = 0; k < V && col + k < a.cols; ++k)
                y[k] = from_f32<U>(inside ? to_f32(x[k]) * a.mul : 0.0f);
        }
    }
}

// ---- the gradient's order of tokens -------------------------------------------
// A counting sort in which every work group has a range of rows and looks
// through all the tokens: how many name a row before its range says where in
// the order its own tokens start, so no work group needs another's counts.
// Wave w looks at the w-th sixteenth of the tokens.  It counts each row's;
// sums over the waves and rows before give where its own tokens of a row go;
// and in a second pass it puts them there, in the order in which they come.
constexpr int EG_LOADS = 16;        // indexes of a lane in flight

// The rows of 64 * EG_LOADS tokens from t on, -1 for those that count for none.
__device__ __forceinline__ void rows_of(const EgSortArgs &a, int64_t t, int64_t end, int lane,
                                        int32_t (&row)[EG_LOADS]) {
#pragma unroll
    for (int k = 0; k < EG_LOADS; ++k) {
        const int64_t i = t + 64 * k + lane;
        int64_t v = -1;
        if (i < end) v = index_at(a.idx, a.wide, i);
        row[k] = v >= 0 && v < a.rows && v != a.skip ? static_cast<int32_t>(v) : -1;
    }
}

__global__ __launch_bounds__(EG_SORT_BLOCK) void k_embed_sort(const EgSortArgs a) {
    constexpr int NW = EG_SORT_BLOCK / 64;
    extern __shared__ int32_t count[];          // [NW][rows_per]
    __shared__ int32_t before[NW];
    __shared__ int32_t scan[NW];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int R = a.rows_per;
    const int32_t row0 = static_cast<int32_t>(blockIdx.x) * R;
    const int n_rows = static_cast<int>(a.rows - row0 < R ? a.rows - row0 : R);
    const int64_t per = (a.T + NW * 64 - 1) / (NW * 64) * 64;
    const int64_t t0 = wave * per, t1 = t0 + per < a.T ? t0 + per : a.T;
    for (int i = threadIdx.x; i < NW * R; i += EG_SORT_BLOCK) count[i] = 0;
    __syncthreads();
    int32_t *mine = count + wave * R;
    int32_t less = 0;
    int32_t row[EG_LOADS];
    for (int64_t t = t0; t < t1; t += 64 * EG_LOADS) {
        rows_of(a, t, t1, lane, row);
#pragma unroll
        for (int k = 0; k < EG_LOADS; ++k) {
            if (row[k] >= 0 && row[k] < row0) ++less;
            const uint32_t key = static_cast<uint32_t>(row[k]) - static_cast<uint32_t>(row0);
            if (key < static_cast<uint32_t>(n_rows)) atomicAdd(&mine[key], 1);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) less += __shfl_xor(less, o, 64);
    if (lane == 0) before[wave] = less;
    __syncthreads();
    // thread r: row r's tokens in each wave's part, as starts
    int32_t total = 0;
    const int r = threadIdx.x;
    if (r < n_rows)
        for (int w = 0; w < NW; ++w) {
            const int32_t c = count[w * R + r];
            count[w * R + r] = total;
            total += c;
        }
    int32_t upto = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(upto, o, 64);
        if (lane >= o) upto += u;
    }
    if (lane == 63) scan[wave] = upto;
    __syncthreads();
    int32_t at = upto - total;
    for (int w = 0; w < NW; ++w) {
        at += before[w];
        if (w < wave) at += scan[w];
    }
    if (r < n_rows) {
        for (int w = 0; w < NW; ++w) count[w * R + r] += at;
        a.start[row0 + r] = at;
        if (row0 + r == a.rows - 1) a.start[a.rows] = at + total;
    }
    __syncthreads();
    for (int64_t t = t0; t < t1; t += 64 * EG_LOADS) {
        rows_of(a, t, t1, lane, row);
#pragma unroll
        for (int k = 0; k < EG_LOADS; ++k) {
            const uint32_t key = static_cast<uint32_t>(row[k]) - static_cast<uint32_t>(row0);
            const bool own = key < static_cast<uint32_t>(n_rows);
            uint64_t same = __ballot(own);
            if (!same) continue;
            // the lanes whose token names the same row
            for (int b = 1; b < R; b <<= 1) {
                const uint64_t set = __ballot((key & b) != 0);
                same &= (key & b) ? set : ~set;
            }
            if (own) {
                const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
                const int32_t from = mine[key], to = from + rank;
                a.order[to] = static_cast<int32_t>(t + 64 * k + lane);
                if (to % EG_PIECE == 0) a.piece_row[to / EG_PIECE] = row[k];
                if (rank == 0) mine[key] = from + __popcll(same);
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---- the sums -------------------------------------------------------------------
// A row of up to EG_PIECE tokens is summed by one wave (or, where a row has few
// columns, by LPR lanes of one).  The tokens of longer rows are summed piece by
// piece and their sums joined by k_embed_join: a row that is longer than a piece
// and lies in it starts at or before the piece's first token, or else reaches
// past its last, so a piece has at most two such rows, and two places for sums.

// The columns of a lane: a vector of V from `col` on, of which the first `skip`
// belong to the lane before (the last lane of a row whose columns are no
// multiple of V); n > 0: a row of n < V columns.
struct Cols {
    int64_t col;
    int skip, n;
    bool any;
};

template <int V>
__device__ __forceinline__ Cols cols_of(int64_t at, int64_t cols) {
    Cols c;
    c.any = at < cols;
    c.n = cols < V ? static_cast<int>(cols) : 0;
    c.col = c.n || at + V <= cols ? at : cols - V;
    c.skip = static_cast<int>(at - c.col);
    return c;
}

// (left as they are in memory, so that nothing waits for them before their use)
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_cols(const T *row, const Cols &c) {
    if (!c.n) return load_v<true, T, V>(row + c.col);
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = k < c.n ? load_1(row + k) : 0.0f;
    return pack<T, V>(v);
}

// grad's columns of a lane from their sums.
template <typename U, int V>
__device__ __forceinline__ void finish(const EgSumArgs &a, int64_t row, const Cols &c,
                                       float (&s)[V]) {
    if (!c.any) return;
    U *g = static_cast<U *>(a.grad) + row * a.ldg;
    Raw<U, V> old;
    if (a.add) old = load_cols<U, V>(g, c);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        s[k] *= a.mul;
        if (a.add) s[k] += elem<U, V>(old, k);
    }
    if (!c.n && !c.skip) {
        store_v<true, U, V>(g + c.col, pack<U, V>(s));
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (c.n ? k < c.n : k >= c.skip) store_1(g + c.col + k, from_f32<U>(s[k]));
    }
}

template <typename T, int LPR>
struct EgShape {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int SUB = 64 / LPR;                // rows of a wave at once
    static constexpr int GROUP = LPR > 8 ? 8 : LPR - 1; // rows of LPR lanes, one after another
    static constexpr int FLY = LPR > 8 ? 8 : LPR;       // tokens in flight
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

template <typename T, typename U, int LPR>
__global__ __launch_bounds__(EM_BLOCK) void k_embed_sum(const EgSumArgs a) {
    using S = EgShape<T, LPR>;
    constexpr int V = S::V, FLY = S::FLY;
    const int lane = threadIdx.x & 63, l = lane % LPR;
    const int64_t slabs = S::slabs(a.cols);
    const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t wave = block * EM_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t g = wave * S::SUB + (LPR == 64 ? 0 : lane / LPR);
    const int64_t unit = g / slabs, slab = g % slabs;
    const Cols c = cols_of<V>((slab * LPR + l) * V, a.cols);
    const T *dy = static_cast<const T *>(a.dy);

    // s += the tokens first .. end - 1 of the order
    auto sum = [&](int32_t first, int32_t end, float (&s)[V]) {
        for (int32_t at = first; at < end; at += LPR) {
            int32_t have = 0;
            if (at + l < end) have = a.order[at + l];
            const int n = end - at < LPR ? end - at : LPR;
            for (int j = 0; j < n; j += FLY) {
                Raw<T, V> v[FLY];
#pragma unroll
                for (int k = 0; k < FLY; ++k) {
                    const int64_t t = take<LPR>(have, j + k < LPR ? j + k : 0);
                    if (j + k < n && c.any) v[k] = load_cols<T, V>(dy + t * a.ldy, c);
                }
#pragma unroll
                for (int k = 0; k < FLY; ++k)
                    if (j + k < n)
#pragma unroll
                        for (int e = 0; e < V; ++e) s[e] += elem<T, V>(v[k], e);
            }
        }
    };
    auto uniform = [](int32_t v) {
        return LPR == 64 ? __builtin_amdgcn_readfirstlane(v) : v;
    };

    if (unit < a.pieces) {
        const int32_t total = uniform(a.start[a.rows]);
        const int64_t from = unit * EG_PIECE;
        if (from >= total) return;
        const int32_t begin = static_cast<int32_t>(from);
        const int32_t stop = total - begin < EG_PIECE ? total : begin + EG_PIECE;
        const int32_t head = uniform(a.piece_row[unit]);
        const int32_t h0 = uniform(a.start[head]), h1 = uniform(a.start[head + 1]);
        const int64_t place = (unit * 2 * slabs + slab) * (LPR * V) + l * V;
        if (h1 - h0 > EG_PIECE) {
            float s[V] = {};
            sum(begin, h1 < stop ? h1 : stop, s);
            store_v<false, float, V>(a.part + place, pack<float, V>(s));
        }
        if (stop < total) {
            const int32_t tail = uniform(a.piece_row[unit + 1]);
            const int32_t t0 = uniform(a.start[tail]), t1 = uniform(a.start[tail + 1]);
            if (tail != head && t0 < stop && t1 - t0 > EG_PIECE) {
                float s[V] = {};
                sum(t0, stop, s);
                store_v<false, float, V>(a.part + place + slabs * (LPR * V), pack<float, V>(s));
            }
        }
        return;
    }
    const int64_t row0 = (unit - a.pieces) * S::GROUP;
    if (row0 >= a.rows) return;
    const int rows = static_cast<int>(a.rows - row0 < S::GROUP ? a.rows - row0 : S::GROUP);
    const int32_t starts = a.start[row0 + (l < rows ? l : rows)];
    for (int r = 0; r < rows; ++r) {
        const int32_t first = take<LPR>(starts, r), end = take<LPR>(starts, r + 1);
        if (end - first > EG_PIECE || (a.add && first == end)) continue;
        float s[V] = {};
        sum(first, end, s);
        finish<U, V>(a, row0 + r, c, s);
    }
}

// The sums of a long row's pieces, added in their order: a quarter of them by
// each wave, then the quarters.  Work group b looks at the pieces b, b + grid,
// ..., a lane at each, for those in which a long row starts.
template <typename T, typename U, int LPR>
__global__ __launch_bounds__(EM_BLOCK) void k_embed_join(const EgSumArgs a) {
    using S = EgShape<T, LPR>;
    constexpr int V = S::V;
    constexpr int FLY = 4;
    __shared__ float sh[EM_WAVES][V][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t slabs = S::slabs(a.cols);
    const int64_t slab = blockIdx.y;
    const int32_t total = a.start[a.rows];
    const int64_t pieces = (static_cast<int64_t>(total) + EG_PIECE - 1) / EG_PIECE;
    const Cols c = cols_of<V>((slab * LPR + lane) * V, lane < LPR ? a.cols : 0);
    for (int64_t p0 = blockIdx.x; p0 < pieces; p0 += static_cast<int64_t>(gridDim.x) * 64) {
        // the long row that starts in this lane's piece: its first piece's
        // first token, or the one that the next piece starts with
        const int64_t p = p0 + static_cast<int64_t>(gridDim.x) * lane;
        int32_t row = -1;
        if (p < pieces) {
            int32_t r = a.piece_row[p];
            if (a.start[r] < p * EG_PIECE) r = p + 1 < pieces ? a.piece_row[p + 1] : -1;
            else if (a.start[r + 1] - a.start[r] <= EG_PIECE && p + 1 < pieces) r = a.piece_row[p + 1];
            if (r >= 0 && a.start[r] >= p * EG_PIECE && a.start[r] < (p + 1) * EG_PIECE &&
                a.start[r + 1] - a.start[r] > EG_PIECE)
                row = r;
        }
        uint64_t found = __ballot(row >= 0);
        while (found) {
            const int from = __ffsll(static_cast<unsigned long long>(found)) - 1;
            found &= found - 1;
            const int32_t r = __builtin_amdgcn_readlane(row, from);
            const int32_t s0 = __builtin_amdgcn_readfirstlane(a.start[r]);
            const int32_t s1 = __builtin_amdgcn_readfirstlane(a.start[r + 1]);
            const int32_t first = s0 / EG_PIECE, n = (s1 - 1) / EG_PIECE - first + 1;
            const int32_t lo = static_cast<int32_t>(static_cast<int64_t>(n) * w / EM_WAVES);
            const int32_t hi = static_cast<int32_t>(static_cast<int64_t>(n) * (w + 1) / EM_WAVES);
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
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int q = 1; q < EM_WAVES; ++q) s[e] += sh[q][e][lane];
                finish<U, V>(a, r, c, s);
            }
            __syncthreads();
        }
    }
}

int groups(int64_t waves) {
    const int64_t g = (waves + EM_WAVES - 1) / EM_WAVES;
    return static_cast<int>(g < 1 << 20 ? g : 1 << 20);
}

template <typename T>
hipError_t embed_from(const EmArgs &a, gq_dtype out_dt, hipStream_t s) {
    constexpr int64_t slab = 64 * 16 / sizeof(T);
    const int grid = groups(a.T * ((a.cols + slab - 1) / slab));
    if (out_dt == GQ_F32) k_embed<T, float><<<grid, EM_BLOCK, 0, s>>>(a);
    else if (out_dt == GQ_F16) k_embed<T, __half><<<grid, EM_BLOCK, 0, s>>>(a);
    else k_embed<T, bf16_t><<<grid, EM_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, typename U, int LPR>
hipError_t sum_as(const EgSumArgs &a, bool join, hipStream_t s) {
    using S = EgShape<T, LPR>;
    const int64_t slabs = S::slabs(a.cols);
    if (join) {
        const dim3 grid(static_cast<uint32_t>(a.pieces < 256 ? a.pieces : 256),
                        static_cast<uint32_t>(slabs));
        k_embed_join<T, U, LPR><<<grid, EM_BLOCK, 0, s>>>(a);
    } else {
        const int64_t units = a.pieces + (a.rows + S::GROUP - 1) / S::GROUP;
        constexpr int64_t per = S::SUB * EM_WAVES;
        const int64_t blocks = (units * slabs + per - 1) / per;
        // (a grid's side has less than 2^32 work-items)
        const int64_t x = blocks < 1 << 20 ? blocks : 1 << 20;
        const dim3 grid(static_cast<uint32_t>(x), static_cast<uint32_t>((blocks + x - 1) / x));
        k_embed_sum<T, U, LPR><<<grid, EM_BLOCK, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T, typename U>
hipError_t sum_into(const EgSumArgs &a, bool join, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.cols <= 4 * V) return sum_as<T, U, 4>(a, join, s);
    if (a.cols <= 16 * V) return sum_as<T, U, 16>(a, join, s);
    return sum_as<T, U, 64>(a, join, s);
}

template <typename T>
hipError_t sum_from(const EgSumArgs &a, gq_dtype out_dt, bool join, hipStream_t s) {
    if (out_dt == GQ_F32) return sum_into<T, float>(a, join, s);
    if (out_dt == GQ_F16) return sum_into<T, __half>(a, join, s);
    return sum_into<T, bf16_t>(a, join, s);
}

hipError_t sum_any(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, bool join, hipStream_t s) {
    if (dt == GQ_F32) return sum_from<float>(a, out_dt, join, s);
    if (dt == GQ_F16) return sum_from<__half>(a, out_dt, join, s);
    return sum_from<bf16_t>(a, out_dt, join, s);
}

}  // namespace

hipError_t launch_embed(const EmArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    if (dt == GQ_F32) return embed_from<float>(a, out_dt, s);
    if (dt == GQ_F16) return embed_from<__half>(a, out_dt, s);
    return embed_from<bf16_t>(a, out_dt, s);
}

hipError_t launch_embed_sort(const EgSortArgs &a, hipStream_t s) {
    const int64_t grid = (a.rows + a.rows_per - 1) / a.rows_per;
    const size_t lds = sizeof(int32_t) * (EG_SORT_BLOCK / 64) * a.rows_per;
    k_embed_sort<<<static_cast<uint32_t>(grid), EG_SORT_BLOCK, lds, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_embed_sum(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    return sum_any(a, dt, out_dt, false, s);
}

hipError_t launch_embed_join(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s) {
    return sum_any(a, dt, out_dt, true, s);
}

}  // namespace gq
