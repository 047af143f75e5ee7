// gq_embed.hip -- gfx950 kernels of the embedding:
//   k_embed       out[t] = mul * table[idx[t]];
//   k_embed_sort  the tokens in the order of their rows;
//   k_embed_sum   grad[v] (+)= mul * the sum of dy over row v's tokens.
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
__global__ __launch_bounds__(EG_SORT_BLOCK) void k_embed_sort(const EgSortArgs a) {
    constexpr int NW = EG_SORT_BLOCK / 64;
    extern __shared__ int32_t count[];          // [NW][rows_per]
    __shared__ int32_t before[NW];
    __shared__ int32_t scan[NW];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int R = a.rows_per;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R;
    const int n_rows = static_cast<int>(a.rows - row0 < R ? a.rows - row0 : R);
    const int64_t per = (a.T + NW * 64 - 1) / (NW * 64) * 64;
    const int64_t t0 = wave * per, t1 = t0 + per < a.T ? t0 + per : a.T;
    for (int i = threadIdx.x; i < NW * R; i += EG_SORT_BLOCK) count[i] = 0;
    __syncthreads();
    int32_t *mine = count + wave * R;
    int32_t less = 0;
    for (int64_t t = t0 + lane; t < t1; t += 64) {
        const int64_t v = index_at(a.idx, a.wide, t);
        if (v < 0 || v >= a.rows || v == a.skip) continue;
        if (v < row0) ++less;
        else if (v < row0 + n_rows) atomicAdd(&mine[v - row0], 1);
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
    for (int64_t t = t0; t < t1; t += 64) {
        int64_t v = -1;
        if (t + lane < t1) v = index_at(a.idx, a.wide, t + lane);
        const bool own = v >= row0 && v < row0 + n_rows && v != a.skip;
        uint64_t same = __ballot(own);
        if (!same) continue;
        const uint32_t key = own ? static_cast<uint32_t>(v - row0) : 0;
        // the lanes whose token names the same row
        for (int b = 1; b < R; b <<= 1) {
            const uint64_t set = __ballot((key & b) != 0);
            same &= (key & b) ? set : ~set;
        }
        if (own) {
            const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
            const int32_t to = mine[key];
            a.order[to + rank] = static_cast<int32_t>(t + lane);
            if (rank == 0) mine[key] = to + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- the sums -------------------------------------------------------------------
// A wave takes 64 vectors of a row of the gradient.
template <typename T, typename U>
__global__ __launch_bounds__(EM_BLOCK) void k_embed_sum(const EgSumArgs a) {
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V);
    const T *dy = static_cast<const T *>(a.dy);
    U *grad = static_cast<U *>(a.grad);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * EM_WAVES + (threadIdx.x >> 6);
         i < a.rows * slabs; i += static_cast<int64_t>(gridDim.x) * EM_WAVES) {
        const int64_t v = i / slabs, col = (i % slabs * 64 + lane) * V;
        const int32_t first = a.start[v], end = a.start[v + 1];
        if (a.add && first == end) continue;
        U *g = grad + v * a.ldg + col;
        float s[V];
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] = 0.0f;
        if (col + V <= a.cols) {
            for (int32_t j = first; j < end; ++j) {
                const Raw<T, V> r = load_v<true, T, V>(dy + a.order[j] * a.ldy + col);
#pragma unroll
                for (int k = 0; k < V; ++k) s[k] += elem<T, V>(r, k);
            }
            Raw<U, V> old;
            if (a.add) old = load_v<true, U, V>(g);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s[k] *= a.mul;
                if (a.add) s[k] += elem<U, V>(old, k);
            }
            store_v<true, U, V>(g, pack<U, V>(s));
        } else {
            for (int k = 0; k < V && col + k < a.cols; ++k) {
                float one = 0.0f;
                for (int32_t j = first; j < end; ++j)
                    one += to_f32(dy[a.order[j] * a.ldy + col + k]);
                one *= a.mul;
                if (a.add) one += to_f32(g[k]);
                g[k] = from_f32<U>(one);
            }
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

template <typename T>
hipError_t sum_from(const EgSumArgs &a, gq_dtype out_dt, hipStream_t s) {
    constexpr int64_t slab = 64 * 16 / sizeof(T);
    const int grid = groups(a.rows * ((a.cols + slab - 1) / slab));
    if (out_dt == GQ_F32) k_embed_sum<T, float><<<grid, EM_BLOCK, 0, s>>>(a);
    else if (out_dt == GQ_F16) k_embed_sum<T, __half><<<grid, EM_BLOCK, 0, s>>>(a);
    else k_embed_sum<T, bf16_t><<<grid, EM_BLOCK, 0, s>>>(a);
    return hipGetLastError();
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
    if (dt == GQ_F32) return sum_from<float>(a, out_dt, s);
    if (dt == GQ_F16) return sum_from<__half>(a, out_dt, s);
    return sum_from<bf16_t>(a, out_dt, s);
}

}  // namespace gq
