// gq_tensors.hip -- gfx950 kernels over a list of tensors:
//   k_tensors_norm  the 2-norm of all of them together and, where each tensor's
//                   norm is asked for, those of tensors of one tile and the
//                   others' tiles' sums of squares;
//   k_tensors_each  the norms of tensors of several tiles from their sums;
//   k_tensors_clip  x * in_mul * min(1, max_norm / (norm + eps)).
// All of it is bound by HBM: one operation or two per element.
// Squares and their sums are binary64 (the square of a binary32 value is exact
// there and neither overflows nor underflows; the vector units do 64-bit
// multiply-adds faster than HBM delivers elements).
#include "gq_elem.h"
#include "gq_tensors.h"

namespace gq {
namespace {

constexpr int TN_WAVES = TN_BLOCK / 64;
constexpr int TN_NWAVES = TN_NORM_BLOCK / 64;
constexpr int TN_GROUP = 8;         // vectors of a lane in flight in the norm
constexpr int TN_PARTS = 4;         // parts of a tile that the clip takes one by one

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Tile t, the same for all lanes of a wave.
__device__ __forceinline__ TnTile tile_at(const TnTile *tiles, int64_t t) {
    TnTile v = tiles[t];
    const uint64_t p = reinterpret_cast<uint64_t>(v.p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
    v.p = reinterpret_cast<char *>(static_cast<uint64_t>(hi) << 32 | lo);
    v.n_dt = __builtin_amdgcn_readfirstlane(v.n_dt);
    v.only = __builtin_amdgcn_readfirstlane(v.only);
    return v;
}

// This lane's part of the sum of squares of n elements.  Whole tiles are
// loaded whole before the first square, shorter ones in groups of TN_GROUP
// vectors a lane (those past the end are the last one again, and are not
// added); what is left is less than a vector, an element a lane.
template <bool NT, typename T>
__device__ __forceinline__ double squares(const T *p, int n) {
    constexpr int V = 16 / sizeof(T);
    constexpr int S = TN_TILE / V / 64;
    const int lane = threadIdx.x & 63;
    double s0 = 0.0, s1 = 0.0;
    auto add = [&](const Raw<T, V> &r, bool in) {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const double a = in ? elem<T, V>(r, k) : 0.0f, b = in ? elem<T, V>(r, k + 1) : 0.0f;
            s0 = __builtin_fma(a, a, s0);
            s1 = __builtin_fma(b, b, s1);
        }
    };
    if (n == TN_TILE) {
        Raw<T, V> r[S];
#pragma unroll
        for (int s = 0; s < S; ++s) r[s] = load_v<NT, T, V>(p + (s * 64 + lane) * V);
#pragma unroll
        for (int s = 0; s < S; ++s) add(r[s], true);
    } else {
        const int full = n / V, rest = full * V + lane;
        const float last = rest < n ? load_1(p + rest) : 0.0f;
        for (int at = 0; at < full; at += TN_GROUP * 64) {
            Raw<T, V> r[TN_GROUP];
#pragma unroll
            for (int g = 0; g < TN_GROUP; ++g) {
                const int s = at + g * 64 + lane;
                r[g] = load_v<NT, T, V>(p + (s < full ? s : full - 1) * V);
            }
#pragma unroll
            for (int g = 0; g < TN_GROUP; ++g) add(r[g], at + g * 64 + lane < full);
        }
        const double a = last;
        s0 = __builtin_fma(a, a, s0);
    }
    return s0 + s1;
}

__device__ __forceinline__ float norm_of(double sum, float in_mul) {
    return static_cast<float>(static_cast<double>(in_mul) * sqrt(sum));
}

// A wave takes every (waves of the grid)-th tile.  Each work group leaves one
// sum; the last one to finish adds them in their order, so that equal calls
// give equal bits.  335M fp16: 102 us, 6.6 TB/s; 10000 tensors of up to 4096 fp32
// with each one's norm 18.7 us, 4.4 TB/s (a wave takes two or three, each a chain of
// two loads); 2^20 fp32 5.2 us, latency: launch, table, elements, sum and ticket.
template <bool EACH, bool NT>
__global__ __launch_bounds__(TN_NORM_BLOCK) void k_tensors_norm(const TnNormArgs a) {
    __shared__ double sh[TN_NWAVES];
    __shared__ uint32_t done;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    double sum = 0.0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * TN_NWAVES + wave; t < a.n_tiles;
         t += static_cast<int64_t>(gridDim.x) * TN_NWAVES) {
        const TnTile v = tile_at(a.tiles, t);
        const int n = v.n_dt & 0xffff, dt = v.n_dt >> 16;
        double s;
        if (dt == GQ_F32) s = squares<NT>(reinterpret_cast<const float *>(v.p), n);
        else if (dt == GQ_F16) s = squares<NT>(reinterpret_cast<const __half *>(v.p), n);
        else s = squares<NT>(reinterpret_cast<const bf16_t *>(v.p), n);
        if (EACH) {
            s = wave_sum(s);
            if (lane == 0) {
                if (v.only >= 0) a.norms[v.only] = norm_of(s, a.in_mul);
                else a.tile_sums[t] = s;
            }
        }
        sum += s;
    }
    if (!EACH) sum = wave_sum(sum);
    if (lane == 0) sh[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = sh[0];
#pragma unroll
        for (int w = 1; w < TN_NWAVES; ++w) s += sh[w];
        // The sum is on its way past this XCD's L2 cache (agent scope); once it
        // has arrived the ticket may say so.  (An acquire-release ticket would
        // write back and invalidate that cache in every work group: 112 us
        // instead of 38 for 10000 tensors, 82 MB.)
        __hip_atomic_store(&a.parts[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        done = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (done != gridDim.x - 1) return;
    sum = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += TN_NORM_BLOCK)
        sum += __hip_atomic_load(&a.parts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = wave_sum(sum);
    if (lane == 0) sh[wave] = sum;      // read by thread 0 before the barrier above
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = sh[0];
#pragma unroll
        for (int w = 1; w < TN_NWAVES; ++w) s += sh[w];
        a.norm[0] = norm_of(s, a.in_mul);
        __hip_atomic_store(a.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// A wave per tensor of several tiles.
__global__ __launch_bounds__(TN_BLOCK) void k_tensors_each(const TnEachArgs a) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * TN_WAVES + (threadIdx.x >> 6);
    if (i >= a.count) return;
    const int lane = threadIdx.x & 63;
    const TnLong v = a.longs[i];
    double s = 0.0;
    for (int64_t t = v.first + lane; t < v.end; t += 64) s += a.tile_sums[t];
    s = wave_sum(s);
    if (lane == 0) a.norms[v.tensor] = norm_of(s, a.in_mul);
}

// y = x * f, x and y apart or the same memory of one type.  A wave takes a quarter
// of a tile, all of its loads in flight: with as many writes as reads HBM is fastest
// with little of each at once.  60.2M fp32 in place: 77 us, 6.3 TB/s (whole tiles 87,
// halves 79, eighths 75, but 10000 tensors of up to 4096 then 31 instead of 27);
// 335M fp16 into fp32 343 us, 5.9 TB/s; 400M bf16 in place 255 (halves 266).
template <bool NT, typename T, typename U>
__device__ __forceinline__ void scale_part(const T *x, U *y, int n, float f) {
    constexpr int V = sizeof(T) == 4 || sizeof(U) == 4 ? 4 : 8;
    constexpr int G = TN_TILE / TN_PARTS / V / 64;      // vectors of a lane in flight
    const int lane = threadIdx.x & 63;
    const int full = n / V, rest = full * V + lane;
    const float last = rest < n ? load_1(x + rest) : 0.0f;
    if (full > 0) {
        Raw<T, V> r[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {       // (past the end the last one again)
            const int s = g * 64 + lane;
            r[g] = load_v<NT, T, V>(x + (s < full ? s : full - 1) * V);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int s = g * 64 + lane;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = elem<T, V>(r[g], k) * f;
            if (s < full) store_v<NT, U, V>(y + s * V, pack<U, V>(v));
        }
    }
    if (rest < n) store_1(y + rest, last * f);
}

template <bool NT, typename T>
__device__ __forceinline__ void scale_into(const T *x, const TnTile &y, int at, int n, float f) {
    const int dt = y.n_dt >> 16;
    if (dt == GQ_F32) scale_part<NT>(x, reinterpret_cast<float *>(y.p) + at, n, f);
    else if (dt == GQ_F16) scale_part<NT>(x, reinterpret_cast<__half *>(y.p) + at, n, f);
    else scale_part<NT>(x, reinterpret_cast<bf16_t *>(y.p) + at, n, f);
}

template <bool NT>
__global__ __launch_bounds__(TN_BLOCK) void k_tensors_clip(const TnClipArgs a) {
    const double top = static_cast<double>(a.norm[0]) + static_cast<double>(a.eps);
    const double c = top <= a.max_norm ? 1.0 : static_cast<double>(a.max_norm) / top;
    const float f = static_cast<float>(c * static_cast<double>(a.in_mul));
    if (f == 1.0f && a.x == a.y) return;
    const int wave = threadIdx.x >> 6;
    constexpr int PART = TN_TILE / TN_PARTS;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * TN_WAVES + wave; t < a.n_tiles * TN_PARTS;
         t += static_cast<int64_t>(gridDim.x) * TN_WAVES) {
        const TnTile v = tile_at(a.x, t / TN_PARTS), y = tile_at(a.y, t / TN_PARTS);
        const int at = static_cast<int>(t % TN_PARTS) * PART, dt = v.n_dt >> 16;
        const int left = static_cast<int>(v.n_dt & 0xffff) - at, n = left < PART ? left : PART;
        if (n <= 0) continue;
        if (dt == GQ_F32) scale_into<NT>(reinterpret_cast<const float *>(v.p) + at, y, at, n, f);
        else if (dt == GQ_F16) scale_into<NT>(reinterpret_cast<const __half *>(v.p) + at, y, at, n, f);
        else scale_into<NT>(reinterpret_cast<const bf16_t *>(v.p) + at, y, at, n, f);
    }
}

int groups(int64_t waves, int per, int64_t most) {
    const int64_t g = (waves + per - 1) / per;
    return static_cast<int>(g < 1 ? 1 : g < most ? g : most);
}

}  // namespace

hipError_t launch_tensors_norm(const TnNormArgs &a, hipStream_t s) {
    const int grid = groups(a.n_tiles, TN_NWAVES, TN_MAX_GRID);
    if (a.norms && a.once) k_tensors_norm<true, true><<<grid, TN_NORM_BLOCK, 0, s>>>(a);
    else if (a.norms) k_tensors_norm<true, false><<<grid, TN_NORM_BLOCK, 0, s>>>(a);
    else if (a.once) k_tensors_norm<false, true><<<grid, TN_NORM_BLOCK, 0, s>>>(a);
    else k_tensors_norm<false, false><<<grid, TN_NORM_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_tensors_each(const TnEachArgs &a, hipStream_t s) {
    k_tensors_each<<<groups(a.count, TN_WAVES, 1 << 20), TN_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_tensors_clip(const TnClipArgs &a, hipStream_t s) {
    if (a.n_tiles == 0) return hipSuccess;
    const int grid = groups(a.n_tiles * TN_PARTS, TN_WAVES, 1 << 20);
    if (a.once) k_tensors_clip<true><<<grid, TN_BLOCK, 0, s>>>(a);
    else k_tensors_clip<false><<<grid, TN_BLOCK, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gq
