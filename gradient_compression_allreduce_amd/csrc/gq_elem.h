// gq_elem.h -- elements of fp32, fp16 and bfloat16 in device code: vectors of
// them at any element's address, and their conversions to and from binary32.
// Shared by the tensor list and embedding kernels.  Not part of the ABI.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {
namespace {

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v.bits) << 16);
}

// Rounded half to even; a NaN stays one.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    // (keeps the compiler from joining the product that v may be with the
    // conversion, in an instruction that does not round to binary32 between them)
    asm("" : "+v"(v));
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
    const __bf16 b = static_cast<__bf16>(v);
    bf16_t r;
    __builtin_memcpy(&r, &b, 2);
    return r;
}

// V elements as they are in memory, in words (one of 16 bits in a word's lower half).
template <typename T, int V>
struct Raw {
    static constexpr int W = V * sizeof(T) < 4 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[W];
};

typedef unsigned int elem_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int elem_u32x2 __attribute__((ext_vector_type(2)));
// In device memory, at any element.  (Addresses that a kernel reads from memory
// are generic to the compiler, which would access them with slower flat
// instructions; all of these are of device memory.)
typedef elem_u32x4 __attribute__((aligned(2), address_space(1))) elem_u32x4_any;
typedef elem_u32x2 __attribute__((aligned(2), address_space(1))) elem_u32x2_any;

typedef uint32_t __attribute__((address_space(1))) elem_u32;
typedef uint16_t __attribute__((address_space(1))) elem_u16;

// NT: with the non-temporal hint, for what is read or written once.
template <bool NT, typename T, int V>
__device__ __forceinline__ Raw<T, V> load_v(const T *p) {
    Raw<T, V> r;
    static_assert(V == 1 || Raw<T, V>::W == 2 || Raw<T, V>::W % 4 == 0, "1, 8 bytes, or 16 n");
    if constexpr (V == 1 && sizeof(T) == 4) {
        r.w[0] = *(const elem_u32 *)p;
    } else if constexpr (V == 1) {
        r.w[0] = *(const elem_u16 *)p;
    } else if constexpr (Raw<T, V>::W == 2) {
        const elem_u32x2_any *q = (const elem_u32x2_any *)p;
        const elem_u32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
        r.w[0] = v[0];
        r.w[1] = v[1];
    } else {
#pragma unroll
        for (int k = 0; k < Raw<T, V>::W / 4; ++k) {
            const elem_u32x4_any *q = (const elem_u32x4_any *)p + k;
            const elem_u32x4 v = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[4 * k + j] = v[j];
        }
    }
    return r;
}

template <bool NT, typename T, int V>
__device__ __forceinline__ void store_v(T *p, const Raw<T, V> &r) {
    if constexpr (V == 1 && sizeof(T) == 4) {
        *(elem_u32 *)p = r.w[0];
    } else if constexpr (V == 1) {
        *(elem_u16 *)p = static_cast<uint16_t>(r.w[0]);
    } else if constexpr (Raw<T, V>::W == 2) {
        elem_u32x2_any *q = (elem_u32x2_any *)p;
        const elem_u32x2 v = {r.w[0], r.w[1]};
        if (NT) __builtin_nontemporal_store(v, q);
        else *q = v;
    } else {
#pragma unroll
        for (int k = 0; k < Raw<T, V>::W / 4; ++k) {
            elem_u32x4_any *q = (elem_u32x4_any *)p + k;
            const elem_u32x4 v = {r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]};
            if (NT) __builtin_nontemporal_store(v, q);
            else *q = v;
        }
    }
}

// Element k of a vector.
template <typename T, int V>
__device__ __forceinline__ float elem(const Raw<T, V> &r, int k) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(r.w[k]);
    } else {
        const uint16_t b = static_cast<uint16_t>((k & 1) ? r.w[k >> 1] >> 16 : r.w[k >> 1]);
        T t;
        __builtin_memcpy(&t, &b, 2);
        return to_f32(t);
    }
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float (&f)[V]) {
    Raw<T, V> r;
    if constexpr (V == 1 && sizeof(T) == 2) {
        const T a = from_f32<T>(f[0]);
        uint16_t x;
        __builtin_memcpy(&x, &a, 2);
        r.w[0] = x;
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) r.w[k] = __float_as_uint(f[k]);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const T a = from_f32<T>(f[k]), b = from_f32<T>(f[k + 1]);
            uint16_t x, y;
            __builtin_memcpy(&x, &a, 2);
            __builtin_memcpy(&y, &b, 2);
            r.w[k / 2] = x | static_cast<uint32_t>(y) << 16;
        }
    }
    return r;
}

// One element.
template <typename T>
__device__ __forceinline__ float load_1(const T *p) {
    return elem<T, 1>(load_v<false, T, 1>(p), 0);
}

template <typename T>
__device__ __forceinline__ void store_1(T *p, float v) {
    const float f[1] = {v};
    store_v<false, T, 1>(p, pack<T, 1>(f));
}

}  // namespace
}  // namespace gq
