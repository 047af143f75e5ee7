// gq_mx4.h -- the microscaled 4-bit format (MX4) on gfx950, shared by the
// kernels that write and read it, and the argument blocks of its launchers.
// Not part of the ABI.
//
// A block is 32 consecutive elements of a row: one scale byte s standing for
// 2^(s - 127), and 16 bytes of codes, element 2i in the low half of byte i.
// A code is a sign bit over a magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
// Quantizing (max|g| = M over the block):
//   s    = max(0, floor(log2 M) - 2 + 127), from M's exponent field; 0 for
//          M = 0; 255 (NaN) when the block holds inf or NaN, codes then 0;
//   code = g * 2^(127 - s), an exact product except where it underflows to
//          values far below 0.25, rounded half to even to a magnitude, above
//          6 to 6 (the products are below 8); the sign is kept, of zeros too.
// The conversions in both directions are the gfx950 instructions.
// tests/test_gpu_mx4_conversions.py compares them with this definition for
// every code at every scale byte, every binary32 magnitude below 8 at the
// scale 1, and the ends of the rounding intervals with their neighbours at
// every scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

namespace gq {

constexpr int MX_BLOCK = 32;     // elements per scale
constexpr int MX_BYTES = 16;     // code bytes per block

struct MxQArgs {
    const void *x[GQ_MAX_RANKS];
    uint8_t *scale[GQ_MAX_RANKS];
    uint8_t *q[GQ_MAX_RANKS];
    int64_t rows;               // of x
    int64_t cols;
    int64_t ld;                 // elements between the rows of x
    int64_t nb;                 // blocks per row of codes
    float in_mul;
    int32_t W;
};

struct MxRArgs {
    const uint8_t *q[GQ_MAX_RANKS];
    const uint8_t *scale[GQ_MAX_RANKS];
    float *r;                   // NULL or [rows][cols]
    uint8_t *scale_out;         // NULL or [rows][nb]
    uint8_t *q_out;             // NULL or [rows][nb][16]
    int64_t rows;
    int64_t cols;
    int64_t nb;
    int32_t W;
};

hipError_t launch_mx4_quantize(const MxQArgs &a, gq_dtype dt, bool transpose, hipStream_t s);
hipError_t launch_mx4_reduce(const MxRArgs &a, hipStream_t s);

namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte of a block whose largest magnitude has the bit pattern m.
__device__ __forceinline__ uint32_t mx_byte(uint32_t m) {
    if (m >= kInfBits) return 255u;
    const uint32_t f = m >> 23;
    return f > 2u ? f - 2u : 0u;
}

// 2^(127 - s): what an element is multiplied by before it is coded.  0 for
// a NaN block (the caller clears its codes).
__device__ __forceinline__ float mx_mult(uint32_t s) {
    return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx_two(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// Two values below 8 in magnitude to codes in byte B of `old`.
template <int B>
__device__ __forceinline__ uint32_t mx_code2(uint32_t old, float a, float b) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, 1.0f, B);
}

// The two values that byte B of w stands for, before the block's scale.
typedef float f32x2_t __attribute__((ext_vector_type(2)));
template <int B>
__device__ __forceinline__ f32x2_t mx_value2(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
}

}  // namespace
}  // namespace gq
