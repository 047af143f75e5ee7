// gq_tensors.h -- argument blocks and launchers of the tensor list's kernels.
// Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

namespace gq {

// A list's tensors are cut into tiles of this many elements, one wave's work;
// a tensor's last tile is shorter.  Tiles are counted in elements, not bytes,
// so that two lists of the same lengths have the same tiles whatever their types.
constexpr int TN_TILE = 4096;
constexpr int TN_BLOCK = 256;
constexpr int TN_MAX_GRID = 2048;       // work groups of the norm, a partial sum each

struct TnTile {
    char *p;                            // its first element
    uint32_t n;                         // elements, 1 .. TN_TILE
    uint32_t dt;                        // gq_dtype
};

struct TnNormArgs {
    const TnTile *tiles;
    int64_t n_tiles;
    double *parts;                      // [grid] sums of squares
    double *tile_sums;                  // NULL, or [n_tiles] sums of squares
    uint32_t *ticket;                   // 0 between calls
    float *norm;
    float in_mul;
};

struct TnEachArgs {
    const int64_t *first;               // [count + 1] first tile of each tensor
    const double *tile_sums;
    float *norms;
    int64_t count;
    float in_mul;
};

struct TnClipArgs {
    const TnTile *x, *y;                // y == x: in place
    int64_t n_tiles;
    const float *norm;
    float max_norm, eps, in_mul;
};

hipError_t launch_tensors_norm(const TnNormArgs &a, hipStream_t s);
hipError_t launch_tensors_each(const TnEachArgs &a, hipStream_t s);
hipError_t launch_tensors_clip(const TnClipArgs &a, hipStream_t s);

}  // namespace gq
