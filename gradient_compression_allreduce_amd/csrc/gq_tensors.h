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
// The norm's work groups, each of which leaves a partial sum and takes a ticket.
// The tickets are handed out one after another, so few large groups: 10000
// tensors of up to 4096 fp32 take 39 us in 2048 groups of 256, 29 in 1024, 23 in 512
// of 512; 335M fp16 105, 102 and 103.
constexpr int TN_NORM_BLOCK = 512;
constexpr int TN_MAX_GRID = 512;

// Calls that touch more bytes than this go past the caches (non-temporal); those
// below leave them in the 256 MB behind HBM for the call that follows.  Past the
// caches / through them, fp32 in place: clip of 64 MB 22.6 / 20.5 us, of 240 MB 77 / 87
// where other lists came between; norm and clip of one list in turn, 64 MB 37 / 36,
// 240 MB 116 / 107, 500 MB 233 / 280, 2 GB 939 / 1060.
constexpr int64_t TN_CACHED = int64_t{128} << 20;

struct TnTile {
    char *p;                            // its first element
    uint32_t n_dt;                      // elements, 1 .. TN_TILE, and gq_dtype << 16
    int32_t only;                       // the number of its tensor if that has no other tile, or -1
};

struct TnNormArgs {
    const TnTile *tiles;
    int64_t n_tiles;
    double *parts;                      // [grid] sums of squares
    double *tile_sums;                  // [n_tiles] sums of squares, where norms is given
    uint32_t *ticket;                   // 0 between calls
    float *norm;
    float *norms;                       // NULL, or of each tensor
    float in_mul;
    bool once;                          // past the caches
};

// A tensor of several tiles.
struct TnLong {
    int64_t first, end;                 // its tiles
    int64_t tensor;
};

struct TnEachArgs {
    const TnLong *longs;
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
    bool once;                          // past the caches
};

hipError_t launch_tensors_norm(const TnNormArgs &a, hipStream_t s);
hipError_t launch_tensors_each(const TnEachArgs &a, hipStream_t s);
hipError_t launch_tensors_clip(const TnClipArgs &a, hipStream_t s);

}  // namespace gq
