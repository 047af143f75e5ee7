// gq_ortho.h -- types shared by the host side (gq_ortho.cpp) and the kernels
// (gq_ortho.hip) of the orthogonalised update.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

namespace gq {

// One matrix of a plan.  X is the matrix itself or, where it has more rows
// than columns, its transpose: s x l with s <= l, padded with zeros to
// sp x lp (multiples of the plan's tile).  Offsets are fp16 elements of the
// plan's workspace.  X is the sum of two numbers: x, in fp16, which the products
// read, held twice, read and written in turn; and y, most of what x leaves of
// it, in 8 bits (gq_ortho.hip), which only the tile's own work group reads and
// writes.
struct OrMat {
    int64_t off;        // first element in the flat gradient, momentum and output
    int64_t x[2];       // [sp][lp]
    int64_t a;          // [sp][sp]
    int64_t b;          // [sp][sp]
    int64_t low;        // bytes: y, [tiles of X][tile * tile], a tile as or_quad orders it
    int64_t diag;       // floats: the diagonals of G and of Q, sp each
    int64_t chunk;      // elements (a multiple of 4) per partial sum of squares
    int32_t rows, cols;
    int32_t s, l, sp, lp;
    int32_t tr;         // X is the transpose
    int32_t part;       // first partial sum of squares, and how many
    int32_t parts;
    float scale;        // X is stored times this power of two
    float out_mul;
    int32_t align;      // elements that the rows start at multiples of: 8, 4 or 1
};

// A tile of a launch (mat < 0: none, it only keeps the order of the XCDs).
struct OrTile {
    int32_t mat, i, j;
    // G = X X^T: the tile's share of K, in units of 128 columns of X, and where
    // its partial sums go (part < 0: the whole sum is the tile).  Joining:
    // the first of the tile's partial sums and, in count, how many.
    int32_t part, first, count;
};

struct OrArgs {
    const OrMat *mats;
    const OrTile *tiles;
    _Float16 *ws;
    double *part;
    float *sums;        // partial sums of tiles of G, tile * tile floats each
    float *diag;
    uint8_t *low;
    const void *g;
    float *m;           // NULL: no momentum
    void *out;
    float in_mul, mu, eps;
    float a, b, c;      // the step's coefficients
    int32_t nesterov;
    int32_t cur;        // which of x[] is read
    int32_t tile_x;     // of X
    int32_t low_in;     // whether the X that is read has a y, and the one written
    int32_t low_out;
};

// The coefficients (a, b, c) of every step.
struct OrSteps {
    float coef[3 * GQ_ORTHO_MAX_STEPS];
    int32_t steps;
};

enum OrTable { OR_NORM = 0, OR_CAST = 1, OR_GRAM = 2, OR_JOIN = 3, OR_POLY = 4, OR_X = 5, OR_TABLES = 6 };
enum OrMode {
    OR_MM_GRAM = 0, OR_MM_POLY = 1, OR_MM_STEP = 2, OR_MM_LAST = 3, OR_MM_LAST_BF16 = 4, OR_MM_JOIN = 5
};

constexpr int OR_CAST_TILE = 64;
// X has a y while at least this many steps are to come.
constexpr int OR_LOW_STEPS = 3;

hipError_t launch_ortho_norm(const OrArgs &a, int64_t n, gq_dtype dt, hipStream_t s);
hipError_t launch_ortho_cast(const OrArgs &a, int64_t n, gq_dtype dt, hipStream_t s);
// n matrices with s <= OR_SMALL_S and l <= OR_SMALL_L, one work group each.
constexpr int OR_SMALL_S = 64, OR_SMALL_L = 256;
hipError_t launch_ortho_small(const OrArgs &a, const OrSteps &st, int64_t n, gq_dtype dt,
                              gq_dtype out, hipStream_t s);
hipError_t launch_ortho_mm(const OrArgs &a, int64_t n, int tile, OrMode mode, gq_dtype out,
                           hipStream_t s);

}  // namespace gq
