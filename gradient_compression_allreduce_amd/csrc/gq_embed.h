// gq_embed.h -- argument blocks and launchers of the embedding's kernels.
// Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

namespace gq {

struct EmArgs {
    const void *idx;            // [T], int32 or int64
    const void *table;          // [rows][ld]
    void *out;                  // [T][ldo]
    int64_t T, rows, cols, ld, ldo;
    float mul;
    bool wide;                  // idx is int64
};

constexpr int EG_BLOCK = 1024;          // threads of a work group that orders tokens
constexpr int EG_WAVES = EG_BLOCK / 64;
constexpr int EG_SORT_ROWS = 1024;      // most rows of the table per work group
constexpr int EG_PIECE = 64;            // tokens that one wave sums
// Most tokens of a gradient in one launch: where one token makes up 7 to 25% of them
// the work group that has its row sums them all.  Columns 1000, bf16 into fp32, one
// launch / three: 1024 tokens into 20 rows 20 / 32 us, into 30522, added, 12 / 20;
// 2000 tokens 34 / 35 and 16 / 24; 4000 tokens 68 / 26 and 29 / 27.  (All of 2000 tokens
// of 1024 one token: 121 / 21.)
constexpr int EG_SMALL = 2 * EG_BLOCK;
constexpr int EG_SMALL_ROWS = 128;      // most rows of the table per work group there
constexpr int EG_HELD = 16;             // tokens of a lane in flight
constexpr int EG_ZERO = 8;              // rows that a wave clears
constexpr int EG_KEYS = 256;            // the sort's row numbers come in multiples

// A gradient of up to EG_SMALL tokens.
struct EgSmallArgs {
    const void *idx;
    const void *dy;             // [T][ldy]
    void *grad;                 // [rows][ldg]
    int64_t T, rows, cols, ldy, ldg, skip;
    int32_t rows_per;           // rows of a work group
    float mul;
    bool wide, add;
};

// The order of tokens that a gradient is summed in: the tokens of row 0, those
// of row 1, ...; row r's are order[start[r]] .. order[start[r + 1] - 1].  The
// order is cut into pieces of EG_PIECE tokens; the token that piece p starts
// with is one of row piece_row[p].
struct EgSortArgs {
    const void *idx;
    int64_t T, rows, skip;
    uint32_t *keys;             // NULL, or [round256(T)]
    int32_t *start;             // [rows + 1]
    int32_t *order;             // [T]
    int32_t *piece_row;         // [ceil(T / EG_PIECE)]
    char *grad;                 // NULL, or where rows without a token get 0
    int64_t cols, ldg;
    int32_t elem;               // bytes of grad's elements
    int32_t rows_per;           // rows of a work group
    bool wide;
};

struct EgSumArgs {
    const void *dy;             // [T][ldy]
    void *grad;                 // [rows][ldg]
    const int32_t *start, *order, *piece_row;
    float *part;                // [pieces][2][round512(cols)]
    int64_t rows, cols, ldy, ldg;
    int64_t pieces;
    int64_t zero_blocks, mixed_blocks;  // work groups that clear rows, and of all but pieces
    float mul;
    bool add;
    bool zero;                  // rows without a token get 0
};

hipError_t launch_embed(const EmArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s);
hipError_t launch_embed_grad_small(const EgSmallArgs &a, gq_dtype dt, gq_dtype out_dt,
                                   hipStream_t s);
hipError_t launch_embed_sort(const EgSortArgs &a, hipStream_t s);
hipError_t launch_embed_sum(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s);
hipError_t launch_embed_join(const EgSumArgs &a, gq_dtype dt, gq_dtype out_dt, hipStream_t s);

}  // namespace gq
