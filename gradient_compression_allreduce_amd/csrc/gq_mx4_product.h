// gq_mx4_product.h -- argument block and launcher of the MX4 product.  Not
// part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gq.h"

namespace gq {

constexpr int64_t MX_CUS = 256;   // compute units of an MI355X

struct MxPlan {
    int32_t tile;     // rows and columns of C per work group
    int32_t splits;   // parts of K
    int32_t groups;   // 512 elements of K each, per part
};

struct MxPArgs {
    const uint8_t *a, *sa, *b, *sb;
    void *c;
    float *part;      // NULL, or [splits][m][n] partial sums
    int64_t m, n, nb, ldc;
    int32_t groups;
    int32_t splits;
    int32_t vec;      // four columns of C from a multiple of 4 on are aligned
    int32_t add;
};

// split: K may be split (there is a workspace).
MxPlan mx4_product_plan(int64_t m, int64_t n, int64_t k, bool split);
hipError_t launch_mx4_product(const MxPArgs &a, int64_t k, gq_dtype dt, hipStream_t s);

}  // namespace gq
