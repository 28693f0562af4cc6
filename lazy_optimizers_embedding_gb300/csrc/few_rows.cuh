// few_rows.cuh -- products of few fp32 rows with matrices that the tensor unit could read only after they were packed: the matrices
// are read where they lie, once for 16 rows.
#pragma once

#include "product.cuh"

namespace so {

// Packing a matrix and reading its parts takes 16 bytes a value, a pass over it 4, and a group's every 16 rows are a pass.  So the
// experts' products go this way with at most 64 rows and 16 for an expert on the average (there and back, us, this way and packed: 64 rows
// among 37 experts of 515 x 771 91 and 150, 16 among 100 of 1000 x 1000 147 and 197, 64 among 8 of 2048 x 1024 87 and 134; but 64
// rows of one expert 37 and 16 forward), and a table's scores with at most 16 tokens (1M x 64: 16 tokens 126 and 215, 32 tokens 240 and
// 205).  Their gradient does with at most 8 (this way and by the tensor unit, 1M x 64: 1 token 230 and 617, 8 397 and 619, 16 609 and 617;
// 124271 x 515: 223 and 499, 324 and 427, 480 and 433), bf16 rows of odd sizes, whose packing costs half, do not (8 tokens against
// 100000 x 515 94 and 70).
constexpr int64_t kFewRows = 64, kFewTokens = 16, kFewGrad = 8;
inline bool few_rows(int64_t n, int64_t groups) { return n <= kFewRows && n <= 16 * groups; }

// out[t, m] = sum over k of x[t, k] w[e, m, k]: dot products with the matrices' rows; with targets (one group of few tokens) their running
// sums, where `part` is given, or the slopes of the loss.
struct FewDots {
    const float *x, *w;
    int64_t n, m, k;         // tokens, rows of a matrix, their columns
    int groups;
    const int64_t* offsets;
    float* out;
    const int64_t* target;
    const float *lse, *dloss;   // slopes
    float2* part;            // [few_dot_slots][n]
    float* hit;
    int32_t* d_err;
};
int few_dot_slots(int64_t m);
cudaError_t few_dots(const FewDots& D, cudaStream_t s);

// slabs[s][t, m] = sum over part s of the k of x[t, k] w[e, k, m].
struct FewSums {
    const float *x, *w;
    int64_t n, m, k;
    int groups;
    const int64_t* offsets;
    int splits;
    float* slabs;
    int32_t* d_err;
};
int few_sums_splits(int64_t n, int64_t m, int64_t k, int64_t groups);
cudaError_t few_sums(const FewSums& D, cudaStream_t s);

// out[e, a, b] = sum over group e's rows of x[t, a] y[t, b].
struct FewOuter {
    const float *x, *y;
    int64_t n, a, b;
    int groups;
    const int64_t* offsets;
    float* out;
    const int64_t* target;   // rows of x and y whose target is no row of the result are not looked at (or none)
    int32_t* d_err;
};
cudaError_t few_outer(const FewOuter& D, cudaStream_t s);

}  // namespace so
