// vocab_back.cuh -- the interface of the loss's gradient for narrow rows.
#pragma once

#include "product.cuh"

namespace so {

constexpr int64_t kBackCols = 128;   // columns at most

struct BackArgs {
    int32_t n, c, v;
    const float4* tokens;    // see TokenRows
    void *dx, *dw;           // results, or fp32 slabs where there are several parts; nullptr: not wanted
    int32_t dx_splits, dw_splits, out_bf16;
    int32_t release;         // writes slabs only
    const float* unit;       // bf16: what results are multiplied by (see common_unit)
    int32_t dx_items, dw_items;   // filled in by loss_back
    int32_t* d_err;
};

struct BackPlan {
    int dx_splits, dw_splits;
    int64_t tokens;          // entries of the tokens' array
};

BackPlan back_plan(bool f32, int64_t n, int64_t c, int64_t v);
cudaError_t loss_back(const CUtensorMap& x, const CUtensorMap& w, bool f32, BackArgs Q, cudaStream_t s);

}  // namespace so
