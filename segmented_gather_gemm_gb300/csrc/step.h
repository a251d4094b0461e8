// Internal interface of what a decoder does between the projections, the
// attention and the verification (residual and norms, rotary positions,
// appending to the cache, logits to probabilities) between the C-ABI layer
// (step_api.cu) and the kernels.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/csgmv.h"

namespace csgmv {

constexpr int kNormMaxHidden = 16384;

struct NormSide {
    const void *w, *b;  // or NULL
    float eps;
    int kind;
};
struct AddNormParams {
    const void *x, *r, *gate;  // r, gate: or NULL
    void *r_out, *out;         // or NULL
    int64_t x_s, r_s, g_s, ro_s, o_s;  // elements from row to row
    NormSide post, pre;
    float scale;
    int n, hidden;
    int dtype, r_dtype;
};
cudaError_t launch_add_norm(const AddNormParams &p, cudaStream_t stream);

}  // namespace csgmv
