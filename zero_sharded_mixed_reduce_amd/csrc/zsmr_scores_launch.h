// Internal interface between the host code of the scores of logits
// (zsmr_scores_api.cpp) and their gfx950 kernels.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace zsmr {

struct ScoreArgs {
    const void* logits;
    int64_t stride;
    int32_t dtype, id_bytes, top, top_bytes;
    const void* ids;                // or NULL
    int64_t tokens, vocab;
    float scale;
    float *logprob, *lse, *entropy; // lse and entropy: inputs of the gradient; any may be NULL otherwise
    void* top_ids;
    float* top_logprobs;
    // gradient
    const float *dlogprob, *dentropy;
    void* dlogits;
    int64_t dstride;
};
hipError_t launch_logprobs(const ScoreArgs& a, void* ws, hipStream_t stream);
hipError_t launch_logprobs_grad(const ScoreArgs& a, hipStream_t stream);

}  // namespace zsmr
