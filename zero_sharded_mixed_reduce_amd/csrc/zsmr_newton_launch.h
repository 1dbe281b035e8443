// Internal interface between the host code of the orthogonalised update
// (zsmr_newton_api.cpp) and its gfx950 kernels.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "zsmr_launch.h"
#include "zsmr_newton_plan.h"

namespace zsmr {

struct NewtonArgs {
    NsShape shape;
    NsPass pass[ZSMR_MAX_NS_STEPS];     // of a matrix that stays in LDS
    int32_t steps;
    double eps, first;                  // first: the power of two of the first X
    // the matrices, in their own orientation (orthogonalise)
    const void* x;
    int64_t x_stride, x_batch;
    int32_t x_dtype;
    void* out;
    int64_t out_stride, out_batch;
    int32_t out_dtype;
    // the shard step: matrices one behind the other from each pointer on
    StepArgs step;                      // grads, row_stride, nrows, mean, nf, inv_nf, inv_pow2, master, m, p16
    int32_t grad_dtype, param_dtype, nesterov;
    float beta, decay, rate;            // decay: 1 - lr * weight_decay; rate: lr * scale
};
// ops: the products, of matrices that do not
hipError_t launch_orthogonalize(const NewtonArgs& a, const NsOp* ops, int n_ops, void* ws, hipStream_t stream);
hipError_t launch_muon(const NewtonArgs& a, const NsOp* ops, int n_ops, void* ws, hipStream_t stream);

}  // namespace zsmr
