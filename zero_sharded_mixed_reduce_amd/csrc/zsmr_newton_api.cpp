// Host side of the orthogonalised update and its shard step, declared in
// include/zsmr_ops.h: every argument is checked here, then the launches of
// zsmr_newton_launch.h go to the caller's stream.  No device memory is allocated
// and nothing is kept between calls.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "zsmr_newton_launch.h"
#include "zsmr_ops_check.h"

using namespace zsmr;

namespace {

bool format_ok(int32_t d) { return d == ZSMR_FP32 || dtype_ok(d); }
uintptr_t bytes_of(int32_t d) { return d == ZSMR_FP32 ? 4 : 2; }

int32_t check_matrices(int64_t rows, int64_t cols, int64_t count) {
    if (rows < 1 || rows > ZSMR_MAX_SIDE || cols < 1 || cols > ZSMR_MAX_SIDE || rows * cols > ZSMR_MAX_MATRIX || count < 0 ||
        count > ZSMR_MAX_MATRICES)
        return ZSMR_ERR_ARG;
    return ZSMR_OK;
}

int32_t check_newton(const zsmr_newton* ns, NewtonArgs* a) {
    if (!ns || ns->steps < 1 || ns->steps > ZSMR_MAX_NS_STEPS || !std::isfinite(ns->eps) || ns->eps < 0) return ZSMR_ERR_ARG;
    a->steps = ns->steps;
    a->eps = ns->eps;
    return ns_passes(ns->coef, ns->steps, a->pass, &a->first) ? ZSMR_OK : ZSMR_ERR_ARG;
}

// Matrices in memory; distinct: they may not overlap.
int32_t check_strided(const void* p, int32_t dtype, int64_t stride, int64_t batch, int64_t rows, int64_t cols, int64_t count, bool distinct) {
    if (!p) return ZSMR_ERR_ARG;
    if (!format_ok(dtype)) return ZSMR_ERR_DTYPE;
    if (stride < cols || stride > ZSMR_MAX_WIDTH || batch < 0 || batch > (int64_t(1) << 40)) return ZSMR_ERR_ARG;
    // one behind the other, or side by side
    if (distinct && count > 1 && batch < (rows - 1) * stride + cols && (batch < cols || stride < (count - 1) * batch + cols))
        return ZSMR_ERR_ARG;
    return al(p, bytes_of(dtype)) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t zsmr_orthogonalize_workspace(int64_t rows, int64_t cols, int64_t count) {
    if (check_matrices(rows, cols, count)) return -1;
    if (count == 0) return 0;
    // of any result's format
    return std::max(ns_space(ns_shape(rows, cols, count, false)).bytes, ns_space(ns_shape(rows, cols, count, true)).bytes);
}

int32_t zsmr_orthogonalize(const void* x, int32_t x_dtype, int64_t x_stride, int64_t x_batch, void* out, int32_t out_dtype,
                           int64_t out_stride, int64_t out_batch, int64_t rows, int64_t cols, int64_t count, const zsmr_newton* ns,
                           void* ws, int64_t ws_bytes, hipStream_t stream) {
    NewtonArgs a{};
    int32_t st;
    if ((st = check_matrices(rows, cols, count)) || (st = check_newton(ns, &a))) return st;
    if (count == 0) return ZSMR_OK;
    if ((st = check_strided(x, x_dtype, x_stride, x_batch, rows, cols, count, false))) return st;
    if ((st = check_strided(out, out_dtype, out_stride, out_batch, rows, cols, count, true))) return st;
    a.shape = ns_shape(rows, cols, count, out_dtype == ZSMR_FP32);
    if ((st = check_space(ws, ws_bytes, ns_space(a.shape).bytes))) return st;
    a.x = x;
    a.x_stride = x_stride;
    a.x_batch = x_batch;
    a.x_dtype = x_dtype;
    a.out = out;
    a.out_stride = out_stride;
    a.out_batch = out_batch;
    a.out_dtype = out_dtype;
    NsOp ops[kNsMaxOps];
    return done(launch_orthogonalize(a, ops, ns_choose(ns->coef, ns->steps, a.shape, ops), ws, stream));
}

int32_t zero_muon_step(zsmr_ctx* c, int32_t rank, int32_t unit, int64_t begin, int64_t rows, int64_t cols, int64_t count,
                       const void* grads, int64_t row_stride, int64_t base, float* master, float* momentum, void* p16_dst,
                       const zsmr_muon* hp, const zsmr_newton* ns, void* ws, int64_t ws_bytes, hipStream_t stream) {
    NewtonArgs a{};
    int32_t st = check_piece(c, rank, unit);
    if (st || (st = check_matrices(rows, cols, count)) || (st = check_newton(ns, &a))) return st;
    if (!hp || !std::isfinite(hp->lr) || !std::isfinite(hp->beta) || !std::isfinite(hp->weight_decay) || !std::isfinite(hp->scale) ||
        hp->lr < 0 || hp->beta < 0 || hp->beta >= 1 || hp->weight_decay < 0 || hp->scale < 0 || (hp->nesterov != 0 && hp->nesterov != 1))
        return ZSMR_ERR_ARG;
    // factors that the kernels have in fp32
    const double decay = 1.0 - hp->lr * hp->weight_decay, rate = hp->lr * hp->scale;
    if (!(std::fabs(decay) <= FLT_MAX) || !(rate <= FLT_MAX)) return ZSMR_ERR_ARG;
    int64_t len = 0;
    piece(c, rank, unit, nullptr, &len, nullptr);
    const int64_t each = rows * cols, total = count * each;     // at most 2^53
    if (begin < 0 || begin > len || total > len - begin) return ZSMR_ERR_ARG;
    // a replica's all-reduce covers the whole vector and is counted once a step
    if (c->stage == ZSMR_DP && total != len) return ZSMR_ERR_ARG;
    if (count == 0) return ZSMR_OK;
    if ((st = check_grads(c, grads, row_stride, base, len))) return st;
    if (!master || !momentum || !p16_dst) return ZSMR_ERR_ARG;
    if (!al(master, 4) || !al(momentum, 4) || !al(p16_dst, 2)) return ZSMR_ERR_ALIGN;
    // Steps in groups, though the master is fp32: the update is then off by 3e-6 to 2e-4 of
    // its norm, as with products of fp32 operands (zsmr_newton_plan.h), where the quintic
    // itself leaves singular values between 0.7 and 1.2.  14,336 x 4,096 of 8 ranks take
    // 6.7 ms, step by step 10.2; 1,600 x 6,400 of 16 ranks 0.78 and 1.06.
    a.shape = ns_shape(rows, cols, count, false);
    if ((st = check_space(ws, ws_bytes, ns_space(a.shape).bytes))) return st;
    a.step.grads = static_cast<const uint16_t*>(grads) + base + begin;
    a.step.row_stride = row_stride;
    a.step.nrows = c->world;
    set_mean_divisor(a.step, c->world);
    a.step.master = master + begin;
    a.step.m = momentum + begin;
    a.step.p16 = static_cast<uint16_t*>(p16_dst) + begin;
    a.grad_dtype = c->gdt;
    a.param_dtype = c->pdt;
    a.nesterov = hp->nesterov;
    a.beta = (float)hp->beta;
    a.decay = (float)decay;
    a.rate = (float)rate;
    NsOp ops[kNsMaxOps];
    const hipError_t e = launch_muon(a, ops, ns_choose(ns->coef, ns->steps, a.shape, ops), ws, stream);
    if (e != hipSuccess) return hip_fail(e);
    count_reduce(c, rank, total);
    count_cast(c, rank, total);
    return ZSMR_OK;
}

}  // extern "C"
