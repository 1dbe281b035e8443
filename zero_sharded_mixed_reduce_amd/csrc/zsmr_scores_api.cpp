// Host side of the scores of logits, declared in include/zsmr_ops.h: every argument
// is checked here, then the launches of zsmr_scores_launch.h go to the caller's
// stream.  No device memory is allocated and nothing is kept between calls.
#include <cstdint>

#include "zsmr_ops_check.h"
#include "zsmr_scores_launch.h"
#include "zsmr_scores_plan.h"

using namespace zsmr;

namespace {

int32_t check_logits(const void* p, int64_t stride, int32_t dtype, int64_t tokens, int64_t vocab) {
    if (tokens < 0 || tokens > ZSMR_MAX_TOKENS || vocab < 1 || vocab > ZSMR_MAX_WIDTH) return ZSMR_ERR_ARG;
    if (dtype != ZSMR_FP32 && !dtype_ok(dtype)) return ZSMR_ERR_DTYPE;
    if (!p && tokens > 0) return ZSMR_ERR_ARG;
    if (stride < vocab || stride > ZSMR_MAX_WIDTH) return ZSMR_ERR_ARG;
    return al(p, dtype == ZSMR_FP32 ? 4 : 2) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

bool scale_ok(float scale) { return scale >= 0x1p-100f && scale <= 0x1p100f; }

bool top_ok(int64_t vocab, int32_t top) { return top >= 0 && top <= ZSMR_MAX_TOP && top <= vocab; }

}  // namespace

extern "C" {

int64_t zsmr_logprobs_workspace(int64_t tokens, int64_t vocab, int32_t top) {
    if (tokens < 0 || tokens > ZSMR_MAX_TOKENS || vocab < 1 || vocab > ZSMR_MAX_WIDTH || !top_ok(vocab, top)) return -1;
    return score_shape(tokens, vocab, top).bytes;
}

int32_t zsmr_logprobs(const void* logits, int64_t stride, int32_t dtype, const void* ids, int32_t id_bytes, int64_t tokens, int64_t vocab,
                      float scale, float* logprob, float* lse, float* entropy, int32_t top, void* top_ids, int32_t top_bytes,
                      float* top_logprobs, void* ws, int64_t ws_bytes, hipStream_t stream) {
    int32_t st;
    if ((st = check_logits(logits, stride, dtype, tokens, vocab))) return st;
    if (!scale_ok(scale) || !top_ok(vocab, top)) return ZSMR_ERR_ARG;
    if (logprob && (st = check_ids(ids, id_bytes, tokens))) return st;
    if (top && top_ids && top_bytes != 4 && top_bytes != 8) return ZSMR_ERR_ARG;
    if (!al(logprob, 4) || !al(lse, 4) || !al(entropy, 4) || !al(top_logprobs, 4)) return ZSMR_ERR_ALIGN;
    if (top && top_ids && !al(top_ids, top_bytes)) return ZSMR_ERR_ALIGN;
    if ((st = check_space(ws, ws_bytes, score_shape(tokens, vocab, top).bytes))) return st;
    if (!top_ids && !top_logprobs) top = 0;
    if (tokens == 0 || (!logprob && !lse && !entropy && top == 0)) return ZSMR_OK;
    ScoreArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.dtype = dtype;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.tokens = tokens;
    a.vocab = vocab;
    a.scale = scale;
    a.logprob = logprob;
    a.lse = lse;
    a.entropy = entropy;
    a.top = top;
    a.top_ids = top ? top_ids : nullptr;
    a.top_bytes = top_bytes;
    a.top_logprobs = top ? top_logprobs : nullptr;
    return done(launch_logprobs(a, ws, stream));
}

int32_t zsmr_logprobs_grad(const void* logits, int64_t stride, int32_t dtype, const void* ids, int32_t id_bytes, int64_t tokens,
                           int64_t vocab, float scale, const float* lse, const float* entropy, const float* g, const float* h,
                           void* dlogits, int64_t dlogits_stride, hipStream_t stream) {
    int32_t st;
    if ((st = check_logits(logits, stride, dtype, tokens, vocab))) return st;
    if ((st = check_logits(dlogits, dlogits_stride, dtype, tokens, vocab))) return st;
    if (!scale_ok(scale)) return ZSMR_ERR_ARG;
    if (g && (st = check_ids(ids, id_bytes, tokens))) return st;
    if (tokens > 0 && (!lse || (h && !entropy))) return ZSMR_ERR_ARG;
    if (dlogits == logits && tokens > 1 && stride != dlogits_stride) return ZSMR_ERR_ARG;
    if (!al(lse, 4) || !al(entropy, 4) || !al(g, 4) || !al(h, 4)) return ZSMR_ERR_ALIGN;
    if (tokens == 0) return ZSMR_OK;
    ScoreArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.dtype = dtype;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.tokens = tokens;
    a.vocab = vocab;
    a.scale = scale;
    a.lse = const_cast<float*>(lse);
    a.entropy = const_cast<float*>(entropy);
    a.dlogprob = g;
    a.dentropy = h;
    a.dlogits = dlogits;
    a.dstride = dlogits_stride;
    return done(launch_logprobs_grad(a, stream));
}

}  // extern "C"
