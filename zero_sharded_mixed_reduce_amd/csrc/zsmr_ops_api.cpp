// Host side of the operators declared in include/zsmr_ops.h: every argument is
// checked here, then the launches of zsmr_ops_launch.h go to the caller's
// stream.  No device memory is allocated and nothing is kept between calls.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zsmr_ctx.h"
#include "zsmr_ops.h"
#include "zsmr_ops_launch.h"

using namespace zsmr;

namespace {

int32_t done(hipError_t e) { return e == hipSuccess ? ZSMR_OK : hip_fail(e); }

// rows x width elements of 16 bits, stride apart
int32_t check_rows(const void* p, int64_t rows, int64_t width, int64_t stride) {
    if (!p && rows > 0) return ZSMR_ERR_ARG;
    if (stride < width || stride > ZSMR_MAX_WIDTH) return ZSMR_ERR_ARG;
    return al(p, 2) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

int32_t check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
    if (tokens < 0 || tokens > ZSMR_MAX_TOKENS || vocab < 1 || vocab > ZSMR_MAX_VOCAB ||
        width < 1 || width > ZSMR_MAX_WIDTH)
        return ZSMR_ERR_ARG;
    return ZSMR_OK;
}

int32_t check_ids(const void* ids, int32_t id_bytes, int64_t tokens) {
    if ((id_bytes != 4 && id_bytes != 8) || (!ids && tokens > 0)) return ZSMR_ERR_ARG;
    return al(ids, id_bytes) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

int32_t check_space(const void* ws, int64_t ws_bytes, int64_t need) {
    if (need > 0 && (!ws || ws_bytes < need)) return ZSMR_ERR_ARG;
    return al(ws, 16) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

int32_t check_clip(double max_norm, double eps, const float* norm_coef) {
    if (!std::isfinite(max_norm) || max_norm < 0 || !std::isfinite(eps) || eps < 0 || !norm_coef)
        return ZSMR_ERR_ARG;
    return al(norm_coef, 4) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

// Elements of a list tensor, or of a gradient row's pad: what one launch can take in
// chunks (550 GB of 16 bits).
constexpr int64_t kMaxItem = kMaxGroups * kChunk;

// A list's tensors; *total gets their elements, *chunks the chunks they have if the
// list is a long one.
int32_t check_list(const void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                   int32_t n, int64_t* total, int64_t* chunks) {
    *total = *chunks = 0;
    if (n < 0 || (n > 0 && (!ptrs || !numels || !dtypes))) return ZSMR_ERR_ARG;
    for (int32_t i = 0; i < n; ++i) {
        if (numels[i] < 0 || numels[i] > kMaxItem || (!ptrs[i] && numels[i] > 0)) return ZSMR_ERR_ARG;
        if (dtypes[i] != ZSMR_FP32 && !dtype_ok(dtypes[i])) return ZSMR_ERR_DTYPE;
        if (!al(ptrs[i], dtypes[i] == ZSMR_FP32 ? 4 : 2)) return ZSMR_ERR_ALIGN;
        *total += numels[i];
        *chunks += ceil_div(numels[i], kChunk);
        if (*total > ZSMR_MAX_NUMEL || *chunks > INT32_MAX) return ZSMR_ERR_ARG;
    }
    return ZSMR_OK;
}

// Puts work items into the launches of at most BATCH items and kMaxGroups chunks that
// carry them in their arguments; flush(args) launches one.  length: of the whole
// list, or of the row it is flattened into.
template <int BATCH, typename A, typename Item, typename F>
struct Batches {
    A a{};
    F flush;
    hipError_t err = hipSuccess;
    Batches(F f, int64_t length) : flush(f) { a.chunk = chunk_of_list(length); }
    void add(Item it, int64_t n) {
        if (n == 0 || err != hipSuccess) return;
        if (a.chunks + ceil_div(n, a.chunk) > kMaxGroups) go();
        it.chunk0 = a.chunks;
        it.n = n;
        a.it[a.count++] = it;
        a.chunks += (int32_t)ceil_div(n, a.chunk);
        if (a.count == BATCH) go();
    }
    void go() {
        if (a.count && err == hipSuccess) err = flush(a);
        a.count = a.chunks = 0;
    }
};

int32_t clip(const void* const* ptrs, void* const* in_place, const int64_t* numels,
             const int32_t* dtypes, int32_t n, const float* coef, uint16_t* flat,
             int64_t flat_numel, int32_t flat_dtype, int64_t total, hipStream_t stream) {
    int64_t before = 0;
    auto launch = [&](ClipArgs& a) {
        a.before = before;
        before += a.chunks;
        return launch_clip(a, stream);
    };
    Batches<kClipBatch, ClipArgs, ClipItem, decltype(launch)> b(launch, in_place ? total : flat_numel);
    b.a.coef = coef;
    b.a.in_place = in_place != nullptr;
    // from the list's end to its start, which the kernel's reads count on
    int64_t at = 0;
    if (!in_place) {
        ClipItem pad{};
        pad.dst = flat + total;
        pad.src_dtype = pad.dst_dtype = (int16_t)flat_dtype;
        b.add(pad, flat_numel - total);
        at = total;
    }
    for (int32_t i = n - 1; i >= 0; --i) {
        at -= numels[i];
        ClipItem it{};
        it.src = ptrs[i];
        it.dst = in_place ? in_place[i] : flat + at;
        it.src_dtype = (int16_t)dtypes[i];
        it.dst_dtype = (int16_t)(in_place ? dtypes[i] : flat_dtype);
        b.add(it, numels[i]);
    }
    b.go();
    return done(b.err);
}

}  // namespace

extern "C" {

int32_t zsmr_embed_lookup(const void* table, int64_t vocab, int64_t width, int64_t table_stride,
                          int32_t dtype, const void* ids, int32_t id_bytes, int64_t tokens,
                          float scale, void* out, int64_t out_stride, hipStream_t stream) {
    int32_t st;
    if ((st = check_sizes(tokens, vocab, width))) return st;
    if (!dtype_ok(dtype)) return ZSMR_ERR_DTYPE;
    if ((st = check_rows(table, vocab, width, table_stride))) return st;
    if ((st = check_ids(ids, id_bytes, tokens))) return st;
    if ((st = check_rows(out, tokens, width, out_stride))) return st;
    if (tokens == 0) return ZSMR_OK;
    EmbedArgs a{};
    a.src = static_cast<const uint16_t*>(table);
    a.src_stride = table_stride;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.dtype = dtype;
    a.tokens = tokens;
    a.vocab = vocab;
    a.width = width;
    a.scale = scale;
    a.dst = static_cast<uint16_t*>(out);
    a.dst_stride = out_stride;
    return done(launch_embed_lookup(a, stream));
}

int64_t zsmr_embed_grad_workspace(int64_t vocab, int64_t width, int64_t tokens) {
    return check_sizes(tokens, vocab, width) ? -1 : embed_grad_bytes(vocab, width, tokens);
}

int32_t zsmr_embed_grad(const void* dout, int64_t dout_stride, int32_t dtype, const void* ids,
                        int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t width,
                        float scale, int32_t accumulate, void* dtable, int64_t dtable_stride,
                        void* ws, int64_t ws_bytes, hipStream_t stream) {
    int32_t st;
    if ((st = check_sizes(tokens, vocab, width))) return st;
    if (!dtype_ok(dtype)) return ZSMR_ERR_DTYPE;
    if (accumulate != 0 && accumulate != 1) return ZSMR_ERR_ARG;
    if ((st = check_rows(dout, tokens, width, dout_stride))) return st;
    if ((st = check_ids(ids, id_bytes, tokens))) return st;
    if ((st = check_rows(dtable, vocab, width, dtable_stride))) return st;
    if ((st = check_space(ws, ws_bytes, embed_grad_bytes(vocab, width, tokens)))) return st;
    if (tokens == 0 && accumulate) return ZSMR_OK;
    EmbedArgs a{};
    a.src = static_cast<const uint16_t*>(dout);
    a.src_stride = dout_stride;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.dtype = dtype;
    a.tokens = tokens;
    a.vocab = vocab;
    a.width = width;
    a.scale = scale;
    a.accumulate = accumulate;
    a.dst = static_cast<uint16_t*>(dtable);
    a.dst_stride = dtable_stride;
    return done(launch_embed_grad(a, ws, stream));
}

int64_t zsmr_xent_workspace(int64_t tokens, int64_t vocab, int64_t width, int32_t backward) {
    if (check_sizes(tokens, vocab, width) || (backward != 0 && backward != 1)) return -1;
    return xent_bytes(tokens, vocab, width, backward != 0);
}

static int32_t xent_args(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                         int32_t dtype, const void* labels, int32_t id_bytes, int64_t tokens,
                         int64_t vocab, int64_t width, const void* ws, int64_t ws_bytes,
                         bool backward, XentArgs* a) {
    int32_t st;
    if ((st = check_sizes(tokens, vocab, width))) return st;
    if (!dtype_ok(dtype)) return ZSMR_ERR_DTYPE;
    if ((st = check_rows(x, tokens, width, x_stride))) return st;
    if ((st = check_rows(w, vocab, width, w_stride))) return st;
    if ((st = check_ids(labels, id_bytes, tokens))) return st;
    if ((st = check_space(ws, ws_bytes, xent_bytes(tokens, vocab, width, backward)))) return st;
    a->x = static_cast<const uint16_t*>(x);
    a->x_stride = x_stride;
    a->w = static_cast<const uint16_t*>(w);
    a->w_stride = w_stride;
    a->labels = labels;
    a->id_bytes = id_bytes;
    a->dtype = dtype;
    a->tokens = tokens;
    a->vocab = vocab;
    a->width = width;
    return ZSMR_OK;
}

int32_t zsmr_xent_forward(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                          int32_t dtype, const void* labels, int32_t id_bytes, int64_t tokens,
                          int64_t vocab, int64_t width, float* loss, float* lse, float* summary,
                          void* ws, int64_t ws_bytes, hipStream_t stream) {
    XentArgs a{};
    const int32_t st = xent_args(x, x_stride, w, w_stride, dtype, labels, id_bytes, tokens, vocab,
                                 width, ws, ws_bytes, false, &a);
    if (st) return st;
    if (!summary || (tokens > 0 && (!loss || !lse))) return ZSMR_ERR_ARG;
    if (!al(loss, 4) || !al(lse, 4) || !al(summary, 4)) return ZSMR_ERR_ALIGN;
    a.loss = loss;
    a.lse = lse;
    a.summary = summary;
    return done(launch_xent_forward(a, ws, stream));
}

int32_t zsmr_xent_backward(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                           int32_t dtype, const void* labels, int32_t id_bytes, int64_t tokens,
                           int64_t vocab, int64_t width, const float* lse, const float* grad,
                           const float* scale, void* dx, int64_t dx_stride, void* dw,
                           int64_t dw_stride, int32_t accumulate, void* ws, int64_t ws_bytes,
                           hipStream_t stream) {
    XentArgs a{};
    int32_t st = xent_args(x, x_stride, w, w_stride, dtype, labels, id_bytes, tokens, vocab, width,
                           ws, ws_bytes, true, &a);
    if (st) return st;
    if ((!lse && tokens > 0) || (accumulate != 0 && accumulate != 1)) return ZSMR_ERR_ARG;
    if (!al(lse, 4) || !al(grad, 4) || !al(scale, 4)) return ZSMR_ERR_ALIGN;
    if (dx && (st = check_rows(dx, tokens, width, dx_stride))) return st;
    if (dw && (st = check_rows(dw, vocab, width, dw_stride))) return st;
    if ((!dx && !dw) || (tokens == 0 && (!dw || accumulate))) return ZSMR_OK;
    a.lse = const_cast<float*>(lse);
    a.grad = grad;
    a.scale = scale;
    a.dx = static_cast<uint16_t*>(dx);
    a.dx_stride = dx_stride;
    a.dw = static_cast<uint16_t*>(dw);
    a.dw_stride = dw_stride;
    a.accumulate = accumulate;
    return done(launch_xent_backward(a, ws, stream));
}

int64_t zsmr_norm_workspace(int64_t total, int32_t n_tensors) {
    if (total < 0 || total > ZSMR_MAX_NUMEL || n_tensors < 0) return -1;
    // one fp64 a chunk of a list (each tensor ends one) or a tile of a shard
    const int64_t short_list = total < kShortList ? total : kShortList;
    const int64_t lists = std::max(total / kChunk, short_list / kShortChunk) + n_tensors;
    return 8 * std::max(lists, ceil_div(total, kTile));
}

int32_t zsmr_grad_norm(const void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                       int32_t n, double max_norm, double eps, float* norm_coef, void* ws,
                       int64_t ws_bytes, hipStream_t stream) {
    int64_t total = 0, chunks = 0;
    int32_t st = check_list(ptrs, numels, dtypes, n, &total, &chunks);
    if (st) return st;
    if ((st = check_clip(max_norm, eps, norm_coef))) return st;
    if (total <= kShortList) {
        chunks = 0;
        for (int32_t i = 0; i < n; ++i) chunks += ceil_div(numels[i], kShortChunk);
    }
    if ((st = check_space(ws, ws_bytes, chunks * 8))) return st;
    double* partial = static_cast<double*>(ws);
    int64_t at = 0;
    auto launch = [&](NormArgs& a) {
        const hipError_t e = launch_sumsq(a, partial + at, stream);
        at += sumsq_grid(a.chunks);
        return e;
    };
    Batches<kNormBatch, NormArgs, NormItem, decltype(launch)> b(launch, total);
    for (int32_t i = 0; i < n; ++i) {
        NormItem it{};
        it.p = ptrs[i];
        it.dtype = dtypes[i];
        b.add(it, numels[i]);
    }
    b.go();
    if (b.err != hipSuccess) return hip_fail(b.err);
    return done(launch_join(partial, at, nullptr, max_norm, eps, norm_coef, stream));
}

int32_t zsmr_clip_coef(const double* sums, int64_t n, double max_norm, double eps,
                       float* norm_coef, hipStream_t stream) {
    if (n < 0 || (n > 0 && !sums)) return ZSMR_ERR_ARG;
    const int32_t st = check_clip(max_norm, eps, norm_coef);
    if (st) return st;
    if (!al(sums, 8)) return ZSMR_ERR_ALIGN;
    return done(launch_join(sums, n, nullptr, max_norm, eps, norm_coef, stream));
}

int32_t zsmr_clip_grads(void* const* ptrs, const int64_t* numels, const int32_t* dtypes, int32_t n,
                        const float* coef, hipStream_t stream) {
    int64_t total = 0, chunks = 0;
    const int32_t st = check_list(const_cast<const void* const*>(ptrs), numels, dtypes, n, &total, &chunks);
    if (st) return st;
    if (!coef) return ZSMR_ERR_ARG;
    if (!al(coef, 4)) return ZSMR_ERR_ALIGN;
    return clip(const_cast<const void* const*>(ptrs), ptrs, numels, dtypes, n, coef, nullptr, 0, 0, total, stream);
}

int32_t zsmr_clip_flatten(const void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                          int32_t n, const float* coef, void* flat, int64_t flat_numel,
                          int32_t flat_dtype, hipStream_t stream) {
    int64_t total = 0, chunks = 0;
    const int32_t st = check_list(ptrs, numels, dtypes, n, &total, &chunks);
    if (st) return st;
    if (!dtype_ok(flat_dtype)) return ZSMR_ERR_DTYPE;
    if (flat_numel < total || flat_numel - total > kMaxItem || (flat_numel > 0 && !flat)) return ZSMR_ERR_ARG;
    if (!al(flat, 2) || !al(coef, 4)) return ZSMR_ERR_ALIGN;
    return clip(ptrs, nullptr, numels, dtypes, n, coef, static_cast<uint16_t*>(flat), flat_numel,
                flat_dtype, total, stream);
}

int32_t zero_reduce_shard_sumsq(zsmr_ctx* c, int32_t rank, int32_t unit, const void* grads,
                                int64_t row_stride, int64_t base, int32_t mean, float* g_out,
                                double* sumsq, void* ws, int64_t ws_bytes, hipStream_t stream) {
    int32_t st = check_piece(c, rank, unit);
    if (st) return st;
    int64_t len = 0;
    piece(c, rank, unit, nullptr, &len, nullptr);
    if ((st = check_grads(c, grads, row_stride, base, len))) return st;
    if (!g_out || !sumsq || (mean != 0 && mean != 1)) return ZSMR_ERR_ARG;
    if (!al(g_out, 4) || !al(sumsq, 8)) return ZSMR_ERR_ALIGN;
    const int64_t tiles = ceil_div(len, kTile);
    if (tiles > kMaxGroups) return ZSMR_ERR_ARG;        // one launch; 137 GB of g_out
    if ((st = check_space(ws, ws_bytes, tiles * 8))) return st;
    StepArgs a{};
    a.grads = static_cast<const uint16_t*>(grads) + base;
    a.row_stride = row_stride;
    a.nrows = c->world;
    a.mean = mean;
    set_mean_divisor(a, c->world);
    a.g_out = g_out;
    a.n = len;
    // a rank without a part of this unit leaves a sum of zero
    double* partial = static_cast<double*>(ws);
    const hipError_t e = len > 0 ? launch_reduce_sumsq(c->gdt, a, partial, sumsq, stream)
                                 : launch_join(partial, 0, sumsq, 0, 0, nullptr, stream);
    if (e != hipSuccess) return hip_fail(e);
    count_reduce(c, rank, len);
    return ZSMR_OK;
}

int32_t zero_clipped_step(zsmr_ctx* c, int32_t rank, int32_t unit, const float* g,
                          const float* coef, float* master, float* m, float* v, void* p16_dst,
                          int32_t t, const zsmr_adam* hp, hipStream_t stream) {
    int32_t st = check_piece(c, rank, unit);
    if (st) return st;
    StepArgs a{};
    if ((st = check_adam(hp, t, &a.k))) return st;
    if (!g || !master || !m || !v || !p16_dst) return ZSMR_ERR_ARG;
    if (!al(g, 4) || !al(coef, 4) || !al(master, 4) || !al(m, 4) || !al(v, 4) || !al(p16_dst, 2))
        return ZSMR_ERR_ALIGN;
    int64_t len = 0;
    piece(c, rank, unit, nullptr, &len, nullptr);
    if (len == 0) return ZSMR_OK;
    if (ceil_div(len, kTile) > kMaxGroups) return ZSMR_ERR_ARG;
    a.g_in = g;
    a.master = master;
    a.m = m;
    a.v = v;
    a.p16 = static_cast<uint16_t*>(p16_dst);
    a.n = len;
    const hipError_t e = launch_clipped(c->pdt, a, coef, stream);
    if (e != hipSuccess) return hip_fail(e);
    count_cast(c, rank, len);
    return ZSMR_OK;
}

}  // extern "C"
