// Internal interface between the host code of the operators (zsmr_ops_api.cpp)
// and their gfx950 kernels.  Not part of the public ABI.
#pragma once
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "zsmr_launch.h"

namespace zsmr {

// A launch has fewer than 2^32 work items in a dimension; in workgroups of 256:
constexpr int64_t kMaxGroups = ((int64_t(1) << 32) - 1) / 256;
// What is longer is launched in parts: rows of `items` work items each, from the
// first one on, and workgroups.  each(first, count).
template <typename F>
void launch_rows(int64_t rows, int64_t items, F each) {
    const int64_t most = kMaxGroups * 256 / items;
    for (int64_t first = 0; first < rows; first += most) each(first, rows - first < most ? rows - first : most);
}
template <typename F>
void launch_groups(int64_t groups, F each) {
    launch_rows(groups, 256, each);
}

// ---- norm and clipping (zsmr_norm.hip)
// Elements of a list tensor one workgroup handles at a time: few in a short
// list, whose call is as long as one workgroup takes.  Norm and flatten of 54
// tensors of 0.25M fp32 on MI355X: chunks of 16,384 5.1 + 6.6 us, of 2,048 4.7 + 4.7 us.
constexpr int kChunk = 16384, kShortChunk = 2048;
constexpr int64_t kShortList = int64_t(1) << 22;
inline int chunk_of_list(int64_t total) { return total <= kShortList ? kShortChunk : kChunk; }
constexpr int kTile = 2048;         // elements of a shard one workgroup handles
struct NormItem {
    const void* p;
    int64_t n;
    int32_t chunk0;                 // first chunk of this tensor within the launch
    int32_t dtype;
};
struct ClipItem {
    const void* src;
    void* dst;
    int64_t n;
    int32_t chunk0;
    int16_t src_dtype, dst_dtype;   // src NULL: zeros
};
// A launch's tensors travel in its kernel arguments (4 KB), so a list needs no
// device copy that would have to outlive the call.
constexpr int kNormBatch = 160, kClipBatch = 120;
struct NormArgs {
    NormItem it[kNormBatch];
    int32_t count, chunks, chunk;
};
struct ClipArgs {
    ClipItem it[kClipBatch];
    int32_t count, chunks, chunk;
    int64_t before;                 // chunks of the launches before this one
    const float* coef;
    int32_t in_place;
};
int sumsq_grid(int64_t chunks);     // partial sums a launch of so many chunks leaves
hipError_t launch_sumsq(const NormArgs& a, double* partial, hipStream_t stream);
hipError_t launch_clip(const ClipArgs& a, hipStream_t stream);
// total = partial[0..n): sumsq (if not NULL) = total; norm_coef (if not NULL)
hipError_t launch_join(const double* partial, int64_t n, double* sumsq, double max_norm,
                       double eps, float* norm_coef, hipStream_t stream);
// grads, row_stride, nrows, mean, nf, inv_nf, inv_pow2, g_out and n of StepArgs
hipError_t launch_reduce_sumsq(int dtype, const StepArgs& a, double* partial, double* sumsq,
                               hipStream_t stream);
// g_in, master, m, v, p16, n and k of StepArgs
hipError_t launch_clipped(int dtype, const StepArgs& a, const float* coef, hipStream_t stream);

// ---- embedding (zsmr_embed.hip)
struct EmbedArgs {
    const uint16_t* src;            // table (lookup) or dout (gradient)
    int64_t src_stride;
    const void* ids;
    int32_t id_bytes, dtype;
    int64_t tokens, vocab, width;
    float scale;
    int32_t accumulate;
    uint16_t* dst;                  // out (lookup) or dtable (gradient)
    int64_t dst_stride;
};
hipError_t launch_embed_lookup(const EmbedArgs& a, hipStream_t stream);
int64_t embed_grad_bytes(int64_t vocab, int64_t width, int64_t tokens);
hipError_t launch_embed_grad(const EmbedArgs& a, void* ws, hipStream_t stream);

// ---- softmax cross entropy (zsmr_xent.hip)
struct XentArgs {
    const uint16_t* x;
    int64_t x_stride;
    const uint16_t* w;
    int64_t w_stride;
    const void* labels;
    int32_t id_bytes, dtype;
    int64_t tokens, vocab, width;
    float* loss;
    float* lse;
    float* summary;
    const float* grad;
    const float* scale;
    uint16_t* dx;
    int64_t dx_stride;
    uint16_t* dw;
    int64_t dw_stride;
    int32_t accumulate;
};
int64_t xent_bytes(int64_t tokens, int64_t vocab, int64_t width, bool backward);
hipError_t launch_xent_forward(const XentArgs& a, void* ws, hipStream_t stream);
hipError_t launch_xent_backward(const XentArgs& a, void* ws, hipStream_t stream);

}  // namespace zsmr
