"""The host code of the operators under AddressSanitizer and
UndefinedBehaviorSanitizer: ``csrc/zsmr_ops_api.cpp`` is built with g++ together
with a stand-in for the kernel launches that records them.  Placeholder device
addresses; no GPU.

* A gradient list's launches cover every element of every tensor once, in
  chunks that stay inside it; the flattened row's destinations follow each
  other, its pad fills the rest; the partial sums fit the workspace the library
  names.
* The clipped step's launches carry the piece the layout gives, and a failing
  launch counts nothing.
"""
import os
import shutil

import pytest

from tests import test_host_sanitizers as base

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <vector>
#include "zsmr_ctx.h"
#include "zsmr_ops.h"
#include "zsmr_ops_launch.h"
#define CHECK(c) do { if (!(c)) { std::printf("CHECK failed line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

static std::vector<zsmr::NormArgs> g_norm;
static std::vector<zsmr::ClipArgs> g_clip;
static std::vector<int64_t> g_norm_at;
struct Join { const double* partial; int64_t n; double* sumsq; double max_norm, eps; float* out; };
static std::vector<Join> g_join;
static std::vector<zsmr::StepArgs> g_step;
static hipError_t g_result = hipSuccess;
static double* g_base;
const char* hipGetErrorString(hipError_t) { return "launch refused by the stand-in"; }
namespace zsmr {
int sumsq_grid(int64_t chunks) { return (int)std::min<int64_t>(chunks, 2048); }
hipError_t launch_sumsq(const NormArgs& a, double* partial, hipStream_t) { g_norm.push_back(a); g_norm_at.push_back(partial - g_base); return g_result; }
hipError_t launch_clip(const ClipArgs& a, hipStream_t) { g_clip.push_back(a); return g_result; }
hipError_t launch_join(const double* p, int64_t n, double* s, double m, double e, float* o, hipStream_t) { g_join.push_back({p, n, s, m, e, o}); return g_result; }
hipError_t launch_reduce_sumsq(int, const StepArgs& a, double*, double*, hipStream_t) { g_step.push_back(a); return g_result; }
hipError_t launch_clipped(int, const StepArgs& a, const float*, hipStream_t) { g_step.push_back(a); return g_result; }
hipError_t launch_embed_lookup(const EmbedArgs&, hipStream_t) { return g_result; }
int64_t embed_grad_bytes(int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_embed_grad(const EmbedArgs&, void*, hipStream_t) { return g_result; }
int64_t xent_bytes(int64_t, int64_t, int64_t, bool) { return 0; }
hipError_t launch_xent_forward(const XentArgs&, void*, hipStream_t) { return g_result; }
hipError_t launch_xent_backward(const XentArgs&, void*, hipStream_t) { return g_result; }
// the step's own launches are not reached
hipError_t launch_step(int, int, int, const StepArgs&, hipStream_t) { std::abort(); }
hipError_t launch_copy16(const uint16_t*, uint16_t*, int64_t, hipStream_t) { std::abort(); }
hipError_t launch_copy_blocks(const uint16_t*, uint16_t*, int64_t, int32_t, int64_t, hipStream_t) { std::abort(); }
hipError_t launch_gather16(const uint16_t* const*, int32_t, int64_t, uint16_t*, hipStream_t) { std::abort(); }
void set_launch_shape(int32_t, int32_t, int32_t, int32_t) {}
void set_write_window(int64_t, int64_t, int64_t, int64_t) {}
void set_xcd_balance(int32_t) {}
void describe_step(int, const StepArgs&, StepPlan*) {}
}  // namespace zsmr

static void list(const std::vector<int64_t>& sizes, int32_t dtype, int64_t pad) {
    const int n = (int)sizes.size();
    const int64_t width = dtype == ZSMR_FP32 ? 4 : 2;
    std::vector<const void*> ptrs;
    std::vector<int32_t> dtypes(n, dtype);
    int64_t total = 0, at = 1 << 20;
    for (int64_t s : sizes) { ptrs.push_back(s ? (const void*)at : nullptr); at += s * width + 4; total += s; }
    const int64_t need = zsmr_norm_workspace(total, n);
    CHECK(need >= 0);
    g_base = (double*)(int64_t(1) << 45);
    float* out = (float*)(int64_t(1) << 46);
    uint16_t* flat = (uint16_t*)(int64_t(1) << 47);
    g_norm.clear(); g_norm_at.clear(); g_clip.clear(); g_join.clear();
    CHECK(zsmr_grad_norm(ptrs.data(), sizes.data(), dtypes.data(), n, 1.0, 1e-6, out, g_base, need, nullptr) == ZSMR_OK);
    int64_t partials = 0; size_t seen = 0; std::vector<int64_t> full;
    for (size_t k = 0; k < sizes.size(); ++k) if (sizes[k]) full.push_back((int64_t)k);
    for (size_t l = 0; l < g_norm.size(); ++l) {
        const zsmr::NormArgs& a = g_norm[l];
        CHECK(a.count > 0 && a.count <= zsmr::kNormBatch && g_norm_at[l] == partials);
        int64_t chunk = 0;
        for (int i = 0; i < a.count; ++i) {
            CHECK(a.it[i].p == ptrs[full[seen]] && a.it[i].n == sizes[full[seen]] && a.it[i].dtype == dtype && a.it[i].chunk0 == chunk);
            chunk += (a.it[i].n + a.chunk - 1) / a.chunk;
            ++seen;
        }
        CHECK(chunk == a.chunks);
        partials += zsmr::sumsq_grid(a.chunks);
    }
    CHECK(seen == full.size() && partials * 8 <= need);
    CHECK(g_join.size() == 1 && g_join[0].n == partials && g_join[0].out == out && g_join[0].partial == g_base);
    CHECK(zsmr_clip_flatten(ptrs.data(), sizes.data(), dtypes.data(), n, out, flat, total + pad, ZSMR_FP16, nullptr) == ZSMR_OK);
    // from the end of the row to its start: what is written is contiguous
    uint16_t* end = flat + total + pad; int64_t before = 0;
    for (const zsmr::ClipArgs& a : g_clip) {
        CHECK(a.count > 0 && a.count <= zsmr::kClipBatch && a.before == before && !a.in_place && a.coef == out);
        int64_t chunk = 0;
        for (int i = 0; i < a.count; ++i) {
            CHECK((uint16_t*)a.it[i].dst + a.it[i].n == end && a.it[i].chunk0 == chunk && a.it[i].dst_dtype == ZSMR_FP16);
            end = (uint16_t*)a.it[i].dst;
            chunk += (a.it[i].n + a.chunk - 1) / a.chunk;
        }
        CHECK(chunk == a.chunks);
        before += chunk;
    }
    CHECK(end == flat);
    g_clip.clear();
    std::vector<void*> own;
    for (const void* q : ptrs) own.push_back(const_cast<void*>(q));
    CHECK(zsmr_clip_grads(own.data(), sizes.data(), dtypes.data(), n, out, nullptr) == ZSMR_OK);
    size_t items = 0;
    for (const zsmr::ClipArgs& a : g_clip)
        for (int i = 0; i < a.count; ++i, ++items) CHECK(a.in_place && a.it[i].src == a.it[i].dst && a.it[i].src_dtype == dtype && a.it[i].dst_dtype == dtype);
    CHECK(items == full.size());
}

int main() {
    list({}, ZSMR_BF16, 0);
    list({}, ZSMR_FP32, 9);
    list({0, 1, 0}, ZSMR_FP32, 0);
    list({7, 2048, 2049, 0, 4097}, ZSMR_BF16, 3);
    list(std::vector<int64_t>(161, 5), ZSMR_FP16, 1);
    list(std::vector<int64_t>(400, 1), ZSMR_FP32, 40000);
    list({int64_t(1) << 22}, ZSMR_BF16, 0);
    list({(int64_t(1) << 22) - 1, 1, 1}, ZSMR_BF16, 0);
    list({int64_t(1) << 33, 3, int64_t(1) << 20}, ZSMR_FP32, 7);
    list(std::vector<int64_t>(300, 100001), ZSMR_BF16, 20001);

    zsmr_ctx* c = nullptr;
    CHECK(zero_init_shards(&c, 100003, 3, ZSMR_ZERO2, ZSMR_BF16, ZSMR_FP16, 1, nullptr, 0) == ZSMR_OK);
    const int64_t S = 33335;
    char* const p = (char*)(int64_t(1) << 40);
    double* sum = (double*)(p + 4096);
    const int64_t need = zsmr_norm_workspace(S, 1);
    CHECK(zero_reduce_shard_sumsq(c, 2, 0, p, 3 * S, 2 * S, 1, (float*)p, sum, p, need, nullptr) == ZSMR_OK);
    CHECK(zero_reduce_shard_sumsq(c, 2, 0, p, 3 * S, 2 * S, 1, (float*)p, sum, p, need - 8, nullptr) == ZSMR_ERR_ARG);
    CHECK(g_step.size() == 1 && g_step[0].n == S && g_step[0].nrows == 3 && g_step[0].row_stride == 3 * S && !g_step[0].inv_pow2 &&
          (const char*)g_step[0].grads == p + 4 * S);
    const zsmr_adam hp = {1e-3, 0.9, 0.999, 1e-8};
    CHECK(zero_clipped_step(c, 1, 0, (float*)p, nullptr, (float*)p, (float*)p, (float*)p, p, 2, &hp, nullptr) == ZSMR_OK);
    CHECK(g_step.size() == 2 && g_step[1].n == S && g_step[1].k.c1 == 0.9f);
    zsmr_counters r2{}, r0{};
    CHECK(zero_counters(c, 2, &r2) == ZSMR_OK && zero_counters(c, 0, &r0) == ZSMR_OK);
    CHECK(r2.rs_elems == 2 * S && r2.ag_elems == S && r0.rs_elems == 0 && r0.ag_elems == S);
    g_result = hipErrorInvalidValue;
    CHECK(zero_reduce_shard_sumsq(c, 2, 0, p, 3 * S, 2 * S, 1, (float*)p, sum, p, need, nullptr) == ZSMR_ERR_HIP);
    CHECK(zero_clipped_step(c, 1, 0, (float*)p, nullptr, (float*)p, (float*)p, (float*)p, p, 2, &hp, nullptr) == ZSMR_ERR_HIP);
    CHECK(zero_counters(c, 2, &r0) == ZSMR_OK && r0.rs_elems == r2.rs_elems && r0.ag_elems == r2.ag_elems);
    const int64_t one = 1; const int32_t f32 = ZSMR_FP32; const void* q = p;
    CHECK(zsmr_grad_norm(&q, &one, &f32, 1, 1, 0, (float*)p, p, 64, nullptr) == ZSMR_ERR_HIP);
    CHECK(zsmr_clip_flatten(&q, &one, &f32, 1, nullptr, p, 1, ZSMR_BF16, nullptr) == ZSMR_ERR_HIP);
    zero_destroy(c);
    // a rank without a part of a unit: its sum is joined from nothing
    g_result = hipSuccess;
    const int64_t units[2] = {10, 20};
    CHECK(zero_init_shards(&c, 30, 2, ZSMR_ZERO3_OWNER, ZSMR_BF16, ZSMR_BF16, 0, units, 2) == ZSMR_OK);
    int32_t owner = -1;
    CHECK(zero_unit_owner(c, 1, &owner) == ZSMR_OK);
    g_join.clear();
    CHECK(zero_reduce_shard_sumsq(c, 1 - owner, 1, p, 20, 0, 1, (float*)p, sum, nullptr, 0, nullptr) == ZSMR_OK);
    CHECK(g_join.size() == 1 && g_join[0].n == 0 && g_join[0].sumsq == sum);
    zero_destroy(c);
    std::printf("host checks passed\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("sanitize", [False, True])
def test_host_code_of_the_operators(tmp_path, monkeypatch, sanitize):
    monkeypatch.setattr(base, "DRIVER", DRIVER)
    extra = [os.path.join(base.CSRC, "zsmr_ops_api.cpp")]
    if sanitize:
        extra += ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    exe = base._compile(tmp_path, extra)
    base._run(exe, {"ASAN_OPTIONS": "detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
                    "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1"})
