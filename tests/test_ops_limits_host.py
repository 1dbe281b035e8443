"""The largest sizes of the list calls and of the clipped step, without a GPU: the
host code of ``csrc/zsmr_ops_api.cpp`` built with g++ under the sanitizers against the
recording stand-in for the kernel launches of ``tests/test_ops_host.py``.

* No launch has 2^32 work items, and what none could take is refused before the
  first one.
"""
import shutil

import pytest

from tests import test_host_sanitizers as base
from tests import test_ops_host as host

MAIN = r"""
#include "zsmr_ops_launch.h"
const int64_t MOST = (int64_t(1) << 32) - 1;
static char* const P = (char*)(int64_t(1) << 40);

static void lists() {
    const int64_t T = int64_t(1) << 37, item = zsmr::kMaxGroups * zsmr::kChunk;
    std::vector<int64_t> sizes = {T, 3, T, T - 1, 70000};
    std::vector<void*> ptrs(5, P);
    std::vector<int32_t> dtypes(5, ZSMR_BF16);
    const float* coef = (float*)P;
    CHECK(zsmr_clip_grads(ptrs.data(), sizes.data(), dtypes.data(), 5, coef, nullptr) == ZSMR_OK);
    int64_t before = 0, items = 0;
    for (const zsmr::ClipArgs& a : g_clip) {
        CHECK(a.chunks > 0 && int64_t(a.chunks) * 256 <= MOST && a.before == before);
        int64_t chunk = 0;
        for (int i = 0; i < a.count; ++i, ++items) {
            CHECK(a.it[i].n == sizes[4 - items] && a.it[i].chunk0 == chunk);
            chunk += (a.it[i].n + a.chunk - 1) / a.chunk;
        }
        CHECK(chunk == a.chunks);
        before += chunk;
    }
    CHECK(items == 5 && g_clip.size() == 3);
    // a short list at the start of a long row
    g_clip.clear();
    const int64_t flat = int64_t(1) << 37;
    CHECK(zsmr_clip_flatten(ptrs.data(), &sizes[1], dtypes.data(), 1, coef, P, flat, ZSMR_BF16, nullptr) == ZSMR_OK);
    CHECK(g_clip.size() == 1 && g_clip[0].count == 2 && int64_t(g_clip[0].chunks) * 256 <= MOST);
    CHECK(g_clip[0].it[0].n == flat - 3 && g_clip[0].it[0].src == nullptr && g_clip[0].it[1].n == 3);
    g_clip.clear(); g_norm.clear(); g_join.clear();
    const int64_t over = item + 1;
    CHECK(zsmr_clip_grads(ptrs.data(), &over, dtypes.data(), 1, coef, nullptr) == ZSMR_ERR_ARG);
    CHECK(zsmr_grad_norm(ptrs.data(), &over, dtypes.data(), 1, 1, 0, (float*)P, P, MOST, nullptr) == ZSMR_ERR_ARG);
    CHECK(zsmr_clip_flatten(ptrs.data(), &over, dtypes.data(), 1, coef, P, over, ZSMR_BF16, nullptr) == ZSMR_ERR_ARG);
    CHECK(zsmr_clip_flatten(ptrs.data(), &sizes[1], dtypes.data(), 1, coef, P, 3 + over, ZSMR_BF16, nullptr) == ZSMR_ERR_ARG);
    CHECK(g_clip.empty() && g_norm.empty() && g_join.empty());
    CHECK(zsmr_clip_grads(ptrs.data(), &item, dtypes.data(), 1, coef, nullptr) == ZSMR_OK && int64_t(g_clip[0].chunks) * 256 <= MOST);
    g_clip.clear();
}

static void pieces() {
    const zsmr_adam hp = {1e-3, 0.9, 0.999, 1e-8};
    for (int over = 0; over < 2; ++over) {
        const int64_t n = zsmr::kMaxGroups * zsmr::kTile + over;
        zsmr_ctx* c = nullptr;
        CHECK(zero_init_shards(&c, n, 1, ZSMR_ZERO2, ZSMR_BF16, ZSMR_BF16, 0, nullptr, 0) == ZSMR_OK);
        g_step.clear();
        const int32_t want = over ? ZSMR_ERR_ARG : ZSMR_OK;
        CHECK(zero_reduce_shard_sumsq(c, 0, 0, P, n, 0, 1, (float*)P, (double*)P, P, zsmr_norm_workspace(n, 1), nullptr) == want);
        CHECK(zero_clipped_step(c, 0, 0, (float*)P, nullptr, (float*)P, (float*)P, (float*)P, P, 1, &hp, nullptr) == want);
        CHECK(g_step.size() == (over ? 0u : 2u));
        zero_destroy(c);
    }
}

int main() {
    lists();
    pieces();
    std::printf("host checks passed\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_largest_sizes(tmp_path, monkeypatch):
    monkeypatch.setattr(base, "DRIVER", host.DRIVER.split("static void list(")[0] + MAIN)
    exe = base._compile(tmp_path, [base.CSRC + "/zsmr_ops_api.cpp", "-Wno-unused-variable", "-fsanitize=address,undefined",
                                   "-fno-sanitize-recover=all"])
    base._run(exe, {"ASAN_OPTIONS": "detect_leaks=1:halt_on_error=1:verify_asan_link_order=0"})
