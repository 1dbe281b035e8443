"""Launches beyond what a grid holds go out in parts: a C++ driver (g++, no GPU)
checks that the parts of ``csrc/zsmr_ops_launch.h`` cover all rows once, in order, and
that none has 2^32 work items."""
import os
import shutil
import subprocess

import pytest

from tests.test_xent_plan import compile_driver

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "zsmr_ops.h"
#include "zsmr_ops_launch.h"
#define CHECK(c) do { if (!(c)) { std::printf("CHECK failed line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

static int parts(int64_t rows, int64_t items) {
    int64_t at = 0;
    int n = 0;
    zsmr::launch_rows(rows, items, [&](int64_t first, int64_t count) {
        CHECK(first == at && count > 0 && first + count <= rows);
        const int64_t groups = (count * items + 255) / 256;
        CHECK(groups > 0 && groups * 256 < (int64_t(1) << 32));
        at += count;
        ++n;
    });
    CHECK(at == rows);
    return n;
}

int main() {
    const int64_t tokens = ZSMR_MAX_TOKENS, vecs = ZSMR_MAX_WIDTH / 8;
    CHECK(parts(0, 1) == 0 && parts(1, 1) == 1 && parts(1, vecs) == 1);
    CHECK(parts(tokens, 1) == 1 && parts(tokens, 255) == 1 && parts(tokens, 256) == 2 && parts(tokens, 257) == 2);
    // 16,383 rows of 2^18 work items are the most of a launch
    CHECK(parts(tokens, vecs) == 1025 && parts(16383, vecs) == 1 && parts(16384, vecs) == 2);
    int64_t groups = 0, launches = 0;
    zsmr::launch_groups(ZSMR_MAX_VOCAB / 16 + 1000, [&](int64_t first, int64_t count) {
        CHECK(first == groups && count * 256 < (int64_t(1) << 32));
        groups += count;
        ++launches;
    });
    CHECK(groups == ZSMR_MAX_VOCAB / 16 + 1000 && launches == 5);
    std::printf("parts passed\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_parts_cover_everything(tmp_path):
    exe = compile_driver(tmp_path, DRIVER, ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"])
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, env=env)
    assert r.returncode == 0 and "parts passed" in r.stdout, r.stdout + r.stderr
