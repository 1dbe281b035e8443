"""What the scores of logits launch, from sizes alone: a C++ driver walks
``csrc/zsmr_scores_plan.h``, which the library's host code follows, to the largest
sizes that ``zsmr_ops.h`` accepts.  No GPU; built with g++, under AddressSanitizer
and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

from tests.test_xent_plan import compile_driver

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "zsmr_scores_plan.h"
#define CHECK(c) do { if (!(c)) { std::printf("CHECK failed line %d: %s (%lld x %lld)\n", __LINE__, #c, (long long)t, (long long)v); std::exit(1); } } while (0)
using namespace zsmr;

static int launches(int64_t t, int64_t v) {
    const ScoreShape s = score_shape(t, v, 20);
    int64_t at = 0;
    int n = 0;
    score_launches(s, t, [&](int64_t first, int64_t count) {
        CHECK(first == at && count > 0);
        CHECK(count * s.waves * 64 < (int64_t(1) << 32));       // a launch has fewer work items
        at += count;
        ++n;
    });
    CHECK(at == t * s.splits);
    return n;
}

// Rows in segments: one launch, whose workgroups one launch of the join follows.
static void segments(int64_t t, int64_t v) {
    const ScoreShape s = score_shape(t, v, 64);
    CHECK(s.splits >= 1 && (s.splits == 1 || t * s.splits <= kScoreSplits));
    CHECK(s.splits == 1 || launches(t, v) == 1);
    CHECK((s.splits - 1) * s.segment < v && s.splits * s.segment >= v);
}

int main() {
    for (int64_t t = 1; t <= 1100; ++t)
        for (int64_t v : {1, 8191, 8192, 65536, 65537, 70000, 100000, 128256, 500000, 2097151, 2097152}) segments(t, v);
    for (int64_t t : {1, 2, 16, 255, 256, 257, 4096, 1 << 20, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, 10000000, 1 << 24})
        for (int64_t v : {1, 500, 8191, 8192, 50257, 128256, 1 << 21}) launches(t, v);
    const int64_t t = 1 << 24, v = 8192;
    CHECK(launches(t, v) == 3 && launches((1 << 23) - 1, v) == 1 && launches(1 << 23, v) == 2 && launches(t, v - 1) == 1);
    std::printf("launches passed\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_launches_hold_their_work_items(tmp_path):
    exe = compile_driver(tmp_path, DRIVER, ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"])
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, env=env)
    assert r.returncode == 0 and "launches passed" in r.stdout, r.stdout + r.stderr
