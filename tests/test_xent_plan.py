"""What the softmax cross entropy launches, from sizes alone: a C++ driver walks
``csrc/zsmr_xent_plan.h``, which the library's host code follows, over every corner
of the sizes that the header ``zsmr_ops.h`` accepts.  No GPU; built with g++, also
under AddressSanitizer and UndefinedBehaviorSanitizer.

* The pieces are whole tiles, at least one, and cover the vocabulary once; the
  tiles of each product cover its sides, its splits all of k.
* No launch has 2^32 work items.
* Every part of the workspace holds what the products put there.
* The shapes of the GPU tests select every form of the product kernel there is.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_mixed_reduce_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "zsmr_xent_plan.h"
using namespace zsmr;
#define CHECK(c) do { if (!(c)) { std::printf("CHECK failed line %d: %s (%lld tokens, vocabulary %lld, width %lld)\n", __LINE__, #c, \
                                              (long long)g_n, (long long)g_v, (long long)g_h); std::exit(1); } } while (0)
static int64_t g_n, g_v, g_h;

static void check(int64_t n, int64_t v, int64_t h) {
    g_n = n; g_v = v; g_h = h;
    const int64_t piece = piece_of(n, v, h), packed = packed_piece(n, v, h);
    CHECK(piece >= BM && piece % BM == 0 && piece <= kMaxPiece);
    CHECK(packed >= BM && packed % BM == 0 && packed <= piece && packed <= 32768);
    CHECK(n * piece * 2 <= std::max(int64_t(1) << 29, n * 512));
    for (int backward = 0; backward < 2; ++backward) {
        const XentSpace s = xent_space(n, v, h, backward);
        CHECK(s.bytes > 0 || n == 0);
        const int64_t ends[] = {s.target, s.x, s.w, backward ? s.mul : s.bytes};
        const int64_t starts[] = {s.stats, s.target, s.x, s.w}, row = ceil_to(h, 8) * 2;
        const int64_t need[] = {tiles_of(v, BM) * n * 8, n * 4, n * row, packed * row};
        for (int i = 0; i < 4; ++i) CHECK(starts[i] % 256 == 0 && ends[i] - starts[i] >= need[i]);
        if (backward) CHECK(s.g - s.mul >= 8 && s.sum - s.g >= n * piece * 2 && s.bytes > s.sum - 1);
    }
    // a call's products; pieces of the largest vocabularies repeat, so their number is bounded by the sizes
    if (v / piece > 600) return;
    for (int pack = 0; pack < 2; ++pack) {
        const int64_t rows = pack ? packed : piece;
        {
            int64_t at = 0;
            forward_products(n, v, h, pack, [&](const ProductShape& p) {
                CHECK(p.grid() * 512 < (int64_t(1) << 32));
                CHECK(p.epi == E_STATS && p.v0 == at && p.v0 % BM == 0 && p.rows > 0);
                CHECK(!pack || p.rows <= packed);
                CHECK(p.m_tiles * BM >= p.rows && (p.m_tiles - 1) * BM < p.rows);
                CHECK(p.n_tiles * p.tile >= n && (p.n_tiles - 1) * p.tile < n && p.splits == 1 && p.k >= h && p.k < h + 8 && p.k_split >= p.k);
                at += p.rows;
            });
            CHECK(at == v);
        }
        int64_t at = 0, seen[4] = {0, 0, 0, 0};
        backward_products(n, v, h, pack, true, true, [&](const ProductShape& p) {
            if (p.epi == (n ? E_GRAD : E_DW)) { CHECK(p.v0 == at); at += p.rows; }
            ++seen[p.epi];
            CHECK(p.rows > 0 && p.rows <= rows && p.v0 + p.rows == at);
            // x and w of 550 GB at most: no card holds more
            CHECK(p.grid() * 512 < (int64_t(1) << 32) || n * h > (int64_t(1) << 38) || v * h > (int64_t(1) << 38));
            CHECK(p.k_split % BK == 0 && p.k_split * p.splits >= p.k && p.splits >= 1);
            const int64_t m = p.epi == E_GRAD ? p.rows : h, across = p.epi == E_DW ? p.rows : n;
            CHECK(p.m_tiles * BM >= m && (p.m_tiles - 1) * BM < m && p.n_tiles * p.tile >= across && (p.n_tiles - 1) * p.tile < across);
            CHECK(p.k >= (p.epi == E_GRAD ? h : p.epi == E_DX ? p.rows : n));
            if (p.epi == E_GRAD) CHECK(p.m_tiles * BM <= rows);         // G's rows hold whole tiles
            if (p.epi == E_DX) {
                CHECK(p.sum_in == (p.v0 > 0) && p.sum_out == (p.splits > 1 || at < v));
                const XentSpace s = xent_space(n, v, h, true);
                CHECK(s.bytes - s.sum >= p.splits * n * ceil_to(h, 4) * 4);
            }
        });
        CHECK(at == v && (!n || (seen[E_DX] == seen[E_DW] && seen[E_GRAD] == seen[E_DW])));
    }
}

int main() {
    const int64_t edges[] = {0, 1, 2, 15, 16, 64, 65, 128, 192, 255, 256, 257, 1000, 4096, 8192, 33500, 50257, 65536, 65537, 65793, 70000, 128256,
                             524287, 524288, 524289, 600000, 1 << 20, (1 << 20) + 1, ZSMR_MAX_WIDTH - 1, ZSMR_MAX_WIDTH, 5000000,
                             ZSMR_MAX_TOKENS - 1, ZSMR_MAX_TOKENS, ZSMR_MAX_VOCAB - 255, ZSMR_MAX_VOCAB};
    int cases = 0;
    for (int64_t n : edges) for (int64_t v : edges) for (int64_t h : edges) {
        if (n > ZSMR_MAX_TOKENS || v < 1 || h < 1 || h > ZSMR_MAX_WIDTH) continue;
        check(n, v, h);
        ++cases;
    }
    uint64_t r = 1;
    auto next = [&](int64_t most) {         // sizes over their logarithm
        r = r * 6364136223846793005ull + 1442695040888963407ull;
        int bits = 0;
        while ((most >> bits) > 1) ++bits;
        const int64_t top = int64_t(1) << ((r >> 33) % (bits + 1));
        r = r * 6364136223846793005ull + 1442695040888963407ull;
        return std::min<int64_t>(most, top + (int64_t)((r >> 20) % top));
    };
    for (int i = 0; i < 5000; ++i) check(next(ZSMR_MAX_TOKENS), next(ZSMR_MAX_VOCAB), next(ZSMR_MAX_WIDTH));
    std::printf("plan checks passed: %d edge cases\n", cases);
    return 0;
}
"""


def compile_driver(tmp_path, source, extra=()):
    src, exe = tmp_path / "plan_driver.cpp", tmp_path / "plan_driver"
    src.write_text(source)
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-I", os.path.join(ROCM, "include"), *extra, str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("sanitize", [False, True])
def test_plan_over_the_accepted_sizes(tmp_path, sanitize):
    extra = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"] if sanitize else []
    exe = compile_driver(tmp_path, DRIVER, extra)
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "plan checks passed" in r.stdout, (r.stdout + r.stderr)[-4000:]


VARIANTS = r"""
#include <cstdio>
#include <cstdlib>
#include "zsmr_xent_plan.h"
using namespace zsmr;
int main(int argc, char** argv) {
    for (int i = 1; i + 2 < argc; i += 3) {
        const int64_t n = std::atoll(argv[i]), v = std::atoll(argv[i + 1]), h = std::atoll(argv[i + 2]);
        auto print = [&](const ProductShape& p) {
            std::printf("%d %d %d %d %s\n", p.epi, p.tile, p.stages, p.once, p.epi != E_DX ? "-" : p.sum_in ? p.sum_out ? "middle" : "last" : p.sum_out ? "first" : "only");
        };
        forward_products(n, v, h, h % 8 != 0, print);
        backward_products(n, v, h, h % 8 != 0, true, true, print);
    }
    return 0;
}
"""
# as zsmr_xent.hip has them: tile, stages, once
TOKEN_TILES = [(64, 2, 1), (64, 4, 0), (128, 3, 1), (128, 3, 0), (192, 2, 0), (256, 2, 0)]


def variants_of(exe, shapes):
    out = subprocess.run([str(exe)] + [str(k) for shape in shapes for k in shape], capture_output=True, text=True, check=True, timeout=60).stdout
    return {tuple(line.split()) for line in out.splitlines()}


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_gpu_tests_shapes_select_every_form(tmp_path):
    from tests.test_gpu_ops_variants import XENT_SHAPES
    exe = compile_driver(tmp_path, VARIANTS)
    seen = variants_of(exe, XENT_SHAPES)
    forms = {v[:4] for v in seen}
    for epi in "012":
        assert forms >= {(epi, str(t), str(s), str(o)) for t, s, o in TOKEN_TILES}, epi
    assert {v for v in forms if v[0] == "3"} == {("3", "128", "3", "0"), ("3", "256", "2", "0")}
    assert len(forms) == 3 * len(TOKEN_TILES) + 2, "a form that zsmr_xent.hip does not have"
    # dx adds what earlier pieces left, and leaves sums for later ones, in each wide tile
    for tile in ("128", "192", "256"):
        assert {v[4] for v in seen if v[:2] == ("2", tile)} == {"only", "first", "middle", "last"}, tile
    # and so does the largest workload of this repository: four pieces, one split
    assert ("2", "256", "2", "0", "last") in variants_of(exe, [(8192, 128256, 4096)])
