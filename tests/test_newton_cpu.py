"""The orthogonalised update, its shard step and the scores of logits on a machine
without a GPU: refusals before anything is launched, sizes of workspaces, what the
binding checks, and the host arithmetic of the plans.  Addresses are placeholders
that nothing reads."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.test_xent_plan import compile_driver
from zero_sharded_mixed_reduce_amd import ops

A, B, C, D, W = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20     # 16-byte aligned
BIG = 1 << 50
L = ops._lib()
ARG, DTYPE, ALIGN = z.ZSMR_ERR_ARG, z.ZSMR_ERR_DTYPE, z.ZSMR_ERR_ALIGN
BF16, F32 = z.ZSMR_BF16, 3


def newton(coefs=ops.NS_COEFS, eps=1e-7, steps=None):
    ns = ops.zsmr_newton(eps, len(coefs) if steps is None else steps, 0)
    for i, triple in enumerate(coefs):
        ns.coef[i][:] = triple
    return ns


NS = newton()
ORTHOGONALIZE = dict(x=A, xd=BF16, xs=180, xb=36000, out=B, od=F32, os=180, ob=36000, rows=200, cols=180, count=3, ns=NS, ws=W, wb=BIG, stream=None)
NAN, INF = float("nan"), float("inf")
BAD_NS = [newton(eps=-1.0), newton(eps=NAN), newton(eps=INF), newton(steps=0), newton(steps=17), newton(((NAN, 0, 0),)), newton(((0, INF, 0),)),
          newton(((182.0, 0, 0),)), newton(((100.0, 0, 0), (2.0, 0, 0))), newton(((1.0, 0, 0), (1e308, 1e308, 1e308))), newton(((1.0, 1e6, -1e6),))]


@pytest.mark.parametrize("change,code", [
    (dict(x=None), ARG), (dict(out=None), ARG), (dict(rows=0), ARG), (dict(cols=0), ARG), (dict(rows=(1 << 18) + 1), ARG), (dict(rows=-1), ARG),
    (dict(rows=1 << 17, cols=(1 << 16) + 1), ARG), (dict(count=-1), ARG), (dict(count=(1 << 20) + 1), ARG), (dict(xs=179), ARG), (dict(os=179), ARG),
    (dict(xs=(1 << 21) + 1), ARG), (dict(xb=-1), ARG), (dict(ob=35999), ARG), (dict(ob=180, os=539), ARG), (dict(ob=179, os=540), ARG),
    (dict(xb=(1 << 40) + 1), ARG), (dict(ns=None), ARG), (dict(ws=None), ARG), (dict(wb=1000), ARG), (dict(xd=4), DTYPE), (dict(od=0), DTYPE),
    (dict(x=A + 1), ALIGN), (dict(out=B + 2), ALIGN), (dict(x=A + 2, xd=F32), ALIGN), (dict(ws=W + 8), ALIGN)] + [(dict(ns=ns), ARG) for ns in BAD_NS])
def test_orthogonalize_refusals(change, code):
    assert L.zsmr_orthogonalize(*(ORTHOGONALIZE | change).values()) == code


def test_nothing_to_orthogonalize():
    assert L.zsmr_orthogonalize(*(ORTHOGONALIZE | dict(count=0, x=None, out=None, ws=None, wb=0)).values()) == 0
    assert z.zsmr_orthogonalize_workspace(10, 10, 0) == 0


def test_workspaces():
    # X twice and two inner matrices, 4 bytes an element; three more inner matrices where steps go in groups
    assert 0 <= z.zsmr_orthogonalize_workspace(4096, 4096) - 4 * 4 * 4096 ** 2 < 1e5
    assert 0 <= z.zsmr_orthogonalize_workspace(4096, 8192) - (4 + 5) * 4 * 4096 ** 2 < 1e5
    assert z.zsmr_orthogonalize_workspace(300, 150, 7) == z.zsmr_orthogonalize_workspace(150, 300, 7) == z.zero_muon_workspace(150, 300, 7) > 0
    assert z.zsmr_orthogonalize_workspace(128, 128, 1000) == 0      # in a CU's LDS
    # a group's matrices at a time
    assert z.zsmr_orthogonalize_workspace(1024, 1024, 1 << 20) < 6.5e8
    assert z.zsmr_orthogonalize_workspace(1, 1, 1 << 20) < 6.5e8
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, -1), ((1 << 18) + 1, 1, 1), (1 << 17, 1 << 17, 1), (1, 1, (1 << 20) + 1)):
        with pytest.raises(z.ZsmrError):
            z.zsmr_orthogonalize_workspace(*bad)
    assert z.zsmr_logprobs_workspace(0, 10) == z.zsmr_logprobs_workspace(8192, 128256, 20) == 0
    assert z.zsmr_logprobs_workspace(1, 128256, 20) >= 16 + 8 * 20
    for bad in ((-1, 10, 0), (1, 0, 0), (1, 10, 11), (1, 100, 65), (1, 100, -1), ((1 << 24) + 1, 10, 0), (1, (1 << 21) + 1, 0)):
        with pytest.raises(z.ZsmrError):
            z.zsmr_logprobs_workspace(*bad)


def test_muon_refusals_count_nothing():
    hp = lambda **kw: ops.zsmr_muon(**(dict(lr=0.02, beta=0.9, weight_decay=0.1, scale=1.0, nesterov=1, pad=0) | kw))  # noqa: E731
    ctx = z.zero_init_shards(201000, 3, z.ZSMR_ZERO3_OWNER, "bf16", units=[1000, 200000])
    z.zero_set_unit_owners(ctx, [2, 0])
    ok = dict(ctx=ctx.handle, rank=0, unit=1, begin=100, rows=200, cols=300, count=3, grads=A, stride=200000, base=0, master=B, momentum=C, p16=D,
              hp=hp(), ns=NS, ws=W, wb=BIG, stream=None)
    bad = [(dict(ctx=None), ARG), (dict(rank=3), ARG), (dict(rank=1), ARG), (dict(unit=2), ARG), (dict(begin=-1), ARG), (dict(begin=20001), ARG),
           (dict(rows=0), ARG), (dict(count=4), ARG), (dict(count=-1), ARG), (dict(grads=None), ARG), (dict(stride=199999), ARG), (dict(base=-1), ARG),
           (dict(master=None), ARG), (dict(momentum=None), ARG), (dict(p16=None), ARG), (dict(hp=None), ARG), (dict(ns=None), ARG), (dict(ws=None), ARG),
           (dict(wb=100), ARG), (dict(rows=1 << 18, cols=1 << 15, count=1 << 20), ARG), (dict(grads=A + 1), ALIGN), (dict(master=B + 2), ALIGN),
           (dict(momentum=C + 1), ALIGN), (dict(p16=D + 1), ALIGN), (dict(ws=W + 4), ALIGN)]
    bad += [(dict(hp=hp(**{k: v})), ARG) for k, v in (("lr", -1.0), ("lr", NAN), ("beta", 1.0), ("beta", -0.1), ("weight_decay", INF),
                                                      ("weight_decay", -1.0), ("scale", -1.0), ("scale", NAN), ("nesterov", 2))]
    bad += [(dict(ns=ns), ARG) for ns in BAD_NS]
    for change, code in bad:
        assert L.zero_muon_step(*(ok | change).values()) == code, change
    # no matrices, also on a rank that holds nothing
    assert L.zero_muon_step(*(ok | dict(count=0, grads=None, master=None, momentum=None, p16=None, ws=None)).values()) == 0
    assert L.zero_muon_step(*(ok | dict(rank=1, begin=0, count=0)).values()) == 0
    whole = z.zero_init_shards(1000, 2, z.ZSMR_DP, "bf16")
    dp = ok | dict(ctx=whole.handle, unit=0, begin=0, rows=10, cols=50, count=1)
    assert L.zero_muon_step(*dp.values()) == ARG            # half of a replica's vector
    assert all(z.zero_counters(c, r)["traffic_elems"] == 0 for c in (ctx, whole) for r in range(2))


LOGPROBS = dict(logits=A, stride=100, dtype=F32, ids=B, id_bytes=8, n=5, vocab=100, scale=1.0, logprob=C, lse=C, entropy=C, top=4, top_ids=D,
                top_bytes=8, top_logprobs=D, ws=W, wb=BIG, stream=None)
GRAD = dict(logits=A, stride=100, dtype=F32, ids=B, id_bytes=8, n=5, vocab=100, scale=1.0, lse=C, entropy=C, g=C, h=C, dlogits=D, ds=100, stream=None)
COMMON = [(dict(logits=None), ARG), (dict(stride=99), ARG), (dict(stride=(1 << 21) + 1), ARG), (dict(dtype=0), DTYPE), (dict(dtype=4), DTYPE),
          (dict(ids=None), ARG), (dict(id_bytes=2), ARG), (dict(n=-1), ARG), (dict(n=(1 << 24) + 1), ARG), (dict(vocab=0), ARG),
          (dict(vocab=(1 << 21) + 1), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(scale=1e31), ARG), (dict(scale=1e-31), ARG),
          (dict(logits=A + 2), ALIGN), (dict(ids=B + 4), ALIGN), (dict(lse=C + 2), ALIGN), (dict(entropy=C + 1), ALIGN)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(top=-1), ARG), (dict(top=65, vocab=100), ARG), (dict(top=11, vocab=10), ARG), (dict(top_bytes=2), ARG), (dict(logprob=C + 2), ALIGN),
    (dict(top_ids=D + 4), ALIGN), (dict(top_logprobs=D + 2), ALIGN), (dict(vocab=10 ** 6, stride=10 ** 6, wb=10), ARG),
    (dict(vocab=10 ** 6, stride=10 ** 6, ws=None), ARG), (dict(ws=W + 8), ALIGN)])
def test_logprobs_refusals(change, code):
    assert L.zsmr_logprobs(*(LOGPROBS | change).values()) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(dlogits=None), ARG), (dict(ds=99), ARG), (dict(lse=None), ARG), (dict(entropy=None), ARG), (dict(dlogits=A, ds=101), ARG),
    (dict(dlogits=D + 1), ALIGN), (dict(g=C + 2), ALIGN), (dict(h=C + 2), ALIGN)])
def test_logprobs_grad_refusals(change, code):
    assert L.zsmr_logprobs_grad(*(GRAD | change).values()) == code


def test_no_scores_launch_nothing():
    assert L.zsmr_logprobs(*(LOGPROBS | dict(n=0, logits=None, ids=None)).values()) == 0
    assert L.zsmr_logprobs(*(LOGPROBS | dict(logprob=None, ids=None, lse=None, entropy=None, top=0)).values()) == 0
    assert L.zsmr_logprobs(*(LOGPROBS | dict(logprob=None, ids=None, lse=None, entropy=None, top_ids=None, top_logprobs=None)).values()) == 0
    assert L.zsmr_logprobs_grad(*(GRAD | dict(n=0, logits=None, ids=None, lse=None, entropy=None, dlogits=None)).values()) == 0


def test_binding_checks_tensors_before_the_library():
    x, ws = torch.zeros(2, 6, 8), torch.zeros(64, dtype=torch.uint8)
    for bad, kw, why in (((x, x[:1], ws), {}, "out"), ((x, x[:, :5], ws), {}, "out"), ((x[0, 0], x, ws), {}, "a matrix or a stack"),
                         ((x.long(), x, ws), {}, "fp16, bf16 or fp32"), ((x.mT, x.mT, ws), {}, "contiguous"), ((x, x, ws[::2]), {}, "workspace"),
                         ((x.as_strided((2, 6, 8), (48, 7, 1)), x, ws), {}, "overlap"), ((x, x, ws), {"coefs": ()}, "coefs"),
                         ((x, x, ws), {"coefs": ((1.0, 2.0),)}, "coefs"), ((x, x, ws), {"coefs": ((1.0, 2.0, 3.0),) * 17}, "coefs"),
                         ((x, x, ws), {"coefs": 3}, None), ((x, x, ws), {}, "host memory")):
        with pytest.raises((ValueError, TypeError), match=why):
            z.zsmr_orthogonalize(*bad, stream=0, **kw)
    ctx = z.zero_init_shards(200, 2, z.ZSMR_ZERO2, "bf16")
    rows, f, h = torch.zeros(2, 200, dtype=torch.bfloat16), torch.zeros(100), torch.zeros(100, dtype=torch.bfloat16)
    ok = dict(ctx=ctx, rank=1, unit=0, begin=4, rows=8, cols=12, count=1, grads=rows, row_stride=200, base_elem=100, master=f, momentum=f, p16_dst=h, ws=ws,
              lr=0.1, stream=0)
    for change, why in ((dict(grads=rows[:1]), "grads"), (dict(base_elem=101), "grads"), (dict(master=f[:99]), "master"), (dict(momentum=h), "momentum"),
                        (dict(p16_dst=h[1:]), "p16_dst"), (dict(count=1 << 64), "int64"), (dict(rank=1 << 40), "int32"), ({}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zero_muon_step(**(ok | change))
    with pytest.raises(z.ZsmrError) as e:       # past the piece: the library's own check
        z.zero_muon_step(**(ok | dict(begin=5, grads=A, master=B, momentum=C, p16_dst=D, ws=W)))
    assert e.value.code == ARG
    t, ids, n3 = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    top, val = torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, 4)
    ok = dict(logits=t, ids=ids, logprob=n3, lse=n3, entropy=n3, ws=ws, stream=0)
    for change, why in ((dict(logits=t[0]), "logits"), (dict(logits=t.t()), "token ids|contiguous"), (dict(logits=t.double()), "logits"),
                        (dict(ids=ids[:2]), "token ids"), (dict(ids=ids.float()), "token ids"), (dict(lse=n3[:2]), "lse"),
                        (dict(entropy=n3.double()), "entropy"), (dict(top_ids=top.float()), "top_ids"), (dict(top_ids=top[:2]), "top_ids"),
                        (dict(top_ids=top, top_logprobs=val[:, :3].contiguous()), "top_logprobs"), (dict(top_logprobs=val.t()), "top_logprobs"),
                        (dict(top_ids=torch.zeros(3, 65, dtype=torch.int64)), "top_ids"), ({}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_logprobs(**(ok | change))
    ok = dict(logits=t, ids=ids, lse=n3, entropy=n3, dlogits=t, stream=0)
    for change, why in ((dict(dlogits=t[:2]), "dlogits"), (dict(dlogits=t.half()), "format"), (dict(dlogprob=n3[:1]), "dlogprob"),
                        (dict(dentropy=ids), "dentropy"), ({}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_logprobs_grad(**(ok | change))


PLAN = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "zsmr_newton_plan.h"
#include "zsmr_scores_plan.h"
#define CHECK(c) do { if (!(c)) { std::printf("CHECK failed line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)
using namespace zsmr;

static void grids(const NsShape& s, int64_t products) {
    for (int kind : {N_INNER, N_UPDATE, N_LAST})
        for (int64_t steps : {s.mp / 32, s.np / 32}) {
            for (int gram = 0; gram < (kind == N_INNER && steps == s.np / 32 ? 2 : 1); ++gram) {
                const NsGrid g = ns_grid(s, kind, products, steps, gram);
                CHECK((int64_t)g.p_tiles * 128 >= (kind == N_INNER ? s.m : s.n) && (int64_t)g.q_tiles * 128 >= s.m);
                CHECK(g.tiles == (kind == N_INNER ? (int64_t)g.q_tiles * (g.q_tiles + 1) / 2 : (int64_t)g.p_tiles * g.q_tiles));
                int64_t at = 0;
                for (int i = 0; i < g.parts; ++i) {
                    const NsPart& p = g.part[i];
                    CHECK(p.first == at && p.count > 0 && p.form >= NS_WIDE && p.form <= NS_PAIR);
                    CHECK(ns_groups(p) * 512 < (int64_t(1) << 32) && p.first + p.count <= INT32_MAX / 4);
                    at += p.count;
                }
                CHECK(g.parts >= 1 && g.parts <= 2 && at == (int64_t)g.tiles * products && g.us > 0);
                // split steps: one launch, every part has some, and the sums fit X's other copy
                CHECK(g.split == 1 ? g.split_steps == steps : gram && g.parts == 1 && g.split <= kNsMaxSplit);
                CHECK((int64_t)g.split * g.split_steps >= steps && (int64_t)(g.split - 1) * g.split_steps < steps);
                CHECK(g.split == 1 || at * g.split * kNsTileBytes <= products * s.m * s.np * 4);
            }
        }
}

static void shape(int64_t rows, int64_t cols, int64_t count) {
    for (int fp32 = 0; fp32 < 2; ++fp32) {
        const NsShape s = ns_shape(rows, cols, count, fp32);
        CHECK(s.m <= s.n && s.m * s.n == rows * cols && s.tall == (rows > cols));
        CHECK(s.mp >= s.m && s.mp % 32 == 0 && s.np >= s.n && s.np % 32 == 0);
        CHECK(s.group >= 1 && s.group <= count && s.parts >= 1);
        CHECK(s.group == 1 || s.group * s.m * s.n <= kNsGroupElems);
        const NsSpace w = ns_space(s);
        if (s.small) {      // a form that holds it
            CHECK(s.m <= (s.small == 3 ? 128 : 64) && s.n <= (s.small == 1 ? 64 : s.small == 2 ? 256 : 128) && w.bytes == 0);
            continue;
        }
        int64_t end = 0;
        for (int i = 0; i < kNsMatrices; ++i) {
            const bool x = i == M_X0 || i == M_X1, used = x || i == M_A || i == M_Q0 || s.grouped;
            CHECK(w.matrix[i] >= end && w.matrix[i] % 256 == 0);
            end = w.matrix[i] + (used ? s.group * s.m * (x ? s.np : s.mp) * 4 : 0);
        }
        CHECK(w.partial >= end && w.partial % 256 == 0 && w.inverse >= w.partial + s.group * s.parts * 8 && w.bytes >= w.inverse + s.group * 8);
        // work items of a launch, byte offsets within an operand's tile
        CHECK(s.group * s.parts < (int64_t(1) << 24) && s.group * ((s.m + 63) / 64) * ((s.np + 63) / 64) * 256 < (int64_t(1) << 32));
        CHECK(256 * s.np * 4 < (int64_t(1) << 31));
        grids(s, 1);
        grids(s, s.group);
        grids(s, 2 * s.group);
    }
}

static void scores(int64_t tokens, int64_t vocab, int64_t top) {
    const ScoreShape s = score_shape(tokens, vocab, top);
    CHECK(s.splits >= 1 && s.segment % kScoreBlock == 0 && s.segment * s.splits >= vocab && s.segment * (s.splits - 1) < vocab);
    CHECK(s.splits == 1 ? s.bytes == 0 : s.bytes >= tokens * s.splits * (16 + 8 * top));
    CHECK(s.splits == 1 || tokens * s.splits <= 4096);
}

// The power of two that a factor rounded to fp32 stands for.
static double power(double x) {
    const double p = std::exp2(std::round(std::log2(x)));
    CHECK(std::fabs(x / p - 1) < 1e-6);
    return p;
}

// Every matrix stays in fp16's range: the polynomial on singular values, in double.
static void scales(const double (*coef)[3], int steps) {
    NsPass pass[ZSMR_MAX_NS_STEPS];
    double first = 0;
    CHECK(ns_passes(coef, steps, pass, &first));
    CHECK(first >= 16384 && first <= 32768);
    for (int k = 0; k <= 10000; ++k) {
        double x = k / 10000.0, sx = first;
        for (int i = 0; i < steps; ++i) {
            const double a = x * x, sa = pass[i].a_mul * sx * sx, b = coef[i][1] * a + coef[i][2] * a * a;
            CHECK(a * sa <= 32800);
            const double sb = power(coef[i][2] != 0 ? pass[i].b_mul * sa * sa / coef[i][2] : coef[i][1] != 0 ? pass[i].b_old * sa / coef[i][1] : 32768);
            CHECK(std::fabs(b) * sb <= 32800);
            const double y = coef[i][0] * x + b * x, next = pass[i].x_mul * sb * sx;
            CHECK(std::fabs(pass[i].x_old - coef[i][0] * next / sx) <= 1e-6 * std::fabs(pass[i].x_old));
            CHECK(i + 1 == steps ? next == 1 : std::fabs(y) * next <= 32800);
            x = std::fabs(y);
            sx = next;
        }
    }
}

// A list of products on one singular value: every matrix is a number.
static void lists(const double (*coef)[3], int steps) {
    NsPass pass[ZSMR_MAX_NS_STEPS];
    double first = 0;
    CHECK(ns_passes(coef, steps, pass, &first));
    for (int grouped = 0; grouped < 2; ++grouped) {
        NsOp ops[kNsMaxOps + 1];
        const int n = ns_ops(coef, steps, grouped, ops);
        CHECK(n > 0 && n <= kNsMaxOps && (grouped || n == 3 * steps) && ops[n - 1].kind == N_LAST);
        for (int k = 0; k <= 1000; ++k) {
            const double s = k / 1000.0;
            double v[kNsMatrices], want = s;
            bool has[kNsMatrices] = {true};
            v[M_X0] = s * first;
            for (int i = 0; i < n; ++i) {
                const NsOp& o = ops[i];
                CHECK(has[o.p] && has[o.q] && (o.old < 0 || has[o.old]) && (o.old2 < 0 || has[o.old2]));
                // nothing is written that the launch reads
                CHECK(o.dst != o.p && o.dst != o.q && o.dst != o.old && o.dst != o.old2);
                if (o.paired) {
                    const NsOp& t = ops[i + 1];
                    CHECK(!t.paired && t.kind == N_INNER && t.dst != o.dst && t.dst != o.p && t.dst != o.q && t.dst != o.old && t.dst != o.old2);
                    CHECK(o.dst != t.p && o.dst != t.q && o.dst != t.old && o.dst != t.old2);
                    CHECK((o.p == M_X0 || o.p == M_X1) == (t.p == M_X0 || t.p == M_X1));
                }
                const double r = o.mul * v[o.p] * v[o.q] + (o.old < 0 ? 0 : o.old_mul * v[o.old]) + (o.old2 < 0 ? 0 : o.old2_mul * v[o.old2]);
                CHECK(std::fabs(r) <= 32900);
                v[o.dst] = r;
                has[o.dst] = true;
            }
            for (int i = 0; i < steps; ++i) want *= coef[i][0] + want * want * (coef[i][1] + want * want * coef[i][2]);
            CHECK(std::fabs(v[ops[n - 1].dst] - want) <= 2e-4 * (1 + std::fabs(want)));
        }
    }
}

int main() {
    for (int64_t r : {1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 767, 1003, 1024, 1600, 2048, 4096, 6400, 14336, 65536, 262144})
        for (int64_t c : {1, 5, 32, 64, 100, 128, 129, 192, 193, 320, 1000, 1600, 2049, 4096, 5000, 14336, 32768, 262144})
            for (int64_t n : {1, 2, 7, 64, 1000, 16385, 1048576})
                if (r * c <= ZSMR_MAX_MATRIX) shape(r, c, n);
    for (int64_t t : {1, 2, 3, 16, 63, 64, 129, 255, 256, 511, 1023, 1024, 1025, 8192, 16777216})
        for (int64_t v : {1, 2, 500, 511, 512, 513, 2048, 4095, 4096, 4097, 50257, 128256, 2097152})
            for (int64_t k : {0, 1, 20, 64}) scores(t, v, k);
    const double quintic[5][3] = {{3.4445, -4.7750, 2.0315}, {3.4445, -4.7750, 2.0315}, {3.4445, -4.7750, 2.0315}, {3.4445, -4.7750, 2.0315}, {3.4445, -4.7750, 2.0315}};
    const double cubic[3][3] = {{1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}}, line[2][3] = {{180, 0, 0}, {0.001, 0, 0}}, none[2][3] = {{0, 0, 0}, {2, -1, 0.3}};
    const double odd[4][3] = {{-3, 2, -1}, {0.1, 0.5, -0.2}, {1, -1, 0.1}, {0, 0, 0.3}};
    scales(quintic, 5);
    scales(cubic, 3);
    scales(line, 2);
    scales(none, 2);
    scales(odd, 4);
    const double soft[16][3] = {{2, -1.5, 0.5}, {2, -1.5, 0.5}, {2, -1.5, 0.5}, {2, -1.5, 0.5}, {1.875, -1.25, 0.375}, {1.875, -1.25, 0.375}, {1.875, -1.25, 0.375},
                                {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}, {1.5, -0.5, 0}};
    const double steep[4][3] = {{20, -30, 12}, {15, -20, 6}, {3, -3, 1}, {2, -1.5, 0.5}};
    lists(quintic, 5);
    lists(cubic, 3);
    lists(none, 2);
    lists(odd, 4);
    lists(soft, 16);
    lists(steep, 1);
    lists(steep + 2, 2);
    for (int steps = 1; steps <= 5; ++steps) lists(quintic, steps);
    NsOp ops[kNsMaxOps];
    CHECK(ns_ops(quintic, 5, true, ops) == 18 && ns_group_steps(true, true, quintic, 5, 1.0) == 3 && ns_group_steps(true, false, quintic, 2, 1.2) == 2);
    CHECK(ns_group_steps(true, true, steep, 4, 1.0) == 1 && ns_group_steps(false, true, quintic, 5, 1.0) == 1);
    // groups where they are sooner, never for fp32 results
    auto chosen = [&](int64_t m, int64_t n, int64_t count, bool fp32 = false) { return ns_choose(quintic, 5, ns_shape(m, n, count, fp32), ops); };
    CHECK(chosen(767, 1003, 1) == 15 && chosen(1003, 767, 1) == 15 && chosen(1600, 6400, 1) == 18 && chosen(140, 2000, 1) == 18);
    CHECK(chosen(1600, 6400, 1, true) == 15 && chosen(4096, 4096, 1) == 15 && chosen(513, 2050, 1) == 18 && chosen(2300, 200, 1) == 18);
    CHECK(chosen(130, 2100, 2) == 18 && chosen(1000, 513, 20) == 18);
    std::printf("plans passed\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_plans(tmp_path):
    exe = compile_driver(tmp_path, PLAN, ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"])
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "plans passed" in r.stdout, r.stdout + r.stderr


def test_structures_match_the_header():
    assert ctypes.sizeof(ops.zsmr_newton) == 16 + 16 * 24 and ctypes.sizeof(ops.zsmr_muon) == 40
