"""The operators around the step on a machine without a GPU: the library exports
what ``include/zsmr_ops.h`` declares, workspaces have the sizes they need, and
every refusal returns its code before anything is launched.  Addresses are
placeholders that nothing reads."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from zero_sharded_mixed_reduce_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, W = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20     # 16-byte aligned
BIG = 1 << 40
L = ops._lib()
ARG, DTYPE, ALIGN = z.ZSMR_ERR_ARG, z.ZSMR_ERR_DTYPE, z.ZSMR_ERR_ALIGN
BF16 = z.ZSMR_BF16


def test_every_declared_symbol_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "zsmr_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*int\d+_t\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(ops.SIGNATURES)
    lib = ctypes.CDLL(z.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
        assert getattr(z, n) is getattr(ops, n)
    with pytest.raises(AttributeError):
        z.zsmr_no_such_call


def test_workspace_sizes():
    assert z.zsmr_norm_workspace(0, 0) == 0
    # a tensor of 1 and one of a chunk and 1: three partial sums; a shard of the same length: nine tiles
    assert z.zsmr_norm_workspace(16386, 2) >= 9 * 8
    assert z.zsmr_norm_workspace(10, 7) >= 7 * 8
    t, h = 1000, 768
    assert z.zsmr_embed_grad_workspace(50257, h, t) >= 4 * 4 * t + -(-t // 64) * 2 * h * 4
    # forward: a (maximum, sum) pair a token for every 256 vocabulary rows at least
    assert z.zsmr_xent_workspace(8192, 50257, 768, backward=False) >= 8192 * 197 * 8
    assert z.zsmr_xent_workspace(8192, 50257, 768) > z.zsmr_xent_workspace(8192, 50257, 768, backward=False)
    # the logits of 8,192 tokens over 128,256 rows would take 4.2 GB in fp32
    assert z.zsmr_xent_workspace(8192, 128256, 4096) < 1.5e9
    for bad in ((-1, 10, 10), (10, 0, 10), (10, 10, 0), ((1 << 24) + 1, 10, 10), (10, (1 << 30) + 1, 10), (10, 10, (1 << 21) + 1)):
        with pytest.raises(z.ZsmrError):
            z.zsmr_xent_workspace(*bad)
        with pytest.raises(z.ZsmrError):
            z.zsmr_embed_grad_workspace(bad[1], bad[2], bad[0])
    for bad in ((-1, 0), (0, -1)):
        with pytest.raises(z.ZsmrError):
            z.zsmr_norm_workspace(*bad)


# argument names in order, a call that would be accepted, and what each change gives
LOOKUP = dict(table=A, vocab=100, width=64, ts=64, dtype=BF16, ids=B, id_bytes=8, n=5, scale=1.0, out=C, os=64, stream=None)
EMBED_GRAD = dict(dout=A, ds=64, dtype=BF16, ids=B, id_bytes=8, n=5, vocab=100, width=64, scale=1.0, acc=0, dtable=C, ts=64,
                  ws=W, wb=BIG, stream=None)
FORWARD = dict(x=A, xs=64, w=B, wst=64, dtype=BF16, labels=C, id_bytes=8, n=5, vocab=100, width=64, loss=D, lse=D, summary=D, ws=W,
               wb=BIG, stream=None)
BACKWARD = dict(x=A, xs=64, w=B, wst=64, dtype=BF16, labels=C, id_bytes=8, n=5, vocab=100, width=64, lse=D, grad=None, scale=None,
                dx=D, dxs=64, dw=D, dws=64, acc=0, ws=W, wb=BIG, stream=None)
CASES = {
    "zsmr_embed_lookup": (LOOKUP, [
        (dict(table=None), ARG), (dict(out=None), ARG), (dict(ids=None), ARG), (dict(vocab=0), ARG), (dict(vocab=(1 << 30) + 1), ARG),
        (dict(width=0), ARG), (dict(width=65), ARG), (dict(ts=63), ARG), (dict(os=(1 << 21) + 1), ARG), (dict(n=-1), ARG),
        (dict(n=(1 << 24) + 1), ARG), (dict(id_bytes=2), ARG), (dict(dtype=3), DTYPE), (dict(dtype=0), DTYPE),
        (dict(table=A + 1), ALIGN), (dict(ids=B + 4), ALIGN), (dict(ids=B + 2, id_bytes=4), ALIGN), (dict(out=C + 1), ALIGN)]),
    "zsmr_embed_grad": (EMBED_GRAD, [
        (dict(dout=None), ARG), (dict(dtable=None), ARG), (dict(ids=None), ARG), (dict(vocab=0), ARG), (dict(ds=63), ARG),
        (dict(ts=63), ARG), (dict(acc=2), ARG), (dict(ws=None), ARG), (dict(wb=100), ARG), (dict(n=-1), ARG), (dict(id_bytes=0), ARG),
        (dict(dtype=3), DTYPE), (dict(dout=A + 1), ALIGN), (dict(dtable=C + 1), ALIGN), (dict(ws=W + 8), ALIGN)]),
    "zsmr_xent_forward": (FORWARD, [
        (dict(x=None), ARG), (dict(w=None), ARG), (dict(labels=None), ARG), (dict(loss=None), ARG), (dict(lse=None), ARG),
        (dict(summary=None), ARG), (dict(ws=None), ARG), (dict(wb=16), ARG), (dict(xs=63), ARG), (dict(wst=63), ARG), (dict(vocab=0), ARG),
        (dict(width=0), ARG), (dict(n=-1), ARG), (dict(id_bytes=1), ARG), (dict(dtype=3), DTYPE), (dict(x=A + 1), ALIGN),
        (dict(w=B + 1), ALIGN), (dict(lse=D + 2), ALIGN), (dict(loss=D + 1), ALIGN), (dict(summary=D + 1), ALIGN), (dict(ws=W + 4), ALIGN)]),
    "zsmr_xent_backward": (BACKWARD, [
        (dict(x=None), ARG), (dict(w=None), ARG), (dict(labels=None), ARG), (dict(lse=None), ARG), (dict(acc=-1), ARG), (dict(dxs=63), ARG),
        (dict(dws=63), ARG), (dict(ws=None), ARG), (dict(wb=1000), ARG), (dict(dtype=7), DTYPE), (dict(dx=D + 1), ALIGN),
        (dict(dw=D + 1), ALIGN), (dict(grad=D + 2), ALIGN), (dict(scale=D + 2), ALIGN), (dict(lse=D + 3), ALIGN)]),
    "zsmr_clip_coef": (dict(sums=A, n=4, max_norm=1.0, eps=1e-6, out=B, stream=None), [
        (dict(sums=None), ARG), (dict(n=-1), ARG), (dict(max_norm=-1.0), ARG), (dict(max_norm=float("nan")), ARG),
        (dict(max_norm=float("inf")), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(out=None), ARG),
        (dict(sums=A + 4), ALIGN), (dict(out=B + 2), ALIGN)]),
}


@pytest.mark.parametrize("name,change,code", [(n, c, e) for n, (_, changes) in CASES.items() for c, e in changes])
def test_refusals(name, change, code):
    args = CASES[name][0]
    assert set(change) <= set(args)
    assert getattr(L, name)(*(args | change).values()) == code


def test_calls_with_nothing_to_do_launch_nothing():
    assert L.zsmr_embed_lookup(*(LOOKUP | dict(n=0, ids=None, out=None)).values()) == 0
    assert L.zsmr_embed_grad(*(EMBED_GRAD | dict(n=0, ids=None, dout=None, acc=1)).values()) == 0
    assert L.zsmr_xent_backward(*(BACKWARD | dict(dx=None, dw=None)).values()) == 0
    assert L.zsmr_xent_backward(*(BACKWARD | dict(n=0, x=None, labels=None, lse=None, acc=1)).values()) == 0
    assert L.zsmr_clip_grads(None, None, None, 0, A, None) == 0
    assert L.zsmr_clip_flatten(None, None, None, 0, None, None, 0, BF16, None) == 0


def _arrays(ptrs, numels, dtypes):
    keep = np.array(ptrs, dtype=np.int64), np.array(numels, dtype=np.int64), np.array(dtypes, dtype=np.int32)
    return keep, [a.ctypes.data for a in keep] + [len(ptrs)]


@pytest.mark.parametrize("ptrs,numels,dtypes,code", [
    ([A, 0], [4, 4], [3, 3], ARG), ([A], [-1], [3], ARG), ([A], [(1 << 56) + 1], [2], ARG), ([A], [4], [4], DTYPE), ([A], [4], [0], DTYPE),
    ([A + 2], [4], [3], ALIGN), ([A + 1], [4], [2], ALIGN), ([A, B], [1 << 46, 1 << 46], [2, 2], ARG)])
def test_list_refusals(ptrs, numels, dtypes, code):
    keep, args = _arrays(ptrs, numels, dtypes)
    assert L.zsmr_grad_norm(*args, 1.0, 1e-6, B, W, BIG, None) == code
    assert L.zsmr_clip_grads(*args, B, None) == code
    assert L.zsmr_clip_flatten(*args, B, C, 1 << 60 >> 4, BF16, None) == code


def test_list_calls_refuse_their_other_arguments():
    keep, args = _arrays([A, B], [20000, 3], [3, 2])
    assert L.zsmr_grad_norm(*args, 1.0, 1e-6, None, W, BIG, None) == ARG
    assert L.zsmr_grad_norm(*args, -1.0, 1e-6, C, W, BIG, None) == ARG
    assert L.zsmr_grad_norm(*args, 1.0, float("inf"), C, W, BIG, None) == ARG
    assert L.zsmr_grad_norm(*args, 1.0, 1e-6, C, W, 16, None) == ARG            # three chunks
    assert L.zsmr_grad_norm(*args, 1.0, 1e-6, C, W + 8, BIG, None) == ALIGN
    assert L.zsmr_grad_norm(None, None, None, -1, 1.0, 1e-6, C, W, BIG, None) == ARG
    assert L.zsmr_grad_norm(None, None, None, 1, 1.0, 1e-6, C, W, BIG, None) == ARG
    assert L.zsmr_clip_grads(*args, None, None) == ARG
    assert L.zsmr_clip_grads(*args, C + 2, None) == ALIGN
    assert L.zsmr_clip_flatten(*args, C, D, 20002, BF16, None) == ARG           # one element short
    assert L.zsmr_clip_flatten(*args, C, None, 20003, BF16, None) == ARG
    assert L.zsmr_clip_flatten(*args, C, D, 20003, 3, None) == DTYPE
    assert L.zsmr_clip_flatten(*args, C, D + 1, 20003, BF16, None) == ALIGN


def test_clipped_step_refusals_count_nothing():
    ctx = z.zero_init_shards(1000, 4, z.ZSMR_ZERO2, "bf16")
    h, hp = ctx.handle, z._hp(1e-3)
    ok = dict(ctx=h, rank=1, unit=0, grads=A, stride=1000, base=250, mean=1, g=B, sumsq=C, ws=W, wb=BIG, stream=None)
    for change, code in [(dict(ctx=None), ARG), (dict(rank=4), ARG), (dict(unit=1), ARG), (dict(grads=None), ARG), (dict(stride=249), ARG),
                         (dict(base=-1), ARG), (dict(mean=2), ARG), (dict(g=None), ARG), (dict(sumsq=None), ARG), (dict(ws=None), ARG),
                         (dict(wb=7), ARG), (dict(grads=A + 1), ALIGN), (dict(g=B + 2), ALIGN), (dict(sumsq=C + 4), ALIGN)]:
        assert L.zero_reduce_shard_sumsq(*(ok | change).values()) == code, change
    ok = dict(ctx=h, rank=1, unit=0, g=A, coef=B, master=C, m=D, v=W, p16=A, t=1, hp=hp, stream=None)
    for change, code in [(dict(ctx=None), ARG), (dict(rank=-1), ARG), (dict(g=None), ARG), (dict(master=None), ARG), (dict(m=None), ARG),
                         (dict(v=None), ARG), (dict(p16=None), ARG), (dict(t=0), ARG), (dict(hp=z._hp(-1.0)), ARG),
                         (dict(hp=z._hp(1e-3, (1.0, 0.9))), ARG), (dict(coef=B + 1), ALIGN), (dict(p16=A + 1), ALIGN), (dict(v=W + 2), ALIGN)]:
        assert L.zero_clipped_step(*(ok | change).values()) == code, change
    assert all(z.zero_counters(ctx, r)["traffic_elems"] == 0 for r in range(4))


def test_binding_checks_tensors_before_the_library():
    """Shapes, formats and strides are refused by name before any address is
    taken, and a tensor in host memory never reaches the library."""
    t, ids = torch.zeros(10, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    out, f3 = torch.zeros(3, 16, dtype=torch.bfloat16), torch.zeros(3)
    ws = torch.zeros(64, dtype=torch.uint8)
    for bad, why in (((t.float(), ids, out), "16-bit"), ((t, ids, out[:2]), "2 x 16"), ((t, ids, out.half()), "format"),
                     ((t, ids, out[:, :8]), "3 x 8"), ((t.t(), ids, out), "contiguous"), ((t[0], ids, out), "matrix"),
                     ((t.as_strided((10, 16), (8, 1)), ids, out), "overlap"), ((t, ids.float(), out), "token ids"),
                     ((t, ids[None], out), "token ids"), ((t, torch.zeros(6, dtype=torch.int64)[::2], out), "token ids"),
                     ((t, ids, out), "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_embed_lookup(*bad, stream=0)
    for bad, why in (((out, ids, t[:, :8], ws), "3 x 16"), ((out, ids, t, ws[::2]), "workspace"), ((out, ids, t, ws), "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_embed_grad(*bad, stream=0)
    for bad, why in (((out, t, ids, f3, f3[:2], f3, ws), "lse"), ((out, t, ids, f3.double(), f3, f3, ws), "loss"),
                     ((out, t, ids, f3, f3, f3[:2], ws), "summary"), ((out, t, ids, f3, f3, f3, ws), "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_xent_forward(*bad, stream=0)
    for bad, kw, why in (((out, t, ids, f3, None, t[:5], ws), {}, "dw"), ((out, t, ids, f3, out[:2], None, ws), {}, "dx"),
                         ((out, t, ids, f3, out, t, ws), {"grad": f3[:1]}, "grad"), ((out, t, ids, f3, out, t, ws), {"scale": ids}, "scale"),
                         ((out, t, ids, f3, None, None, ws), {}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_xent_backward(*bad, stream=0, **kw)
    i64, i32 = np.zeros(2, np.int64), np.zeros(2, np.int32)
    for bad in ([t.t()], (i64, i64[:1], i32), (i64, i32, i32), (i64, i64, i64), (np.zeros(4, np.int64)[::2], i64, i32), (i64[None], i64, i32)):
        with pytest.raises(ValueError, match="tensor list"):
            z.zsmr_grad_norm(bad, 1.0, f3, ws, stream=0)
        with pytest.raises(ValueError, match="tensor list"):
            z.zsmr_clip_grads(bad, f3, stream=0)
    for flat, why in ((f3, "flat"), (out.t(), "flat"), (out, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zsmr_clip_flatten((i64[:0], i64[:0], i32[:0]), None, flat, stream=0)
    with pytest.raises(ValueError, match="sums"):
        z.zsmr_clip_coef(f3.double(), 4, 1.0, f3, stream=0)
    ctx = z.zero_init_shards(1000, 4, z.ZSMR_ZERO2, "bf16")
    rows, shard, sums = torch.zeros(4000, dtype=torch.bfloat16), torch.zeros(250), torch.zeros(1, dtype=torch.float64)
    for change, why in ((dict(base_elem=751), "grads"), (dict(g_out=shard[:249]), "g_out"), (dict(sumsq=shard), "sumsq"), (dict(rank=1 << 32), "int32"),
                        (dict(row_stride=1 << 63), "int64"), ({}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zero_reduce_shard_sumsq(**(dict(ctx=ctx, rank=0, unit=0, grads=rows, row_stride=1000, base_elem=0, mean=True, g_out=shard,
                                              sumsq=sums, ws=ws, stream=0) | change))
    for change, why in ((dict(g=shard[:249]), "g"), (dict(m=shard.bfloat16()), "m"), (dict(p16_dst=rows[:249]), "p16_dst"), (dict(coef=sums), "coef"),
                        (dict(t=1 << 31), "int32"), ({}, "host memory")):
        with pytest.raises(ValueError, match=why):
            z.zero_clipped_step(**(dict(ctx=ctx, rank=0, unit=0, g=shard, coef=shard, master=shard, m=shard, v=shard, p16_dst=rows, t=1, lr=1e-3,
                                        stream=0) | change))
    assert z.zero_counters(ctx, 0)["traffic_elems"] == 0
    for call in (lambda: ops._ops.embed_lookup(t), lambda: ops._ops.embed_lookup(1, 2, 3, 4, 5), lambda: z.zsmr_embed_lookup(t, None, out, stream=0)):
        with pytest.raises((TypeError, AttributeError, ValueError)):
            call()
