"""Cases that measure the operators around the shard step: the embedding
lookup and its gradient, the softmax cross entropy of the output head with its
gradient, the global gradient norm with clipping, and the clipped shard step.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
with the entry points of ``zero_sharded_mixed_reduce_amd``.  Sizes are those of
the repository's workloads: a flat vector of 65,536 parameters on 4 ranks,
GPT-2 small (vocabulary 50,257, width 768, 124,439,808 parameters), one rank's
share of 7.5e9 parameters on 64 ranks, and the Llama-3-8B shape's
embedding/head unit (vocabulary 128,256, width 4,096)."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = {"fp16": 1, "bf16": 2, "fp32": 3}       # the library's format codes
MAX_NORM, EPS = 1.0, 1e-6
LR, BETAS, ADAM_EPS, STEP = 1e-4, (0.9, 0.999), 1e-8, 100


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decoding step of 64 sequences: latency
        {"name": "lookup_decode", "op": "lookup", "tokens": 64, "vocab": 128256, "width": 4096, "dtype": "bf16", "scale": 1.0},
        # a training batch's prompt through the embedding unit, scaled by sqrt(width)
        {"name": "lookup_batch", "op": "lookup", "tokens": 16384, "vocab": 128256, "width": 4096, "dtype": "bf16", "scale": 64.0},
        # tied embedding of GPT-2 small: added to the head's gradient, touched rows only, odd token count
        {"name": "embed_grad_tied", "op": "embed_grad", "tokens": 1023, "vocab": 50257, "width": 768, "dtype": "fp16", "scale": 1.0, "accumulate": True},
        # the embedding half of the largest unit: the whole gradient row segment is written
        {"name": "embed_grad_batch", "op": "embed_grad", "tokens": 16384, "vocab": 128256, "width": 4096, "dtype": "bf16", "scale": 64.0, "accumulate": False},
        # scoring a few positions: the head's weights are read once
        {"name": "xent_score", "op": "xent_forward", "tokens": 16, "vocab": 128256, "width": 4096, "dtype": "bf16"},
        # a small odd batch on GPT-2 small's head, loss and gradients
        {"name": "xent_small", "op": "xent", "tokens": 129, "vocab": 50257, "width": 768, "dtype": "fp16"},
        # an ordinary batch on GPT-2 small's head
        {"name": "xent_gpt2s", "op": "xent", "tokens": 8192, "vocab": 50257, "width": 768, "dtype": "bf16"},
        # the Llama-3-8B shape's head, one sequence of 8,192
        {"name": "xent_llama8b", "op": "xent", "tokens": 8192, "vocab": 128256, "width": 4096, "dtype": "bf16"},
        # a small model's tensors into its fp16 gradient row: latency
        {"name": "clip_flatten_small", "op": "clip_flatten", "layers": 4, "width": 61, "vocab": 101, "dtype": "fp32", "out": "fp16"},
        # GPT-2 small's 148 fp32 gradient tensors into a rank's bf16 row
        {"name": "clip_flatten_gpt2s", "op": "clip_flatten", "layers": 12, "width": 768, "vocab": 50257, "dtype": "fp32", "out": "bf16"},
        # the whole simulated world of 4 ranks, 65,536 parameters: launches and latency
        {"name": "clipped_step_psi65k", "op": "clipped_step", "shard": 16384, "world": 4, "ranks": 4, "dtype": "fp16"},
        # one rank of 64 of a 7.5e9-parameter model
        {"name": "clipped_step_share64", "op": "clipped_step", "shard": 117187500, "world": 64, "ranks": 1, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "xent_forward", "xent", "clip_flatten", "clipped_step"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("lookup", "embed_grad"):
        case = {"op": op, "tokens": _log(rng, 1, 16384), "vocab": _log(rng, 500, 128256), "width": 8 * _log(rng, 8, 512), "dtype": dtype,
                "scale": rng.choice([1.0, 0.125, 22.5])}
        if rng.random() < 0.3:
            case["width"] += rng.choice([1, 2, 4])
        return case | ({"accumulate": rng.random() < 0.5} if op == "embed_grad" else {})
    if op == "xent_forward":
        return {"op": op, "tokens": _log(rng, 1, 4096), "vocab": _log(rng, 500, 128256), "width": 8 * _log(rng, 16, 512), "dtype": dtype}
    if op == "xent":
        return {"op": op, "tokens": _log(rng, 1, 8192), "vocab": _log(rng, 500, 128256), "width": 8 * _log(rng, 16, 512), "dtype": dtype}
    if op == "clip_flatten":
        return {"op": op, "layers": _log(rng, 1, 12), "width": _log(rng, 24, 1024), "vocab": _log(rng, 100, 50257),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "out": dtype}
    world = rng.choice([1, 2, 3, 4, 8, 16, 32, 64])
    return {"op": op, "shard": _log(rng, 1000, 20_000_000), "world": world, "ranks": rng.choice([1, 1, min(2, world)]), "dtype": dtype}


# ----------------------------------------------------------------- inputs --
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)


def _tokens(g, n, vocab):
    """Token ids as text has them: frequency falls as one over rank, and the
    ranks lie anywhere in the vocabulary; about one in fifty is padding (-1)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab)).long().clamp_(1, vocab) - 1
    step = next(p for p in (48271, 40692, 16807) if math.gcd(p, vocab) == 1)
    ids = (rank * step + 7) % vocab
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, -1, ids)


def _shapes(case):
    """The tensors of a GPT-2-like model: two embeddings, twelve tensors a
    layer, the final norm."""
    h, shapes = case["width"], [(case["vocab"], case["width"]), (1024, case["width"])]
    shapes += [(h,), (h,), (h, 3 * h), (3 * h,), (h, h), (h,), (h,), (h,), (h, 4 * h), (4 * h,), (4 * h, h), (h,)] * case["layers"]
    return shapes + [(h,), (h,)]


def prepare(case, seed):
    g, dtype = _rng(seed), DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("lookup", "embed_grad"):
        t, v, h = case["tokens"], case["vocab"], case["width"]
        state["ids"] = _tokens(g, t, v)
        state["out"] = torch.empty(t, h, device="cuda", dtype=dtype)
        if case["op"] == "lookup":
            state["table"] = _normal(g, (v, h), 0.02, dtype)
        else:
            state["dout"] = _normal(g, (t, h), 1e-3, dtype)
            # tied: the head's gradient is there already; else the row segment's old content does not matter
            state["dtable"] = _normal(g, (v, h), 1e-3, dtype)
    elif case["op"] in ("xent", "xent_forward"):
        t, v, h = case["tokens"], case["vocab"], case["width"]
        state["x"] = _normal(g, (t, h), 1.0, dtype)
        # logits of a model in training: standard deviation about 2
        state["w"] = _normal(g, (v, h), 2.0 / math.sqrt(h), dtype)
        state["labels"] = _tokens(g, t, v)
        state["labels"][0] = 1      # never all padding
    elif case["op"] == "clip_flatten":
        tensors = [_normal(g, s, 1e-2, dtype) for s in _shapes(case)]
        total = sum(x.numel() for x in tensors)
        state["tensors"] = tensors
        # what a program keeps of its gradient buffers: their addresses, sizes and formats
        state["list"] = (np.array([x.data_ptr() for x in tensors], dtype=np.int64), np.array([x.numel() for x in tensors], dtype=np.int64),
                         np.full(len(tensors), CODES[case["dtype"]], dtype=np.int32))
        state["flat"] = torch.empty(-(-total // 8) * 8, device="cuda", dtype=DTYPES[case["out"]])
    else:
        s, n, k = case["shard"], case["world"], case["ranks"]
        state["grads"] = _normal(g, (n, k * s), 1e-3, dtype)
        state["master"] = _normal(g, (k * s,), 0.02, torch.float32)
        state["m"] = _normal(g, (k * s,), 1e-4, torch.float32)
        state["v"] = _normal(g, (k * s,), 3e-4, torch.float32).square_()
        state["p16"] = torch.empty(k * s, device="cuda", dtype=dtype)
        state["reduced"] = torch.empty(k * s, device="cuda")
        # the other ranks' sums of squares, as received; this program's ranks fill theirs in
        state["sums"] = torch.rand(n, generator=g, device="cuda", dtype=torch.float64).add_(0.5).mul_(s * 1e-6 / n)
    return state


# ------------------------------------------------------------- plain forms --
def _plain_lookup(s):
    ids = s["ids"]
    rows = s["table"][ids.clamp(min=0)].float() * s["case"]["scale"]
    return {"out": torch.where(ids[:, None] >= 0, rows, 0.0).to(s["table"].dtype)}


def _plain_embed_grad(s):
    case, keep = s["case"], s["ids"] >= 0
    total = torch.zeros(case["vocab"], case["width"], device="cuda")
    total.index_add_(0, s["ids"].clamp(min=0), torch.where(keep[:, None], s["dout"].float(), 0.0))
    total *= case["scale"]
    if case["accumulate"]:
        total += s["dtable"]
    s["dtable"].copy_(total)
    return {"dtable": s["dtable"]}


def _plain_xent(s, backward):
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"]
    logits = x @ w.t()
    keep = labels >= 0
    count = keep.sum()
    at = labels.clamp(min=0)[:, None]
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp_().sum(1, keepdim=True).log_() + top
    loss = torch.where(keep, (lse - logits.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0], "mean": (loss.double().sum() / count).float()}
    if backward:
        p = logits.sub_(lse).exp_()
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p *= torch.where(keep, 1.0 / count, 0.0)[:, None]
        out["dx"] = (p @ w).to(s["x"].dtype)
        out["dw"] = (p.t() @ x).to(s["w"].dtype)
    return out


def _plain_clip_flatten(s):
    total = torch.stack([x.double().square().sum() for x in s["tensors"]]).sum()
    norm = total.sqrt().float()
    coef = (MAX_NORM / (norm + EPS)).clamp(max=1.0)
    flat = torch.cat([x.reshape(-1).float() for x in s["tensors"]]) * coef
    s["flat"].zero_()
    s["flat"][:flat.numel()] = flat
    return {"norm": norm, "coef": coef, "flat": s["flat"]}


def _plain_clipped_step(s):
    case, (b1, b2) = s["case"], BETAS
    g = torch.sum(s["grads"], 0, dtype=torch.float32) / case["world"]
    sums = s["sums"].clone()
    sums[:case["ranks"]] = g.double().square().view(case["ranks"], -1).sum(1)
    norm = sums.sum().sqrt().float()
    coef = (MAX_NORM / (norm + EPS)).clamp(max=1.0)
    g *= coef
    s["m"].mul_(b1).add_(g, alpha=1 - b1)
    s["v"].mul_(b2).add_(g.square() * (1 - b2))
    step = (s["m"] / (1 - b1 ** STEP)) * LR / ((s["v"] / (1 - b2 ** STEP)).sqrt() + ADAM_EPS)
    s["master"] -= step
    s["p16"].copy_(s["master"])
    return {"norm": norm, "coef": coef, "master": s["master"], "m": s["m"], "v": s["v"], "p16": s["p16"]}


# ----------------------------------------------------- the framework's calls --
def _scratch(s, name, size):
    """A workspace that a program keeps between calls."""
    if name not in s:
        s[name] = torch.empty(max(size, 1), device="cuda", dtype=torch.uint8)
    return s[name]


def _own(s):
    import zero_sharded_mixed_reduce_amd as z
    case = s["case"]
    if case["op"] == "lookup":
        z.zsmr_embed_lookup(s["table"], s["ids"], s["out"], scale=case["scale"])
        return {"out": s["out"]}
    if case["op"] == "embed_grad":
        ws = _scratch(s, "ws", z.zsmr_embed_grad_workspace(case["vocab"], case["width"], case["tokens"]))
        z.zsmr_embed_grad(s["dout"], s["ids"], s["dtable"], ws, scale=case["scale"], accumulate=case["accumulate"])
        return {"dtable": s["dtable"]}
    if case["op"] in ("xent", "xent_forward"):
        t, backward = case["tokens"], case["op"] == "xent"
        loss, lse, summary = torch.empty(t, device="cuda"), torch.empty(t, device="cuda"), torch.empty(3, device="cuda")
        ws = _scratch(s, "ws", z.zsmr_xent_workspace(t, case["vocab"], case["width"], backward=backward))
        z.zsmr_xent_forward(s["x"], s["w"], s["labels"], loss, lse, summary, ws)
        out = {"loss": loss, "lse": lse, "mean": summary[0]}
        if backward:
            out["dx"], out["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
            # the mean's gradient: one over the number of tokens that count, as the forward pass left it on the device
            z.zsmr_xent_backward(s["x"], s["w"], s["labels"], lse, out["dx"], out["dw"], ws, scale=summary[1:2])
        return out
    if case["op"] == "clip_flatten":
        norm_coef = torch.empty(2, device="cuda")
        ws = _scratch(s, "ws", z.zsmr_norm_workspace(int(s["list"][1].sum()), len(s["list"][1])))
        z.zsmr_grad_norm(s["list"], MAX_NORM, norm_coef, ws, eps=EPS)
        z.zsmr_clip_flatten(s["list"], norm_coef[1:], s["flat"])
        return {"norm": norm_coef[0], "coef": norm_coef[1], "flat": s["flat"]}
    n, k, size = case["world"], case["ranks"], case["shard"]
    if "ctx" not in s:
        s["ctx"] = z.zero_init_shards(n * size, n, z.ZSMR_ZERO2, case["dtype"])
    norm_coef, sums = torch.empty(2, device="cuda"), s["sums"].clone()
    ws = _scratch(s, "ws", z.zsmr_norm_workspace(size, 1))
    for r in range(k):
        z.zero_reduce_shard_sumsq(s["ctx"], r, 0, s["grads"], k * size, r * size, True, s["reduced"][r * size:], sums[r:], ws)
    z.zsmr_clip_coef(sums, n, MAX_NORM, norm_coef, eps=EPS)
    for r in range(k):
        a = r * size
        z.zero_clipped_step(s["ctx"], r, 0, s["reduced"][a:], norm_coef[1:], s["master"][a:], s["m"][a:], s["v"][a:], s["p16"][a:], STEP, LR, BETAS, ADAM_EPS)
    return {"norm": norm_coef[0], "coef": norm_coef[1], "master": s["master"], "m": s["m"], "v": s["v"], "p16": s["p16"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "lookup":
        return _plain_lookup(state)
    if op == "embed_grad":
        return _plain_embed_grad(state)
    if op in ("xent", "xent_forward"):
        return _plain_xent(state, op == "xent")
    return _plain_clip_flatten(state) if op == "clip_flatten" else _plain_clipped_step(state)


# --------------------------------------------------------- work and truth --
def work(case):
    size = {"fp32": 4}.get(case["dtype"], 2)
    if case["op"] == "lookup":
        t, h = case["tokens"], case["width"]
        return {"bytes": 2 * t * h * size + 8 * t, "flops": t * h}
    if case["op"] == "embed_grad":
        t, h = case["tokens"], case["width"]
        # added to: the touched rows (at most one a token) are read and written
        rows = 2 * min(t, case["vocab"]) if case["accumulate"] else case["vocab"]
        return {"bytes": t * h * size + rows * h * size + 8 * t, "flops": t * h}
    if case["op"] in ("xent", "xent_forward"):
        t, v, h = case["tokens"], case["vocab"], case["width"]
        n = 1 if case["op"] == "xent_forward" else 3      # logits; the two gradients
        return {"bytes": (t + v) * h * size * (1 if n == 1 else 2) + 16 * t, "flops": 2 * n * t * v * h}
    if case["op"] == "clip_flatten":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": n * (size + 2), "flops": 3 * n}
    n = case["shard"] * case["ranks"]
    return {"bytes": n * (2 * case["world"] + 26), "flops": n * (case["world"] + 16)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        padded = torch.cat([s["table"].double() * case["scale"], torch.zeros(1, case["width"], device="cuda", dtype=torch.float64)])
        return {"out": torch.nn.functional.embedding(s["ids"] % (case["vocab"] + 1), padded)}
    if case["op"] == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        ids, rows = s["ids"][order], s["dout"].double()[order]
        rows, ids = rows[ids >= 0], ids[ids >= 0]
        # differences of running sums at the ends of each token's run
        sums = torch.cat([torch.zeros(1, case["width"], device="cuda", dtype=torch.float64), rows.cumsum(0)])
        edge = torch.searchsorted(ids, torch.arange(case["vocab"] + 1, device="cuda"))
        grad = (sums[edge[1:]] - sums[edge[:-1]]) * case["scale"]
        return {"dtable": grad + s["dtable"].double() if case["accumulate"] else grad}
    if case["op"] in ("xent", "xent_forward"):
        backward = case["op"] == "xent"
        x, w = s["x"].double().requires_grad_(backward), s["w"].double().requires_grad_(backward)
        logits = x @ w.t()
        loss = torch.nn.functional.cross_entropy(logits, s["labels"], ignore_index=-1, reduction="none")
        mean = loss.sum() / (s["labels"] >= 0).sum()
        out = {"loss": loss.detach(), "lse": torch.logsumexp(logits.detach(), 1), "mean": mean.detach()}
        if backward:
            out["dx"], out["dw"] = torch.autograd.grad(mean, (x, w))
        return out
    if case["op"] == "clip_flatten":
        flat = torch.nn.functional.pad(torch.cat([x.reshape(-1) for x in s["tensors"]]).double(), (0, s["flat"].numel() - sum(x.numel() for x in s["tensors"])))
        norm = torch.linalg.vector_norm(flat)
        coef = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + EPS))
        return {"norm": norm, "coef": coef, "flat": flat * coef}
    g = torch.mean(s["grads"], 0, dtype=torch.float64)
    sums = s["sums"].tolist()
    sums[:case["ranks"]] = [float(torch.dot(part, part)) for part in g.split(case["shard"])]
    norm = math.sqrt(math.fsum(sums))
    coef = min(1.0, MAX_NORM / (norm + EPS))
    m = torch.lerp(g * coef, s["m"].double(), BETAS[0])
    v = torch.lerp((g * coef) ** 2, s["v"].double(), BETAS[1])
    master = s["master"].double() - LR * (m / (1 - BETAS[0] ** STEP)) / (torch.sqrt(v / (1 - BETAS[1] ** STEP)) + ADAM_EPS)
    one = lambda value: torch.tensor(value, device="cuda", dtype=torch.float64)  # noqa: E731
    return {"norm": one(norm), "coef": one(coef), "master": master, "m": m, "v": v, "p16": master}
