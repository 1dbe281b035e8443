"""Cases that measure the matrix optimizer step and the scores of logits: the
orthogonalised update (Newton-Schulz products), the shard step that applies it
(reduce, momentum, orthogonalise, update, cast), and the log probabilities of given
tokens with entropy and top alternatives, with their gradient.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
with the entry points of ``zero_sharded_mixed_reduce_amd``.  Sizes are those of
the repository's workloads: a flat vector of 65,536 parameters on 4 ranks,
GPT-2 XL (width 1,600), GPT-2's vocabulary of 50,257, the Llama-3-8B shape (width
4,096, its MLP's 14,336, vocabulary 128,256), and odd ones."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# the odd quintic that raises small singular values and keeps large ones about 1
COEFS = ((3.4445, -4.7750, 2.0315),) * 5
NS_EPS = 1e-7
LR, BETA, DECAY = 1e-3, 0.95, 0.1


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the query and key heads of a layer, one matrix each: latency
        {"name": "orthogonal_heads", "op": "orthogonal", "rows": 64, "cols": 64, "count": 24, "dtype": "bf16", "out": "bf16"},
        # an odd matrix, taller than wide, of a small model whose gradients are fp32
        {"name": "orthogonal_ragged", "op": "orthogonal", "rows": 1003, "cols": 767, "count": 1, "dtype": "fp32", "out": "fp16"},
        # the projections of GPT-2 XL's attention: four square matrices of a layer
        {"name": "orthogonal_gpt2xl", "op": "orthogonal", "rows": 1600, "cols": 1600, "count": 4, "dtype": "fp32", "out": "bf16"},
        # a square projection of the Llama-3-8B shape
        {"name": "orthogonal_llama8b", "op": "orthogonal", "rows": 4096, "cols": 4096, "count": 1, "dtype": "bf16", "out": "bf16"},
        # 65,536 parameters as four matrices, one rank's unit of a world of 4: latency
        {"name": "muon_psi65k", "op": "muon", "rows": 128, "cols": 128, "count": 4, "world": 4, "dtype": "fp16"},
        # the first matrix of GPT-2 XL's MLP, on its owner, 16 ranks' gradients
        {"name": "muon_gpt2xl", "op": "muon", "rows": 1600, "cols": 6400, "count": 1, "world": 16, "dtype": "bf16"},
        # the MLP's way out of the Llama-3-8B shape, taller than wide as x @ w stores it, 8 ranks' gradients
        {"name": "muon_llama8b", "op": "muon", "rows": 14336, "cols": 4096, "count": 1, "world": 8, "dtype": "bf16"},
        # a decoding step of 16 sequences: 20 alternatives each
        {"name": "scores_decode", "op": "scores", "tokens": 16, "vocab": 128256, "dtype": "bf16", "top": 20, "scale": 1.0},
        # a prompt's tokens scored, 5 alternatives, tempered, fp32 logits of an odd vocabulary
        {"name": "scores_prompt", "op": "scores", "tokens": 1023, "vocab": 50257, "dtype": "fp32", "top": 5, "scale": 1.25},
        # a small odd batch of a policy's update: log probabilities, entropy, gradient of both
        {"name": "policy_small", "op": "policy", "tokens": 129, "vocab": 50257, "dtype": "fp16", "scale": 1.0},
        # the same over 8,192 tokens of the largest vocabulary
        {"name": "policy_llama8b", "op": "policy", "tokens": 8192, "vocab": 128256, "dtype": "bf16", "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, dtype = rng.choice(["orthogonal", "muon", "scores", "policy"]), rng.choice(["bf16", "fp16"])
    if op in ("orthogonal", "muon"):
        rows, cols = _log(rng, 8, 4096), _log(rng, 8, 4096)
        if rng.random() < 0.6:          # most weights are aligned
            rows, cols = -(-rows // 16) * 16, -(-cols // 16) * 16
        # about as much as one square matrix of 4,096 at most
        count = min(_log(rng, 1, 64), max(1, 2 ** 24 // (rows * cols)))
        if op == "orthogonal":
            return {"op": op, "rows": rows, "cols": cols, "count": count, "dtype": rng.choice([dtype, "fp32"]), "out": dtype}
        return {"op": op, "rows": rows, "cols": cols, "count": count, "world": rng.choice([1, 2, 4, 8, 16]), "dtype": dtype}
    case = {"op": op, "tokens": _log(rng, 1, 4096), "vocab": _log(rng, 500, 128256), "dtype": rng.choice([dtype, "fp32"]),
            "scale": rng.choice([1.0, 1.0, 0.5, 1.25])}
    return case | ({"top": min(_log(rng, 1, 64), case["vocab"])} if op == "scores" else {})


# ----------------------------------------------------------------- inputs --
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _gradients(g, n, rows, cols, sigma, dtype):
    """n gradients of a matrix: a few directions that all of them share, of falling
    strength, under noise of each one's own."""
    rank = min(16, rows, cols)
    left = torch.randn(rows, rank, generator=g, device="cuda") / (1.0 + torch.arange(rank, device="cuda"))
    shared = left @ torch.randn(rank, cols, generator=g, device="cuda")
    out = torch.empty(n, rows, cols, device="cuda", dtype=dtype)
    for i in range(n):
        torch.randn(rows, cols, generator=g, device="cuda", out=(noise := torch.empty(rows, cols, device="cuda")))
        out[i] = noise.add_(shared).mul_(sigma)
    return out


def _ids(g, n, vocab):
    """The given tokens; about one in fifty is padding (-1)."""
    ids = torch.randint(vocab, (n,), generator=g, device="cuda")
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, -1, ids)


def _logits(g, case, ids):
    """Logits of a trained model: standard deviation 2, the given token often near
    the top, a quarter of the rows with half of the vocabulary masked by -infinity
    (tokens that a grammar bars) and a quarter by the type's lowest value."""
    t, v, dtype = case["tokens"], case["vocab"], DTYPES[case["dtype"]]
    x = torch.randn(t, v, generator=g, device="cuda", dtype=dtype).mul_(2.0)
    at = ids.clamp(min=0)[:, None]
    given = torch.rand(t, 1, generator=g, device="cuda").mul_(12.0).to(dtype)
    barred = torch.rand(v, generator=g, device="cuda") < 0.5
    x[1::4] = torch.where(barred, float("-inf"), x[1::4])
    x[2::4] = torch.where(barred, torch.finfo(dtype).min, x[2::4])
    return x.scatter_(1, at, given)


def prepare(case, seed):
    g, state = _rng(seed), {"case": case}
    if case["op"] == "orthogonal":
        state["x"] = torch.stack([_gradients(g, 1, case["rows"], case["cols"], 1e-3, DTYPES[case["dtype"]])[0] for _ in range(case["count"])])
    elif case["op"] == "muon":
        r, c, k, n = case["rows"], case["cols"], case["count"], case["world"]
        size = r * c
        state["grads"] = torch.empty(n, k * size, device="cuda", dtype=DTYPES[case["dtype"]])
        state["momentum"] = torch.empty(k * size, device="cuda")
        for i in range(k):
            # the momentum follows the same directions as the new gradients
            got = _gradients(g, n + 1, r, c, 1e-3, torch.float32).view(n + 1, size)
            state["grads"][:, i * size:(i + 1) * size] = got[:n]
            state["momentum"][i * size:(i + 1) * size] = got[n] * 4.0
        state["master"] = torch.randn(k * size, generator=g, device="cuda").mul_(0.02)
        state["p16"] = torch.empty(k * size, device="cuda", dtype=DTYPES[case["dtype"]])
    else:
        state["ids"] = _ids(g, case["tokens"], case["vocab"])
        state["logits"] = _logits(g, case, state["ids"])
        if case["op"] == "policy":
            # advantages and the entropy bonus, over the tokens
            state["dlogprob"] = torch.randn(case["tokens"], generator=g, device="cuda").div_(case["tokens"])
            state["dentropy"] = torch.full((case["tokens"],), -0.01 / case["tokens"], device="cuda")
    return state


# ------------------------------------------------------------- plain forms --
def _newton_schulz(x, coefs):
    """x: count x rows x cols."""
    tall = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if tall else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + NS_EPS).to(x.dtype)
    for a, b, c in coefs:
        gram = x @ x.mT.contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _plain_orthogonal(s):
    return {"out": _newton_schulz(s["x"].float(), COEFS).to(DTYPES[s["case"]["out"]])}


def _update_scale(case):
    """An update as large as Adam's: elements of 0.2 in root mean square."""
    return 0.2 * math.sqrt(max(case["rows"], case["cols"]))


def _plain_muon(s):
    case = s["case"]
    g = torch.sum(s["grads"], 0, dtype=torch.float32) / case["world"]
    s["momentum"].mul_(BETA).add_(g)
    u = g.add_(s["momentum"], alpha=BETA).view(case["count"], case["rows"], case["cols"])
    s["master"].mul_(1 - LR * DECAY).sub_(_newton_schulz(u, COEFS).reshape(-1), alpha=LR * _update_scale(case))
    s["p16"].copy_(s["master"])
    return {"master": s["master"], "momentum": s["momentum"], "p16": s["p16"]}


def _plain_scores(s):
    case, ids = s["case"], s["ids"]
    z = s["logits"].float()
    # keys in the order of the logits, ties by the lowest index
    bits = (z + 0.0).view(torch.int32)
    keys = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * 2 ** 32 + (2 ** 31 - 1 - torch.arange(case["vocab"], device="cuda"))
    z = z * case["scale"]
    top = z.amax(1, keepdim=True)
    e = (z - top).exp_()
    total = e.sum(1, keepdim=True)
    lse = total.log() + top
    mean = torch.where(e > 0, e * z, 0.0).sum(1, keepdim=True) / total
    given = torch.where(ids >= 0, (z.gather(1, ids.clamp(min=0)[:, None]) - lse)[:, 0], 0.0)
    out = {"logprob": given, "entropy": (lse - mean)[:, 0], "lse": lse[:, 0]}
    if case["op"] == "scores":
        at = 2 ** 31 - 1 - torch.topk(keys, case["top"]).values % 2 ** 32
        value = z.gather(1, at) - lse
        out["top_ids"] = torch.where(value > float("-inf"), at, -1)
        out["top_logprobs"] = value
    return out


def _plain_policy(s):
    out, z = _plain_scores(s), s["logits"].float() * s["case"]["scale"]
    logp = z - out["lse"][:, None]
    p = logp.exp()
    bonus = torch.where(p > 0, p * (logp + out["entropy"][:, None]), 0.0) * s["dentropy"][:, None]
    weight = torch.where(s["ids"] >= 0, s["dlogprob"], 0.0)[:, None]
    d = -p * weight
    d.scatter_add_(1, s["ids"].clamp(min=0)[:, None], weight)
    out["dlogits"] = ((d - bonus) * s["case"]["scale"]).to(s["logits"].dtype)
    return out


# ----------------------------------------------------- the framework's calls --
def _scratch(s, size):
    """A workspace that a program keeps between calls."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(size, 1), device="cuda", dtype=torch.uint8)
    return s["ws"]


def _own(s):
    import zero_sharded_mixed_reduce_amd as z
    case = s["case"]
    if case["op"] == "orthogonal":
        ws = _scratch(s, z.zsmr_orthogonalize_workspace(case["rows"], case["cols"], case["count"]))
        out = torch.empty_like(s["x"], dtype=DTYPES[case["out"]])
        z.zsmr_orthogonalize(s["x"], out, ws, coefs=COEFS, eps=NS_EPS)
        return {"out": out}
    if case["op"] == "muon":
        if "ctx" not in s:
            # every rank owns such a unit; this program is rank 0
            n = case["count"] * case["rows"] * case["cols"]
            s["ctx"] = z.zero_init_shards(case["world"] * n, case["world"], z.ZSMR_ZERO3_OWNER, case["dtype"], units=[n] * case["world"])
        ws = _scratch(s, z.zero_muon_workspace(case["rows"], case["cols"], case["count"]))
        z.zero_muon_step(s["ctx"], 0, 0, 0, case["rows"], case["cols"], case["count"], s["grads"], s["grads"].shape[1], 0, s["master"],
                         s["momentum"], s["p16"], ws, LR, beta=BETA, weight_decay=DECAY, scale=_update_scale(case), nesterov=True,
                         coefs=COEFS, eps=NS_EPS)
        return {"master": s["master"], "momentum": s["momentum"], "p16": s["p16"]}
    t, top = case["tokens"], case.get("top", 0)
    logprob, lse, entropy = torch.empty(3, t, device="cuda")
    out = {"logprob": logprob, "entropy": entropy, "lse": lse}
    if top:
        out["top_ids"] = torch.empty(t, top, device="cuda", dtype=torch.int64)
        out["top_logprobs"] = torch.empty(t, top, device="cuda")
    ws = _scratch(s, z.zsmr_logprobs_workspace(t, case["vocab"], top))
    z.zsmr_logprobs(s["logits"], s["ids"], logprob, lse, entropy, ws, top_ids=out.get("top_ids"), top_logprobs=out.get("top_logprobs"),
                    scale=case["scale"])
    if case["op"] == "policy":
        out["dlogits"] = torch.empty_like(s["logits"])
        z.zsmr_logprobs_grad(s["logits"], s["ids"], lse, entropy, out["dlogits"], dlogprob=s["dlogprob"], dentropy=s["dentropy"],
                             scale=case["scale"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"orthogonal": _plain_orthogonal, "muon": _plain_muon, "scores": _plain_scores, "policy": _plain_policy}[state["case"]["op"]](state)


# --------------------------------------------------------- work and truth --
def work(case):
    size = {"fp32": 4}.get(case["dtype"], 2)
    if case["op"] in ("orthogonal", "muon"):
        m, n = sorted((case["rows"], case["cols"]))
        k = case["count"]
        # a pass: half of the symmetric X X^T and of its square, and the product with X
        flops = len(COEFS) * k * (m * m * n + m ** 3 + 2 * m * m * n)
        if case["op"] == "orthogonal":
            return {"bytes": k * m * n * (size + 2), "flops": flops}
        # the ranks' gradients; master and momentum in and out; the working copy
        return {"bytes": k * m * n * (2 * case["world"] + 18), "flops": flops}
    t, v = case["tokens"], case["vocab"]
    if case["op"] == "scores":
        return {"bytes": t * v * size + t * (20 + 12 * case["top"]), "flops": 5 * t * v}
    return {"bytes": 2 * t * v * size + 28 * t, "flops": 14 * t * v}


def _exact_polar(x):
    """Through products of the transposed operands, in 64 bits."""
    x = x.double()
    wide = x if x.shape[-2] <= x.shape[-1] else x.transpose(-1, -2)
    y = (wide / (torch.linalg.vector_norm(wide, dim=(-2, -1), keepdim=True) + NS_EPS)).contiguous()
    eye = torch.eye(y.shape[-2], device=y.device, dtype=y.dtype)
    for a, b, c in COEFS:
        q = torch.matmul(y, y.transpose(-1, -2).contiguous())
        y = torch.matmul(a * eye + torch.matmul(q, b * eye + c * q), y)
    return y if x.shape[-2] <= x.shape[-1] else y.transpose(-1, -2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonal":
        return {"out": _exact_polar(s["x"])}
    if case["op"] == "muon":
        g = torch.mean(s["grads"], 0, dtype=torch.float64)
        momentum = s["momentum"].double() * BETA + g
        update = _exact_polar((g + BETA * momentum).view(case["count"], case["rows"], case["cols"]))
        master = s["master"].double() * (1 - LR * DECAY) - LR * _update_scale(case) * update.reshape(-1)
        return {"master": master, "momentum": momentum, "p16": master}
    parts = []
    for first in range(0, case["tokens"], 1024):        # 64 bits of all rows at once are much memory
        rows = slice(first, first + 1024)
        raw = s["logits"][rows].double()
        ids = s["ids"][rows]
        x = (raw * case["scale"]).requires_grad_(case["op"] == "policy")
        logp = torch.log_softmax(x, 1)
        p = logp.exp()
        entropy = -torch.where(p > 0, p * logp.clamp(min=-1e300), torch.zeros_like(p)).sum(1)
        given = torch.where(ids >= 0, logp.gather(1, ids.clamp(min=0).unsqueeze(1)).squeeze(1), torch.zeros_like(entropy))
        out = {"logprob": given.detach(), "entropy": entropy.detach(), "lse": torch.logsumexp(x.detach(), 1)}
        if case["op"] == "scores":
            order = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            best = logp.gather(1, order)
            out |= {"top_ids": torch.where(torch.isinf(best), torch.full_like(order, -1), order), "top_logprobs": best}
        else:
            # d entropy / dx = -p (log p + entropy), written out: a masked logit has no derivative that autograd could find
            q = p.detach()
            d = torch.where(ids >= 0, s["dlogprob"][rows].double(), torch.zeros_like(entropy.detach()))
            slope = torch.nn.functional.one_hot(ids.clamp(min=0), case["vocab"]).double().sub_(q).mul_(d.unsqueeze(1))
            slope -= s["dentropy"][rows].double().unsqueeze(1) * torch.where(q > 0, q * (logp.detach().clamp(min=-1e300) + entropy.detach().unsqueeze(1)), torch.zeros_like(q))
            out["dlogits"] = slope * case["scale"]
        parts.append(out)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
