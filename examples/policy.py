"""A policy over tokens trained by its own samples, its matrix with the orthogonalised step.

The policy is an embedding, a square matrix and an output head: the logits of the next
token are head . (matrix . embedding[token]).  The three are the units of a flat
parameter vector that N simulated ranks own whole (stage 3 with owners).  A step of the
whole world:

  each rank r, its own tokens:
    zsmr_embed_lookup    hidden states from the 16-bit working copy; two products
    zsmr_logprobs        log probabilities of the sampled tokens, the entropy, and the
                         policy's likeliest tokens
    zsmr_logprobs_grad   the logits' gradient of  -mean(advantage logprob) - bonus mean(entropy)
    zsmr_embed_grad      the embedding's gradient into its segment of gradient row r; the
                         matrix's and the head's are products
  each unit's owner:
    zero_muon_step       the matrix: momentum, orthogonalised, applied and cast
    zero_fused_step      the others: Adam

A sampled token is worth 1 where it is the fixed random successor of its input.

    python examples/policy.py [--vocab 500] [--width 128] [--tokens 2048] [--world 4] [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_sharded_mixed_reduce_amd as z  # noqa: E402

EMBEDDING, MATRIX, HEAD = range(3)


class Policy:
    def __init__(self, vocab: int, width: int, tokens: int, world: int, lr: float, muon_lr: float, bonus: float, top: int = 4):
        dev, bf16 = "cuda", torch.bfloat16
        self.vocab, self.width, self.world, self.lr, self.muon_lr, self.bonus, self.t = vocab, width, world, lr, muon_lr, bonus, 0
        units = [vocab * width, width * width, vocab * width]
        shapes = [(vocab, width), (width, width), (vocab, width)]
        n = sum(units)
        self.at = [0, units[0], units[0] + units[1]]
        self.ctx = z.zero_init_shards(n, world, z.ZSMR_ZERO3_OWNER, "bf16", units=units)
        self.master, self.m, self.v = (torch.empty(n, device=dev) for _ in range(3))
        self.params = torch.empty(n, device=dev, dtype=bf16)            # working copy
        self.grads = torch.zeros(world, n, device=dev, dtype=bf16)      # a row for each rank
        self.owner = [z.zero_unit_owner(self.ctx, u) for u in range(3)]
        theta = torch.randn(n, device=dev) * width ** -0.5
        for u, o in enumerate(self.at):
            z.zero_init_state(self.ctx, self.owner[u], u, theta[o:], self.master[o:], self.m[o:], self.v[o:], self.params[o:])
        cut = [slice(o, o + size) for o, size in zip(self.at, units)]
        self.weights = [self.params[c].view(s) for c, s in zip(cut, shapes)]
        self.weight_grads = [self.grads[:, c].unflatten(1, s) for c, s in zip(cut, shapes)]
        self.x = torch.empty(tokens, width, device=dev, dtype=bf16)
        self.logprob, self.lse, self.entropy = (torch.empty(tokens, device=dev) for _ in range(3))
        self.top_ids = torch.empty(tokens, top, device=dev, dtype=torch.int64)
        self.top_logprobs = torch.empty(tokens, top, device=dev)
        self.dlogits = torch.empty(tokens, vocab, device=dev, dtype=bf16)
        size = max(z.zsmr_logprobs_workspace(tokens, vocab, top), z.zsmr_embed_grad_workspace(vocab, width, tokens),
                   z.zero_muon_workspace(width, width))
        self.ws = torch.empty(size, device=dev, dtype=torch.uint8)      # the calls follow each other on one stream

    def logits(self, tokens):
        """Into self.x the embeddings; returns the hidden states and the logits."""
        z.zsmr_embed_lookup(self.weights[EMBEDDING], tokens, self.x)
        hidden = self.x @ self.weights[MATRIX].t()
        return hidden, hidden @ self.weights[HEAD].t()

    def backward(self, r: int, tokens, hidden, logits, actions, advantage):
        """The scores of rank r's samples, and its gradient row."""
        z.zsmr_logprobs(logits, actions, self.logprob, self.lse, self.entropy, self.ws, self.top_ids, self.top_logprobs)
        z.zsmr_logprobs_grad(logits, actions, self.lse, self.entropy, self.dlogits, -advantage / len(tokens),
                             torch.full_like(self.entropy, -self.bonus / len(tokens)))
        dhidden = self.dlogits @ self.weights[HEAD]
        dx = dhidden @ self.weights[MATRIX]
        self.weight_grads[HEAD][r] = self.dlogits.t() @ hidden
        self.weight_grads[MATRIX][r] = dhidden.t() @ self.x
        z.zsmr_embed_grad(dx, tokens, self.weight_grads[EMBEDDING][r], self.ws)

    def update(self):
        self.t += 1
        for u, o in enumerate(self.at):
            rest = (self.grads, self.grads.shape[1], o, self.master[o:], self.m[o:])
            if u == MATRIX:
                z.zero_muon_step(self.ctx, self.owner[u], u, 0, self.width, self.width, 1, *rest, self.params[o:], self.ws, self.muon_lr)
            else:
                z.zero_fused_step(self.ctx, self.owner[u], u, *rest, self.v[o:], self.params[o:], self.t, self.lr)

    def step(self, tokens, successor, g):
        """tokens: a row for each rank.  Returns the mean reward, the mean entropy and how
        often the successor is among the likeliest tokens, on the device."""
        sums = torch.zeros(3, device="cuda")
        for r in range(self.world):
            hidden, logits = self.logits(tokens[r])
            actions = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=g).squeeze(1)
            reward = (actions == successor[tokens[r]]).float()
            self.backward(r, tokens[r], hidden, logits, actions, reward - reward.mean())
            known = (self.top_ids == successor[tokens[r]][:, None]).any(1).float()
            sums += torch.stack([reward.mean(), self.entropy.mean(), known.mean()])
        self.update()
        return sums / self.world


def train(vocab=500, width=128, tokens=2048, world=4, steps=60, lr=3e-3, muon_lr=0.02, bonus=0.01, seed=0, say=print):
    """Mean rewards of the steps."""
    torch.manual_seed(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    policy = Policy(vocab, width, tokens, world, lr, muon_lr, bonus)
    successor = torch.randperm(vocab, device="cuda", generator=g)
    rewards = []
    for t in range(1, steps + 1):
        reward, entropy, known = policy.step(torch.randint(vocab, (world, tokens), device="cuda", generator=g), successor, g).tolist()
        rewards.append(reward)
        if t == 1 or t % 10 == 0:
            say(f"step {t}: reward {reward:.4f}, entropy {entropy:.3f}, successor among the likeliest {known:.3f}")
    return rewards


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("vocab", 500), ("width", 128), ("tokens", 2048), ("world", 4), ("steps", 60)):
        parser.add_argument(f"--{name}", type=int, default=value)
    train(**vars(parser.parse_args()))
