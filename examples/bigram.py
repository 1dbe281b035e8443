"""A next-token model trained through the ZeRO step, with clipping.

The model is an embedding and an output head (logits = head . embedding[token]),
the two halves of the unit that a language model's flat parameter vector starts
and ends with.  Its parameters are one flat vector of 2 * vocab * width
elements, sharded over N simulated ranks at stage 2.  A step of the whole world:

  each rank r, its own tokens:
    zsmr_embed_lookup   hidden states from the 16-bit working copy
    zsmr_xent_forward   loss of the next token, logits never kept
    zsmr_xent_backward  the head's gradient into its segment of gradient row r
    zsmr_embed_grad     the embedding's gradient into its segment
  each rank's shard:
    zero_reduce_shard_sumsq   mean gradient over the ranks, and its sum of squares
  zsmr_clip_coef              the global norm and the clipping coefficient
  each rank's shard:
    zero_clipped_step         Adam on the clipped gradient, cast into the working copy

The tokens follow a fixed random successor table nine times of ten, so the loss
falls from log(vocab) towards the table's entropy.

    python examples/bigram.py [--vocab 5000] [--width 256] [--tokens 2048] [--world 4] [--steps 60]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_sharded_mixed_reduce_amd as z  # noqa: E402


class Bigram:
    def __init__(self, vocab: int, width: int, tokens: int, world: int, max_norm: float, lr: float):
        dev = "cuda"
        self.vocab, self.world, self.max_norm, self.lr, self.t = vocab, world, max_norm, lr, 0
        half = vocab * width
        self.ctx = z.zero_init_shards(2 * half, world, z.ZSMR_ZERO2, "bf16", pad=True)
        info = self.ctx.info()
        self.padded, self.shard = info["padded_numel"], info["shard_numel"]
        self.master, self.m, self.v = (torch.empty(self.padded, device=dev) for _ in range(3))
        self.params = torch.empty(self.padded, device=dev, dtype=torch.bfloat16)       # working copy
        self.grads = torch.zeros(world, self.padded, device=dev, dtype=torch.bfloat16)  # a row for each rank
        theta = torch.zeros(self.padded, device=dev)
        theta[:2 * half].normal_(std=width ** -0.5)
        for r in range(world):
            o = r * self.shard
            z.zero_init_state(self.ctx, r, 0, theta[o:], self.master[o:], self.m[o:], self.v[o:], self.params[o:])
        self.embedding, self.head = self.params[:2 * half].view(2, vocab, width)
        self.embedding_grad, self.head_grad = self.grads[:, :2 * half].unflatten(1, (2, vocab, width)).unbind(1)
        self.x, self.dx = (torch.empty(tokens, width, device=dev, dtype=torch.bfloat16) for _ in range(2))
        self.loss, self.lse = (torch.empty(tokens, device=dev) for _ in range(2))
        self.summary = torch.empty(world, 3, device=dev)
        self.reduced = torch.empty(self.padded, device=dev)
        self.sums = torch.empty(world, device=dev, dtype=torch.float64)
        self.norm_coef = torch.empty(2, device=dev)
        size = max(z.zsmr_xent_workspace(tokens, vocab, width), z.zsmr_embed_grad_workspace(vocab, width, tokens),
                   z.zsmr_norm_workspace(self.shard, 1))
        self.ws = torch.empty(size, device=dev, dtype=torch.uint8)      # the calls follow each other on one stream

    def step(self, tokens, labels):
        """tokens, labels: one row for each rank.  Returns the mean loss and
        {norm, coefficient}, on the device."""
        self.t += 1
        for r in range(self.world):
            z.zsmr_embed_lookup(self.embedding, tokens[r], self.x)
            z.zsmr_xent_forward(self.x, self.head, labels[r], self.loss, self.lse, self.summary[r], self.ws)
            z.zsmr_xent_backward(self.x, self.head, labels[r], self.lse, self.dx, self.head_grad[r], self.ws,
                                 scale=self.summary[r, 1:2])
            z.zsmr_embed_grad(self.dx, tokens[r], self.embedding_grad[r], self.ws)
        for r in range(self.world):
            o = r * self.shard
            z.zero_reduce_shard_sumsq(self.ctx, r, 0, self.grads, self.padded, o, True, self.reduced[o:], self.sums[r:],
                                      self.ws)
        z.zsmr_clip_coef(self.sums, self.world, self.max_norm, self.norm_coef)
        for r in range(self.world):
            o = r * self.shard
            z.zero_clipped_step(self.ctx, r, 0, self.reduced[o:], self.norm_coef[1:], self.master[o:], self.m[o:], self.v[o:],
                                self.params[o:], self.t, self.lr)
        return self.summary[:, 0].mean(), self.norm_coef


def batch(successor, world: int, tokens: int, g):
    """Tokens and their successors; every hundredth label is padding (-1)."""
    vocab = len(successor)
    x = torch.randint(vocab, (world, tokens), device="cuda", generator=g)
    y = torch.where(torch.rand(world, tokens, device="cuda", generator=g) < 0.9, successor[x],
                    torch.randint(vocab, (world, tokens), device="cuda", generator=g))
    y[:, ::100] = -1
    return x, y


def train(vocab=5000, width=256, tokens=2048, world=4, steps=60, max_norm=0.03, lr=1e-2, seed=0, say=print):
    """Losses and gradient norms of the steps."""
    torch.manual_seed(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    model = Bigram(vocab, width, tokens, world, max_norm, lr)
    successor = torch.randperm(vocab, device="cuda", generator=g)
    say(f"{2 * vocab * width} parameters on {world} ranks, log(vocab) = {math.log(vocab):.3f}")
    losses, norms = [], []
    for t in range(1, steps + 1):
        loss, norm_coef = model.step(*batch(successor, world, tokens, g))
        losses.append(loss.item())
        norms.append(norm_coef[0].item())
        if t == 1 or t % 10 == 0:
            say(f"step {t}: loss {losses[-1]:.4f}, gradient norm {norms[-1]:.4f}, coefficient {norm_coef[1].item():.4f}")
    return losses, norms


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("vocab", 5000), ("width", 256), ("tokens", 2048), ("world", 4), ("steps", 60)):
        parser.add_argument(f"--{name}", type=int, default=value)
    train(**vars(parser.parse_args()))
