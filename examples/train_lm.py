"""Trains a small language model from token ids to clipped gradients on the
library's operators: the blocks of train_block.py between

  embedding             token ids to the FP32 residual stream, scaled
  swiglu                the MLPs' activation, its input kept in 8 bits
  linear_cross_entropy  the output head and its loss; the logits are not kept

The embedding and the output head share one weight: the head's gradient is
formed first, and the embedding's is added to the rows of the batch's tokens.

  python examples/train_lm.py --steps 10

Synthetic data: every token is followed by the same other one most of the time.
Each document's first tokens are a prompt, which is no target.  Tokens and widths
must be multiples of 128.
"""
import argparse
import time

import torch

import train_block
from train_block import fgs


class Block(train_block.Block):
    """A transformer block whose MLP keeps half as much for its backward pass."""

    def activate(self, gate_up):
        return fgs.swiglu(gate_up)


class Model(torch.nn.Module):
    def __init__(self, vocab: int, width: int, heads: int, kv_heads: int, hidden: int, layers: int, device):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.randn(vocab, width, device=device) * width ** -0.5)
        self.scale = float(width) ** 0.5
        self.first = torch.nn.Parameter(torch.ones(width, device=device))
        self.blocks = torch.nn.ModuleList(Block(width, heads, kv_heads, hidden, device) for _ in range(layers))

    def forward(self, tokens, targets, cu_seqlens):
        """The loss of each token, and the embedded tokens, whose gradient add_embedding_gradient() takes."""
        embedded = fgs.embedding_fwd(tokens, self.weight.detach(), self.scale).requires_grad_()
        nothing = torch.zeros_like(embedded, dtype=torch.bfloat16)
        x, n = fgs.residual_norm(nothing, embedded, w_pre=self.first)      # the stream, and its norm for the first block
        for block in self.blocks:
            x, n = block(x, n, cu_seqlens)
        return fgs.linear_cross_entropy(n, self.weight, targets), embedded

    def add_embedding_gradient(self, embedded, tokens):
        fgs.embedding_bwd(embedded.grad, tokens, self.weight.shape[0], self.scale, out=self.weight.grad)


def batch(vocab, tokens, generator, device):
    """Token ids, targets and the documents' offsets."""
    follows = torch.arange(vocab).roll(7919 % vocab)
    ids = torch.randint(0, vocab, (tokens + 1,), generator=generator)
    known = torch.rand(tokens, generator=generator) < 0.8
    for i in range(tokens):
        if known[i]:
            ids[i + 1] = follows[ids[i]]
    cuts = [0, tokens // 5, tokens // 2, tokens]
    targets = ids[1:].clone()
    for begin, end in zip(cuts, cuts[1:]):
        targets[begin:begin + (end - begin) // 4] = -100      # a prompt
        targets[end - 1] = -100                               # the next token is another document's
    return ids[:-1].to(device), targets.to(device), torch.tensor(cuts, dtype=torch.int32, device=device)


def train(steps=10, tokens=1024, vocab=4099, width=512, heads=8, kv_heads=2, hidden=1024, layers=2, max_norm=1.0,
          lr=2e-3, seed=0, say=print):
    """The losses and the gradients' norms of `steps` steps."""
    torch.manual_seed(seed)
    device = torch.device("cuda")
    model = Model(vocab, width, heads, kv_heads, hidden, layers, device)
    params = list(model.parameters())
    optimizer = torch.optim.AdamW(params, lr=lr)
    ids, targets, cu_seqlens = batch(vocab, tokens, torch.Generator().manual_seed(seed), device)
    count = int((targets >= 0).sum())
    losses, norms = [], []
    for step in range(steps):
        begin = time.perf_counter()
        each, embedded = model(ids, targets, cu_seqlens)
        loss = each.sum() / count
        loss.backward()
        model.add_embedding_gradient(embedded, ids)
        norm = fgs.clip_grad_norm([p.grad for p in params if p.grad is not None], max_norm)
        optimizer.step()
        optimizer.zero_grad()
        losses.append(float(loss.detach()))
        norms.append(float(norm))
        say(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {norms[-1]:.4f}  "
            f"{1e3 * (time.perf_counter() - begin):.1f} ms")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 10), ("tokens", 1024), ("vocab", 4099), ("width", 512), ("heads", 8), ("kv-heads", 2),
                        ("hidden", 1024), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    train(**vars(ap.parse_args()))
