"""Trains a small stack of transformer blocks on packed documents, the linear
layers in scaled FP8 and everything around them on the library's other
operators:

  attention        causal, grouped heads, documents of different lengths in
                   one pack
  residual_norm    the boundary between two blocks: norm of the block's
                   output, its gate, the FP32 residual stream and the norm
                   for the next block
  clip_grad_norm   the gradients' global norm and clipping, in place

  python examples/train_block.py --steps 10

Synthetic data: fixed random targets for fixed random inputs, so the loss
falls from step to step.  Tokens and widths must be multiples of 128.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fine_grained_scaled_amd as fgs  # noqa: E402


class Boundary(torch.nn.Module):
    """r = x + gate * norm(y), n = norm(r)."""

    def __init__(self, width: int, device):
        super().__init__()
        self.w_post = torch.nn.Parameter(torch.ones(width, device=device))
        self.w_pre = torch.nn.Parameter(torch.ones(width, device=device))
        self.gate = torch.nn.Parameter(torch.full((width,), 0.5, device=device))

    def forward(self, y, x):
        return fgs.residual_norm(y, x, w_pre=self.w_pre, w_post=self.w_post, gate=self.gate)


class Block(torch.nn.Module):
    """Attention and a gated MLP over the stream x and its norm n."""

    def __init__(self, width: int, heads: int, kv_heads: int, hidden: int, device):
        super().__init__()
        self.split = [heads, kv_heads, kv_heads]
        self.dim = width // heads
        self.qkv = fgs.Linear(width, (heads + 2 * kv_heads) * self.dim, device=device)
        self.out = fgs.Linear(width, width, device=device)
        self.up = fgs.Linear(width, 2 * hidden, device=device)
        self.down = fgs.Linear(hidden, width, device=device)
        self.after_attention, self.after_mlp = Boundary(width, device), Boundary(width, device)

    def forward(self, x, n, cu_seqlens):
        tokens, width = n.shape
        q, k, v = self.qkv(n).view(tokens, -1, self.dim).split(self.split, 1)    # views: nothing is copied
        y = self.out(fgs.attention(q, k, v, cu_seqlens).view(tokens, width))
        x, n = self.after_attention(y, x)
        return self.after_mlp(self.down(self.activate(self.up(n))), x)

    def activate(self, gate_up):
        a, b = gate_up.chunk(2, 1)
        return torch.nn.functional.silu(a) * b


def train(steps=10, tokens=1024, width=512, heads=8, kv_heads=2, hidden=1024, layers=2, max_norm=1.0, lr=2e-3, seed=0,
          say=print):
    """The losses and the gradients' norms of `steps` steps."""
    torch.manual_seed(seed)
    device = torch.device("cuda")
    blocks = torch.nn.ModuleList(Block(width, heads, kv_heads, hidden, device) for _ in range(layers))
    params = list(blocks.parameters())
    optimizer = torch.optim.AdamW(params, lr=lr)
    cuts = torch.randperm(tokens - 1)[:6].sort().values + 1                      # seven documents
    cu_seqlens = torch.cat([torch.tensor([0]), cuts, torch.tensor([tokens])]).to(torch.int32).to(device)
    x0 = torch.randn(tokens, width, device=device)
    n0 = torch.nn.functional.normalize(x0, dim=1).mul(width ** 0.5).to(torch.bfloat16)
    target = torch.randn(tokens, width, device=device)
    losses, norms = [], []
    for step in range(steps):
        begin = time.perf_counter()
        x, n = x0, n0
        for block in blocks:
            x, n = block(x, n, cu_seqlens)
        loss = (n.float() - target).square().mean()
        loss.backward()
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
    for name, value in (("steps", 10), ("tokens", 1024), ("width", 512), ("heads", 8), ("kv-heads", 2),
                        ("hidden", 1024), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    train(**vars(ap.parse_args()))
