"""Trains a small causal transformer on a synthetic copy task.

Every block runs on the library's training operators in both directions
(layer norm, attention, linear layers whose inputs are kept in 8 bits), and
the library's Muon step with its AdamW fallback applies the gradients.  With
--experts the hidden layers are experts, two for each token; with --bits 8 the
linear layers' products run in 8 bits and AdamW's states are kept in 8.

    python examples/train_block.py [--steps 60] [--dim 256] [--heads 4] [--seq 128] [--experts 8] [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_orthogonalized_muon_gb300 as muon  # noqa: E402
from newton_schulz_orthogonalized_muon_gb300 import nn  # noqa: E402


class Experts(torch.nn.Module):
    """Two experts of hidden size 2 dim for each token, weighted by the router."""

    def __init__(self, dim, experts):
        super().__init__()
        self.experts = experts
        self.router = torch.nn.Linear(dim, experts, bias=False, dtype=torch.bfloat16)
        self.up, self.down = nn.ExpertLinear(experts, dim, 2 * dim), nn.ExpertLinear(experts, 2 * dim, dim)

    def forward(self, x):
        flat = x.flatten(0, 1)
        share, chosen = self.router(flat).float().topk(2)
        # rows in the order of their experts, and where each expert's begin
        sorted_, order = chosen.flatten().sort(stable=True)
        offsets = torch.searchsorted(sorted_, torch.arange(self.experts + 1, device=x.device), out_int32=True)
        y = self.down(torch.nn.functional.gelu(self.up(flat[order // 2], offsets)), offsets)
        back = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=x.device))
        return (y[back].unflatten(0, (-1, 2)) * share.softmax(-1).to(y.dtype)[..., None]).sum(1).view_as(x)


class Block(torch.nn.Module):
    def __init__(self, dim, heads, experts=0, products8=False):
        super().__init__()
        self.heads = heads
        self.norm_1, self.norm_2 = nn.LayerNorm(dim), nn.LayerNorm(dim)
        self.qkv, self.proj = nn.Linear8(dim, 3 * dim, products8=products8), nn.Linear8(dim, dim, products8=products8)
        if experts:
            self.mlp = Experts(dim, experts)
        else:
            self.up, self.down = (nn.Linear8(dim, 4 * dim, products8=products8),
                                  nn.Linear8(4 * dim, dim, products8=products8))

    def forward(self, x):
        b, s, d = x.shape
        q, k, v = self.qkv(self.norm_1(x)).view(b, s, 3, self.heads, d // self.heads).unbind(2)
        x = x + self.proj(nn.attention(q, k, v, causal=True).reshape(b, s, d))
        if hasattr(self, "mlp"):
            return x + self.mlp(self.norm_2(x))
        return x + self.down(torch.nn.functional.gelu(self.up(self.norm_2(x))))


class Model(torch.nn.Module):
    def __init__(self, vocab, seq, dim, heads, layers, experts=0, products8=False):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, dim, dtype=torch.bfloat16)
        self.embed_pos = torch.nn.Embedding(seq, dim, dtype=torch.bfloat16)
        self.blocks = torch.nn.ModuleList(Block(dim, heads, experts, products8) for _ in range(layers))
        self.norm = nn.LayerNorm(dim)
        self.lm_head = nn.Linear8(dim, vocab)

    def forward(self, tokens):
        x = self.embed(tokens) + self.embed_pos.weight[:tokens.shape[1]]
        for block in self.blocks:
            x = block(x)
        return self.lm_head(self.norm(x))


def train(steps=60, dim=256, heads=4, seq=128, batch=16, vocab=64, layers=2, seed=0, log=print, experts=0, bits=16):
    """The losses of `steps` steps.  The second half of each sequence repeats
    the first; only it is scored."""
    torch.manual_seed(seed)
    model = Model(vocab, seq, dim, heads, layers, experts, bits == 8).cuda()
    heads_of = {f"blocks.{i}.qkv.weight": 3 for i in range(layers)}       # q, k and v orthogonalised apart
    # an expert's matrix each, with the update scale of one
    heads_of |= {f"blocks.{i}.mlp.{n}.weight": experts for i in range(layers) for n in ("up", "down") if experts}
    scale = {n: 2 * dim for n in heads_of if ".mlp." in n}
    opt = muon.Muon(model.named_parameters(), lr=0.02, wd=0.0, adamw_lr=3e-3, split_heads=heads_of, scale_dims=scale,
                    adamw_states=8 if bits == 8 else 32)
    losses = []
    for step in range(steps):
        half = torch.randint(vocab, (batch, seq // 2), device="cuda")
        tokens = torch.cat([half, half], 1)
        logits = model(tokens[:, :-1]).float()
        loss = torch.nn.functional.cross_entropy(logits[:, seq // 2 - 1:].flatten(0, 1), tokens[:, seq // 2:].flatten())
        loss.backward()
        opt.step()
        opt.zero_grad()
        losses.append(loss.item())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step}: loss {losses[-1]:.4f}")
    if muon.default_handle().check() != 0:
        raise RuntimeError("the device error word is set")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 60), ("dim", 256), ("heads", 4), ("seq", 128), ("experts", 0), ("bits", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    train(**vars(ap.parse_args()))
