"""A small student distilled from a teacher's top logits, trained with the 8-bit
optimizer: every operator of the training step as it would be used.

    python examples/distill_step.py [--steps 150]

Each step embeds the last tokens of a context, runs blocks of norm, gated
feed-forward product and gated residual, compares the logits with a fixed
teacher's sixteen largest (and, in part, with the next token), and steps
AdamW8bitSR on the bf16 parameters.
"""
import argparse
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_blockwise_adamw_gb300 import nn as q8nn           # noqa: E402
from bit_blockwise_adamw_gb300.optim import AdamW8bitSR    # noqa: E402


class Student(nn.Module):
    def __init__(self, vocab, dim, d_ff, blocks, context, device):
        super().__init__()
        kw = dict(dtype=torch.bfloat16, device=device)
        self.embed = nn.Parameter(torch.randn(vocab, dim, device=device).mul_(0.5).bfloat16())
        self.mix = nn.Linear(context * dim, dim, bias=False, **kw)
        self.first = q8nn.BlockNorm(dim, post=None, gate=False, device=device)
        self.ff = nn.ModuleList([q8nn.GatedFeedForward(dim, d_ff, device=device) for _ in range(blocks)])
        self.norm = nn.ModuleList([q8nn.BlockNorm(dim, device=device) for _ in range(blocks)])
        self.head = nn.Linear(dim, vocab, bias=False, **kw)

    def forward(self, tokens):
        r, z = self.first(torch.zeros(*tokens.shape[:-1], self.head.in_features, dtype=torch.bfloat16, device=tokens.device),
                          self.mix(self.embed[tokens].flatten(-2)))
        for ff, norm in zip(self.ff, self.norm):
            r, z = norm(r, ff(z))
        return self.head(z)


def train(steps=150, batch=512, vocab=2003, dim=256, d_ff=704, blocks=3, context=4, top=16, lr=4e-3, seed=0, device="cuda"):
    """The mean loss of each step."""
    torch.manual_seed(seed)
    student = Student(vocab, dim, d_ff, blocks, context, device)
    with torch.no_grad():                            # a teacher that depends on the context: a wide random layer
        key = torch.randn(vocab, 64, device=device)
        mix = torch.randn(context * 64, 256, device=device) / 16
        out = torch.randn(256, vocab, device=device) / 4
    opt = AdamW8bitSR(student.parameters(), lr=lr, weight_decay=0.01, seed=seed)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab // 20, (batch, context), device=device)
        teacher = torch.tanh(key[tokens].flatten(-2) @ mix) @ out
        logits, ids = teacher.topk(top, -1)
        loss = q8nn.distill_topk(student(tokens), ids, logits, labels=ids[:, 0], temperature=2.0, kd_weight=0.8,
                                 ce_weight=0.2).mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=150)
    a = ap.parse_args()
    losses = train(a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.4f" % (i, losses[i]))
    print("last ten: %.4f" % (sum(losses[-10:]) / len(losses[-10:])))


if __name__ == "__main__":
    main()
