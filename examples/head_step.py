"""The head of a model through a rollout step and a training step.

Rollout: the final RMS norm of the sequences' last hidden states, the 4-bit
head times these few tokens, the most probable token of each.  Training: the
same norm over a batch, token losses of the BF16 head without its logits, the
gradients of head, hidden states and norm weight, a plain gradient step, and
the head quantized again for the next rollout.

    python examples/head_step.py [--steps 20] [--vocab 2000] [--hidden 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rollout_x128_act_gb300 as jq  # noqa: E402

EPS = 1e-6


class Head:
    """Norm weight and head in FP32, with the BF16 and NVFP4 copies that the kernels read."""

    def __init__(self, vocab, hidden, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm = torch.ones(hidden, device=device)
        self.weight = 0.02 * torch.randn((vocab, hidden), generator=g, device=device)
        self.sync()

    def sync(self):
        """The copies of the current weights: what training reads and what the rollout reads."""
        self.norm16 = self.norm.to(torch.bfloat16)
        self.weight16 = self.weight.to(torch.bfloat16)
        self.weight4 = jq.quant_nvfp4(self.weight16, scope_amax=jq.amax_bf16(self.weight16))

    def rollout(self, x):
        """BF16 hidden states of up to 16 sequences -> (tokens, logits)."""
        y, _, _ = jq.norm_fwd(x, self.norm16, eps=EPS, kind=jq.NORM_RMS)
        logits = jq.gemv_nvfp4(y, self.weight4)
        return logits.argmax(1), logits

    def grads(self, x, target, weight):
        """Loss of each token of a batch, and the gradients of sum(weight * loss)."""
        y, _, rstd = jq.norm_fwd(x, self.norm16, eps=EPS, kind=jq.NORM_RMS)
        loss, lse = jq.linear_ce(y, self.weight16, target)
        dy, dhead = jq.linear_ce_bwd(y, self.weight16, target, lse, weight)
        dx, dnorm, _ = jq.norm_bwd(dy, x, self.norm16, None, rstd, kind=jq.NORM_RMS)
        return loss, dx, dhead, dnorm

    def step(self, x, target, rate):
        """One gradient step on the mean loss of the rows with a target; that loss."""
        count = (target >= 0).sum()
        weight = (1.0 / count).expand(target.shape[0]).contiguous()
        loss, _, dhead, dnorm = self.grads(x, target, weight)
        self.weight -= rate * dhead
        self.norm -= rate * dnorm
        self.sync()
        return loss.sum() / count


def main(steps=20, vocab=2000, hidden=256, tokens=512, rate=2.0, seed=0):
    """Teaches the head a fixed token for each of 64 hidden states; returns the losses and the rollout's hits."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    states = torch.randn((64, hidden), generator=g, device="cuda").to(torch.bfloat16)
    answer = torch.randint(0, vocab, (64,), generator=g, device="cuda")
    head, losses = Head(vocab, hidden, seed), []
    for _ in range(steps):
        pick = torch.randint(0, 64, (tokens,), generator=g, device="cuda")
        target = answer[pick]
        target[: tokens // 8] = -100  # prompt tokens
        losses.append(float(head.step(states[pick], target, rate)))
    hits = sum(int((head.rollout(states[i:i + 16])[0] == answer[i:i + 16]).sum()) for i in range(0, 64, 16))
    return losses, hits


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--hidden", type=int, default=256)
    a = ap.parse_args()
    losses, hits = main(a.steps, a.vocab, a.hidden)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  loss {v:.4f}")
    print(f"rollout with the 4-bit head: {hits} of 64 answers")
