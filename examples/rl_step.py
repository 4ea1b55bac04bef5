"""A rollout and two training steps of a small model: a mixture-of-experts layer and the head of head_step.py.

Rollout: few hidden states through the NVFP4 layer, the norm and the 4-bit head; the tokens that they pick.
Training on packed answers: token losses of the head, the clipped policy loss with its KL term, and its gradient
through head and norm; or the distance to a teacher's top logits and its gradient.

    python examples/rl_step.py [--vocab 2000] [--hidden 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import rollout_x128_act_gb300 as jq  # noqa: E402
from head_step import EPS, Head  # noqa: E402


class Layer:
    """A mixture-of-experts layer with a residual connection, NVFP4 weights and a BF16 router."""

    def __init__(self, hidden, inter=128, experts=16, topk=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5
            return w.to(torch.bfloat16)

        self.router = weights(experts, hidden)
        self.w13 = jq.quant_nvfp4_experts(weights(experts, 2 * inter, hidden))
        self.w2 = jq.quant_nvfp4_experts(weights(experts, hidden, inter))
        self.topk = topk

    def __call__(self, x):
        """BF16 hidden states of up to 16 sequences."""
        y, _, _ = jq.moe_nvfp4(x, self.router, self.w13, self.w2, self.topk, out_dtype=torch.float32)
        return (x + y).to(torch.bfloat16)


def rollout(layer, head, x):
    """(tokens, logits) of up to 16 sequences' hidden states."""
    return head.rollout(layer(x))


def _head_backward(head, x, y, rstd, dy, dhead):
    dx, dnorm, _ = jq.norm_bwd(dy, x, head.norm16, None, rstd, kind=jq.NORM_RMS)
    return dx, dhead, dnorm


def token_losses(head, x, tokens):
    """Minus the log-probabilities of the tokens."""
    y, _, _ = jq.norm_fwd(x, head.norm16, eps=EPS, kind=jq.NORM_RMS)
    return jq.linear_ce(y, head.weight16, tokens)[0]


def policy_grads(head, x, tokens, old, adv, offsets, ref=None, mask=None, kl=0.0):
    """The policy loss's six numbers and its gradients (hidden states, head, norm weight)."""
    y, _, rstd = jq.norm_fwd(x, head.norm16, eps=EPS, kind=jq.NORM_RMS)
    nll, lse = jq.linear_ce(y, head.weight16, tokens)
    how = dict(seg_offsets=offsets, nll_ref=ref, mask=mask, kl=kl, mean=jq.POLICY_MEAN_SEGMENTS)
    out, seg = jq.policy_loss(nll, old, adv, **how)
    dnll = jq.policy_loss_bwd(nll, old, adv, out, seg, **how)
    dy, dhead = jq.linear_ce_bwd(y, head.weight16, tokens, lse, dnll)
    return (out,) + _head_backward(head, x, y, rstd, dy, dhead)


def distill_grads(head, x, ids, teacher, weight):
    """Each row's distance to the teacher, and the gradients of sum(weight * distance)."""
    y, _, rstd = jq.norm_fwd(x, head.norm16, eps=EPS, kind=jq.NORM_RMS)
    loss, lse, logp = jq.linear_distill(y, head.weight16, ids, teacher)
    dy, dhead = jq.linear_distill_bwd(y, head.weight16, ids, teacher, lse, logp, weight)
    return (loss,) + _head_backward(head, x, y, rstd, dy, dhead)


def main(vocab=2000, hidden=256, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer, head, teacher = Layer(hidden, seed=seed), Head(vocab, hidden, seed), Head(vocab, hidden, seed + 7)
    prompts = torch.randn((16, hidden), generator=g, device="cuda").to(torch.bfloat16)
    tokens, _ = rollout(layer, head, prompts)
    print("rollout:", tokens.tolist())
    # packed answers: 8 sequences, the first tokens of each are the prompt's
    lengths = torch.randint(5, 60, (8,), generator=g, device="cuda")
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), lengths.cumsum(0)))
    n = int(offsets[-1])
    x = torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[offsets[:-1]] = False
    old = token_losses(head, x, tokens)
    adv = torch.randn(8, generator=g, device="cuda")
    for step in range(3):
        out, _, dhead, dnorm = policy_grads(head, x, tokens, old, adv, offsets, old, mask, kl=0.05)
        print(f"policy step {step}: loss {float(out[0]):+.4f}  mean KL {float(out[2]):.5f}  "
              f"clipped {int(out[3])} of {int(out[4])} tokens")
        head.weight -= 5.0 * dhead
        head.norm -= 5.0 * dnorm
        head.sync()
    y, _, _ = jq.norm_fwd(x, teacher.norm16, eps=EPS, kind=jq.NORM_RMS)
    top, ids = (y.float() @ teacher.weight.T).topk(32, dim=1)
    weight = torch.full((n,), 1.0 / n, device="cuda")
    for step in range(3):
        loss, _, dhead, dnorm = distill_grads(head, x, ids, top, weight)
        print(f"distillation step {step}: {float(loss.mean()):.4f}")
        head.weight -= 5.0 * dhead
        head.norm -= 5.0 * dnorm
        head.sync()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--hidden", type=int, default=256)
    a = ap.parse_args()
    main(a.vocab, a.hidden)
