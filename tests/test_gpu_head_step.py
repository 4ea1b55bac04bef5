"""The head's operators together: a rollout step with the 4-bit head, a training step with its gradients
against the same formulas in binary64, and a few steps that have to learn."""
import os
import sys

import pytest
import torch

import rollout_x128_act_gb300 as jq
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import head_step  # noqa: E402

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8  # BF16


def _batch(n, vocab, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((n, hidden), generator=g, device="cuda") * 2).to(torch.bfloat16)
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    target[::5] = -100
    return x, target, torch.randn(n, generator=g, device="cuda") / n


def test_gradients_of_the_whole_head():
    """The chain's gradient in binary64 from the same BF16 weights.  Each BF16 tensor on the way (y, d, dy, dx)
    rounds by at most 2^-8 of its value: in the 2-norm four such roundings, and y's enters the loss twice."""
    n, vocab, hidden = 200, 1500, 256
    head = head_step.Head(vocab, hidden, seed=3)
    x, target, weight = _batch(n, vocab, hidden, 4)
    loss, dx, dhead, dnorm = head.grads(x, target, weight)
    ok = target >= 0
    X = x.double().requires_grad_()
    N, W = head.norm16.double().requires_grad_(), head.weight16.double().requires_grad_()
    y = X / (X.square().mean(1, keepdim=True) + head_step.EPS).sqrt() * N
    z = y @ W.T
    ref = torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    (ref * weight.double())[ok].sum().backward()
    size = (y.abs() @ W.abs().T).amax(1)  # a logit moves by y's rounding
    assert bool(((loss.double() - ref).abs()[ok] <= (2 * HALF * size + 1e-5 * size)[ok]).all())
    assert bool((loss[~ok] == 0).all()) and bool((dx[~ok] == 0).all())
    for got, want in ((dx, X.grad), (dhead, W.grad), (dnorm, N.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 6 * HALF


def test_rollout_picks_the_dequantized_heads_token():
    head = head_step.Head(777, 512, seed=5)
    x, _, _ = _batch(16, 777, 512, 6)
    token, logits = head.rollout(x)
    W = jq.dequant_nvfp4_bf16(head.weight4["q"], head.weight4["sb"], head.weight4["sg"]).double()
    y, _, _ = jq.norm_fwd(x, head.norm16, eps=head_step.EPS, kind=jq.NORM_RMS)
    z, size = y.double() @ W.T, y.double().abs() @ W.abs().T
    assert bool(((logits.double() - z).abs() <= (1e-5 + HALF) * size).all())  # W is rounded to BF16 here only
    assert torch.equal(token, logits.argmax(1))


def test_a_few_steps_learn():
    losses, hits = head_step.main(steps=20)
    assert losses[0] > 7 and losses[-1] < 0.2 * losses[0]
    assert hits >= 60


def test_helpers_on_another_stream():
    """The helpers' `stream` argument: same results, workspaces and outputs allocated for that stream."""
    head = head_step.Head(900, 256, seed=7)
    x, target, weight = _batch(300, 900, 256, 8)
    y, _, rstd = jq.norm_fwd(x, head.norm16, eps=1e-6, kind=jq.NORM_RMS)
    loss, lse = jq.linear_ce(y, head.weight16, target)
    dy, dw = jq.linear_ce_bwd(y, head.weight16, target, lse, weight)
    dx, dn, _ = jq.norm_bwd(dy, x, head.norm16, None, rstd, kind=jq.NORM_RMS)
    z = jq.gemv_nvfp4(y[:4], head.weight4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, _, rstd1 = jq.norm_fwd(x, head.norm16, eps=1e-6, kind=jq.NORM_RMS, stream=side)
    loss1, lse1 = jq.linear_ce(y1, head.weight16, target, stream=side)
    dy1, dw1 = jq.linear_ce_bwd(y1, head.weight16, target, lse1, weight, stream=side)
    dx1, dn1, _ = jq.norm_bwd(dy1, x, head.norm16, None, rstd1, kind=jq.NORM_RMS, stream=side)
    z1 = jq.gemv_nvfp4(y1[:4], head.weight4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((y, y1), (loss, loss1), (dy, dy1), (dw, dw1), (dx, dx1), (dn, dn1), (z, z1)):
        assert torch.equal(a, b)
