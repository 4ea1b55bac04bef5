"""The losses and the mixture-of-experts layer together, as a rollout step and a training step use them: gradients of
the whole chains against the same formulas in binary64."""
import os
import subprocess
import sys

import pytest
import torch

import rollout_x128_act_gb300 as jq
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import head_step  # noqa: E402
import rl_step  # noqa: E402

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8  # BF16


def _norm(x, w):
    return x / (x.square().mean(1, keepdim=True) + head_step.EPS).sqrt() * w


def _leaves(head, x):
    return x.double().requires_grad_(), head.weight16.double().requires_grad_(), head.norm16.double().requires_grad_()


def _same_gradients(got, leaves):
    """Each BF16 tensor on the way (y, d, dy, dx) rounds by at most 2^-8 of its value: in the 2-norm four such
    roundings, and y's enters the loss twice."""
    for a, leaf in zip(got, leaves):
        assert float((a.double() - leaf.grad).norm() / leaf.grad.norm()) <= 6 * HALF


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_gradients_of_the_policy_loss_through_the_head(kl):
    """Sampling policy and reference lie near the policy, far from the clip's borders (their distance is 0.2 at
    most, where y's rounding moves a token's loss by less)."""
    n, vocab, hidden = 230, 1500, 256
    head = head_step.Head(vocab, hidden, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randn((n, hidden), generator=g, device="cuda") * 2).to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    offsets = torch.tensor([0, 40, 41, 41, 150, 220], device="cuda")  # 10 rows of padding
    mask = torch.rand(n, generator=g, device="cuda") < 0.8
    adv = torch.randn(5, generator=g, device="cuda")
    nll = rl_step.token_losses(head, x, tokens)
    old = nll + 0.05 * torch.randn(n, generator=g, device="cuda").clamp(-1, 1)
    ref = nll + 0.3 * torch.randn(n, generator=g, device="cuda")
    out, *got = rl_step.policy_grads(head, x, tokens, old, adv, offsets, ref, mask, kl)
    X, W, N = leaves = _leaves(head, x)
    z = _norm(X, N) @ W.T
    loss = torch.logsumexp(z, 1) - z.gather(1, tokens[:, None])[:, 0]
    seg = torch.bucketize(torch.arange(n, device="cuda"), offsets[1:], right=True)
    on = mask & (seg < 5)
    count = torch.zeros(5, dtype=torch.float64, device="cuda").index_add_(0, seg[on], torch.ones_like(loss)[on])
    weight = 1 / (count[seg[on]] * (count > 0).sum())
    d = loss[on] - ref.double()[on]
    surrogate = -adv.double()[seg[on]] * (old.double()[on] - loss[on]).exp()
    total = (weight * (surrogate + kl * (d.exp() - 1 - d))).sum()
    total.backward()
    assert int(out[3]) == 0 and int(out[4]) == int(on.sum())
    assert abs(float(out[0]) - float(total.detach())) <= 4 * HALF * float((weight * (surrogate.abs() + kl)).sum().detach())
    _same_gradients(got, leaves)
    assert bool((got[0][~on] == 0).all())


def test_gradients_of_the_distillation_through_the_head():
    n, vocab, hidden, k = 150, 1200, 256, 20
    head, teacher = head_step.Head(vocab, hidden, seed=5), head_step.Head(vocab, hidden, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.randn((n, hidden), generator=g, device="cuda") * 2).to(torch.bfloat16)
    t, ids = (_norm(x.double(), 1.0) @ teacher.weight16.double().T * 4).topk(k, dim=1)
    ids[::6] = -1  # prompt tokens
    weight = torch.randn(n, generator=g, device="cuda") / n
    loss, *got = rl_step.distill_grads(head, x, ids, t.float(), weight)
    X, W, N = leaves = _leaves(head, x)
    logp = torch.log_softmax(_norm(X, N) @ W.T, 1)
    q = torch.softmax(t.float().double(), 1)
    ref = (q * (q.log() - logp.gather(1, ids.clamp(min=0)))).sum(1)
    on = (ids >= 0).any(1)
    (ref * weight.double())[on].sum().backward()
    size = (_norm(X, N).abs() @ W.abs().T).amax(1)  # a logit moves by y's rounding
    assert bool(((loss.double() - ref).abs() <= 2 * HALF * size + 1e-5 * size)[on].all())
    assert bool((loss[~on] == 0).all())
    _same_gradients(got, leaves)


def test_rollout_goes_through_the_layer():
    """The tokens are those of the layer's, the norm's and the head's own calls; more than 16 sequences are refused."""
    layer, head = rl_step.Layer(512, seed=8), head_step.Head(777, 512, seed=9)
    x = torch.randn((16, 512), generator=torch.Generator(device="cuda").manual_seed(10), device="cuda")
    x = x.to(torch.bfloat16)
    token, logits = rl_step.rollout(layer, head, x)
    y, ids, p = jq.moe_nvfp4(x, layer.router, layer.w13, layer.w2, layer.topk, out_dtype=torch.float32)
    h, _, _ = jq.norm_fwd((x + y).to(torch.bfloat16), head.norm16, eps=head_step.EPS, kind=jq.NORM_RMS)
    assert torch.equal(logits, jq.gemv_nvfp4(h, head.weight4)) and torch.equal(token, logits.argmax(1))
    assert ids.shape == (16, 4) and bool(((p.sum(1) - 1).abs() < 1e-6).all())
    with pytest.raises(jq.JetqError):
        layer(torch.zeros((17, 512), dtype=torch.bfloat16, device="cuda"))


def test_a_whole_step_in_a_graph():
    """Rollout layer, policy loss and distillation with their gradients captured together and replayed."""
    n, vocab, hidden = 96, 600, 128
    head, layer = head_step.Head(vocab, hidden, seed=11), rl_step.Layer(hidden, inter=64, experts=8, topk=2, seed=12)
    g = torch.Generator(device="cuda").manual_seed(13)
    x = torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    old, adv = rl_step.token_losses(head, x, tokens) + 0.1, torch.randn(3, generator=g, device="cuda")
    offsets = torch.tensor([0, 30, 70, 96], device="cuda")
    ids = torch.randint(0, vocab, (n, 8), generator=g, device="cuda")
    teacher = torch.randn((n, 8), generator=g, device="cuda")
    weight = torch.full((n,), 1.0 / n, device="cuda")

    def step():
        return (layer(x[:5]),) + rl_step.policy_grads(head, x, tokens, old, adv, offsets) + \
            rl_step.distill_grads(head, x, ids, teacher, weight)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert jq.jetq_check_device_error() == jq.OK


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "rl_step.py"), "--vocab", "300", "--hidden",
                        "128"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("policy step") == 3 and r.stdout.count("distillation step") == 3
