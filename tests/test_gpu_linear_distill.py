"""Distillation of a linear head from a teacher's top logits against its definition in binary64.

Bounds.  An unlisted logit's FP32 sum is within SUM * sum |x w| of the exact one (SUM = 1e-5, the bound every GEMM
test of this library uses); a listed one is a joined sum of FP32 chains of at most c / 256 products.  The loss moves
by Q times the errors of its logits and of lse; an exponential by the error of its exponent.  d is rounded to BF16
(2^-8 of its value), its sums are within SUM of the sum of magnitudes, a BF16 result is rounded once more.
"""
import math

import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SUM = 1e-5
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24

SIZES = [(1, 1, 8, 1), (1, 1000, 64, 7), (2, 255, 8, 255), (5, 257, 72, 32), (127, 256, 64, 33), (129, 511, 264, 64),
         (256, 513, 128, 2), (300, 1000, 520, 100), (257, 4097, 1032, 256), (513, 300, 2048, 20)]


def _inputs(n, v, c, k, seed, pad=0, gaps=True, spread=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, c + pad), generator=g, device=DEV).to(torch.bfloat16)[:, :c]
    w = (torch.randn((v, c + pad), generator=g, device=DEV) * spread).to(torch.bfloat16)[:, :c]
    ids = torch.rand((n, v), generator=g, device=DEV).topk(min(k, v), dim=1).indices
    ids = torch.cat((ids, torch.full((n, k - ids.shape[1]), -1, device=DEV)), 1)
    t = 2 * torch.randn((n, k), generator=g, device=DEV)
    if gaps and n > 2:
        drop = torch.rand((n, k), generator=g, device=DEV) < 0.2
        drop[1::4] = True  # rows that list nothing
        ids = torch.where(drop, torch.full_like(ids, -100), ids)
        ids[2::8, 0] = v  # outside the vocabulary on the other side
        t = torch.where((ids < 0) | (ids >= v), torch.full_like(t, math.nan), t)
    return x, w, ids, t, torch.randn(n, generator=g, device=DEV)


def _logprobs(t, ids, v):
    """The listed logits as log-probabilities that sum to less than one."""
    on = (ids >= 0) & (ids < v)
    return t - 0.3 - torch.logsumexp(torch.where(on, t, torch.full_like(t, -math.inf)), 1, keepdim=True).clamp(min=-50)


def _teacher(t, ids, v, renorm):
    """(q, log q, listed) in binary64, zero where nothing is listed."""
    on = (ids >= 0) & (ids < v)
    t = torch.where(on, t.double(), torch.full_like(t.double(), -math.inf))
    if renorm:
        total = torch.logsumexp(t, 1, keepdim=True)
        t = torch.where(total > -math.inf, t - total, t)
    q = t.exp()
    return q, torch.where(q > 0, t, torch.zeros_like(t)), on


def _define(x, w, ids, t, scale, renorm):
    z = scale * (x.double() @ w.double().T)
    lse = torch.logsumexp(z, 1)
    q, logq, on = _teacher(t, ids, w.shape[0], renorm)
    logp = torch.where(on, z.gather(1, ids.clamp(0, w.shape[0] - 1)) - lse[:, None], torch.zeros_like(q))
    loss = torch.where(q > 0, q * (logq - logp), torch.zeros_like(q)).sum(1)
    ez = scale * SUM * (x.double().abs() @ w.double().abs().T).amax(1)
    size = (q * (logq.abs() + logp.abs() + 1)).sum(1)
    return z, lse, loss, logp, q, on, ez, size


def _check_fwd(x, w, ids, t, scale=1.0, renorm=True, **kw):
    loss, lse, logp = jq.linear_distill(x, w, ids, t, scale=scale, renorm=renorm, **kw)
    assert jq.jetq_check_device_error() == jq.OK
    _, rlse, rloss, rlogp, q, on, ez, size = _define(x, w, ids, t, scale, renorm)
    one = 8 * HALF_F32
    assert bool(((lse.double() - rlse).abs() <= ez + one * (rlse.abs() + 1)).all())
    assert bool(((logp.double() - rlogp).abs() <= 2 * ez[:, None] + one * (rlogp.abs() + 1)).all())
    assert bool((logp[~on] == 0).all())
    assert bool(((loss.double() - rloss).abs() <= 2 * ez * q.sum(1) + one * size).all())
    assert bool((loss[~on.any(1)] == 0).all())
    return loss, lse, logp


def _check_bwd(x, w, ids, t, lse, logp, dloss, scale=1.0, renorm=True, dw_dtype=torch.float32, **kw):
    dx, dw = jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss, scale=scale, renorm=renorm, dw_dtype=dw_dtype, **kw)
    assert jq.jetq_check_device_error() == jq.OK
    z, _, _, _, q, on, ez, _ = _define(x, w, ids, t, scale, renorm)
    coef = torch.where(on.any(1), dloss.double(), torch.zeros_like(ez))
    p = torch.exp(z - lse.double()[:, None]) * q.sum(1, keepdim=True)
    d = p.clone()
    spread = torch.zeros_like(p).scatter_add_(1, ids.clamp(0, w.shape[0] - 1), torch.where(on, q, torch.zeros_like(q)))
    d, mass = (d - spread) * coef[:, None], (p + spread) * coef.abs()[:, None]
    moved = ez[:, None] + 8 * HALF_F32 * (1 + lse.double().abs()[:, None])  # of an exponent
    off = d.abs() * (HALF_BF16 + SUM) + mass * 2 * moved
    X, W = x.double(), w.double()
    last = HALF_BF16 if dw_dtype is torch.bfloat16 else 2 * HALF_F32
    for got, want, tol, half in ((dx, scale * (d @ W), scale * (off @ W.abs()), HALF_BF16),
                                 (dw, scale * (d.T @ X), scale * (off.T @ X.abs()), last)):
        assert bool(((got.double() - want).abs() <= tol * 1.01 + half * want.abs() + 1e-30).all())
    assert bool((dx[~on.any(1)] == 0).all())
    return dx, dw


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("n,v,c,k", SIZES)
def test_both_directions(n, v, c, k, renorm):
    x, w, ids, t, dloss = _inputs(n, v, c, k, n + v, pad=8 if n % 2 else 0)
    if not renorm:
        t = _logprobs(t, ids, v)
    scale = 0.7 if n % 3 else 1.0
    _, lse, logp = _check_fwd(x, w, ids, t, scale, renorm)
    _check_bwd(x, w, ids, t, lse, logp, dloss, scale, renorm, torch.bfloat16 if n % 2 else torch.float32)


@pytest.mark.parametrize("n", [1, 16, 100, 400])
def test_a_large_vocabulary(n):
    """Several chunks of marks a row (131072 columns and more), single CTAs and pairs, tiles of uneven width."""
    x, w, ids, t, _ = _inputs(n, 140001, 128, 50, n, gaps=n > 2)
    ids[0, :4] = torch.tensor([0, 140000, 131071, 131072], device=DEV)
    t[0] = 1.0
    _check_fwd(x, w, ids, t)


def test_columns_at_the_edges_of_tiles():
    """Every column of a small vocabulary is listed by some row: borders of 32, 128 and 256 columns among them."""
    v, k = 777, 111
    x, w, _, t, dloss = _inputs(7, v, 64, k, 3, gaps=False)
    ids = torch.arange(v, device=DEV).view(7, k)
    _, lse, logp = _check_fwd(x, w, ids, t)
    _check_bwd(x, w, ids, t, lse, logp, dloss)


def test_the_whole_vocabulary_listed():
    """No column is left to the tensor cores' statistics: the sum of the others is empty."""
    x, w, ids, t, dloss = _inputs(9, 200, 96, 200, 4, gaps=False)
    _, lse, logp = _check_fwd(x, w, ids, t)
    assert bool(((logp.double().exp().sum(1) - 1).abs() < 1e-5).all())
    _check_bwd(x, w, ids, t, lse, logp, dloss)


@pytest.mark.parametrize("renorm", [True, False])
def test_a_column_listed_twice(renorm):
    """Its q adds up in the gradient; lse has its term once."""
    x, w, ids, t, dloss = _inputs(50, 700, 128, 12, 5, gaps=False)
    ids[:, 5] = ids[:, 2]
    ids[::2, 9] = ids[::2, 2]
    ids[7, :] = 333
    if not renorm:
        t = _logprobs(t, ids, 700)
    _, lse, logp = _check_fwd(x, w, ids, t, renorm=renorm)
    _check_bwd(x, w, ids, t, lse, logp, dloss, renorm=renorm)


def test_teachers_without_mass():
    """-infinity is a probability of zero; a row of nothing else has no loss, whatever renorm says."""
    x, w, ids, t, dloss = _inputs(20, 400, 64, 6, 6, gaps=False)
    t[3, 2] = t[4, 0] = -math.inf
    t[5] = -math.inf
    for renorm in (True, False):
        tt = t if renorm else t - 4
        loss, lse, logp = _check_fwd(x, w, ids, tt, renorm=renorm)
        assert float(loss[5]) == 0
        dx, _ = _check_bwd(x, w, ids, tt, lse, logp, dloss, renorm=renorm)
        assert bool((dx[5] == 0).all())


def test_rows_without_a_loss_may_hold_anything():
    x, w, ids, t, dloss = _inputs(140, 600, 72, 9, 7)
    none = ~((ids >= 0) & (ids < 600)).any(1)
    _, lse, logp = _check_fwd(x, w, ids, t)
    dx, dw = _check_bwd(x, w, ids, t, lse, logp, dloss)
    for value in (math.nan, math.inf):
        x2, lse2, logp2, dloss2 = x.clone(), lse.clone(), logp.clone(), dloss.clone()
        for a in (x2, lse2, logp2, dloss2):
            a[none] = value
        dx2, dw2 = jq.linear_distill_bwd(x2, w, ids, t, lse2, logp2, dloss2)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        loss3, lse3, _ = jq.linear_distill(x2, w, ids, t)
        assert bool((loss3[none] == 0).all()) and torch.equal(lse3[~none], lse[~none])


def test_a_number_missing_shows_in_its_row():
    x, w, ids, t, _ = _inputs(30, 300, 64, 5, 8, gaps=False)
    t[2, 1] = math.nan
    x[4, 3] = math.nan
    loss, lse, _ = jq.linear_distill(x, w, ids, t)
    bad = torch.zeros(30, dtype=torch.bool, device=DEV)
    bad[2] = bad[4] = True
    assert torch.equal(loss.isnan(), bad) and bool(lse[4].isnan()) and bool(lse[~bad].isfinite().all())


def test_student_and_teacher_nearly_agree():
    """Losses of 1e-5 to 1e-3 of confident rows.  The listed logits' chains are c / 256 products long, what is not
    listed has the mass R: the error is Q ((c / 256 + 2) 2^-24 max sum |x w| + R SUM max sum |x w|) and FP32
    rounding of the terms (8 of them), most of which the mass weighs down."""
    n, v, c, k = 200, 3000, 1024, 24
    g = torch.Generator(device=DEV).manual_seed(11)
    w = (torch.randn((v, c), generator=g, device=DEV) * 0.03).to(torch.bfloat16)
    near = torch.randint(0, v, (n,), generator=g, device=DEV)
    x = (torch.randn((n, c), generator=g, device=DEV) + 14 * w[near].float()).to(torch.bfloat16)
    z = x.double() @ w.double().T
    top, ids = z.topk(k, dim=1)
    t = (top + 0.02 * torch.randn((n, k), generator=g, device=DEV)).float()
    loss, lse, logp = jq.linear_distill(x, w, ids, t)
    _, rlse, rloss, rlogp, q, _, ez, size = _define(x, w, ids, t, 1.0, True)
    rest = 1 - rlogp.exp().sum(1)
    tight = ez / SUM * ((c / 256 + 2) * HALF_F32 + rest * SUM) + 8 * HALF_F32 * (q * (rlogp.abs() + 1)).sum(1)
    assert bool(((loss.double() - rloss).abs() <= 2 * tight).all())
    assert float((loss.double() - rloss).norm() / rloss.norm()) < float(2 * tight.norm() / rloss.norm())
    dx, dw = _check_bwd(x, w, ids, t, lse, logp, torch.ones(n, device=DEV))


def test_gradient_against_differences():
    """The kernel's losses at x + h u and x - h u (h u in whole BF16 steps) against dx . u: the logits move by
    |delta z| < 0.2, so the third-order rest is below 0.2^3 / 3 a row, next to the roundings of dx (2^-8)."""
    n, v, c, k = 40, 500, 256, 16
    x, w, ids, t, _ = _inputs(n, v, c, k, 12, gaps=False, spread=0.05)
    x = (x.float() * 64).round().div(64).clamp(-3, 3).to(torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(13)
    u = torch.randint(-1, 2, (n, c), generator=g, device=DEV).float() / 64
    up, down = (x.float() + u).to(torch.bfloat16), (x.float() - u).to(torch.bfloat16)
    step = (up.double() - down.double()) / 2
    loss, lse, logp = jq.linear_distill(x, w, ids, t)
    dx, _ = jq.linear_distill_bwd(x, w, ids, t, lse, logp, torch.ones(n, device=DEV))
    slope = (dx.double() * step).sum(1)
    change = (jq.linear_distill(up, w, ids, t)[0].double() - jq.linear_distill(down, w, ids, t)[0].double()) / 2
    dz = (step @ w.double().T).abs().amax(1)
    bound = dz ** 3 + 2 * HALF_BF16 * (dx.double().abs() * step.abs()).sum(1) + 1e-5
    mid = (up.double() + down.double()) / 2 - x.double()  # where the grid of BF16 is coarser
    bound = bound + 2 * (mid @ w.double().T).abs().amax(1)
    assert bool(((change - slope).abs() <= bound).all())


def test_strided_lists_and_pieces_of_the_vocabulary():
    x, w, ids, t, dloss = _inputs(130, 1500, 136, 10, 14)
    wide_i = torch.full((130, 17), 5, dtype=torch.int64, device=DEV)
    wide_t = torch.full((130, 23), math.nan, device=DEV)
    wide_i[:, :10], wide_t[:, 4:14] = ids, t
    a = jq.linear_distill(x, w, ids, t)
    b = jq.linear_distill(x, w, wide_i[:, :10], wide_t[:, 4:14])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    small = torch.empty(jq.jetq_linear_distill_bwd_workspace_bytes(130, 1500, 136, 10, True), dtype=torch.uint8,
                        device=DEV)
    _check_bwd(x, w, wide_i[:, :10], wide_t[:, 4:14], a[1], a[2], dloss, workspace=small)
    dx, dw = jq.linear_distill_bwd(x, w, ids, t, a[1], a[2], dloss)
    total = torch.ones((1500, 136), device=DEV)
    dx2, dw2 = jq.linear_distill_bwd(x, w, ids, t, a[1], a[2], dloss, dw=total, accumulate=True)
    assert torch.equal(dx, dx2) and dw2 is total
    assert bool(((dw2.double() - 1 - dw.double()).abs() <= HALF_F32 * (1 + dw.double().abs()) * 1.01).all())


def test_nothing_listed_and_no_rows():
    x, w, ids, t, dloss = _inputs(33, 300, 64, 4, 15, gaps=False)
    ids[:] = -1
    loss, lse, logp = _check_fwd(x, w, ids, t)
    dx, dw = jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss)
    assert bool((loss == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())
    dw = torch.ones((300, 64), device=DEV)
    jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss, dw=dw, accumulate=True)
    assert bool((dw == 1).all())
    e = torch.empty(0, device=DEV)
    loss, lse, logp = jq.linear_distill(x[:0], w, ids[:0], t[:0])
    assert loss.numel() == lse.numel() == logp.numel() == 0
    dx, dw = jq.linear_distill_bwd(x[:0], w, ids[:0], t[:0], e, torch.empty((0, 4), device=DEV), e)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_repeatable_captured_and_on_another_stream():
    x, w, ids, t, dloss = _inputs(200, 2000, 264, 30, 16)
    first = jq.linear_distill(x, w, ids, t)
    grads = jq.linear_distill_bwd(x, w, ids, t, first[1], first[2], dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = jq.linear_distill(x, w, ids, t, stream=side)
    other += jq.linear_distill_bwd(x, w, ids, t, other[1], other[2], dloss, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first + grads, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = jq.linear_distill(x, w, ids, t)
        out += jq.linear_distill_bwd(x, w, ids, t, out[1], out[2], dloss)
    for _ in range(3):
        for o in out:
            o.fill_(3)
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(first + grads, out))
    ids.copy_(ids.flip(0))  # other columns under the same graph
    t.copy_(t.flip(0))
    g.replay()
    again = jq.linear_distill(x, w, ids, t)
    assert all(torch.equal(p, q) for p, q in zip(again, out[:3]))


def test_workspaces_that_hold_anything():
    x, w, ids, t, dloss = _inputs(150, 900, 72, 11, 17)
    ws = torch.full((jq.jetq_linear_distill_workspace_bytes(150, 900, 72, 11),), 255, dtype=torch.uint8, device=DEV)
    a, b = jq.linear_distill(x, w, ids, t, workspace=ws), jq.linear_distill(x, w, ids, t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ws = torch.full((jq.jetq_linear_distill_bwd_workspace_bytes(150, 900, 72, 11),), 255, dtype=torch.uint8,
                    device=DEV)
    c = jq.linear_distill_bwd(x, w, ids, t, a[1], a[2], dloss, workspace=ws)
    d = jq.linear_distill_bwd(x, w, ids, t, a[1], a[2], dloss)
    assert all(torch.equal(p, q) for p, q in zip(c, d))
