"""The distillation's dx takes the listed columns, which hold nearly all of a confident token's d, with more than the
BF16 of the tensor cores' operand.

Bound.  A listed entry of d enters dx as its BF16 value and the FP32 rest of it, whose sum is off by 2^-24 of the entry
and the errors of its two terms (2 ulp of an exponential each: 2^-20 of their magnitudes); an unlisted one, and every
one in dw, is rounded to BF16, 2^-8 of it.  Sums are within SUM of the sum of magnitudes, exponents within SUM of
theirs, and the result is rounded once.
"""
import math

import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SUM = 1e-5
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24


def _case(n, v, c, k, seed, columns=None):
    """A student and a teacher of its k best columns (or of the columns given), which differ by a factor of about 2."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, c), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((v, c), generator=g, device=DEV) * (2.0 / math.sqrt(c))).to(torch.bfloat16)
    z = x.double() @ w.double().T
    ids = z.topk(k, dim=1).indices if columns is None else columns(n, v, k, g)
    t = z.gather(1, ids).float() + 0.7 * torch.randn((n, k), generator=g, device=DEV)
    if n > 4:  # rows of fewer entries, and without any
        drop = torch.rand((n, k), generator=g, device=DEV) < 0.15
        drop[::7] = True
        ids = torch.where(drop, torch.full_like(ids, -1), ids)
    lse = torch.logsumexp(z, 1)
    logp = torch.where(ids >= 0, z.gather(1, ids.clamp(min=0)) - lse[:, None], torch.zeros_like(t, dtype=torch.float64))
    return x, w, ids, t, lse.float(), logp.float(), torch.rand(n, generator=g, device=DEV) / n


def _define(x, w, ids, t, lse, logp, dloss, scale=1.0):
    """d in binary64 (from the same lse and logp), which of it is listed, and how far each entry may be off."""
    n, v = x.shape[0], w.shape[0]
    on = (ids >= 0) & (ids < v)
    tt = torch.where(on, t.double(), torch.full_like(t.double(), -math.inf))
    q = torch.where(on.any(1, keepdim=True), (tt - torch.logsumexp(tt, 1, keepdim=True)).exp(), torch.zeros_like(tt))
    z = scale * (x.double() @ w.double().T)
    p = (z - lse.double()[:, None]).exp() * on.any(1, keepdim=True)
    ez = scale * SUM * (x.double().abs() @ w.double().abs().T).amax(1, keepdim=True)
    ez = ez + 2.0 ** -22 * (1 + lse.double().abs()[:, None])
    spread = torch.zeros_like(p).scatter_add_(1, ids.clamp(0, v - 1), torch.where(on, q, torch.zeros_like(q)))
    listed = torch.zeros_like(p).scatter_add_(1, ids.clamp(0, v - 1), on.double()) > 0
    at = torch.where(on, logp.double().exp(), torch.zeros_like(q))
    exact = torch.zeros_like(p).scatter_reduce_(1, ids.clamp(0, v - 1), at, "amax")
    p = torch.where(listed, exact, p)
    d = (p - spread) * dloss.double()[:, None]
    size = (p + spread) * dloss.double().abs()[:, None]
    own = torch.where(listed, 2.0 ** -20 * size, size * 2 * ez) + SUM * d.abs()
    return d, own + torch.where(listed, torch.zeros_like(d), d.abs() * HALF_BF16), own + d.abs() * HALF_BF16


def _check(x, w, ids, t, lse, logp, dloss, scale=1.0, dw_dtype=torch.float32, **kw):
    dx, dw = jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss, scale=scale, dw_dtype=dw_dtype, **kw)
    assert jq.jetq_check_device_error() == jq.OK
    d, off, off16 = _define(x, w, ids, t, lse, logp, dloss, scale)
    X, W = x.double(), w.double()
    for got, want, tol, half in ((dx, scale * (d @ W), scale * (off @ W.abs()), HALF_BF16),
                                 (dw, scale * (d.T @ X), scale * (off16.T @ X.abs()),
                                  HALF_BF16 if dw.dtype is torch.bfloat16 else 2 * HALF_F32)):
        assert bool(((got.double() - want).abs() <= 1.01 * tol + half * want.abs() + 1e-30).all())
    return dx, dw


SIZES = [(1, 300, 64, 5), (3, 64, 8, 64), (40, 1000, 136, 20), (130, 700, 64, 100), (257, 4097, 264, 32),
         (513, 257, 72, 256), (1000, 3001, 1032, 16), (2049, 1300, 128, 40)]


@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,c,k", SIZES)
def test_listed_entries_keep_their_rest(n, v, c, k, dw_dtype):
    """The whole vocabulary listed and few of it, rows and columns off the tiles, single CTAs and pairs."""
    a = _case(n, v, c, k, n + v)
    _check(*a, scale=1.0 if n % 2 else 0.8, dw_dtype=dw_dtype)


def test_every_column_listed_leaves_the_rounding_of_the_result():
    """dx off its definition by no more than the definition rounded to BF16 is, and 1e-4 of it."""
    a = _case(200, 96, 128, 96, 5)
    ids = torch.arange(96, device=DEV).expand(200, 96).contiguous()
    z = a[0].double() @ a[1].double().T
    logp = (z - torch.logsumexp(z, 1, keepdim=True)).float()
    want = _define(a[0], a[1], ids, a[3], a[4], logp, a[6])[0] @ a[1].double()
    dx, _ = jq.linear_distill_bwd(a[0], a[1], ids, a[3], a[4], logp, a[6])
    rounded = (want.to(torch.bfloat16).double() - want).norm()
    assert float((dx.double() - want).norm()) <= float(rounded + 1e-4 * want.norm())


@pytest.mark.parametrize("columns", ["the same for all", "64 columns", "scattered and common"])
def test_common_columns(columns):
    """Columns that every token lists."""
    def pick(n, v, k, g):
        if columns == "the same for all":
            return torch.randperm(v, generator=g, device=DEV)[:k].expand(n, k).contiguous()
        if columns == "64 columns":
            return (128 + torch.rand((n, 64), generator=g, device=DEV).argsort(1)[:, :k]).contiguous()
        rest = 5 + torch.rand((n, v - 5), generator=g, device=DEV).argsort(1)[:, :k - 5]
        return torch.cat((torch.arange(5, device=DEV).expand(n, 5), rest), 1)

    a = _case(900, 1000, 96, 30, 6, pick)
    for dw_dtype in (torch.float32, torch.bfloat16):
        _check(*a, dw_dtype=dw_dtype)


def test_a_column_listed_twice_counts_once():
    x, w, ids, t, lse, logp, dloss = _case(60, 500, 64, 9, 7)
    ids[:, 4], logp[:, 4] = ids[:, 1], logp[:, 1]
    ids[::3, 8], logp[::3, 8] = ids[::3, 1], logp[::3, 1]
    _check(x, w, ids, t, lse, logp, dloss)


def test_pieces_of_the_vocabulary_strides_and_accumulation():
    n, v, c, k = 300, 2500, 136, 24
    x, w, ids, t, lse, logp, dloss = _case(n, v, c, k, 8)
    dx, dw = _check(x, w, ids, t, lse, logp, dloss)
    small = torch.full((jq.jetq_linear_distill_bwd_workspace_bytes(n, v, c, k, smallest=True),), 255, dtype=torch.uint8,
                       device=DEV)
    _check(x, w, ids, t, lse, logp, dloss, workspace=small)
    wide = torch.full((n, 200), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + c] = x
    wide_w = torch.full((v, 152), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_w[:, :c] = w
    wide_i = torch.full((n, 40), 3, dtype=torch.int64, device=DEV)
    wide_i[:, :k] = ids
    dx2, dw2 = jq.linear_distill_bwd(wide[:, 8:8 + c], wide_w[:, :c], wide_i[:, :k], t, lse, logp, dloss)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    start = torch.randn((v, c), device=DEV)
    into = start.clone()
    jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss, dw=into, accumulate=True)
    assert bool(((into - start).double() - dw.double()).abs().max() <= 2 ** -22 * (start.abs() + dw.abs()).max())


def test_two_tokens_of_a_large_vocabulary_with_the_smallest_workspace():
    n, v, c, k = 2, 140001, 64, 16
    a = _case(n, v, c, k, 9)
    dx, dw = _check(*a)
    small = torch.empty(jq.jetq_linear_distill_bwd_workspace_bytes(n, v, c, k, smallest=True), dtype=torch.uint8,
                        device=DEV)
    _check(*a, workspace=small)


def test_a_number_missing_stays_in_its_row_and_columns():
    x, w, ids, t, lse, logp, dloss = _case(90, 600, 64, 8, 10)
    ids[5] = torch.arange(8, device=DEV) * 70
    dx, dw = jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss)
    logp[5, 2] = float("nan")
    dx2, dw2 = jq.linear_distill_bwd(x, w, ids, t, lse, logp, dloss)
    rows, cols = torch.arange(90, device=DEV) != 5, torch.arange(600, device=DEV) != 140
    assert torch.equal(dx[rows], dx2[rows]) and torch.equal(dw[cols], dw2[cols])
    assert bool(dx2[5].isnan().all()) and bool(dw2[140].isnan().all())


def test_repeatable_captured_and_on_another_stream():
    a = _case(700, 2000, 264, 40, 11)
    first = jq.linear_distill_bwd(*a)
    for _ in range(10):
        assert all(torch.equal(p, q) for p, q in zip(first, jq.linear_distill_bwd(*a)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = jq.linear_distill_bwd(*a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = jq.linear_distill_bwd(*a)
    for _ in range(5):
        for o in out:
            o.fill_(3)
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(first, out))
    a[6].mul_(0.3)  # another loss's gradient under the same graph
    g.replay()
    assert all(torch.equal(p, q) for p, q in zip(jq.linear_distill_bwd(*a), out))
