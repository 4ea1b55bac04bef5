"""Softmax cross entropy of a linear head against its definition in binary64.

Bounds.  A logit's FP32 sum is within SUM * sum |x w| of the exact one (SUM =
1e-5, the bound every GEMM test of this library uses); the loss and lse follow
from two logits, plus FP32 rounding of values of lse's size.  d is rounded to
BF16 (2^-8 of its value), its sums again within SUM of the sum of magnitudes,
an exponential moves by the error of its exponent, and a BF16 result is
rounded once more (2^-8 of its value).
"""
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SUM = 1e-5
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24

SIZES = [(1, 1, 8), (1, 1000, 64), (2, 255, 8), (5, 257, 72), (127, 256, 64), (129, 511, 264), (256, 513, 128),
         (300, 1000, 520), (257, 4097, 1032), (513, 300, 2048)]


def _inputs(n, v, c, seed, pad=0, ignored=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, c + pad), generator=g, device=DEV).to(torch.bfloat16)[:, :c]
    w = (torch.randn((v, c + pad), generator=g, device=DEV) * 0.3).to(torch.bfloat16)[:, :c]
    target = torch.randint(0, v, (n,), generator=g, device=DEV)
    if ignored and n > 2:
        target[1::4] = -100
        target[2::8] = v  # outside the vocabulary on the other side
    dloss = torch.randn(n, generator=g, device=DEV)
    return x, w, target, dloss


def _define(x, w, target, scale):
    """(z, lse, loss, bound of a logit's error) in binary64."""
    z = scale * (x.double() @ w.double().T)
    lse = torch.logsumexp(z, 1)
    ok = (target >= 0) & (target < w.shape[0])
    zt = z.gather(1, target.clamp(0, w.shape[0] - 1)[:, None])[:, 0]
    loss = torch.where(ok, lse - zt, torch.zeros_like(lse))
    ez = scale * SUM * (x.double().abs() @ w.double().abs().T).amax(1)
    return z, lse, loss, ok, ez


def _d(z, lse, target, ok, dloss):
    p = torch.exp(z - lse[:, None])
    coef = torch.where(ok, dloss.double(), torch.zeros_like(lse))
    d = p * coef[:, None]
    row = torch.arange(z.shape[0], device=z.device)[ok]
    d[row, target[ok]] -= coef[ok]
    return p * coef.abs()[:, None], d


def _check_fwd(x, w, target, scale):
    loss, lse = jq.linear_ce(x, w, target, scale=scale)
    assert jq.jetq_check_device_error() == jq.OK
    _, rlse, rloss, ok, ez = _define(x, w, target, scale)
    tol = 2 * ez + 8 * HALF_F32 * (rlse.abs() + rloss.abs() + 1)
    assert bool(((lse.double() - rlse).abs() <= tol).all())
    assert bool(((loss.double() - rloss).abs() <= tol).all())
    assert bool((loss[~ok] == 0).all())
    return lse


def _bounds(x, w, target, scale, dloss, lse):
    """dx, dw in binary64 and what the kernels may be off by before their last rounding."""
    z, _, _, ok, ez = _define(x, w, target, scale)
    pg, d = _d(z, lse.double(), target, ok, dloss)
    moved = ez[:, None] + 8 * HALF_F32 * (1 + lse.double().abs()[:, None])  # of the exponent
    off = d.abs() * (HALF_BF16 + SUM) + pg * 2 * moved
    X, W = x.double(), w.double()
    return (scale * (d @ W), scale * (off @ W.abs())), (scale * (d.T @ X), scale * (off.T @ X.abs()))


def _check_bwd(x, w, target, scale, dloss, lse, dw_dtype, workspace=None):
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss, scale=scale, dw_dtype=dw_dtype, workspace=workspace)
    assert jq.jetq_check_device_error() == jq.OK
    assert dx.dtype == torch.bfloat16 and dw.dtype == dw_dtype
    (rx, tx), (rw, tw) = _bounds(x, w, target, scale, dloss, lse)
    last = HALF_BF16 if dw_dtype == torch.bfloat16 else HALF_F32
    assert bool(((dx.double() - rx).abs() <= tx * 1.01 + HALF_BF16 * rx.abs() + 1e-30).all())
    assert bool(((dw.double() - rw).abs() <= tw * 1.01 + last * rw.abs() + 1e-30).all())
    return dx, dw


@pytest.mark.parametrize("n,v,c", SIZES)
@pytest.mark.parametrize("scale", [1.0, 1.7])
def test_forward(n, v, c, scale):
    x, w, target, _ = _inputs(n, v, c, seed=n + v + c, pad=8 * (n % 3))
    _check_fwd(x, w, target, scale)


@pytest.mark.parametrize("n,v,c", SIZES)
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_backward(n, v, c, dw_dtype):
    x, w, target, dloss = _inputs(n, v, c, seed=n + v + c + 1, pad=8 * (n % 3))
    lse = _check_fwd(x, w, target, 0.8)
    _check_bwd(x, w, target, 0.8, dloss, lse, dw_dtype)


# several tiles a CTA or pair (152 SMs): single CTAs with three tiles of rows; pairs with one and with three folds of K;
# pairs in two raster groups, the second one ragged
BATCHES = [(333, 50257, 136), (1000, 30011, 72), (700, 20011, 1032), (1100, 6000, 520), (8500, 3000, 64)]


@pytest.mark.parametrize("n,v,c", BATCHES)
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_several_tiles_a_worker(n, v, c, dw_dtype):
    """The ring, the accumulators and a row's inputs are carried from tile to tile."""
    x, w, target, dloss = _inputs(n, v, c, seed=n + v + c)
    lse = _check_fwd(x, w, target, 1.1)
    _check_bwd(x, w, target, 1.1, dloss, lse, dw_dtype)


def test_backward_in_small_pieces():
    """The smallest workspace (256 vocabulary rows a piece) and one in between give the same gradient."""
    x, w, target, dloss = _inputs(200, 3000, 136, seed=5)
    _, lse = jq.linear_ce(x, w, target)
    small = jq.jetq_linear_ce_bwd_workspace_bytes(200, 3000, 136, True)
    large = jq.jetq_linear_ce_bwd_workspace_bytes(200, 3000, 136)
    assert small < large
    for size in (small, (small + large) // 2, large):
        _check_bwd(x, w, target, 1.0, dloss, lse, torch.float32, torch.empty(size, dtype=torch.uint8, device=DEV))


def test_rows_on_and_off_the_lines():
    """x in rows of whole 128-byte lines, off them, and in a view that starts off them: the same bits."""
    x, w, target, dloss = _inputs(200, 600, 136, seed=15)
    _check_fwd(x, w, target, 1.0)
    loss, lse = jq.linear_ce(x, w, target)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss)
    wide = torch.full((200, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    for at in (0, 8, 64):
        wide[:, at:at + 136] = x
        loss1, lse1 = jq.linear_ce(wide[:, at:at + 136], w, target)
        dx1, dw1 = jq.linear_ce_bwd(wide[:, at:at + 136], w, target, lse, dloss)
        assert torch.equal(loss, loss1) and torch.equal(lse, lse1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_rows_without_a_loss():
    x, w, target, dloss = _inputs(70, 300, 64, seed=6, ignored=False)
    target[:] = -100
    loss, lse = jq.linear_ce(x, w, target)
    assert bool((loss == 0).all()) and bool(torch.isfinite(lse).all())
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    target[3] = 7  # an infinite or NaN weight of an ignored row is not looked at
    bad = dloss.clone()
    bad[5], bad[6] = float("inf"), float("nan")
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, bad)
    dx1, dw1 = jq.linear_ce_bwd(x, w, target, lse, dloss)
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    assert bool((dx[[i for i in range(70) if i != 3]] == 0).all()) and bool((dx[3] != 0).any())


@pytest.mark.parametrize("n", [70, 200])
def test_rows_without_a_loss_may_hold_anything(n):
    """NaN and infinities in the hidden states, lse and dloss of ignored rows reach no gradient and no other row."""
    x, w, target, dloss = _inputs(n, 300, 72, seed=16)
    loss, lse = jq.linear_ce(x, w, target)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss)
    out = (target < 0) | (target >= 300)
    assert 0 < int(out.sum()) < n
    bad, blse, bloss = x.clone(), lse.clone(), dloss.clone()
    bad[out] = float("nan")
    bad[out.nonzero()[0, 0], 3:] = float("inf")
    blse[out], bloss[out] = float("-inf"), float("nan")
    loss1, lse1 = jq.linear_ce(bad, w, target)
    dx1, dw1 = jq.linear_ce_bwd(bad, w, target, blse, bloss)
    assert torch.equal(loss, loss1) and torch.equal(lse[~out], lse1[~out])
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1) and bool((dx1[out] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_weight_of_a_row_with_a_loss(bad):
    """It shows in its own row of dx; the other rows' gradients stay what they are."""
    x, w, target, dloss = _inputs(12, 300, 64, seed=13, ignored=False)
    _, lse = jq.linear_ce(x, w, target)
    dx, _ = jq.linear_ce_bwd(x, w, target, lse, dloss / dloss.abs().max())
    one = dloss / dloss.abs().max()
    one[4] = bad
    dx1, _ = jq.linear_ce_bwd(x, w, target, lse, one)
    keep = [i for i in range(12) if i != 4]
    assert not bool(torch.isfinite(dx1[4].float()).any())
    assert torch.equal(dx1[keep], dx[keep])
    target[:] = -1
    target[4] = 0  # the only loss
    dx1, _ = jq.linear_ce_bwd(x, w, target, lse, one)
    assert not bool(torch.isfinite(dx1[4].float()).any()) and bool((dx1[keep] == 0).all())


def test_confident_token_keeps_its_relative_precision():
    """One logit far above the others: loss = sum of the others over it, far below FP32's step at lse."""
    v, c = 512, 8
    w = torch.zeros((v, c), dtype=torch.bfloat16, device=DEV)
    w[5, 0] = 1.0
    x = torch.zeros((1, c), dtype=torch.bfloat16, device=DEV)
    x[0, 0] = 30.0
    loss, lse = jq.linear_ce(x, w, torch.tensor([5], device=DEV))
    want = torch.log1p((v - 1) * torch.exp(torch.tensor(-30.0, dtype=torch.float64))).item()
    assert abs(loss.item() - want) <= 16 * 30 * HALF_F32 * want
    assert abs(lse.item() - 30.0) <= 8 * 30 * HALF_F32


def test_large_logits_and_nan():
    x, w, target, _ = _inputs(64, 700, 64, seed=8, ignored=False)
    _check_fwd((x.float() * 64).to(torch.bfloat16), w, target, 4.0)  # exponents far outside FP32's range
    x[9, 3] = float("nan")
    loss, lse = jq.linear_ce(x, w, target)
    bad = torch.isnan(loss)
    assert bool(bad[9]) and int(bad.sum()) == 1 and bool(torch.isnan(lse[9]))


@pytest.mark.parametrize("n", [60, 300])
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_confident_tokens(n, dw_dtype):
    """Tokens whose loss is 1e-3 to 1e-5, at a hidden size where the logit's sum is long: d at the target is -(1 - p),
    so its exponent has to be good to a small part of the loss, not of the logit.  The target's exponent counts 2^-40
    of the logit's magnitudes (a compensated sum and its one rounding, at most 4 * 2^-24 of the exponent); the other
    columns' are bounded as everywhere."""
    v, c = 2000, 4096
    g = torch.Generator(device=DEV).manual_seed(n)
    w = (torch.randn((v, c), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    target = torch.randperm(v, generator=g, device=DEV)[:n]  # a row of dw has one token's target
    row = w[target].float()
    lean = torch.linspace(15.3, 20.0, n, device=DEV)[:, None]
    x = (torch.randn((n, c), generator=g, device=DEV) + lean * row / row.square().sum(1, keepdim=True)).to(torch.bfloat16)
    dloss = 0.5 + torch.rand(n, generator=g, device=DEV)
    loss, lse = jq.linear_ce(x, w, target)
    assert float(loss.max()) > 3e-4 and float(loss.min()) < 3e-5
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss, dw_dtype=dw_dtype)
    assert jq.jetq_check_device_error() == jq.OK
    X, W, rows = x.double(), w.double(), torch.arange(n, device=DEV)
    e = X @ W.T - lse.double()[:, None]
    coef = dloss.double()[:, None]
    d = torch.exp(e) * coef
    off = d * (HALF_BF16 + SUM + 2 * (SUM * (X.abs() @ W.abs().T) + 8 * HALF_F32 * (1 + lse.double().abs()[:, None])))
    et = e[rows, target]
    d[rows, target] = torch.expm1(et) * coef[:, 0]
    far = 2.0 ** -40 * (X.abs() * W[target].abs()).sum(1) + 4 * HALF_F32 * et.abs()
    off[rows, target] = d[rows, target].abs() * (HALF_BF16 + SUM) + coef[:, 0] * 2 * far
    last = HALF_BF16 if dw_dtype == torch.bfloat16 else HALF_F32
    rx, rw = d @ W, d.T @ X
    assert bool(((dx.double() - rx).abs() <= off @ W.abs() * 1.01 + HALF_BF16 * rx.abs() + 1e-30).all())
    assert bool(((dw.double() - rw).abs() <= off.T @ X.abs() * 1.01 + last * rw.abs() + 1e-30).all())
    # a whole row: each of its two roundings moves it by at most 2^-8 of its terms, which add up to at most twice d
    assert float(((dx.double() - rx).norm(dim=1) / rx.norm(dim=1)).max()) <= 4 * HALF_BF16


@pytest.mark.parametrize("n", [1, 60, 300])
@pytest.mark.parametrize("scale", [1.0, 1.3])
def test_lse_of_confident_tokens(n, scale):
    """lse of a token that its target leads is the target's logit plus the loss: FP32's step at lse (2^-24 of it) and
    the loss's own error, a small part of a small loss.  The backward pass subtracts it from the same logit, so a larger
    error of lse would be one of 1 - p."""
    v, c = 2000, 4096
    g = torch.Generator(device=DEV).manual_seed(n + 7)
    w = (torch.randn((v, c), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    target = torch.randperm(v, generator=g, device=DEV)[:n]
    row = w[target].float()
    lean = torch.linspace(15.3, 20.0, n, device=DEV)[:, None]
    x = (torch.randn((n, c), generator=g, device=DEV) + lean * row / row.square().sum(1, keepdim=True)).to(torch.bfloat16)
    loss, lse = jq.linear_ce(x, w, target, scale=scale)
    assert jq.jetq_check_device_error() == jq.OK
    _, rlse, rloss, _, ez = _define(x, w, target, torch.tensor(scale).item())  # the entry point takes a float
    part = rloss * (4 * ez + 16 * HALF_F32 * (1 + rlse.abs()))  # both exponents' errors, relative to the loss
    assert bool(((loss.double() - rloss).abs() <= part).all())
    assert bool(((lse.double() - rlse).abs() <= HALF_F32 * rlse.abs() + part).all())


@pytest.mark.parametrize("n,v", [(200, 129), (4, 1000), (4, 129), (300, 4097)])
def test_nan_in_a_partial_slice(n, v):
    """NaN in the vocabulary's last, partly filled columns reaches every row; NaN in a hidden state reaches its row."""
    x, w, target, _ = _inputs(n, v, 64, seed=17, ignored=False)
    target[0] = -100
    bad = w.clone()
    bad[v - 1, 5] = float("nan")
    loss, lse = jq.linear_ce(x, bad, target)
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(loss[1:]).all()) and loss[0].item() == 0
    x[:2, 7] = float("nan")
    loss, lse = jq.linear_ce(x, w, target)
    assert bool(torch.isnan(lse[:2]).all()) and bool(torch.isfinite(lse[2:]).all())
    assert loss[0].item() == 0 and bool(torch.isnan(loss[1])) and bool(torch.isfinite(loss[2:]).all())


def test_accumulate_into_dw():
    x, w, target, dloss = _inputs(150, 400, 72, seed=9)
    _, lse = jq.linear_ce(x, w, target)
    _, dw = jq.linear_ce_bwd(x, w, target, lse, dloss)
    base = torch.randn((400, 76), device=DEV)
    acc = base.clone()[:, :72]
    jq.linear_ce_bwd(x, w, target, lse, dloss, dw=acc, accumulate=True)
    want = base[:, :72].double() + dw.double()
    assert bool(((acc.double() - want).abs() <= HALF_F32 * want.abs() + 1e-30).all())


def test_gradient_against_differences():
    """The kernels' gradient along a direction is the loss's central difference in binary64."""
    x, w, target, dloss = _inputs(40, 600, 64, seed=10)
    scale = 0.9
    _, lse = jq.linear_ce(x, w, target, scale=scale)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss, scale=scale)
    g = torch.Generator(device=DEV).manual_seed(1)
    ux = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
    uw = torch.randn(w.shape, generator=g, device=DEV, dtype=torch.float64)
    ok = (target >= 0) & (target < 600)

    def total(h):
        z = scale * ((x.double() + h * ux) @ (w.double() + h * uw).T)
        loss = torch.logsumexp(z, 1) - z.gather(1, target.clamp(0, 599)[:, None])[:, 0]
        return (loss * dloss.double())[ok].sum()

    h = 1e-5
    slope = (total(h) - total(-h)) / (2 * h)
    (rx, tx), (rw, tw) = _bounds(x, w, target, scale, dloss, lse)
    got = (dx.double() * ux).sum() + (dw.double() * uw).sum()
    tol = ((tx * 1.01 + HALF_BF16 * rx.abs()) * ux.abs()).sum() + ((tw * 1.01 + HALF_F32 * rw.abs()) * uw.abs()).sum()
    third = 1e-6 * (1 + slope.abs())  # the difference's own error
    assert abs(got - slope) <= tol + third


def test_repeatable_streams_and_graph():
    x, w, target, dloss = _inputs(333, 2000, 264, seed=11)
    loss, lse = jq.linear_ce(x, w, target)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss1, lse1 = jq.linear_ce(x, w, target)
        dx1, dw1 = jq.linear_ce_bwd(x, w, target, lse1, dloss)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, loss1) and torch.equal(lse, lse1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss2, lse2 = jq.linear_ce(x, w, target)
        dx2, dw2 = jq.linear_ce_bwd(x, w, target, lse2, dloss)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_no_tokens():
    w = torch.randn((300, 64), device=DEV).to(torch.bfloat16)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    target = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = jq.linear_ce(x, w, target)
    assert loss.shape == lse.shape == (0,)
    dw = torch.ones((300, 64), device=DEV)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, loss, dw=dw)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_offsets_past_32_bits():
    """A head of 2.5e9 weights: the last rows are where they belong, in the losses and in both gradients."""
    n, v, c = 24, 600_011, 4096
    g = torch.Generator(device=DEV).manual_seed(14)
    x = torch.randn((n, c), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.empty((v, c), dtype=torch.bfloat16, device=DEV)
    for a in range(0, v, 50_000):
        b = min(v, a + 50_000)
        w[a:b] = torch.randn((b - a, c), generator=g, device=DEV) * 0.05
    target = torch.randint(0, v, (n,), generator=g, device=DEV)
    target[:4] = torch.tensor([v - 1, v - 2, 0, 2 ** 31 // c + 1], device=DEV)
    dloss = torch.randn(n, generator=g, device=DEV)
    loss, lse = jq.linear_ce(x, w, target)
    dx, dw = jq.linear_ce_bwd(x, w, target, lse, dloss, dw_dtype=torch.bfloat16)
    assert jq.jetq_check_device_error() == jq.OK
    X = x.double()
    rlse = torch.full((n,), -float("inf"), dtype=torch.float64, device=DEV)
    size = torch.zeros(n, dtype=torch.float64, device=DEV)
    rx, tx = torch.zeros_like(X), torch.zeros_like(X)
    coef = dloss.double()
    rows = torch.arange(n, device=DEV)
    pieces = [(a, min(v, a + 50_000)) for a in range(0, v, 50_000)]
    for a, b in pieces:
        W = w[a:b].double()
        rlse = torch.logaddexp(rlse, torch.logsumexp(X @ W.T, 1))
        size = torch.maximum(size, (X.abs() @ W.abs().T).amax(1))
    zt = (X * w[target].double()).sum(1)
    tol = 2 * SUM * size + 8 * HALF_F32 * (rlse.abs() + (rlse - zt).abs() + 1)
    assert bool(((lse.double() - rlse).abs() <= tol).all())
    assert bool(((loss.double() - (rlse - zt)).abs() <= tol).all())
    moved = (SUM * size + 8 * HALF_F32 * (1 + lse.double().abs()))[:, None]
    for a, b in pieces:
        W = w[a:b].double()
        p = torch.exp(X @ W.T - lse.double()[:, None])
        d = p * coef[:, None]
        here = rows[(target >= a) & (target < b)]
        d[here, target[here] - a] -= coef[here]
        off = d.abs() * (HALF_BF16 + SUM) + p * coef.abs()[:, None] * 2 * moved
        rx += d @ W
        tx += off @ W.abs()
        rw, tw = d.T @ X, off.T @ X.abs()
        assert bool(((dw[a:b].double() - rw).abs() <= tw * 1.01 + HALF_BF16 * rw.abs() + 1e-30).all())
    assert bool(((dx.double() - rx).abs() <= tx * 1.01 + HALF_BF16 * rx.abs() + 1e-30).all())
