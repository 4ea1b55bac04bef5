"""Layer norm and RMS norm, forward and backward, against binary64.

Bounds, with u = 2^-24 (FP32): sums run over at most 100 additions in
sequence, a row's mean is off by that many u of its mean magnitude, and what
follows from it by the same factor of the magnitudes that enter; the last
rounding adds half a step of the output's type (2^-8 of a BF16 value, u of an
FP32 one).  dw and db add one u of the summed magnitudes for every 300 rows (a
group's rows are added in sequence).
"""
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
LAST = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
KINDS = [jq.NORM_LAYER, jq.NORM_RMS]
DTYPES = [torch.bfloat16, torch.float32]
# every group width (1 to 16 warps a row), their edges, odd widths, wide rows, one row and many
SIZES = [(1, 1), (3, 7), (1, 4096), (5, 512), (257, 513), (64, 1024), (33, 1111), (301, 2048), (40, 4095), (17, 8192),
         (9, 8193), (3, 20001), (3000, 64), (2500, 136)]


def _rows(n, c, dtype, g, pad=0, mu=0.3):
    step = 8 if dtype == torch.bfloat16 else 4
    ld = -(-c // step) * step + pad
    t = torch.full((n, ld), float("nan"), dtype=dtype, device=DEV)  # the padding of a row is never used
    t[:, :c] = (torch.randn((n, c), generator=g, device=DEV) * 1.5 + mu).to(dtype)
    return t[:, :c]


def _inputs(n, c, dtype, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, dy = _rows(n, c, dtype, g, pad), _rows(n, c, dtype, g, 2 * pad, 0.0)
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(dtype)
    b = torch.randn(c, generator=g, device=DEV).to(dtype)
    return x, dy, w, b


def _check_fwd(x, w, b, eps, kind):
    y, mean, rstd = jq.norm_fwd(x, w, b, eps=eps, kind=kind)
    assert jq.jetq_check_device_error() == jq.OK
    X = x.double()
    m = X.mean(1, keepdim=True) if kind == jq.NORM_LAYER else torch.zeros_like(X[:, :1])
    r = 1 / ((X - m).square().mean(1, keepdim=True) + eps).sqrt()
    W = w.double() if w is not None else 1.0
    ref = (X - m) * r * W + (b.double() if b is not None else 0.0)
    size = X.abs().mean(1, keepdim=True)
    tol = LAST[x.dtype] * ref.abs() + 100 * U * ((r * (size + (X - m).abs()) * W).abs() + 2 * ref.abs())
    if b is not None:
        tol = tol + 100 * U * b.double().abs()
    assert y.dtype == x.dtype and bool(((y.double() - ref).abs() <= tol).all())
    assert bool(((rstd.double() - r[:, 0]).abs() <= 100 * U * r[:, 0]).all())
    if kind == jq.NORM_LAYER:
        assert bool(((mean.double() - m[:, 0]).abs() <= 100 * U * size[:, 0]).all())
    else:
        assert mean is None
    return mean, rstd


def _define_bwd(dy, x, w, mean, rstd, kind):
    X, DY, r = x.double(), dy.double(), rstd.double()[:, None]
    m = mean.double()[:, None] if kind == jq.NORM_LAYER else torch.zeros_like(r)
    h, t = (X - m) * r, DY * (w.double() if w is not None else 1.0)
    dx = r * (t - h * (t * h).mean(1, keepdim=True) - (t.mean(1, keepdim=True) if kind == jq.NORM_LAYER else 0.0))
    size = h.abs() + (X.abs() + m.abs()) * r
    off = 100 * U * r * (t.abs() + t.abs().mean(1, keepdim=True) + size * (t.abs() * size).mean(1, keepdim=True))
    steps = (100 + x.shape[0] / 300) * U
    return (dx, off), ((DY * h).sum(0), steps * (DY.abs() * size).sum(0)), (DY.sum(0), steps * DY.abs().sum(0))


def _check_bwd(dy, x, w, mean, rstd, kind, bias):
    dx, dw, db = jq.norm_bwd(dy, x, w, mean, rstd, kind=kind, bias=bias)
    assert jq.jetq_check_device_error() == jq.OK
    (rx, tx), (rw, tw), (rb, tb) = _define_bwd(dy, x, w, mean, rstd, kind)
    assert dx.dtype == x.dtype and bool(((dx.double() - rx).abs() <= tx + LAST[x.dtype] * rx.abs()).all())
    assert dw.dtype == torch.float32 and bool(((dw.double() - rw).abs() <= tw).all())
    if bias:
        assert bool(((db.double() - rb).abs() <= tb).all())
    else:
        assert db is None
    return dx, dw, db


@pytest.mark.parametrize("n,c", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward_and_backward(n, c, kind, dtype):
    x, dy, w, b = _inputs(n, c, dtype, seed=n + c, pad=8 * (c % 2))
    layer = kind == jq.NORM_LAYER
    mean, rstd = _check_fwd(x, w, b if layer else None, 1e-5, kind)
    _check_bwd(dy, x, w, mean, rstd, kind, layer)


@pytest.mark.parametrize("kind", KINDS)
def test_without_parameters(kind):
    x, dy, _, _ = _inputs(100, 384, torch.bfloat16, seed=3)
    mean, rstd = _check_fwd(x, None, None, 1e-6, kind)
    _check_bwd(dy, x, None, mean, rstd, kind, False)


@pytest.mark.parametrize("c", [8, 9, 63, 64, 65, 127, 128, 129, 200, 256, 257, 383, 511, 512])
@pytest.mark.parametrize("dtype", DTYPES)
def test_short_rows(c, dtype):
    """Rows of up to 512 columns: every number of lanes and vectors a row, whole and partial ones."""
    for n, kind in ((1, jq.NORM_LAYER), (37, jq.NORM_RMS), (1003, jq.NORM_LAYER)):
        x, dy, w, b = _inputs(n, c, dtype, seed=n + c)
        layer = kind == jq.NORM_LAYER
        mean, rstd = _check_fwd(x, w, b if layer else None, 1e-5, kind)
        _check_bwd(dy, x, w, mean, rstd, kind, layer)


def test_many_rows():
    x, dy, w, b = _inputs(30011, 264, torch.bfloat16, seed=4)
    mean, rstd = _check_fwd(x, w, b, 1e-5, jq.NORM_LAYER)
    _check_bwd(dy, x, w, mean, rstd, jq.NORM_LAYER, True)


@pytest.mark.parametrize("n,c", [(4000, 1111), (6001, 2048), (2500, 4096), (1501, 8192)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_more_rows_than_the_rings_hold(n, c, kind, dtype):
    """Every group of warps takes many rows: the rings' stages are filled again in both passes."""
    x, dy, w, b = _inputs(n, c, dtype, seed=n + c)
    layer = kind == jq.NORM_LAYER
    mean, rstd = _check_fwd(x, w, b if layer else None, 1e-5, kind)
    _check_bwd(dy, x, w, mean, rstd, kind, layer)


@pytest.mark.parametrize("c", [128, 1111, 2048, 9000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_parameters_off_the_vectors(c, dtype):
    """w and b need the alignment of an element only."""
    x, dy, w, b = _inputs(30, c, dtype, seed=c)
    both = torch.empty(2 * c + 3, dtype=dtype, device=DEV)
    w1, b1 = both[1:c + 1].copy_(w), both[c + 2:2 * c + 2].copy_(b)
    assert w1.data_ptr() % 16 and b1.data_ptr() % 16
    y, mean, rstd = jq.norm_fwd(x, w1, b1)
    y2, mean2, rstd2 = jq.norm_fwd(x, w, b)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    for p, q in zip(jq.norm_bwd(dy, x, w1, mean, rstd, bias=True), jq.norm_bwd(dy, x, w, mean, rstd, bias=True)):
        assert torch.equal(p, q)
    _check_fwd(x, w1, b1, 1e-5, jq.NORM_LAYER)


@pytest.mark.parametrize("dtype", DTYPES)
def test_mean_far_above_the_spread(dtype):
    """The variance is summed around the mean: an offset of 64 spreads costs no precision beyond its own rounding."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = _rows(50, 1000, dtype, g, mu=100.0)
    _check_fwd(x, None, None, 1e-5, jq.NORM_LAYER)


def test_constant_and_special_rows():
    x = torch.zeros((4, 256), device=DEV)
    x[1] = 3.0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    y, mean, rstd = jq.norm_fwd(x, None, None, eps=1e-5)
    assert bool((y[:2] == 0).all()) and mean[1].item() == 3.0
    assert abs(rstd[0].item() - 1e-5 ** -0.5) <= 8 * U * 1e-5 ** -0.5
    assert bool(torch.isnan(y[2:]).any(1).all())  # and no other row is touched
    y, _, rstd = jq.norm_fwd(x[:1], None, None, eps=0.0, kind=jq.NORM_RMS)
    assert rstd[0].item() == float("inf")


def test_in_place():
    x, dy, w, b = _inputs(77, 520, torch.bfloat16, seed=6)
    y, mean, rstd = jq.norm_fwd(x, w, b)
    z = x.clone()
    jq.jetq_norm_fwd(jq.NORM_LAYER, z, w, b, 1e-5, z, torch.empty_like(mean), torch.empty_like(rstd))
    assert torch.equal(y, z)
    dx, dw, db = jq.norm_bwd(dy, x, w, mean, rstd, bias=True)
    d = dy.clone()
    ws = torch.empty(jq.jetq_norm_bwd_workspace_bytes(jq.OUT_BF16, 77, 520), dtype=torch.uint8, device=DEV)
    jq.jetq_norm_bwd(jq.NORM_LAYER, d, x, w, mean, rstd, d, torch.empty_like(dw), torch.empty_like(db), ws)
    assert torch.equal(dx, d)


def _same_layout(t):
    """A copy in rows of the same stride (Tensor.clone would pack them)."""
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
    return out.copy_(t)


@pytest.mark.parametrize("c", [64, 300, 511, 520, 1111, 8192, 8193, 12000, 20001])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_every_alias_gives_the_same_bits(c, kind, dtype):
    """y = x, dx = dy and dx = x: outputs, statistics and parameter gradients as of separate tensors."""
    n, layer = 41, kind == jq.NORM_LAYER
    x, dy, w, b = _inputs(n, c, dtype, seed=c)
    b = b if layer else None
    y, mean, rstd = jq.norm_fwd(x, w, b, kind=kind)
    z, mean1, rstd1 = _same_layout(x), torch.empty_like(rstd) if layer else None, torch.empty_like(rstd)
    jq.jetq_norm_fwd(kind, z, w, b, 1e-5, z, mean1, rstd1)
    assert torch.equal(y, z) and torch.equal(rstd, rstd1) and (not layer or torch.equal(mean, mean1))
    dx, dw, db = jq.norm_bwd(dy, x, w, mean, rstd, kind=kind, bias=layer)
    ws = torch.empty(jq.jetq_norm_bwd_workspace_bytes(jq._out_dtype(x), n, c), dtype=torch.uint8, device=DEV)
    for alias in ("dy", "x"):
        t = dict(dy=_same_layout(dy), x=_same_layout(x))
        dw1, db1 = torch.empty_like(dw), torch.empty_like(db) if layer else None
        jq.jetq_norm_bwd(kind, t["dy"], t["x"], w, mean, rstd, t[alias], dw1, db1, ws)
        assert torch.equal(dx, t[alias]), alias
        assert torch.equal(dw, dw1) and (not layer or torch.equal(db, db1)), alias


@pytest.mark.parametrize("n,c", [(50, 1111), (1, 1111), (7, 63), (1, 1), (3, 8195)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_any_layout(n, c, dtype):
    """Dense rows of odd width, as autograd hands them back, and a view off the 16 bytes: the bits of padded rows."""
    x, dy, w, b = _inputs(n, c, dtype, seed=n * c)
    want = jq.norm_fwd(x, w, b)
    want += jq.norm_bwd(dy, x, w, want[1], want[2], bias=True)
    wide = torch.empty((2, n, c + 3), dtype=dtype, device=DEV)
    off = [t[:, 1:c + 1].copy_(v) for t, v in zip(wide, (x, dy))]
    for xs, dys in ((x.contiguous(), dy.contiguous()), off):
        got = jq.norm_fwd(xs, w, b)
        got += jq.norm_bwd(dys, xs, w, got[1], got[2], bias=True)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        assert torch.equal(xs, x) and torch.equal(dys, dy)


def test_gradient_against_differences():
    x, dy, w, b = _inputs(20, 96, torch.float32, seed=7)
    _, mean, rstd = jq.norm_fwd(x, w, b)
    dx, dw, db = jq.norm_bwd(dy, x, w, mean, rstd, bias=True)
    g = torch.Generator(device=DEV).manual_seed(8)
    ux = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
    uw, ub = (torch.randn(96, generator=g, device=DEV, dtype=torch.float64) for _ in range(2))

    def total(s):
        X = x.double() + s * ux
        h = X - X.mean(1, keepdim=True)
        h = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt()
        return ((h * (w.double() + s * uw) + b.double() + s * ub) * dy.double()).sum()

    s = 1e-5
    slope = (total(s) - total(-s)) / (2 * s)
    got = (dx.double() * ux).sum() + (dw.double() * uw).sum() + (db.double() * ub).sum()
    (rx, tx), (rw, tw), (rb, tb) = _define_bwd(dy, x, w, mean, rstd, jq.NORM_LAYER)
    tol = ((tx + U * rx.abs()) * ux.abs()).sum() + (tw * uw.abs()).sum() + (tb * ub.abs()).sum()
    # the forward's own rounding of mean and rstd, and the difference's error
    assert abs(got - slope) <= tol + 200 * U * (dx.double() * ux).abs().sum() + 1e-6 * (1 + slope.abs())


def test_backward_of_the_quantizers_rmsnorm():
    """rstd of the fused RMSNorm quantizer feeds the backward pass."""
    x, dy, w, _ = _inputs(130, 256, torch.bfloat16, seed=9)
    x, dy = x.contiguous(), dy.contiguous()
    q = jq.quant_act_rmsnorm(x, w, eps=1e-6)
    _check_bwd(dy, x, w, None, q["rstd"], jq.NORM_RMS, False)


def test_repeatable_streams_and_graph():
    x, dy, w, b = _inputs(999, 1032, torch.bfloat16, seed=10)
    y, mean, rstd = jq.norm_fwd(x, w, b)
    grads = jq.norm_bwd(dy, x, w, mean, rstd, bias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, mean1, rstd1 = jq.norm_fwd(x, w, b)
        grads1 = jq.norm_bwd(dy, x, w, mean1, rstd1, bias=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, mean2, rstd2 = jq.norm_fwd(x, w, b)
        grads2 = jq.norm_bwd(dy, x, w, mean2, rstd2, bias=True)
    graph.replay()
    torch.cuda.synchronize()
    for other in ((y1, mean1, rstd1) + grads1, (y2, mean2, rstd2) + grads2):
        assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd) + grads, other))


def test_no_rows():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    y, mean, rstd = jq.norm_fwd(x, None, None)
    assert y.shape == (0, 256) and mean.shape == rstd.shape == (0,)
    dx, dw, db = jq.norm_bwd(x, x, None, mean, rstd, bias=True)
    assert dx.shape == (0, 256) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("n,c", [(300_007, 8192), (9_000_001, 256), (150_001, 16384)])
def test_offsets_past_32_bits(n, c):
    """2.3e9 elements and more: the first and the last rows, and dw as a sum over pieces in binary64."""
    x, dy = (torch.empty((n, c), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(11)
    pieces = [(a, min(n, a + (1 << 26) // c)) for a in range(0, n, (1 << 26) // c)]
    for a, b in pieces:
        x[a:b] = torch.randn((b - a, c), generator=g, device=DEV)
        dy[a:b] = torch.randn((b - a, c), generator=g, device=DEV)
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(torch.bfloat16)
    y, _, rstd = jq.norm_fwd(x, w, None, eps=1e-5, kind=jq.NORM_RMS)
    dx, dw, _ = jq.norm_bwd(dy, x, w, None, rstd, kind=jq.NORM_RMS)
    assert jq.jetq_check_device_error() == jq.OK
    rw, tw = (torch.zeros(c, dtype=torch.float64, device=DEV) for _ in range(2))
    for a, b in pieces:
        X, r = x[a:b].double(), rstd[a:b].double()[:, None]
        ref = X * r * w.double()
        assert bool(((y[a:b].double() - ref).abs() <= (2.0 ** -8 + 4 * U) * ref.abs()).all())
        (rx, tx), (pw, _), _ = _define_bwd(dy[a:b], x[a:b], w, None, rstd[a:b], jq.NORM_RMS)
        assert bool(((dx[a:b].double() - rx).abs() <= tx + 2.0 ** -8 * rx.abs()).all())
        rw += pw
        tw += (dy[a:b].double().abs() * 2 * (X * r).abs()).sum(0)
    assert bool(((dw.double() - rw).abs() <= (100 + n / 300) * U * tw).all())
