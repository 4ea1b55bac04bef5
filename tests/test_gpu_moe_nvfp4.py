"""The mixture-of-experts layer for few tokens against its definition in binary64.

Bounds.  Every FP32 sum is within SUM = 1e-5 of the sum of its terms' magnitudes (the bound every GEMM test of this
library uses).  silu's slope is below 1.1.  An activation enters the second product as two BF16 numbers (2^-16 of its
value) for a BF16 result, as three (2^-24) for an FP32 one; p, silu and the scales add 10 roundings of 2^-24; the
result is rounded once.  The choice of experts is checked within the logits' own bound, and the layer's output for
the experts that were chosen.
"""
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SUM = 1e-5
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _layer(m, e, h, i, seed, spread=1.0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((m, h + pad), generator=g, device=DEV).to(torch.bfloat16)[:, :h]
    router = (torch.randn((e, h + pad), generator=g, device=DEV) * spread * h ** -0.5).to(torch.bfloat16)[:, :h]
    w13 = jq.quant_nvfp4_experts((torch.randn((e, 2 * i, h), generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16))
    w2 = jq.quant_nvfp4_experts((torch.randn((e, h, i), generator=g, device=DEV) * i ** -0.5).to(torch.bfloat16))
    return x, router, w13, w2


def _values(w, e):
    """Expert e's weight in binary64."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)
    code = torch.stack((w["q"][e] & 15, w["q"][e] >> 4), -1).flatten(-2).long()
    scale = w["sb"][e].view(torch.float8_e4m3fn).double() * w["sg"][e].double()
    return grid[code] * scale.repeat_interleave(16, -1)


def _check(x, router, w13, w2, topk, renorm, out_dtype, y, ids, p):
    """The three outputs against the definition."""
    m, h = x.shape
    X, R = x.double(), router.double()
    logits, el = X @ R.T, SUM * (X.abs() @ R.abs().T).amax(1, keepdim=True)
    # distinct, in falling order, and none left out that is larger
    assert bool((ids >= 0).all()) and bool((ids < router.shape[0]).all())
    mine = logits.gather(1, ids)
    assert all(len(set(r)) == topk for r in ids.tolist())
    assert bool((mine[:, :-1] - mine[:, 1:] >= -2 * el).all())
    rest = logits.scatter(1, ids, -torch.inf).amax(1, keepdim=True)
    assert bool((rest <= mine[:, -1:] + 2 * el).all())
    total = torch.logsumexp(mine if renorm else logits, 1, keepdim=True)
    want = (mine - total).exp()
    ep = want * (2 * el + 8 * HALF_F32)
    assert bool(((p.double() - want).abs() <= ep).all())
    ry, tol = torch.zeros_like(X), torch.zeros_like(X)
    parts = 2.0 ** -16 if out_dtype is torch.bfloat16 else HALF_F32
    for e in set(ids.flatten().tolist()):
        t, j = (ids == e).nonzero(as_tuple=True)
        A, B = _values(w13, e), _values(w2, e)
        gu, size = X[t] @ A.T, SUM * (X[t].abs() @ A.abs().T)
        gate, up = gu.chunk(2, 1)
        eg, eu = size.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        a = silu * up
        ea = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + (parts + 10 * HALF_F32) * a.abs()
        w = want[t, j][:, None]
        ry[t] += w * (a @ B.T)
        tol[t] += (w * (ea + SUM * a.abs()) + ep[t, j][:, None] * a.abs()) @ B.abs().T
    half = HALF_BF16 if out_dtype is torch.bfloat16 else HALF_F32
    assert bool(((y.double() - ry).abs() <= 1.01 * tol + half * ry.abs() + 1e-30).all())


SIZES = [(1, 1, 32, 32, 1), (1, 8, 256, 128, 2), (2, 5, 288, 64, 5), (3, 20, 1056, 352, 3), (4, 33, 512, 96, 4),
         (5, 7, 160, 224, 2), (8, 16, 512, 96, 16), (9, 40, 160, 64, 5), (12, 3, 2048, 768, 1), (16, 2, 256, 64, 2),
         (16, 128, 2048, 768, 8), (13, 256, 96, 32, 16), (7, 12, 4096, 32, 3), (16, 17, 2560, 160, 6)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("m,e,h,i,topk", SIZES)
def test_the_layer(m, e, h, i, topk, renorm, out_dtype):
    """One token to sixteen, all tokens on the same experts (e = topk), several row blocks a CTA, rows of y in more
    CTAs than SMs, shares of K that are empty (h = 32) or end in a part of a step."""
    x, router, w13, w2 = _layer(m, e, h, i, m * 100 + e, pad=8 if m % 2 else 0)
    y, ids, p = jq.moe_nvfp4(x, router, w13, w2, topk, renorm, out_dtype)
    assert y.dtype is out_dtype and p.shape == ids.shape == (m, topk)
    _check(x, router, w13, w2, topk, renorm, out_dtype, y, ids, p)


def test_sixteen_tokens_that_all_take_the_same_experts():
    """Two tiles of tokens for one expert, next to experts with one token."""
    x, router, w13, w2 = _layer(16, 32, 512, 128, 5, spread=0.1)
    bias = torch.ones(512, device=DEV)
    x = (x.float() + 0.5 * bias).to(torch.bfloat16)
    router[7] = router[19] = 0.05  # far above the others for every token
    for out_dtype in (torch.bfloat16, torch.float32):
        y, ids, p = jq.moe_nvfp4(x, router, w13, w2, 4, True, out_dtype)
        assert bool((ids == 7).any(1).all()) and bool((ids == 19).any(1).all())
        _check(x, router, w13, w2, 4, True, out_dtype, y, ids, p)


def test_equal_logits_take_the_lower_index():
    x, router, w13, w2 = _layer(3, 70, 64, 32, 6)
    x[1] = 0  # all 70 logits are equal
    router[40] = router[3]
    router[69] = router[3]
    y, ids, p = jq.moe_nvfp4(x, router, w13, w2, 16)
    assert ids[1].tolist() == list(range(16))
    assert bool((p[1] == 1 / 16).all()) and bool((y[1] == 0).all())
    for row in ids.tolist():
        at = [row.index(k) for k in (3, 40, 69) if k in row]
        assert at == sorted(at)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_number_missing_shows_in_its_token(value):
    x, router, w13, w2 = _layer(6, 20, 128, 64, 7)
    y, ids, p = jq.moe_nvfp4(x, router, w13, w2, 4)
    x2 = x.clone()
    x2[2, 5] = value
    y2, ids2, p2 = jq.moe_nvfp4(x2, router, w13, w2, 4)
    keep = torch.arange(6, device=DEV) != 2
    assert torch.equal(y2[keep], y[keep]) and torch.equal(ids2[keep], ids[keep]) and torch.equal(p2[keep], p[keep])
    assert not bool(y2[2].isfinite().any())
    assert bool((ids2 >= 0).all()) and bool((ids2 < 20).all()) and len(set(ids2[2].tolist())) == 4


def test_an_experts_missing_number_stays_with_its_tokens():
    x, router, w13, w2 = _layer(9, 24, 128, 64, 8)
    y, ids, _ = jq.moe_nvfp4(x, router, w13, w2, 3, out_dtype=torch.float32)
    e = int(ids[4, 1])
    w2["sg"][e] = float("nan")
    y2, _, _ = jq.moe_nvfp4(x, router, w13, w2, 3, out_dtype=torch.float32)
    hit = (ids == e).any(1)
    assert bool(y2[hit].isnan().all()) and torch.equal(y2[~hit], y[~hit])


def test_one_expert_is_the_few_token_products():
    """e = topk = 1: the layer is two few-token products (FP32) with silu between them, p = 1."""
    x, router, w13, w2 = _layer(4, 1, 256, 128, 9)
    y, _, p = jq.moe_nvfp4(x, router, w13, w2, 1, out_dtype=torch.float32)
    gu = jq.gemv_nvfp4(x, dict(q=w13["q"][0], sb=w13["sb"][0], sg=w13["sg"]))
    gate, up = gu.double().chunk(2, 1)
    B = _values(w2, 0)
    a = gate * torch.sigmoid(gate) * up
    assert bool((p == 1).all())
    assert bool(((y.double() - a @ B.T).abs() <= 4 * SUM * (a.abs() @ B.abs().T) + 1e-6 * (a.abs() @ B.abs().T)).all())


def test_no_tokens_strided_rows_and_absent_outputs():
    x, router, w13, w2 = _layer(6, 10, 128, 64, 10)
    y, ids, p = jq.moe_nvfp4(x[:0], router, w13, w2, 2)
    assert y.shape == (0, 128) and ids.shape == p.shape == (0, 2)
    y, ids, p = jq.moe_nvfp4(x, router, w13, w2, 2)
    wide_x = torch.full((6, 200), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_x[:, 8:136] = x
    wide_r = torch.full((10, 144), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_r[:, :128] = router
    out = torch.full((6, 131), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((jq.jetq_moe_nvfp4_workspace_bytes(6, 10, 128, 64, 2),), 255, dtype=torch.uint8, device=DEV)
    jq.jetq_moe_nvfp4(wide_x[:, 8:136], wide_r[:, :128], 2, True, w13["q"], w13["sb"], w13["sg"], w2["q"], w2["sb"],
                      w2["sg"], out[:, 1:129], None, None, ws)
    assert torch.equal(out[:, 1:129], y)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 129:] == 7).all())


def test_repeatable_captured_and_on_another_stream():
    x, router, w13, w2 = _layer(11, 64, 1024, 256, 11)
    first = jq.moe_nvfp4(x, router, w13, w2, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = jq.moe_nvfp4(x, router, w13, w2, 6, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # two layers in a row, the second reads the first
        a = jq.moe_nvfp4(x, router, w13, w2, 6)
        b = jq.moe_nvfp4(a[0], router, w13, w2, 6)
    for _ in range(20):
        for t in a + b:
            t.fill_(3)
        g.replay()
        assert all(torch.equal(s, t) for s, t in zip(first, a))
        assert all(torch.equal(s, t) for s, t in zip(jq.moe_nvfp4(first[0], router, w13, w2, 6), b))
    x.copy_(x.flip(0))  # other tokens under the same graph
    g.replay()
    assert all(torch.equal(s, t) for s, t in zip(jq.moe_nvfp4(x, router, w13, w2, 6), a))


def test_layers_that_share_a_workspace():
    """Calls in stream order on one workspace, different choices each."""
    x, router, w13, w2 = _layer(16, 48, 512, 160, 12)
    ws = torch.empty(jq.jetq_moe_nvfp4_workspace_bytes(16, 48, 512, 160, 8), dtype=torch.uint8, device=DEV)
    rows = [x[:k].flip(0) if k % 2 else x[-k:] for k in (16, 1, 7, 12, 3, 16)]
    alone = [jq.moe_nvfp4(r, router, w13, w2, 8) for r in rows]
    for _ in range(10):
        shared = [jq.moe_nvfp4(r, router, w13, w2, 8, workspace=ws) for r in rows]
        for a, b in zip(alone, shared):
            assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("m,e,h,i,topk", [
    (2, 2, 16384, 64, 1), (1, 2, 64, 16384, 2), (16, 3, 16384, 32, 2), (5, 4, 8192, 96, 2), (9, 6, 128, 8192, 3),
    (16, 40, 4096, 256, 8), (7, 9, 96, 4096, 4)])
def test_wide_layers(m, e, h, i, topk):
    """Rows of up to 16384 values: rings of one to five buffers, each given back before it is filled again, shared by
    all warps, two groups or eight."""
    x, router, w13, w2 = _layer(m, e, h, i, 13)
    for out_dtype in (torch.bfloat16, torch.float32):
        y, ids, p = jq.moe_nvfp4(x, router, w13, w2, topk, True, out_dtype)
        assert jq.jetq_check_device_error() == jq.OK
        _check(x, router, w13, w2, topk, True, out_dtype, y, ids, p)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_tokens_of_any_magnitude(size):
    """x times 2^k gives gate and up times 2^k: both products see the same FP16 values, whatever k is (up is scaled
    back by a power of two; gate is kept at the size where silu is not linear by its weights' scale)."""
    x, router, w13, w2 = _layer(3, 6, 128, 64, 14)
    k = 2.0 ** round(torch.tensor(size).log2().item())
    w13s = dict(w13, sg=w13["sg"] / k)
    a = jq.moe_nvfp4(x, router, w13, w2, 6, out_dtype=torch.float32)
    b = jq.moe_nvfp4((x.float() * k).to(torch.bfloat16), (router.float() / k).to(torch.bfloat16), w13s, w2, 6,
                     out_dtype=torch.float32)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    x, router, w13, w2 = _layer(16, 40, 512, 160, 15)
    want = [jq.moe_nvfp4(x[:9], router, w13, w2, 5), jq.moe_nvfp4(x, router, w13, w2, 7)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(30):
        got[0].append(jq.moe_nvfp4(x[:9], router, w13, w2, 5, stream=streams[0]))
        got[1].append(jq.moe_nvfp4(x, router, w13, w2, 7, stream=streams[1]))
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, w))
