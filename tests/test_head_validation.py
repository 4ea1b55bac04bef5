"""Refusals of the head's entry points (linear cross entropy, norms, few-token
NVFP4 product): decided on the host before any CUDA call, so no GPU is needed.
Sizes of workspaces, and the tensor helpers' checks."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
F = ctypes.c_float
FAKE = P(4096)  # never dereferenced: every call below fails validation first
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from rollout_x128_act_gb300 import build

    build.build()
    import rollout_x128_act_gb300 as jq

    return jq.lib()


def _ce_fwd(L, **k):
    a = dict(x=FAKE, n=4, c=64, ldx=64, w=FAKE, v=300, ldw=64, target=FAKE, scale=1.0, loss=FAKE, lse=FAKE, ws=FAKE,
             bytes=BIG)
    a.update(k)
    return L.jetq_linear_ce_fwd(a["x"], a["n"], a["c"], a["ldx"], a["w"], a["v"], a["ldw"], a["target"],
                                F(a["scale"]), a["loss"], a["lse"], a["ws"], ctypes.c_size_t(a["bytes"]), None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(v=0), INVALID), (dict(c=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(target=None), INVALID), (dict(loss=None), INVALID), (dict(lse=None), INVALID),
    (dict(ws=None), INVALID), (dict(bytes=100), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(c=60), SHAPE), (dict(ldx=56), SHAPE), (dict(ldw=56), SHAPE), (dict(v=1 << 31), SHAPE),
    (dict(n=1 << 31), SHAPE), (dict(n=1 << 29, v=1 << 29), SHAPE),
    (dict(n=1 << 29, c=1 << 16, ldx=1 << 16, ldw=1 << 16), SHAPE),
    (dict(x=P(4104)), ALIGN), (dict(w=P(4104)), ALIGN), (dict(ldx=68), ALIGN), (dict(ldw=68), ALIGN),
    (dict(target=P(4100)), ALIGN), (dict(loss=P(4098)), ALIGN), (dict(ws=P(4104)), ALIGN),
])
def test_linear_ce_forward_refuses(L, change, status):
    assert _ce_fwd(L, **change) == status


def test_linear_ce_forward_of_no_tokens(L):
    assert _ce_fwd(L, n=0, x=None, target=None, loss=None, lse=None, ws=None, bytes=0) == OK


def _ce_bwd(L, **k):
    a = dict(x=FAKE, n=4, c=64, ldx=64, w=FAKE, v=300, ldw=64, target=FAKE, scale=1.0, lse=FAKE, dloss=FAKE, dx=FAKE,
             lddx=64, dw=FAKE, dt=0, lddw=64, acc=0, ws=FAKE, bytes=BIG)
    a.update(k)
    return L.jetq_linear_ce_bwd(a["x"], a["n"], a["c"], a["ldx"], a["w"], a["v"], a["ldw"], a["target"],
                                F(a["scale"]), a["lse"], a["dloss"], a["dx"], a["lddx"], a["dw"], a["dt"], a["lddw"],
                                a["acc"], a["ws"], ctypes.c_size_t(a["bytes"]), None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(lse=None), INVALID), (dict(dloss=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(ws=None), INVALID), (dict(dt=2), INVALID), (dict(acc=1, dt=1), INVALID),
    (dict(acc=2), INVALID), (dict(lddx=56), SHAPE), (dict(lddw=56), SHAPE), (dict(lddw=66), ALIGN),
    (dict(dt=1, lddw=68), ALIGN), (dict(lddx=68), ALIGN), (dict(dx=P(4104)), ALIGN), (dict(dw=P(4104)), ALIGN),
    (dict(dloss=P(4098)), ALIGN), (dict(ws=P(4104)), ALIGN),
])
def test_linear_ce_backward_refuses(L, change, status):
    assert _ce_bwd(L, **change) == status


def test_linear_ce_workspaces(L):
    assert L.jetq_linear_ce_workspace_bytes(0, 300, 64) == 0
    assert L.jetq_linear_ce_workspace_bytes(4, 300, 64) >= 2 * 2 * 4 * 8 + 4 * 4  # a pair every 128 columns, a logit
    assert L.jetq_linear_ce_workspace_bytes(4096, 131072, 4096) == 2 * 512 * 4096 * 8 + 4096 * 4
    assert L.jetq_linear_ce_bwd_workspace_bytes(0, 300, 64, 0) == 0
    small = L.jetq_linear_ce_bwd_workspace_bytes(4096, 131072, 4096, 1)
    large = L.jetq_linear_ce_bwd_workspace_bytes(4096, 131072, 4096, 0)
    assert 4096 * 256 * 2 < small < large < 4096 * 131072 * 2  # never the whole vocabulary's logits


def _fwd(L, **k):
    a = dict(kind=0, dt=1, x=FAKE, n=4, c=65, ldx=72, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, ldy=72, mean=FAKE, rstd=FAKE)
    a.update(k)
    return L.jetq_norm_fwd(a["kind"], a["dt"], a["x"], a["n"], a["c"], a["ldx"], a["w"], a["b"], F(a["eps"]), a["y"],
                           a["ldy"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=2), INVALID), (dict(dt=2), INVALID), (dict(n=-1), INVALID), (dict(c=0), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(rstd=None), INVALID), (dict(mean=None), INVALID),
    (dict(kind=1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(ldx=64), SHAPE), (dict(ldy=64), SHAPE), (dict(c=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), SHAPE),
    (dict(x=P(4104)), ALIGN), (dict(ldx=68), ALIGN), (dict(ldy=68), ALIGN), (dict(w=P(4097)), ALIGN),
    (dict(b=P(4097)), ALIGN), (dict(rstd=P(4098)), ALIGN), (dict(dt=0, w=P(4098)), ALIGN),
])
def test_norm_forward_refuses(L, change, status):
    assert _fwd(L, **change) == status


def _bwd(L, **k):
    a = dict(kind=0, dt=0, dy=FAKE, lddy=68, x=FAKE, n=4, c=65, ldx=68, w=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, lddx=68,
             dw=FAKE, db=FAKE, ws=FAKE, bytes=BIG)
    a.update(k)
    return L.jetq_norm_bwd(a["kind"], a["dt"], a["dy"], a["lddy"], a["x"], a["n"], a["c"], a["ldx"], a["w"], a["mean"],
                           a["rstd"], a["dx"], a["lddx"], a["dw"], a["db"], a["ws"], ctypes.c_size_t(a["bytes"]),
                           None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=-1), INVALID), (dict(dt=7), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(rstd=None), INVALID), (dict(mean=None), INVALID), (dict(ws=None), INVALID),
    (dict(kind=1), INVALID),  # RMS norm has no bias
    (dict(lddy=64), SHAPE), (dict(lddx=64), SHAPE), (dict(ldx=64), SHAPE),
    (dict(lddy=66), ALIGN), (dict(dy=P(4104)), ALIGN), (dict(dw=P(4098)), ALIGN), (dict(db=P(4098)), ALIGN),
    (dict(ws=P(4104)), ALIGN), (dict(dt=1), ALIGN),  # 68 elements are not 16-byte rows of BF16
])
def test_norm_backward_refuses(L, change, status):
    assert _bwd(L, **change) == status


def test_norm_of_no_rows_and_workspaces(L):
    assert _fwd(L, n=0, x=None, y=None, mean=None, rstd=None) == OK
    assert L.jetq_norm_bwd_workspace_bytes(1, 0, 64) == 0
    for n, c in ((1, 1), (100, 512), (5, 20001)):  # at least one partial row of dw and db
        assert L.jetq_norm_bwd_workspace_bytes(1, n, c) >= 8 * c


def _gemv(L, **k):
    a = dict(q=FAKE, sb=FAKE, sg=FAKE, n=5, k=64, x=FAKE, m=2, ldx=64, y=FAKE, dt=0, ldy=5)
    a.update(k)
    return L.jetq_gemv_nvfp4(a["q"], a["sb"], a["sg"], a["n"], a["k"], a["x"], a["m"], a["ldx"], a["y"], a["dt"],
                             a["ldy"], None)


@pytest.mark.parametrize("change,status", [
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(m=-1), INVALID), (dict(dt=3), INVALID), (dict(q=None), INVALID),
    (dict(sb=None), INVALID), (dict(sg=None), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(m=17), SHAPE), (dict(k=48), SHAPE), (dict(ldx=56), SHAPE), (dict(ldy=4), SHAPE),
    (dict(q=P(4104)), ALIGN), (dict(sb=P(4097)), ALIGN), (dict(sg=P(4098)), ALIGN), (dict(x=P(4104)), ALIGN),
    (dict(ldx=68), ALIGN), (dict(y=P(4098)), ALIGN), (dict(dt=1, y=P(4097)), ALIGN),
])
def test_gemv_refuses(L, change, status):
    assert _gemv(L, **change) == status


def test_gemv_of_no_tokens(L):
    assert _gemv(L, m=0, x=None, y=None) == OK


def test_tensor_helpers_refuse_host_tensors(L):
    import rollout_x128_act_gb300 as jq

    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="x: a CUDA tensor"):
        jq.linear_ce(x, x, t)
    with pytest.raises(ValueError, match="x: a CUDA tensor"):
        jq.linear_ce_bwd(x, x, t, None, None)
    with pytest.raises(ValueError, match="x: a CUDA tensor"):
        jq.norm_fwd(x)
    with pytest.raises(ValueError, match="x: a CUDA tensor"):
        jq.norm_bwd(x, x, None, None, None)
    with pytest.raises(ValueError, match="x: a CUDA tensor"):
        jq.gemv_nvfp4(x, dict(q=None, sb=None, sg=None))


class _Fake:
    """What the checks look at, of a CUDA tensor that does not exist."""

    is_cuda = True

    def __init__(self, shape, dtype, stride):
        self.shape, self.dtype, self._stride = torch.Size(shape), dtype, stride

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        dense, step = True, 1
        for size, stride in zip(reversed(self.shape), reversed(self._stride)):
            dense, step = dense and (size == 1 or stride == step), step * size
        return dense


def test_tensor_checks(monkeypatch, L):
    import rollout_x128_act_gb300 as jq

    monkeypatch.setattr(jq.torch, "Tensor", _Fake)
    bf, f32 = torch.bfloat16, torch.float32
    jq._want(_Fake((4, 8), bf, (16, 1)), "x", bf, (4, 8), rows=True)
    jq._want(_Fake((4, 8), f32, (8, 1)), "x", (bf, f32))
    jq._want(_Fake((1, 8), f32, (3, 1)), "x", f32, rows=True)  # one row: its stride is not used
    for t, dtype, shape, rows, what in (
            (_Fake((4, 8), f32, (8, 1)), bf, None, True, "is wanted, got torch.float32"),
            (_Fake((4, 8), bf, (8, 1)), bf, (4, 9), True, "shape"),
            (_Fake((4, 8), bf, (1, 4)), bf, None, True, "strides"),
            (_Fake((4, 8), bf, (0, 1)), bf, None, True, "strides"),
            (_Fake((2, 4, 8), bf, (32, 8, 1)), bf, None, True, "strides"),
            (_Fake((8,), f32, (2,)), f32, (8,), False, "contiguous")):
        with pytest.raises(ValueError, match=what):
            jq._want(t, "x", dtype, shape, rows)


def test_rows_are_padded_where_their_layout_asks_for_it():
    import rollout_x128_act_gb300 as jq

    for dtype, step in ((torch.bfloat16, 8), (torch.float32, 4)):
        base = torch.arange(40 * 24, dtype=torch.float32).to(dtype).view(40, 24)
        assert base.data_ptr() % 16 == 0
        for x, same in ((base, True), (base[:, :step], True), (base[3:, step:], True), (base[:, :17], True),
                        (base[:, 1:], False), (base[:, :17].contiguous(), False), (base.view(-1)[:23].view(1, 23), False),
                        (torch.as_strided(base, (1, 16), (3, 1)), False), (torch.empty((0, 17), dtype=dtype), False)):
            y = jq._aligned_rows(x)
            assert (y is x) == same and torch.equal(x, y)
            assert y.data_ptr() % 16 == 0 and y.stride(0) % step == 0 and y.stride(0) >= y.shape[1]
