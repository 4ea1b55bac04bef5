"""Refusals of the losses' and the mixture-of-experts layer's entry points: decided on the host before any CUDA
call, so no GPU is needed.  Sizes of workspaces, and the tensor helpers' checks."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
F = ctypes.c_float
FAKE = P(4096)  # never dereferenced: every call below fails validation first
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from rollout_x128_act_gb300 import build

    build.build()
    import rollout_x128_act_gb300 as jq

    return jq.lib()


# ------------------------------------------------------------------ policy loss

def _policy(L, back, **k):
    a = dict(nll=FAKE, old=FAKE, ref=None, adv=FAKE, per=0, mask=None, n=9, off=FAKE, nseg=3, level=0, mean=0,
             scale=1.0, low=0.2, high=0.2, dual=0.0, kl=0.1, out=FAKE, seg=FAKE, ws=FAKE, bytes=BIG, dloss=None,
             dnll=FAKE)
    a.update(k)
    common = (a["nll"], a["old"], a["ref"], a["adv"], a["per"], a["mask"], a["n"], a["off"], a["nseg"], a["level"],
              a["mean"], F(a["scale"]), F(a["low"]), F(a["high"]), F(a["dual"]), F(a["kl"]), a["out"], a["seg"])
    if back:
        return L.jetq_policy_loss_bwd(*common, a["dloss"], a["dnll"], None)
    return L.jetq_policy_loss_fwd(*common, a["ws"], ctypes.c_size_t(a["bytes"]), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(nll=None), INVALID), (dict(old=None), INVALID), (dict(adv=None), INVALID),
    (dict(per=2), INVALID), (dict(nseg=0), INVALID), (dict(level=2), INVALID), (dict(mean=3), INVALID),
    (dict(mean=-1), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(kl=NAN), INVALID),
    (dict(low=-0.1), INVALID), (dict(low=1.5), INVALID), (dict(low=NAN), INVALID), (dict(high=-0.1), INVALID),
    (dict(high=INF), INVALID), (dict(dual=0.5), INVALID), (dict(dual=-1.0), INVALID), (dict(dual=NAN), INVALID),
    (dict(out=None), INVALID), (dict(seg=None), INVALID), (dict(n=1 << 41), SHAPE), (dict(nseg=1 << 31), SHAPE),
    (dict(nll=P(4098)), ALIGN), (dict(old=P(4097)), ALIGN), (dict(ref=P(4098)), ALIGN), (dict(adv=P(4098)), ALIGN),
    (dict(off=P(4100)), ALIGN), (dict(seg=P(4100)), ALIGN), (dict(out=P(4098)), ALIGN),
])
def test_policy_loss_refuses(L, back, change, status):
    assert _policy(L, back, **change) == status


@pytest.mark.parametrize("change,status", [(dict(ws=None), INVALID), (dict(bytes=64), INVALID),
                                           (dict(ws=P(4104)), ALIGN)])
def test_policy_loss_workspace_refused(L, change, status):
    assert _policy(L, False, **change) == status


@pytest.mark.parametrize("change,status", [(dict(dnll=None), INVALID), (dict(dnll=P(4098)), ALIGN),
                                           (dict(dloss=P(4098)), ALIGN)])
def test_policy_loss_backward_refuses(L, change, status):
    assert _policy(L, True, **change) == status


def test_policy_loss_backward_of_no_tokens(L):
    assert _policy(L, True, n=0, nll=None, old=None, adv=None, dnll=None) == OK


def test_policy_loss_workspaces(L):
    size = L.jetq_policy_loss_workspace_bytes
    assert size(0, 3) == size(9, 0) == size(1 << 41, 3) == 0
    assert size(1, 1) >= 16 + 2 * 32 + 40  # a piece for each window of 128 and for each sequence
    assert size(1 << 20, 100) >= 16 + (8192 + 100) * 32
    assert size(1 << 20, 100) < (1 << 20)  # far less than the tokens' own


def test_policy_loss_helper_checks_its_tensors():
    import rollout_x128_act_gb300 as jq

    cpu = torch.zeros(4)
    with pytest.raises(ValueError):
        jq.policy_loss(cpu, cpu, cpu)
    with pytest.raises(ValueError):
        jq.policy_loss_bwd(cpu, cpu, cpu, None, None)


# ------------------------------------------------------------------ distillation

def _distill(L, back, **k):
    a = dict(x=FAKE, n=4, c=64, ldx=64, w=FAKE, v=300, ldw=64, ids=FAKE, ldi=8, t=FAKE, ldt=8, k=8, renorm=1,
             scale=1.0, loss=FAKE, lse=FAKE, logp=FAKE, dloss=FAKE, dx=FAKE, lddx=64, dw=FAKE, dt=0, lddw=64, acc=0,
             ws=FAKE, bytes=BIG)
    a.update(k)
    common = (a["x"], a["n"], a["c"], a["ldx"], a["w"], a["v"], a["ldw"], a["ids"], a["ldi"], a["t"], a["ldt"], a["k"],
              a["renorm"], F(a["scale"]))
    if back:
        return L.jetq_linear_distill_bwd(*common, a["lse"], a["logp"], a["dloss"], a["dx"], a["lddx"], a["dw"],
                                         a["dt"], a["lddw"], a["acc"], a["ws"], ctypes.c_size_t(a["bytes"]), None)
    return L.jetq_linear_distill_fwd(*common, a["loss"], a["lse"], a["logp"], a["ws"], ctypes.c_size_t(a["bytes"]),
                                     None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(v=0), INVALID), (dict(c=0), INVALID), (dict(k=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(ids=None), INVALID), (dict(t=None), INVALID), (dict(renorm=2), INVALID),
    (dict(lse=None), INVALID), (dict(logp=None), INVALID), (dict(ws=None), INVALID), (dict(bytes=100), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID),
    (dict(c=60), SHAPE), (dict(ldx=56), SHAPE), (dict(ldw=56), SHAPE), (dict(k=257, ldi=300, ldt=300), SHAPE),
    (dict(ldi=7), SHAPE), (dict(ldt=7), SHAPE), (dict(v=1 << 31), SHAPE), (dict(n=1 << 31), SHAPE),
    (dict(x=P(4104)), ALIGN), (dict(w=P(4104)), ALIGN), (dict(ids=P(4100)), ALIGN), (dict(t=P(4098)), ALIGN),
    (dict(ws=P(4104)), ALIGN), (dict(logp=P(4098)), ALIGN),
])
def test_distillation_refuses(L, back, change, status):
    assert _distill(L, back, **change) == status


@pytest.mark.parametrize("change,status", [(dict(dloss=None), INVALID), (dict(dx=None), INVALID),
                                           (dict(dw=None), INVALID), (dict(acc=1, dt=1), INVALID),
                                           (dict(lddx=56), SHAPE), (dict(lddw=66), ALIGN), (dict(dx=P(4104)), ALIGN)])
def test_distillation_backward_refuses(L, change, status):
    assert _distill(L, True, **change) == status


def test_distillation_of_no_rows(L):
    assert _distill(L, False, n=0, x=None, ids=None, t=None, loss=None, lse=None, logp=None, ws=None, bytes=0) == OK


def test_distillation_workspaces(L):
    size, back = L.jetq_linear_distill_workspace_bytes, L.jetq_linear_distill_bwd_workspace_bytes
    for f in (size, lambda *a: back(*a, 0), lambda *a: back(*a, 1)):
        assert f(0, 300, 64, 8) == f(4, 300, 64, 0) == f(4, 300, 64, 257) == 0
    # the cross entropy's, a bit a logit, 8 bytes an entry
    more = size(4096, 131072, 4096, 64) - L.jetq_linear_ce_workspace_bytes(4096, 131072, 4096)
    assert 4096 * 131072 // 8 + 4096 * 64 * 8 <= more <= 4096 * 131072 // 8 + 4096 * 64 * 8 + (1 << 16)
    assert back(4096, 131072, 4096, 64, 1) < back(4096, 131072, 4096, 64, 0)
    entries = back(4096, 131072, 4096, 64, 0) - L.jetq_linear_ce_bwd_workspace_bytes(4096, 131072, 4096, 0)
    assert entries == 4096 * 64 * 8


def test_distillation_helper_checks_its_tensors():
    import rollout_x128_act_gb300 as jq

    x, i, t = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 8), dtype=torch.int64), torch.zeros((4, 8))
    with pytest.raises(ValueError):
        jq.linear_distill(x, x, i, t)
    with pytest.raises(ValueError):
        jq.linear_distill_bwd(x, x, i, t, t[:, 0], t, t[:, 0])


# ------------------------------------------------------------------ mixture of experts

def _moe(L, **k):
    a = dict(x=FAKE, m=4, h=64, ldx=64, router=FAKE, ldr=64, e=8, topk=2, renorm=1, q13=FAKE, sb13=FAKE, sg13=FAKE,
             i=32, q2=FAKE, sb2=FAKE, sg2=FAKE, y=FAKE, dt=1, ldy=64, ids=FAKE, p=FAKE, ws=FAKE, bytes=BIG)
    a.update(k)
    return L.jetq_moe_nvfp4(a["x"], a["m"], a["h"], a["ldx"], a["router"], a["ldr"], a["e"], a["topk"], a["renorm"],
                            a["q13"], a["sb13"], a["sg13"], a["i"], a["q2"], a["sb2"], a["sg2"], a["y"], a["dt"],
                            a["ldy"], a["ids"], a["p"], a["ws"], ctypes.c_size_t(a["bytes"]), None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(h=0), INVALID), (dict(i=0), INVALID), (dict(e=0), INVALID), (dict(topk=0), INVALID),
    (dict(renorm=2), INVALID), (dict(dt=2), INVALID), (dict(x=None), INVALID), (dict(router=None), INVALID),
    (dict(q13=None), INVALID), (dict(sb13=None), INVALID), (dict(sg13=None), INVALID), (dict(q2=None), INVALID),
    (dict(sb2=None), INVALID), (dict(sg2=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID),
    (dict(bytes=64), INVALID),
    (dict(m=17), SHAPE), (dict(e=257), SHAPE), (dict(topk=9), SHAPE), (dict(e=64, topk=17), SHAPE),
    (dict(h=48, ldx=48, ldr=48, ldy=48), SHAPE), (dict(i=48), SHAPE), (dict(ldx=56), SHAPE), (dict(ldr=56), SHAPE),
    (dict(ldy=63), SHAPE), (dict(i=16416), SHAPE), (dict(h=16416, ldx=16416, ldr=16416, ldy=16416), SHAPE),
    (dict(x=P(4104)), ALIGN), (dict(ldx=68), ALIGN), (dict(router=P(4104)), ALIGN), (dict(ldr=68), ALIGN),
    (dict(q13=P(4104)), ALIGN), (dict(q2=P(4104)), ALIGN), (dict(sb13=P(4104)), ALIGN), (dict(sb2=P(4104)), ALIGN),
    (dict(sg13=P(4098)), ALIGN), (dict(sg2=P(4098)), ALIGN), (dict(y=P(4097)), ALIGN), (dict(y=P(4098), dt=0), ALIGN),
    (dict(ids=P(4100)), ALIGN), (dict(p=P(4098)), ALIGN), (dict(ws=P(4104)), ALIGN),
])
def test_moe_refuses(L, change, status):
    assert _moe(L, **change) == status


def test_moe_of_no_tokens(L):
    assert _moe(L, m=0, x=None, y=None, ids=None, p=None, ws=None, bytes=0) == OK


def test_moe_workspaces(L):
    size = L.jetq_moe_nvfp4_workspace_bytes
    assert size(0, 8, 64, 32, 2) == size(17, 8, 64, 32, 2) == size(4, 257, 64, 32, 2) == size(4, 8, 64, 32, 17) == 0
    # logits, x in 16 bits, three 16-bit numbers an activation
    assert size(16, 128, 2048, 768, 8) >= 16 * 128 * 4 + 16 * 2048 * 2 + 16 * 8 * 768 * 6


def test_moe_helper_checks_its_tensors():
    import rollout_x128_act_gb300 as jq

    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        jq.moe_nvfp4(x, x, {}, {}, 2)
