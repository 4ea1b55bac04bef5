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
