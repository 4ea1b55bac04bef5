"""What the tensor helpers refuse before anything is launched, on tensors that exist in name only (no GPU is needed)."""
import pytest
import torch
from torch._subclasses import FakeTensorMode

import rollout_x128_act_gb300 as jq


class Launched(Exception):
    pass


@pytest.fixture
def cuda(monkeypatch):
    """Tensors of a device 0 that is the current one; launches raise Launched."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    def launch(*args, **kw):
        raise Launched

    for name in ("jetq_linear_distill_fwd", "jetq_linear_distill_bwd", "jetq_moe_nvfp4", "jetq_policy_loss_fwd",
                 "jetq_linear_ce_fwd", "jetq_linear_ce_bwd", "jetq_norm_bwd", "jetq_gemm_fprop_ws",
                 "jetq_quant_nvfp4", "jetq_amax_bf16"):
        monkeypatch.setattr(jq, name, launch)
    monkeypatch.setattr(jq, "jetq_decode_workspace_bytes", lambda n, d, c: 1024)
    monkeypatch.setattr(jq, "_aligned_rows", lambda t: t)  # looks at the address, which these have not
    from rollout_x128_act_gb300 import build

    build.build()
    with FakeTensorMode():
        yield


def _t(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=device)


def _experts(e, r, c):
    return dict(q=_t(e, r, c // 2, dtype=torch.uint8), sb=_t(e, r, c // 16, dtype=torch.uint8),
                sg=_t(e, dtype=torch.float32))


F32, I64, U8 = torch.float32, torch.int64, torch.uint8
CALLS = {
    "linear_distill": lambda ws: jq.linear_distill(_t(4, 64), _t(300, 64), _t(4, 8, dtype=I64), _t(4, 8, dtype=F32),
                                                   workspace=ws),
    "linear_distill_bwd": lambda ws: jq.linear_distill_bwd(
        _t(4, 64), _t(300, 64), _t(4, 8, dtype=I64), _t(4, 8, dtype=F32), _t(4, dtype=F32), _t(4, 8, dtype=F32),
        _t(4, dtype=F32), workspace=ws),
    "moe_nvfp4": lambda ws: jq.moe_nvfp4(_t(4, 64), _t(8, 64), _experts(8, 64, 64), _experts(8, 64, 32), 2,
                                         workspace=ws),
    "policy_loss": lambda ws: jq.policy_loss(_t(9, dtype=F32), _t(9, dtype=F32), _t(9, dtype=F32), workspace=ws),
    "linear_ce": lambda ws: jq.linear_ce(_t(4, 64), _t(300, 64), _t(4, dtype=I64), workspace=ws),
    "linear_ce_bwd": lambda ws: jq.linear_ce_bwd(_t(4, 64), _t(300, 64), _t(4, dtype=I64), _t(4, dtype=F32),
                                                 _t(4, dtype=F32), workspace=ws),
    "norm_bwd": lambda ws: jq.norm_bwd(_t(4, 64), _t(4, 64), _t(64), _t(4, dtype=F32), _t(4, dtype=F32),
                                       workspace=ws),
    "fprop": lambda ws: jq.fprop(_t(4, 128, dtype=U8), _t(1, 4, dtype=F32), _t(128, 128, dtype=U8),
                                 _t(1, 1, dtype=F32), workspace=ws),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", ["host", "another device", "one element many times", "every other byte"])
def test_a_workspace_that_the_kernels_may_not_write(cuda, call, bad):
    """Its address goes to kernels that write as many bytes as its elements have."""
    n = 1 << 26
    ws = {"host": lambda: _t(n, dtype=U8, device="cpu"), "another device": lambda: _t(n, dtype=U8, device="cuda:1"),
          "one element many times": lambda: _t(1, dtype=U8).expand(n),
          "every other byte": lambda: _t(2 * n, dtype=U8)[::2]}[bad]()
    with pytest.raises(ValueError):
        CALLS[call](ws)


@pytest.mark.parametrize("call", CALLS)
def test_a_workspace_of_the_right_kind(cuda, call):
    with pytest.raises(Launched):
        CALLS[call](_t(1 << 26, dtype=U8))
    with pytest.raises(Launched):
        CALLS[call](_t(1 << 20, 16, dtype=F32))
    with pytest.raises(Launched):
        CALLS[call](None)


def test_experts_that_quant_nvfp4_experts_takes(cuda):
    """BF16 [e x r x c] with consecutive elements along the last axis; experts and rows may lie apart."""
    for w in (_t(3, 32, 64), _t(3, 32, 72)[:, :, :64], _t(6, 32, 64)[::2], _t(3, 64, 64)[:, ::2], _t(3, 1, 64),
              _t(1, 32, 64).expand(3, 32, 64)):
        with pytest.raises(Launched):
            jq.quant_nvfp4_experts(w)


@pytest.mark.parametrize("bad", ["FP32", "FP16", "two axes", "strided last axis", "transposed", "host",
                                 "another device", "rows that overlap"])
def test_experts_that_quant_nvfp4_experts_refuses(cuda, bad):
    """Their bits would be read as those of a dense BF16 tensor."""
    w = {"FP32": lambda: _t(3, 32, 64, dtype=F32), "FP16": lambda: _t(3, 32, 64, dtype=torch.float16),
         "two axes": lambda: _t(32, 64), "strided last axis": lambda: _t(3, 32, 128)[:, :, ::2],
         "transposed": lambda: _t(3, 64, 32).transpose(1, 2), "host": lambda: _t(3, 32, 64, device="cpu"),
         "another device": lambda: _t(3, 32, 64, device="cuda:1"),
         "rows that overlap": lambda: _t(3, 1, 64).expand(3, 32, 64)}[bad]()
    with pytest.raises(ValueError):
        jq.quant_nvfp4_experts(w)
