"""Few-token product with NVFP4 weights against the dequantized product in binary64.

Bounds: products of codes, scales and activations are exact in FP32's range,
so only the sum rounds: within 1e-5 * sum |w x|, as for every GEMM of the
library, and half a step of a BF16 output (2^-8 of its value).
"""
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SUM = 1e-5
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _dequant(w):
    table = torch.cat((GRID, -GRID)).to(DEV)
    codes = torch.stack((w["q"] & 15, w["q"] >> 4), 2).flatten(1).long()
    step = w["sb"].view(torch.float8_e4m3fn).double() * w["sg"].double()
    return table[codes] * step.repeat_interleave(16, 1)


def _weight(n, k, seed):
    """Every code and scales over E4M3's whole range (its subnormals and 448 among them)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    sb = torch.randint(0, 127, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8)
    return dict(q=q, sb=sb, sg=torch.tensor([3.1e-4], device=DEV))


def _check(x, w, out_dtype):
    y = jq.gemv_nvfp4(x, w, out_dtype=out_dtype)
    torch.cuda.synchronize()
    W, X = _dequant(w), x.double()
    ref, size = X @ W.T, X.abs() @ W.abs().T
    last = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    assert y.dtype == out_dtype
    assert bool(((y.double() - ref).abs() <= SUM * size + last * ref.abs()).all())
    return y


@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 17, 64), (2, 16, 96), (3, 100, 128), (8, 33, 1056), (9, 48, 2048),
                                   (16, 257, 160), (1, 1536, 2048), (5, 768, 4128), (13, 40, 12288)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_product(m, n, k, out_dtype):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = torch.randn((m, k + 8 * (m % 2)), generator=g, device=DEV).to(torch.bfloat16)[:, :k]
    _check(x, _weight(n, k, n * k), out_dtype)


def test_quantized_weight_and_wide_activations():
    """A weight from the library's quantizer; activations over many binades."""
    g = torch.Generator(device=DEV).manual_seed(1)
    w = (torch.randn((200, 512), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    q = jq.quant_nvfp4(w, scope_amax=jq.amax_bf16(w))
    x = torch.randn((4, 512), generator=g, device=DEV) * torch.exp2(
        torch.randint(-60, 60, (4, 512), generator=g, device=DEV).float())
    _check(x.to(torch.bfloat16), q, torch.float32)


def test_each_code_and_scale_is_exact():
    """One nonzero activation: y is the dequantized weight itself, for all 16 codes and all finite scales."""
    scales = torch.arange(127, device=DEV, dtype=torch.uint8)
    codes = torch.arange(8, device=DEV, dtype=torch.uint8)
    q = (2 * codes + 16 * (2 * codes + 1)).repeat(127, 2)  # codes 0..15, twice: 32 columns
    w = dict(q=q.contiguous(), sb=scales[:, None].repeat(1, 2).contiguous(), sg=torch.ones(1, device=DEV))
    W = _dequant(w)
    for col in range(0, 32, 16):
        x = torch.zeros((16, 32), dtype=torch.bfloat16, device=DEV)
        x[torch.arange(16), col + torch.arange(16)] = 1.0
        y = jq.gemv_nvfp4(x, w)
        assert torch.equal(y.double(), W[:, col:col + 16].T)


def test_tokens_do_not_mix():
    """A NaN or infinite activation stays in its own row, and a batch's rows are each token's own product."""
    w = _weight(64, 256, 2)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((16, 256), generator=g, device=DEV).to(torch.bfloat16)
    y = jq.gemv_nvfp4(x, w)
    for i in (0, 7, 8, 15):
        assert torch.equal(jq.gemv_nvfp4(x[i:i + 1], w)[0], y[i])
    x[5, 9], x[12, 0] = float("nan"), float("inf")
    z = jq.gemv_nvfp4(x, w)
    keep = [i for i in range(16) if i not in (5, 12)]
    assert torch.equal(z[keep], y[keep]) and bool(torch.isnan(z[5]).all())
    assert bool((~torch.isfinite(z[12])).all())


def test_stream_graph_strided_output_and_no_tokens():
    w = _weight(100, 512, 4)
    x = torch.randn((3, 512), device=DEV).to(torch.bfloat16)
    y = jq.gemv_nvfp4(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = jq.gemv_nvfp4(x, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = jq.gemv_nvfp4(x, w)
    graph.replay()
    out = torch.full((3, 103), 7.0, device=DEV)
    jq.jetq_gemv_nvfp4(w["q"], w["sb"], w["sg"], x, out[:, 1:101])
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(y, y2) and torch.equal(y, out[:, 1:101])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 101:] == 7).all())
    assert jq.gemv_nvfp4(x[:0], w).shape == (0, 100)


def test_offsets_past_32_bits():
    """A weight of 2.5e9 bytes of codes: its first and its last rows."""
    n, k = 1_200_003, 4096
    q = torch.randint(0, 256, (n, k // 2), device=DEV, dtype=torch.uint8)
    sb = torch.randint(0, 127, (n, k // 16), device=DEV, dtype=torch.uint8)
    w = dict(q=q, sb=sb, sg=torch.tensor([3.1e-4], device=DEV))
    x = torch.randn((3, k), device=DEV).to(torch.bfloat16)
    y = jq.gemv_nvfp4(x, w)
    for a in (0, 2 ** 31 // (k // 2) - 20, n - 40):
        W = _dequant(dict(q=q[a:a + 40], sb=sb[a:a + 40], sg=w["sg"]))
        ref, size = x.double() @ W.T, x.double().abs() @ W.abs().T
        assert bool(((y[:, a:a + 40].double() - ref).abs() <= SUM * size + 2.0 ** -24 * ref.abs()).all())
