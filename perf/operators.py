"""The head of a model as training and rollout run it: cases, plain forms and definitions.

Three operators, each with the directions that a training step or a rollout
step needs:

  ce_fwd, ce_bwd      token losses (log-probabilities) of a linear head with
                      softmax over a large vocabulary, without keeping the
                      logits; gradients of the hidden states and of the head
  norm_fwd, norm_bwd  layer norm and RMS norm; backward pass with the weight's
                      and the bias's gradient
  gemv                few-token product with NVFP4 weights (E2M1 codes, one
                      E4M3 scale per 16 values, one FP32 scale) and BF16
                      activations

`listed()` and `draw()` give cases, `prepare()` what a caller has in hand,
`run()` one pass (plain torch operations, or the library's calls where `own`
is true), `exact()` the definitions in binary64, `work()` the bytes and
operations that a pass cannot do without.
"""
import math

import torch

own = False

_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        import rollout_x128_act_gb300

        _LIB = rollout_x128_act_gb300
    return _LIB


# ------------------------------------------------------------------ cases

def listed():
    return [
        # scoring the one token a rollout has just sampled: a head of 32000 rows is read once
        dict(name="ce_fwd_token", op="ce_fwd", n=1, v=32000, c=4096, scale=1.0, uniform=True),
        # log-probabilities of a short ragged answer, vocabulary of odd length, sampling temperature 0.7
        dict(name="ce_fwd_answer", op="ce_fwd", n=333, v=50257, c=2048, scale=1.0 / 0.7, uniform=True),
        # log-probabilities of a training micro-batch at the dense 8B hidden size
        dict(name="ce_fwd_batch", op="ce_fwd", n=4096, v=131072, c=4096, scale=1.0, uniform=True),
        # gradient of a small ragged batch with per-token weights (advantages), odd everything
        dict(name="ce_bwd_ragged", op="ce_bwd", n=1000, v=50257, c=1032, scale=1.0, uniform=False),
        # gradient of the training micro-batch, mean loss
        dict(name="ce_bwd_batch", op="ce_bwd", n=4096, v=131072, c=4096, scale=1.0, uniform=True),
        # the final norm of one decoded token
        dict(name="norm_fwd_token", op="norm_fwd", kind="rms", dtype="bf16", n=1, c=4096, bias=False),
        # the norm of a training batch
        dict(name="norm_fwd_batch", op="norm_fwd", kind="layer", dtype="bf16", n=16384, c=4096, bias=True),
        # its backward pass, at the 30B-A3B hidden size
        dict(name="norm_bwd_batch", op="norm_bwd", kind="rms", dtype="bf16", n=32768, c=2048, bias=False),
        # FP32 activations, odd width and row count
        dict(name="norm_bwd_odd", op="norm_bwd", kind="layer", dtype="f32", n=3001, c=1111, bias=True),
        # one token through an expert's gate/up projection
        dict(name="gemv_expert", op="gemv", m=1, n=1536, k=2048, out="bf16"),
        # one token through a dense 8B up projection
        dict(name="gemv_up", op="gemv", m=1, n=12288, k=4096, out="bf16"),
        # eight sequences in flight through the down projection
        dict(name="gemv_down8", op="gemv", m=8, n=4096, k=12288, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce_fwd", "ce_bwd", "norm_fwd", "norm_bwd", "gemv"])
    if op in ("ce_fwd", "ce_bwd"):
        n = _log_int(rng, 1 if op == "ce_fwd" else 64, 4096)
        v = _log_int(rng, 1000, 131072)
        c = 8 * _log_int(rng, 32, 512)
        return dict(op=op, n=n, v=v, c=c, scale=round(rng.uniform(0.7, 1.5), 3), uniform=rng.random() < 0.5)
    if op in ("norm_fwd", "norm_bwd"):
        kind = rng.choice(["layer", "rms"])
        return dict(op=op, kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), n=_log_int(rng, 1, 32768),
                    c=_log_int(rng, 64, 8192), bias=kind == "layer" and rng.random() < 0.8)
    return dict(op=op, m=rng.randint(1, 16), n=_log_int(rng, 256, 16384), k=32 * _log_int(rng, 16, 512),
                out=rng.choice(["bf16", "f32"]))


def work(case):
    op = case["op"]
    if op in ("ce_fwd", "ce_bwd"):
        n, v, c = case["n"], case["v"], case["c"]
        if op == "ce_fwd":  # x, w, targets in; loss, lse out
            return {"bytes": 2 * n * c + 2 * v * c + 16 * n, "flops": 2 * n * v * c}
        # x, w, targets, lse, dloss in; dx, dw out; the logits again, then the two products
        return {"bytes": 4 * n * c + 4 * v * c + 16 * n, "flops": 6 * n * v * c}
    if op in ("norm_fwd", "norm_bwd"):
        n, c, e = case["n"], case["c"], 2 if case["dtype"] == "bf16" else 4
        stats = (8 if case["kind"] == "layer" else 4) * n
        params = (2 if case["bias"] else 1) * c
        if op == "norm_fwd":
            return {"bytes": 2 * n * c * e + stats + params * e, "flops": 8 * n * c}
        return {"bytes": 3 * n * c * e + stats + c * e + params * 4, "flops": 14 * n * c}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": n * k // 2 + n * k // 16 + 2 * m * k + (2 if case["out"] == "bf16" else 4) * m * n,
            "flops": 2 * m * n * k}


# ------------------------------------------------------------------ inputs

_DEV = "cuda"
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes by code


def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed) * 7919 + 17)


def _rows(n, c, dtype, g, sigma=1.0, mu=0.0):
    """[n x c] values in rows whose stride keeps every row 16-byte aligned."""
    step = 8 if dtype == torch.bfloat16 else 4
    ld = -(-c // step) * step
    t = torch.empty((n, ld), dtype=dtype, device=_DEV)
    t.copy_(torch.randn((n, ld), generator=g, device=_DEV).mul_(sigma).add_(mu))
    return t[:, :c]


def _prepare_ce(case, seed):
    n, v, c = case["n"], case["v"], case["c"]
    g = _gen(seed)
    w = torch.empty((v, c), dtype=torch.bfloat16, device=_DEV)
    for a in range(0, v, 16384):  # in pieces: no large FP32 copy
        b = min(v, a + 16384)
        w[a:b] = torch.randn((b - a, c), generator=g, device=_DEV) * 0.02
    target = torch.randint(0, v, (n,), generator=g, device=_DEV)
    # normed hidden states that lean towards their token's row, from not at all to a logit that rivals all others'
    # sum: unsure and confident tokens
    lean = (math.log(v) + 1.0) * torch.rand((n, 1), generator=g, device=_DEV)
    row = w[target].float()
    x = torch.randn((n, c), generator=g, device=_DEV) + lean * row / row.square().sum(1, keepdim=True)
    x = (x * (c / x.square().sum(1, keepdim=True)).sqrt()).to(torch.bfloat16)
    if n > 8:  # prompt tokens carry no loss
        target[: n // 8] = -100
    s = dict(case=case, x=x, w=w, target=target)
    if case["op"] == "ce_bwd":
        valid = target >= 0
        s["dloss"] = (torch.ones(n, device=_DEV) if case["uniform"] else torch.randn(n, generator=g, device=_DEV)) / n
        lse = torch.empty(n, device=_DEV)
        for a in range(0, n, 512):
            z = (x[a:a + 512].float() @ w.float().T) * case["scale"]
            top = z.amax(1, keepdim=True)
            lse[a:a + 512] = ((z - top).exp().sum(1).log() + top[:, 0])
        s["lse"] = torch.where(valid, lse, torch.zeros_like(lse))
    return s


def _prepare_norm(case, seed):
    n, c = case["n"], case["c"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    g = _gen(seed)
    s = dict(case=case, x=_rows(n, c, dtype, g, 1.5, 0.3),
             w=(1.0 + 0.1 * torch.randn(c, generator=g, device=_DEV)).to(dtype), b=None, eps=1e-5)
    if case["bias"]:
        s["b"] = (0.1 * torch.randn(c, generator=g, device=_DEV)).to(dtype)
    if case["op"] == "norm_bwd":
        s["dy"] = _rows(n, c, dtype, g, 1e-2)
        x = s["x"].double()
        s["mean"] = x.mean(1).float() if case["kind"] == "layer" else None
        var = (x - x.mean(1, keepdim=True)).square().mean(1) if case["kind"] == "layer" else x.square().mean(1)
        s["rstd"] = (1.0 / (var + s["eps"]).sqrt()).float()
    return s


def _prepare_gemv(case, seed):
    m, n, k = case["m"], case["n"], case["k"]
    g = _gen(seed)
    w = torch.randn((n, k), generator=g, device=_DEV) * 0.02
    sg = (w.abs().amax() / 2688.0).reshape(1)
    blocks = w.view(n, k // 16, 16)
    sb = (blocks.abs().amax(2) / 6.0 / sg).to(torch.float8_e4m3fn)
    step = (sb.float() * sg).unsqueeze(2)
    ratio = torch.where(step > 0, blocks / step, torch.zeros_like(blocks))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=_DEV)
    code = torch.bucketize(ratio.abs(), edges).to(torch.uint8) + 8 * (ratio < 0).to(torch.uint8)
    code = code.view(n, k)
    x = torch.randn((m, k), generator=g, device=_DEV).to(torch.bfloat16)
    return dict(case=case, x=x, w=dict(q=(code[:, 0::2] + 16 * code[:, 1::2]).contiguous(),
                                       sb=sb.view(torch.uint8).contiguous(), sg=sg))


def prepare(case, seed):
    op = case["op"]
    if op in ("ce_fwd", "ce_bwd"):
        return _prepare_ce(case, seed)
    if op in ("norm_fwd", "norm_bwd"):
        return _prepare_norm(case, seed)
    return _prepare_gemv(case, seed)


# ------------------------------------------------------------------ plain forms (32 bits)

def _plain_logits(s):
    return (s["x"].float() @ s["w"].float().T) * s["case"]["scale"]


def _plain_ce_fwd(s):
    z, target = _plain_logits(s), s["target"]
    valid = target >= 0
    top = z.amax(1, keepdim=True)
    zt = z.gather(1, target.clamp(min=0).unsqueeze(1))[:, 0]
    lse = (z - top).exp_().sum(1).log() + top[:, 0]
    zero = torch.zeros_like(lse)
    return dict(loss=torch.where(valid, lse - zt, zero), lse=lse)


def _plain_ce_bwd(s):
    target, scale = s["target"], s["case"]["scale"]
    valid = target >= 0
    d = _plain_logits(s).sub_(s["lse"].unsqueeze(1)).exp_()
    row = torch.arange(target.numel(), device=d.device)
    d[row, target.clamp(min=0)] -= 1.0
    d *= torch.where(valid, s["dloss"] * scale, torch.zeros_like(s["dloss"])).unsqueeze(1)
    return dict(dx=(d @ s["w"].float()).to(torch.bfloat16), dw=(d.T @ s["x"].float()).to(torch.bfloat16))


def _plain_norm_fwd(s):
    x = s["x"].float()
    layer = s["case"]["kind"] == "layer"
    mean = x.mean(1) if layer else None
    h = x - mean.unsqueeze(1) if layer else x
    rstd = 1.0 / (h.square().mean(1) + s["eps"]).sqrt()
    y = h * rstd.unsqueeze(1) * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    layer = s["case"]["kind"] == "layer"
    h = (x - s["mean"].unsqueeze(1)) * rstd if layer else x * rstd
    t = dy * s["w"].float()
    dx = t - h * (t * h).mean(1, keepdim=True)
    if layer:
        dx = dx - t.mean(1, keepdim=True)
    return dict(dx=(dx * rstd).to(s["x"].dtype), dw=(dy * h).sum(0), db=dy.sum(0) if s["b"] is not None else None)


def _plain_gemv(s):
    w = s["w"]
    code = torch.stack((w["q"] & 15, w["q"] >> 4), 2).flatten(1).long()
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=code.device)
    step = w["sb"].view(torch.float8_e4m3fn).float() * w["sg"]
    full = grid[code] * step.repeat_interleave(16, 1)
    return (s["x"].float() @ full.T).to(torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"ce_fwd": _plain_ce_fwd, "ce_bwd": _plain_ce_bwd, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd, "gemv": _plain_gemv}[op](s)
    jq = _lib()
    if op == "ce_fwd":
        loss, lse = jq.linear_ce(s["x"], s["w"], s["target"], scale=s["case"]["scale"])
        return dict(loss=loss, lse=lse)
    if op == "ce_bwd":
        dx, dw = jq.linear_ce_bwd(s["x"], s["w"], s["target"], s["lse"], s["dloss"], scale=s["case"]["scale"],
                                  dw_dtype=torch.bfloat16)
        return dict(dx=dx, dw=dw)
    if op == "norm_fwd":
        kind = jq.NORM_LAYER if s["case"]["kind"] == "layer" else jq.NORM_RMS
        y, mean, rstd = jq.norm_fwd(s["x"], s["w"], s["b"], eps=s["eps"], kind=kind)
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "norm_bwd":
        kind = jq.NORM_LAYER if s["case"]["kind"] == "layer" else jq.NORM_RMS
        dx, dw, db = jq.norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], kind=kind, bias=s["b"] is not None)
        return dict(dx=dx, dw=dw, db=db)
    return jq.gemv_nvfp4(s["x"], s["w"], out_dtype=torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32)


# ------------------------------------------------------------------ definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ce_fwd", "ce_bwd"):
        x, target = s["x"].double(), s["target"]
        n, v = case["n"], case["v"]
        hot = torch.arange(n, device=x.device)[target >= 0]
        if op == "ce_fwd":
            lse = torch.full((n,), -math.inf, dtype=torch.float64, device=x.device)
            zt = torch.zeros(n, dtype=torch.float64, device=x.device)
            for a in range(0, v, 8192):
                z = case["scale"] * torch.mm(x, s["w"][a:a + 8192].double().T)
                lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
                here = hot[(target[hot] >= a) & (target[hot] < a + 8192)]
                zt[here] = z[here, target[here] - a]
            loss = torch.zeros_like(lse)
            loss[hot] = lse[hot] - zt[hot]
            return dict(loss=loss, lse=lse)
        coef = torch.zeros(n, dtype=torch.float64, device=x.device)
        coef[hot] = s["dloss"][hot].double() * case["scale"]
        dx, dw = torch.zeros_like(x), []
        for a in range(0, v, 8192):
            w = s["w"][a:a + 8192].double()
            p = coef[:, None] * torch.exp(case["scale"] * torch.mm(x, w.T) - s["lse"].double()[:, None])
            here = hot[(target[hot] >= a) & (target[hot] < a + 8192)]
            p[here, target[here] - a] -= coef[here]
            dx += torch.mm(p, w)
            dw.append(torch.mm(p.T, x))
        return dict(dx=dx, dw=torch.cat(dw))
    if op in ("norm_fwd", "norm_bwd"):
        x, w = s["x"].double(), s["w"].double()
        n, c = x.shape
        layer = case["kind"] == "layer"
        if op == "norm_fwd":
            mean = x.sum(1) / c if layer else torch.zeros(n, dtype=torch.float64, device=x.device)
            rstd = ((x - mean[:, None]).pow(2).sum(1) / c + s["eps"]).rsqrt()
            y = torch.einsum("nc,n,c->nc", x - mean[:, None], rstd, w)
            return dict(y=y if s["b"] is None else y + s["b"].double(), mean=mean if layer else None, rstd=rstd)
        dy, rstd = s["dy"].double(), s["rstd"].double()
        h = torch.einsum("nc,n->nc", x - s["mean"].double()[:, None] if layer else x, rstd)
        along = torch.einsum("nc,nc,c->n", dy, h, w) / c
        dx = dy * w - along[:, None] * h - (torch.mv(dy, w)[:, None] / c if layer else 0.0)
        return dict(dx=rstd[:, None] * dx, dw=torch.einsum("nc,nc->c", dy, h),
                    db=dy.sum(0) if s["b"] is not None else None)
    q, n, k = s["w"]["q"], case["n"], case["k"]
    table = torch.tensor([(-1.0 if i & 8 else 1.0) * _GRID[i & 7] for i in range(16)], dtype=torch.float64,
                         device=q.device)
    even, odd = table[(q % 16).int()], table[(q // 16).int()]
    x = s["x"].double()
    xe, xo = x[:, 0::2].reshape(-1, k // 16, 8), x[:, 1::2].reshape(-1, k // 16, 8)
    scale = s["w"]["sb"].view(torch.float8_e4m3fn).double() * s["w"]["sg"].double()
    part = torch.einsum("nbi,mbi->mnb", even.view(n, k // 16, 8), xe)
    part += torch.einsum("nbi,mbi->mnb", odd.view(n, k // 16, 8), xo)
    return torch.einsum("mnb,nb->mn", part, scale)
