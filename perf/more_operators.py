"""The losses of reinforcement learning and distillation, and a mixture-of-experts layer in decoding: cases,
plain forms and definitions.

  policy        clipped policy-gradient loss of packed sequences with a KL term against a reference policy, and
                its gradient with respect to the token losses (minus log-probabilities); ratios of tokens or of
                whole sequences
  distill_fwd,  KL divergence of a linear head's softmax from a teacher known by its top logits, without keeping
  distill_bwd   the student's logits; gradients of the hidden states and of the head
  moe           a whole mixture-of-experts layer (router, gate/up, SwiGLU, down, weighted sum) for 1 to 16 tokens
                with NVFP4 expert weights

`listed()` and `draw()` give cases, `prepare()` what a caller has in hand, `run()` one pass (plain torch
operations, or the library's calls where `own` is true), `exact()` the definitions in binary64, `work()` the
bytes and operations that a pass cannot do without.
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
        # one prompt's group of 8 short answers, KL term, means of sequences
        dict(name="policy_group", op="policy", n=1531, nseg=8, level="token", mean="segs", adv="seg", ref=True,
             mask=True, low=0.2, high=0.2, dual=0.0, kl=0.04),
        # a rollout step's 512 answers of about 1024 tokens, wider upper clip, mean over all tokens, no reference
        dict(name="policy_batch", op="policy", n=524288, nseg=512, level="token", mean="tokens", adv="seg", ref=False,
             mask=True, low=0.2, high=0.28, dual=0.0, kl=0.0),
        # few long answers with an advantage a token, KL term and a bound on negative advantages' ratios
        dict(name="policy_long", op="policy", n=1000003, nseg=24, level="token", mean="tokens", adv="token", ref=True,
             mask=True, low=0.2, high=0.2, dual=3.0, kl=0.001),
        # 8192 answers with one ratio a sequence, clipped tightly
        dict(name="policy_seqs", op="policy", n=4194304, nseg=8192, level="segment", mean="segs", adv="seg", ref=True,
             mask=False, low=0.0003, high=0.0004, dual=0.0, kl=0.01),
        # the distance to the teacher at one sampled token: the head is read once
        dict(name="distill_fwd_token", op="distill_fwd", n=1, v=32000, c=4096, k=32, scale=1.0, renorm=True),
        # a training micro-batch at the dense 8B hidden size, teacher's 64 best of the whole vocabulary
        dict(name="distill_fwd_batch", op="distill_fwd", n=2048, v=131072, c=4096, k=64, scale=1.0, renorm=False),
        # gradient of a small ragged batch, temperature 1.5, odd everything
        dict(name="distill_bwd_ragged", op="distill_bwd", n=777, v=50257, c=1032, k=20, scale=1.0 / 1.5, renorm=True),
        # gradient of the micro-batch
        dict(name="distill_bwd_batch", op="distill_bwd", n=2048, v=131072, c=4096, k=64, scale=1.0, renorm=False),
        # one token through a layer of the 30B-A3B shape
        dict(name="moe_token", op="moe", m=1, e=128, h=2048, inter=768, topk=8, renorm=True, out="bf16"),
        # five sequences, a small layer of odd sizes, FP32 out
        dict(name="moe_small", op="moe", m=5, e=20, h=1056, inter=352, topk=3, renorm=False, out="f32"),
        # sixteen sequences in flight
        dict(name="moe_tokens16", op="moe", m=16, e=128, h=2048, inter=768, topk=8, renorm=True, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "policy", "distill_fwd", "distill_bwd", "moe", "moe"])
    if op == "policy":
        n = _log_int(rng, 64, 1 << 22)
        level = rng.choice(["token", "token", "segment"])
        tight = level == "segment" and rng.random() < 0.7
        return dict(op=op, n=n, nseg=_log_int(rng, 1, max(1, n // 8)) if n < 65536 else _log_int(rng, 8, n // 128),
                    level=level, mean=rng.choice(["tokens", "segs", "sum"]), adv=rng.choice(["seg", "token"]),
                    ref=rng.random() < 0.6, mask=rng.random() < 0.6, low=0.0003 if tight else 0.2,
                    high=0.0004 if tight else rng.choice([0.2, 0.28]), dual=rng.choice([0.0, 0.0, 3.0]),
                    kl=rng.choice([0.001, 0.04]))
    if op in ("distill_fwd", "distill_bwd"):
        n = _log_int(rng, 1 if op == "distill_fwd" else 64, 2048)
        return dict(op=op, n=n, v=_log_int(rng, 1000, 131072), c=8 * _log_int(rng, 32, 512), k=_log_int(rng, 1, 128),
                    scale=round(rng.uniform(0.5, 1.5), 3), renorm=rng.random() < 0.5)
    e = _log_int(rng, 4, 128)
    return dict(op=op, m=rng.randint(1, 16), e=e, h=32 * _log_int(rng, 8, 64), inter=32 * _log_int(rng, 4, 24),
                topk=rng.randint(1, min(e, 8)), renorm=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


def work(case):
    op = case["op"]
    if op == "policy":
        n, s = case["n"], case["nseg"]
        token = 8 + (4 if case["ref"] else 0) + (1 if case["mask"] else 0) + (4 if case["adv"] == "token" else 0)
        return {"bytes": n * (token + 4) + s * (8 + (4 if case["adv"] == "seg" else 0)) + 24, "flops": 40 * n}
    if op in ("distill_fwd", "distill_bwd"):
        n, v, c, k = case["n"], case["v"], case["c"], case["k"]
        if op == "distill_fwd":  # x, w, ids, teacher in; loss, lse, log-probabilities at the ids out
            return {"bytes": 2 * n * c + 2 * v * c + 16 * n * k + 8 * n, "flops": 2 * n * v * c}
        # x, w, ids, teacher, log-probabilities, lse, dloss in; dx, dw out; the logits again, then the two products
        return {"bytes": 4 * n * c + 4 * v * c + 16 * n * k + 8 * n, "flops": 6 * n * v * c}
    m, e, h, i, k = case["m"], case["e"], case["h"], case["inter"], case["topk"]
    used = e * (1.0 - (1.0 - k / e) ** m)  # experts that some token takes, on average
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": int(used * 3 * h * i * 9 / 16) + 2 * e * h + m * (2 * h + out * h + 12 * k),
            "flops": 6 * m * k * h * i + 2 * m * e * h}


# ------------------------------------------------------------------ inputs

_DEV = "cuda"
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes by code


def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed) * 6151 + 29)


def _prepare_policy(case, seed):
    n, s = case["n"], case["nseg"]
    g = _gen(seed)
    # ragged lengths (some sequences may be empty), and rows behind the last sequence: a padded batch
    used = n - n // 50
    share = torch.randn(s, generator=g, device=_DEV).mul_(0.7).exp_().double()
    ends = (share.cumsum(0) / share.sum() * used).round_().long()
    ends[-1] = used
    off = torch.cat((torch.zeros(1, dtype=torch.int64, device=_DEV), ends))
    old = torch.empty(n, device=_DEV).exponential_(1.5, generator=g)
    nll = old + 0.12 * torch.randn(n, generator=g, device=_DEV)
    st = dict(case=case, off=off, old=old, nll=nll, ref=None, mask=None)
    if case["ref"]:
        st["ref"] = old + 0.2 * torch.randn(n, generator=g, device=_DEV)
    if case["mask"]:  # prompt tokens and tool output
        st["mask"] = torch.rand(n, generator=g, device=_DEV) < 0.8
    st["adv"] = torch.randn(n if case["adv"] == "token" else s, generator=g, device=_DEV)
    return st


def _student_logits(x, w, scale):
    return (x.float() @ w.float().T).mul_(scale)


def _prepare_distill(case, seed):
    n, v, c, k = case["n"], case["v"], case["c"], case["k"]
    g = _gen(seed)
    w = torch.empty((v, c), dtype=torch.bfloat16, device=_DEV)
    for a in range(0, v, 16384):  # in pieces: no large FP32 copy
        b = min(v, a + 16384)
        w[a:b] = torch.randn((b - a, c), generator=g, device=_DEV) * 0.02
    # normed hidden states that lean towards some row of the head: unsure and confident tokens
    near = torch.randint(0, v, (n,), generator=g, device=_DEV)
    lean = (math.log(v) + 1.0) * torch.rand((n, 1), generator=g, device=_DEV)
    row = w[near].float()
    x = torch.randn((n, c), generator=g, device=_DEV) + lean * row / row.square().sum(1, keepdim=True)
    x = (x * (c / x.square().sum(1, keepdim=True)).sqrt()).to(torch.bfloat16)
    # the teacher's logits are the student's, moved; its best k of them are known
    ids = torch.empty((n, k), dtype=torch.int64, device=_DEV)
    teacher = torch.empty((n, k), device=_DEV)
    lse, logp = torch.empty(n, device=_DEV), torch.empty((n, k), device=_DEV)
    for a in range(0, n, 512):
        z = _student_logits(x[a:a + 512], w, case["scale"])
        t = z + 0.5 * torch.randn(z.shape, generator=g, device=_DEV)
        top, at = t.topk(k, dim=1)
        if not case["renorm"]:  # log-probabilities over the whole vocabulary
            m = t.amax(1, keepdim=True)
            top = top - ((t - m).exp_().sum(1, keepdim=True).log() + m)
        m = z.amax(1, keepdim=True)
        lse[a:a + 512] = ((z - m).exp().sum(1, keepdim=True).log() + m)[:, 0]
        logp[a:a + 512] = z.gather(1, at) - lse[a:a + 512, None]
        ids[a:a + 512], teacher[a:a + 512] = at, top
    if n > 8:  # prompt tokens carry no loss; some rows have fewer entries than others
        ids[: n // 8] = -1
        short = torch.randint(1, k + 1, (n,), generator=g, device=_DEV)
        ids.masked_fill_(torch.arange(k, device=_DEV)[None] >= short[:, None], -1)
    st = dict(case=case, x=x, w=w, ids=ids, teacher=teacher)
    if case["op"] == "distill_bwd":
        st["lse"] = lse
        st["logp"] = torch.where(ids >= 0, logp, torch.zeros_like(logp))
        st["dloss"] = torch.full((n,), 1.0 / n, device=_DEV)
    return st


def _quant_experts(e, rows, cols, g):
    """Random weights [e x rows x cols] in NVFP4: codes, scales of 16 values, a scale an expert."""
    q = torch.empty((e, rows, cols // 2), dtype=torch.uint8, device=_DEV)
    sb = torch.empty((e, rows, cols // 16), dtype=torch.uint8, device=_DEV)
    sg = torch.empty(e, device=_DEV)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=_DEV)
    step = max(1, (1 << 24) // (rows * cols))
    for a in range(0, e, step):
        b = min(e, a + step)
        w = torch.randn((b - a, rows, cols // 16, 16), generator=g, device=_DEV) * cols ** -0.5
        top = w.abs().amax(3)
        scope = top.amax((1, 2)) / 2688.0
        scale = (top / 6.0 / scope[:, None, None]).to(torch.float8_e4m3fn)
        unit = (scale.float() * scope[:, None, None]).unsqueeze(3)
        w = torch.where(unit > 0, w / unit, torch.zeros_like(w))
        code = (torch.bucketize(w.abs(), edges).to(torch.uint8) + 8 * (w < 0).to(torch.uint8)).flatten(2)
        q[a:b] = code[:, :, 0::2] + 16 * code[:, :, 1::2]
        sb[a:b] = scale.view(torch.uint8)
        sg[a:b] = scope
    return dict(q=q, sb=sb, sg=sg)


def _prepare_moe(case, seed):
    m, e, h, i = case["m"], case["e"], case["h"], case["inter"]
    g = _gen(seed)
    return dict(case=case, x=torch.randn((m, h), generator=g, device=_DEV).to(torch.bfloat16),
                router=(torch.randn((e, h), generator=g, device=_DEV) * (1.5 * h ** -0.5)).to(torch.bfloat16),
                w13=_quant_experts(e, 2 * i, h, g), w2=_quant_experts(e, h, i, g))


def prepare(case, seed):
    op = case["op"]
    if op == "policy":
        return _prepare_policy(case, seed)
    if op in ("distill_fwd", "distill_bwd"):
        return _prepare_distill(case, seed)
    return _prepare_moe(case, seed)


# ------------------------------------------------------------------ plain forms (32 bits)

def _plain_policy(s):
    case, off = s["case"], s["off"]
    n, nseg = case["n"], case["nseg"]
    seg = torch.bucketize(torch.arange(n, device=off.device), off[1:], right=True)  # nseg: behind the last
    on = seg < nseg
    if s["mask"] is not None:
        on = on & s["mask"]
    idx = seg.clamp(max=nseg - 1)
    adv = s["adv"] if case["adv"] == "token" else s["adv"][idx]
    logr = s["old"].double() - s["nll"].double()  # in 64 bits: which side of the clip's border
    zero = torch.zeros(n, device=off.device)

    def seg_sum(x):
        out = torch.zeros(nseg, dtype=x.dtype, device=x.device)
        return out.index_add_(0, idx, torch.where(on, x, torch.zeros_like(x)))

    count = seg_sum(torch.ones(n, device=off.device))
    tokens, segs = count.sum(), (count > 0).sum().float()
    if case["level"] == "segment":
        logr = (seg_sum(logr) / count.clamp(min=1.0))[idx]
    ratio, border = logr.exp().float(), logr.exp()
    low, high = border < 1.0 - case["low"], border > 1.0 + case["high"]
    clipped = torch.where(adv < 0, low, high)
    bound = torch.where(adv < 0, torch.full_like(ratio, 1.0 - case["low"]), torch.full_like(ratio, 1.0 + case["high"]))
    if case["dual"] > 0:
        over = (adv < 0) & (border > case["dual"])
        clipped = clipped | over
        bound = torch.where(over, torch.full_like(ratio, case["dual"]), bound)
    loss = -adv * torch.where(clipped, bound, ratio)
    grad = torch.where(clipped, zero, adv * ratio)
    if case["level"] == "segment":
        grad = (seg_sum(grad.double()) / count.clamp(min=1.0)).float()[idx]
    if case["mean"] == "tokens":
        weight = (on / tokens.clamp(min=1.0)).float()
    elif case["mean"] == "segs":
        weight = torch.where(on, 1.0 / (count[idx].clamp(min=1.0) * segs.clamp(min=1.0)), zero)
    else:
        weight = on.float()
    dnll, kl = grad, zero
    if s["ref"] is not None:
        d = s["nll"].double() - s["ref"].double()  # in 64 bits: exp(d) - 1 - d cancels
        kl = (d.exp() - 1.0 - d).float()
        dnll = grad + case["kl"] * torch.expm1(d).float()
    # long sums of either sign, in 64 bits
    surrogate, klsum = (weight.double() * loss).sum(), (weight.double() * kl).sum()
    means = torch.stack((surrogate + case["kl"] * klsum, surrogate, klsum)).float()
    return dict(means=means, counts=torch.stack(((on & clipped).sum().float(), tokens, segs)), dnll=weight * dnll)


def _teacher_probs(s):
    """q [n x k] and log q of the listed entries (zero and zero elsewhere)."""
    on, t = s["ids"] >= 0, s["teacher"].double()
    off = torch.full_like(t, -math.inf)
    t = torch.where(on, t, off)
    if s["case"]["renorm"]:
        top = t.amax(1, keepdim=True).clamp(min=-1e30)
        t = t - top - (t - top).exp().sum(1, keepdim=True).clamp(min=1e-30).log()
    zero = torch.zeros_like(t)
    return torch.where(on, t.exp(), zero), torch.where(on, t, zero)


def _plain_distill_fwd(s):
    x, w = s["x"].float(), s["w"].float()
    z = torch.zeros((x.shape[0], w.shape[0]), device=x.device)
    for a in range(0, x.shape[1], 256):  # short sums: the loss is a small difference of logits
        z.addmm_(x[:, a:a + 256], w[:, a:a + 256].T)
    z *= s["case"]["scale"]
    top = z.amax(1, keepdim=True)
    zt = z.gather(1, s["ids"].clamp(min=0))
    # the n x k values that are left, in 64 bits: logits and log q nearly cancel
    lse = (z - top).exp_().sum(1).double().log() + top[:, 0].double()
    q, logq = _teacher_probs(s)
    logp = torch.where(s["ids"] >= 0, zt.double() - lse[:, None], torch.zeros_like(lse)[:, None])
    return dict(loss=(q * (logq - logp)).sum(1).float(), lse=lse.float(), logp=logp.float())


def _plain_distill_bwd(s):
    ids, scale = s["ids"], s["case"]["scale"]
    q, _ = _teacher_probs(s)
    d = _student_logits(s["x"], s["w"], scale).sub_(s["lse"][:, None]).exp_().mul_(q.sum(1, keepdim=True).float())
    d.scatter_add_(1, ids.clamp(min=0), -q.float())
    d *= (s["dloss"] * scale)[:, None]
    d *= (ids >= 0).any(1, keepdim=True)
    return dict(dx=(d @ s["w"].float()).to(torch.bfloat16), dw=(d.T @ s["x"].float()).to(torch.bfloat16))


def _dequant(w, e):
    """FP32 values of the expert weights e (any shape of indexes)."""
    q = w["q"][e]
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2).int()
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=q.device)
    step = w["sb"][e].view(torch.float8_e4m3fn).float() * w["sg"][e][..., None, None]
    return grid[code] * step.repeat_interleave(16, -1)


def _plain_moe(s):
    case, x = s["case"], s["x"].float()
    logits = (s["x"].double() @ s["router"].double().T).float()  # in 64 bits: which expert is the next
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    k = case["topk"]
    ids, top = ids[:, :k], top[:, :k]
    p = (top - top[:, :1]).exp()
    p = p / (p.sum(1, keepdim=True) if case["renorm"] else (logits - top[:, :1]).exp().sum(1, keepdim=True))
    y = torch.zeros_like(x)
    for j in range(k):  # one choice of every token at a time
        gu = (_dequant(s["w13"], ids[:, j]) @ x[:, :, None])[:, :, 0]
        gate, up = gu.chunk(2, dim=1)
        act = gate / (1.0 + (-gate).exp()) * up
        y += p[:, j:j + 1] * (_dequant(s["w2"], ids[:, j]) @ act[:, :, None])[:, :, 0]
    return dict(y=y.to(torch.bfloat16) if case["out"] == "bf16" else y, ids=ids, p=p)


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"policy": _plain_policy, "distill_fwd": _plain_distill_fwd, "distill_bwd": _plain_distill_bwd,
                "moe": _plain_moe}[op](s)
    jq = _lib()
    if op == "policy":
        kw = dict(seg_offsets=s["off"], nll_ref=s["ref"], mask=s["mask"], clip_low=case["low"],
                  clip_high=case["high"], clip_dual=case["dual"], kl=case["kl"],
                  level={"token": jq.POLICY_TOKEN, "segment": jq.POLICY_SEGMENT}[case["level"]],
                  mean={"tokens": jq.POLICY_MEAN_TOKENS, "segs": jq.POLICY_MEAN_SEGMENTS,
                        "sum": jq.POLICY_SUM}[case["mean"]])
        out, seg = jq.policy_loss(s["nll"], s["old"], s["adv"], **kw)
        return dict(means=out[:3], counts=out[3:], dnll=jq.policy_loss_bwd(s["nll"], s["old"], s["adv"], out, seg, **kw))
    if op == "distill_fwd":
        loss, lse, logp = jq.linear_distill(s["x"], s["w"], s["ids"], s["teacher"], scale=case["scale"],
                                            renorm=case["renorm"])
        return dict(loss=loss, lse=lse, logp=logp)
    if op == "distill_bwd":
        dx, dw = jq.linear_distill_bwd(s["x"], s["w"], s["ids"], s["teacher"], s["lse"], s["logp"], s["dloss"],
                                       scale=case["scale"], renorm=case["renorm"], dw_dtype=torch.bfloat16)
        return dict(dx=dx, dw=dw)
    y, ids, p = jq.moe_nvfp4(s["x"], s["router"], s["w13"], s["w2"], case["topk"], renorm=case["renorm"],
                             out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return dict(y=y, ids=ids, p=p)


# ------------------------------------------------------------------ definitions in 64 bits

def _exact_policy(case, s):
    n, nseg = case["n"], case["nseg"]
    nll, old, adv = s["nll"].double(), s["old"].double(), s["adv"].double()
    lengths = s["off"].diff()
    used = int(lengths.sum())
    owner = torch.repeat_interleave(torch.arange(nseg, device=nll.device), lengths)
    keep = torch.ones(used, dtype=torch.bool, device=nll.device) if s["mask"] is None else s["mask"][:used]
    at = keep.nonzero()[:, 0]  # counted tokens
    own_seg = owner[at]
    a = adv[at] if case["adv"] == "token" else adv[own_seg]

    def total(values):  # of each sequence
        return torch.zeros(nseg, dtype=torch.float64, device=nll.device).scatter_add(0, own_seg, values)

    cnt = total(torch.ones_like(a))
    w = {"tokens": lambda: torch.full_like(a, 1.0 / max(at.numel(), 1)),
         "segs": lambda: 1.0 / cnt[own_seg] / max(int((cnt > 0).sum()), 1),
         "sum": lambda: torch.ones_like(a)}[case["mean"]]()
    r = (old - nll)[at]
    if case["level"] == "segment":
        r = (total(r) / cnt.clamp(min=1))[own_seg]
    r = r.exp()
    # PPO's pessimistic bound, and for negative advantages the second one
    bounded = torch.minimum(r * a, r.clamp(1.0 - case["low"], 1.0 + case["high"]) * a)
    if case["dual"] > 0:
        bounded = torch.where(a < 0, torch.maximum(bounded, case["dual"] * a), bounded)
    active = bounded == r * a
    slope = torch.where(active, a * r, torch.zeros_like(a))
    if case["level"] == "segment":
        slope = (total(slope) / cnt.clamp(min=1))[own_seg]
    surrogate, klsum = -(w * bounded).sum(), torch.zeros((), dtype=torch.float64, device=nll.device)
    if s["ref"] is not None:
        d = (nll - s["ref"].double())[at]
        klsum = (w * (torch.expm1(d) - d)).sum()
        slope = slope + case["kl"] * torch.expm1(d)
    dnll = torch.zeros(n, dtype=torch.float64, device=nll.device)
    dnll[at] = w * slope
    counts = torch.tensor([float((~active).sum()), float(at.numel()), float((cnt > 0).sum())], dtype=torch.float64,
                          device=nll.device)
    return dict(means=torch.stack((surrogate + case["kl"] * klsum, surrogate, klsum)), counts=counts, dnll=dnll)


def _exact_distill(case, s):
    x, ids, n, v = s["x"].double(), s["ids"], case["n"], case["v"]
    listed_ = ids >= 0
    t = s["teacher"].double().masked_fill(~listed_, -math.inf)
    if case["renorm"]:
        t = torch.where(listed_, t - torch.logsumexp(t, 1, keepdim=True), t)
    q = torch.exp(t)
    if case["op"] == "distill_fwd":
        lse = torch.full((n,), -math.inf, dtype=torch.float64, device=x.device)
        zt = torch.zeros_like(q)
        for a in range(0, v, 8192):
            z = case["scale"] * torch.mm(x, s["w"][a:a + 8192].double().T)
            lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
            here = listed_ & (ids >= a) & (ids < a + 8192)
            zt = torch.where(here, z.gather(1, (ids - a).clamp(0, z.shape[1] - 1)), zt)
        logp = torch.where(listed_, zt - lse[:, None], torch.zeros_like(zt))
        return dict(loss=torch.where(listed_, torch.xlogy(q, q) - q * logp, torch.zeros_like(q)).sum(1), lse=lse,
                    logp=logp)
    coef = torch.where(listed_.any(1), s["dloss"].double() * case["scale"], torch.zeros(n, dtype=torch.float64,
                                                                                        device=x.device))
    dx, dw, mass = torch.zeros_like(x), [], q.sum(1)
    for a in range(0, v, 8192):
        w = s["w"][a:a + 8192].double()
        d = mass[:, None] * torch.exp(case["scale"] * torch.mm(x, w.T) - s["lse"].double()[:, None])
        r, j = (listed_ & (ids >= a) & (ids < a + 8192)).nonzero(as_tuple=True)
        d.index_put_((r, ids[r, j] - a), -q[r, j], accumulate=True)
        d = torch.where(coef[:, None] != 0, coef[:, None] * d, torch.zeros_like(d))
        dx += torch.mm(d, w)
        dw.append(torch.mm(d.T, x))
    return dict(dx=dx, dw=torch.cat(dw))


def _exact_moe(case, s):
    m, e, k = case["m"], case["e"], case["topk"]
    x = s["x"].double()
    score = torch.einsum("mh,eh->me", x, s["router"].double())
    prob = torch.softmax(score, 1)
    # ordered by score, the lower index first among equals
    order = [sorted(range(e), key=lambda j: (-row[j], j))[:k] for row in score.tolist()]
    ids = torch.tensor(order, device=x.device)
    p = prob.gather(1, ids)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    table = torch.tensor([(-1.0 if i & 8 else 1.0) * _GRID[i & 7] for i in range(16)], dtype=torch.float64,
                         device=x.device)

    def product(w, j, v):  # expert j's weight times the vector v
        q = w["q"][j]
        full = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
        full[:, 0::2], full[:, 1::2] = table[(q % 16).int()], table[(q // 16).int()]
        part = torch.einsum("nbi,bi->nb", full.view(q.shape[0], -1, 16), v.view(-1, 16))
        return (part * w["sb"][j].view(torch.float8_e4m3fn).double()).sum(1) * w["sg"][j].double()

    y = torch.zeros_like(x)
    for t in range(m):
        for j, weight in zip(order[t], p[t]):
            gu = product(s["w13"], j, x[t])
            gate, up = gu[: case["inter"]], gu[case["inter"]:]
            y[t] += weight * product(s["w2"], j, torch.sigmoid(gate) * gate * up)
    return dict(y=y, ids=ids, p=p)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "policy":
        return _exact_policy(case, s)
    if op in ("distill_fwd", "distill_bwd"):
        return _exact_distill(case, s)
    return _exact_moe(case, s)
