"""The policy loss where FP32 loses most: sums of advantages that nearly cancel, ratios beyond FP32's range, advantages
of zero, the longest chunks.  Against the definition in binary64."""
import math

import numpy as np
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("lengths,clip", [([500000], 0.2), ([2000001], 0.2), ([700001, 3, 600000, 1], 0.2)])
@pytest.mark.parametrize("n_tail", [0, 999])
def test_advantages_that_nearly_cancel(lengths, clip, n_tail):
    """One ratio a sequence, an advantage a token, nothing clipped: gradient and loss are r times the sum of A, which
    is some sqrt(n) where the sums of either sign are n / 2.5.

    Bound, relative to the result itself: 2 ulp of expf and 2^-24 of the mean for r (its sums are compensated), and
    roundings of the sum, its product with r, the division by n and the weight (2^-22 + 6 U, taken as 12 U).  The
    compensated sum of A adds m^2 U^2 of the sum of |A|, m at most 128 + 64 steps one after another."""
    rng = np.random.default_rng(sum(lengths))
    n = sum(lengths) + n_tail
    old = rng.exponential(1.0, n).astype(np.float32)
    nll = (old + 0.15 * rng.standard_normal(n)).astype(np.float32)
    adv = rng.standard_normal(n).astype(np.float32)
    off = np.concatenate(([0], np.cumsum(lengths))).astype(np.int64)
    args = dev(nll), dev(old), dev(adv)
    kw = dict(seg_offsets=dev(off), clip_low=clip, clip_high=clip, level=jq.POLICY_SEGMENT, mean=jq.POLICY_SUM,
              adv_per_token=True)
    out, seg = jq.policy_loss(*args, **kw)
    dnll = jq.policy_loss_bwd(*args, out, seg, **kw).cpu().numpy()
    loss, slack = 0.0, 0.0
    logr = old.astype(np.float64) - nll.astype(np.float64)
    for a, b in zip(off[:-1], off[1:]):
        mean = math.fsum(logr[a:b]) / (b - a)
        assert math.log(1 - clip) < mean < math.log(1 + clip)
        r, total, size = math.exp(mean), math.fsum(adv[a:b].tolist()), math.fsum(np.abs(adv[a:b]).tolist())
        lost = 192.0 ** 2 * U * U * size
        got = dnll[a:b].astype(np.float64)
        assert np.all(got == got[0])
        want = r * total / (b - a)
        assert abs(got[0] - want) <= 12 * U * abs(want) + r * lost / (b - a)
        loss -= r * total
        slack += r * (12 * U * abs(total) + lost)
    assert np.all(dnll[off[-1]:] == 0)
    assert abs(float(out[0]) - loss) <= slack + U * abs(loss)


@pytest.mark.parametrize("by_seg", [False, True])
@pytest.mark.parametrize("length", [1, 3])
def test_ratios_that_overflow_with_a_rest(by_seg, length):
    """Differences of nll above 88.7 that are no FP32 numbers, rests of either sign: the ratio is infinite, and so are
    loss and gradient where nothing bounds it."""
    rng = np.random.default_rng(length)
    nll = rng.uniform(0.1, 0.9, 60).astype(np.float32)
    old = rng.uniform(95.0, 140.0, 60).astype(np.float32)
    diff = old - nll  # FP32
    rest = (old.astype(np.float64) - nll.astype(np.float64)) - diff.astype(np.float64)
    assert (rest < 0).any() and (rest > 0).any()
    off = np.arange(0, 61, length, dtype=np.int64)
    for A, kw in ((-1.0, dict()), (-1.0, dict(clip_dual=3.0)), (1.0, dict())):
        kw = dict(kw, level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN, mean=jq.POLICY_SUM, seg_offsets=dev(off),
                  adv_per_token=True)
        args = dev(nll), dev(old), torch.full((60,), A, device=DEV)
        out, seg = jq.policy_loss(*args, **kw)
        dnll = jq.policy_loss_bwd(*args, out, seg, **kw)
        if A < 0 and "clip_dual" not in kw:
            assert float(out[0]) == math.inf and float(out[3]) == 0
            assert bool((dnll == -math.inf).all())
        else:
            bound = 3.0 if A < 0 else -float(np.float32(1.2))
            assert abs(float(out[0]) - 60 * bound) <= 60 * abs(bound) * 2 * U
            assert float(out[3]) == 60 and bool((dnll == 0).all())


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("by_seg", [False, True])
def test_advantages_of_zero_are_not_clipped(by_seg, per_token):
    """Answers that all earn the same: nothing to bound, whatever the ratio.  A clipped token is one whose A * r the
    bound changes."""
    rng = np.random.default_rng(3)
    nseg, length = 60, 5
    n = nseg * length
    adv_seg = np.float32(rng.choice([0.0, -0.0, 0.0, 1.5, -0.7], nseg))
    adv = np.float32(rng.choice([0.0, -0.0, 0.0, 1.5, -0.7], n)) if per_token else adv_seg
    jump = np.repeat(rng.choice([-0.9, 0.0, 0.9, 2.0], nseg), length) if by_seg else rng.choice([-0.9, 0.0, 0.9, 2.0], n)
    old = rng.exponential(1.0, n).astype(np.float32)
    nll = (old - jump + 0.01 * rng.standard_normal(n)).astype(np.float32)
    mask = rng.random(n) < 0.8
    off = (np.arange(nseg + 1) * length).astype(np.int64)
    A = (adv if per_token else np.repeat(adv_seg, length)).astype(np.float64)
    logr = old.astype(np.float64) - nll.astype(np.float64)
    if by_seg:
        for a, b in zip(off[:-1], off[1:]):
            if mask[a:b].any():
                logr[a:b] = logr[a:b][mask[a:b]].mean()
    r = np.exp(logr)
    low, high, dual = 1 - float(np.float32(0.2)), 1 + float(np.float32(0.2)), 3.0
    for use_dual in (False, True):
        bounded = np.minimum(r * A, np.clip(r, low, high) * A)
        if use_dual:
            bounded = np.where(A < 0, np.maximum(bounded, dual * A), bounded)
        changed = (bounded != r * A) & mask
        assert changed.any() and not (changed & (A == 0)).any()
        kw = dict(seg_offsets=dev(off), mask=dev(mask), clip_dual=dual if use_dual else 0.0, mean=jq.POLICY_MEAN_TOKENS,
                  level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN, adv_per_token=per_token)
        args = dev(nll), dev(old), dev(adv)
        out, seg = jq.policy_loss(*args, **kw)
        assert float(out[3]) == changed.sum()
        dnll = jq.policy_loss_bwd(*args, out, seg, **kw).cpu().numpy()
        if not by_seg:
            assert np.all(dnll[(A == 0) & mask] == 0)
    if not per_token:
        zero = torch.zeros(nseg, device=DEV)
        out, seg = jq.policy_loss(args[0], args[1], zero, **kw)
        assert bool((out[:4] == 0).all())
        assert bool((jq.policy_loss_bwd(args[0], args[1], zero, out, seg, **kw) == 0).all())


@pytest.mark.parametrize("by_seg,per_token", [(False, False), (True, False), (True, True)])
def test_the_longest_chunks(by_seg, per_token):
    """More than 128 * 32 tokens for each of a GPU's 3648 warps (152 SMs): chunks of 32 windows, the most there are.

    A lane then sums KL terms of 128 tokens in FP32, and five shuffles add the lanes: 133 roundings of the sum of the
    terms' magnitudes, and the terms' own 2^-20.  Everything else is compensated (2^-20, as for short chunks)."""
    lengths = [9000001, 0, 1, 6500000, 130]
    n = sum(lengths) + 4097
    g = torch.Generator(device=DEV).manual_seed(7)
    old = torch.empty(n, device=DEV).exponential_(1.0, generator=g)
    nll = old + 0.15 * torch.randn(n, generator=g, device=DEV)
    ref = old + 0.3 * torch.randn(n, generator=g, device=DEV)
    nseg = len(lengths)
    off = torch.tensor([0] + lengths, device=DEV).cumsum(0)
    adv = torch.randn(n if per_token else nseg, generator=g, device=DEV)
    low, high, kl = (float(np.float32(v)) for v in (0.2, 0.28, 0.03))
    kw = dict(seg_offsets=off, nll_ref=ref, clip_low=low, clip_high=high, kl=kl, mean=jq.POLICY_MEAN_TOKENS,
              level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN, adv_per_token=per_token)
    out, seg = jq.policy_loss(nll, old, adv, **kw)
    dnll = jq.policy_loss_bwd(nll, old, adv, out, seg, **kw)
    N = sum(lengths)
    sums, sizes, clipped = np.zeros(2), np.zeros(2), 0
    for s, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        if a == b:
            continue
        A = adv[a:b].double() if per_token else adv[s].double().expand(b - a)
        logr = old[a:b].double() - nll[a:b].double()
        if by_seg:
            logr = logr.mean().expand(b - a)
        r, d = logr.exp(), nll[a:b].double() - ref[a:b].double()
        m = torch.where(A >= 0, r.clamp(max=1 + high), r.clamp(min=1 - low))
        live, k = m == r, torch.expm1(d) - d
        slope = torch.where(live, A * r, torch.zeros_like(A))
        size = slope.abs()
        if by_seg:
            slope, size = slope.mean().expand(b - a), size.mean().expand(b - a)
        slope, size = slope + kl * torch.expm1(d), size + kl * (torch.expm1(d).abs() + d.abs() * d.exp())
        assert bool(((dnll[a:b].double() * N - slope).abs() <= 2.0 ** -20 * size).all())
        sums += [float((-A * m).sum()) / N, float(k.sum()) / N]
        sizes += [float((A * m).abs().sum()) / N, float(k.sum()) / N]
        clipped += int((~live).sum())
    assert bool((dnll[off[-1]:] == 0).all())
    tol = 2.0 ** -20 * sizes + np.array([0.0, 133 * U * sizes[1]])
    assert abs(float(out[1]) - sums[0]) <= tol[0] and abs(float(out[2]) - sums[1]) <= tol[1]
    assert abs(float(out[0]) - sums[0] - kl * sums[1]) <= tol[0] + kl * tol[1]
    assert [float(v) for v in out[3:]] == [float(np.float32(clipped)), float(np.float32(N)), 4.0]
