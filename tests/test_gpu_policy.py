"""The policy loss and its gradient against the definition in binary64.

Tolerances.  A token's ratio is expf (2 ulp) of a difference whose rounding error is kept, times the advantage:
4 roundings of 2^-24 and the 2 ulp; expm1 of the reference term the same, of a difference rounded to 2^-24 of
itself.  Sums of at most 128 tokens are FP32 (9 roundings), the rest compensated.  Weights add 3 roundings.  All of
it is below 2^-20 of the terms' magnitudes.  Counts are whole numbers.
"""
import itertools
import math

import numpy as np
import pytest
import torch

import rollout_x128_act_gb300 as jq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 2.0 ** -20
MEANS = {"tokens": jq.POLICY_MEAN_TOKENS, "segs": jq.POLICY_MEAN_SEGMENTS, "sum": jq.POLICY_SUM}


def reference(nll, old, adv, off, ref, mask, low, high, dual, kl, by_seg, mean, scale, per_token):
    """(out [6], dnll, size of dnll's terms, sizes of the sums) in binary64, a sequence at a time."""
    low, high, dual, kl, scale = (float(np.float32(v)) for v in (low, high, dual, kl, scale))
    nll, old, adv = nll.astype(np.float64), old.astype(np.float64), adv.astype(np.float64)
    n = nll.size
    counted = [np.array([t for t in range(max(a, 0), min(b, n)) if mask is None or mask[t]], dtype=np.int64)
               for a, b in zip(off[:-1], off[1:])]
    N, S = sum(c.size for c in counted), sum(c.size > 0 for c in counted)
    dnll, size = np.zeros(n), np.zeros(n)
    sums, sizes, clipped = np.zeros(2), np.zeros(2), 0
    with np.errstate(over="ignore", invalid="ignore"):
        for s, at in enumerate(counted):
            if at.size == 0:
                continue
            w = {"tokens": scale / N, "segs": scale / (S * at.size), "sum": scale}[mean]
            A = adv[at] if per_token else np.full(at.size, adv[s])
            logr = old[at] - nll[at]
            if by_seg:
                logr = np.full(at.size, math.fsum(logr) / at.size)
            r = np.exp(logr)
            hi = (A >= 0) & (logr > np.log(1.0 + high))
            lo = (A < 0) & (logr < (np.log(1.0 - low) if low < 1 else -np.inf))
            du = (A < 0) & (logr > (np.log(dual) if dual > 0 else np.inf))
            m = np.where(hi, 1.0 + high, np.where(lo, 1.0 - low, np.where(du, dual, r)))
            live = ~(hi | lo | du)
            g = np.where(live, A * np.where(live, r, 0.0), 0.0)
            mag = np.abs(g)
            if by_seg:
                g, mag = np.full(at.size, g.sum() / at.size), np.full(at.size, mag.sum() / at.size)
            k = np.zeros(at.size)
            if ref is not None:
                d = nll[at] - ref[at].astype(np.float64)
                k = np.expm1(d) - d
                g, mag = g + kl * np.expm1(d), mag + abs(kl) * (np.abs(np.expm1(d)) + np.abs(d) * np.exp(d))
            dnll[at], size[at] = w * g, abs(w) * mag
            sums += w * np.array([(-A * m).sum(), k.sum()])
            sizes += abs(w) * np.array([np.abs(A * m).sum(), np.abs(k).sum()])
            clipped += int((~live).sum())
    out = np.array([sums[0] + (kl * sums[1] if ref is not None else 0.0), sums[0], sums[1], clipped, N, S])
    return out, dnll, size, np.array([sizes[0] + abs(kl) * sizes[1], sizes[0], sizes[1]])


def offsets(n, nseg, rng, tail=0, front=0):
    """Ragged sequences, empty ones among them where there are many."""
    cuts = np.sort(rng.integers(front, n - tail + 1, nseg - 1))
    return np.concatenate(([front], cuts, [n - tail])).astype(np.int64)


def data(n, nadv, seed, spread=0.15):
    rng = np.random.default_rng(seed)
    old = rng.exponential(1.0, n).astype(np.float32)
    nll = (old + spread * rng.standard_normal(n)).astype(np.float32)
    ref = (old + 0.3 * rng.standard_normal(n)).astype(np.float32)
    return rng, old, nll, ref, rng.standard_normal(nadv).astype(np.float32)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(nll, old, adv, off=None, ref=None, mask=None, low=0.2, high=0.2, dual=0.0, kl=0.0, by_seg=False,
          mean="tokens", scale=1.0, per_token=None, dloss=None, tol=TOL):
    n = nll.size
    whole = np.array([0, n], dtype=np.int64) if off is None else off
    if per_token is None:
        per_token = adv.size != whole.size - 1
    want, dwant, size, sums = reference(nll, old, adv, whole, ref, mask, low, high, dual, kl, by_seg, mean, scale,
                                        per_token)
    kw = dict(seg_offsets=dev(off), nll_ref=dev(ref), mask=dev(mask), clip_low=low, clip_high=high, clip_dual=dual,
              kl=kl, level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN, mean=MEANS[mean], scale=scale,
              adv_per_token=per_token)
    args = dev(nll), dev(old), dev(adv)
    out, seg = jq.policy_loss(*args, **kw)
    dnll = jq.policy_loss_bwd(*args, out, seg, dloss=dev(dloss), **kw)
    got, dgot = out.double().cpu().numpy(), dnll.double().cpu().numpy()
    factor = 1.0 if dloss is None else float(dloss[0])
    assert np.array_equal(got[3:], want[3:])
    assert np.all(np.abs(got[:3] - want[:3]) <= tol * sums + 1e-37)
    assert np.all(np.abs(dgot - factor * dwant) <= tol * abs(factor) * size + 1e-37)
    return out, seg, dnll, args, kw


MODES = list(itertools.product((False, True), ("tokens", "segs", "sum"), (False, True), (False, True)))


@pytest.mark.parametrize("by_seg,mean,per_token,full", MODES)
def test_every_form(by_seg, mean, per_token, full):
    """full: reference term, mask, bound on negative advantages, rows outside the sequences."""
    n, nseg = 5003, 37
    rng, old, nll, ref, adv = data(n, n if per_token else nseg, 1)
    off = offsets(n, nseg, rng, 101 if full else 0, 13 if full else 0)
    mask = rng.random(n) < 0.7 if full else None
    check(nll, old, adv, off, ref if full else None, mask, 0.02 if by_seg else 0.2, 0.03 if by_seg else 0.28,
          1.05 if full else 0.0, 0.07 if full else 0.0, by_seg, mean, 0.7, dloss=np.float32([-1.5]) if full else None)


@pytest.mark.parametrize("n", [1, 2, 31, 33, 127, 128, 129, 255, 1023, 1025, 4096])
@pytest.mark.parametrize("by_seg", [False, True])
def test_lengths_of_one_sequence(n, by_seg):
    _, old, nll, ref, adv = data(n, 1, n)
    check(nll, old, adv, ref=ref, kl=0.1, by_seg=by_seg)


@pytest.mark.parametrize("lengths", [
    [1] * 700, [0, 0, 5, 0, 0, 0, 123, 0, 1, 0], [128] * 9, [127, 129, 0, 128, 1], [40000, 1, 0, 50000],
    [3] * 300 + [70000] + [0] * 200 + [2] * 400, [33000] * 5, [0] * 5000 + [700] + [0] * 5000, [1] * 2000 + [0] * 4000])
@pytest.mark.parametrize("by_seg,mean", [(False, "segs"), (True, "tokens")])
def test_ragged_sequences(lengths, by_seg, mean):
    """Sequences of one token, empty ones, ends on a window's border, some that a whole block has to join."""
    off = np.concatenate(([0], np.cumsum(lengths))).astype(np.int64)
    n = int(off[-1]) + 77
    _, old, nll, ref, adv = data(n, len(lengths), sum(lengths))
    check(nll, old, adv, off, ref, None, 0.01, 0.01, 0.0, 0.05, by_seg, mean)


def test_many_sequences_in_many_blocks():
    n, nseg = 300000, 5000
    rng, old, nll, ref, adv = data(n, nseg, 5)
    check(nll, old, adv, offsets(n, nseg, rng), ref, rng.random(n) < 0.5, 0.2, 0.2, 0.0, 0.01, False, "segs")
    check(nll, old, adv, offsets(n, nseg, rng), ref, rng.random(n) < 0.5, 0.003, 0.004, 0.0, 0.01, True, "segs")


@pytest.mark.parametrize("nseg", [1, 25, 3000])
@pytest.mark.parametrize("by_seg", [False, True])
def test_chunks_of_several_windows(by_seg, nseg):
    """More windows than warps run at a time: a lane sums 3 windows (12 more roundings than a single one's 9)."""
    n = 1300003
    rng, old, nll, ref, adv = data(n, n if nseg == 25 else nseg, 40 + nseg)
    check(nll, old, adv, offsets(n, nseg, rng, 5000, 700), ref, rng.random(n) < 0.9, 0.003, 0.004, 0.0, 0.02, by_seg,
          "segs", tol=2 * TOL)


@pytest.mark.parametrize("by_seg", [False, True])
def test_a_policy_that_is_still_its_sampling_policy(by_seg):
    """Ratios of 1: each token of a sequence adds the same -A, and the advantages of the sequences nearly cancel.
    The sums are compensated: 4 roundings of 2^-24 of the mean magnitude, however long a sequence is."""
    n, nseg = 1200000, 6
    rng, old, nll, _, adv = data(n, nseg, 50)
    adv = np.float32([0.1, -0.1, 0.3, -0.3, 0.7, -0.7])
    check(old, old, adv, (np.arange(nseg + 1) * (n // nseg)).astype(np.int64), by_seg=by_seg, tol=4 * 2.0 ** -24)


@pytest.mark.parametrize("by_seg", [False, True])
def test_what_is_not_counted_may_hold_anything(by_seg):
    n, nseg = 1000, 7
    rng, old, nll, ref, adv = data(n, n, 8)
    off = offsets(n, nseg, rng, 90, 40)
    mask = rng.random(n) < 0.5
    mask[off[2]:off[3]] = False  # a sequence without a counted token
    out, seg, dnll, _, kw = check(nll, old, adv, off, ref, mask, kl=0.1, by_seg=by_seg, mean="segs")
    bad = ~mask
    bad[:40] = bad[-90:] = True
    for value in (math.nan, math.inf, -math.inf, -3.4e38):
        args = []
        for a in (nll, old, ref, adv):
            b = a.copy()
            b[bad] = value
            args.append(dev(b))
        kw["nll_ref"] = args[2]
        out2, seg2 = jq.policy_loss(args[0], args[1], args[3], **kw)
        dnll2 = jq.policy_loss_bwd(args[0], args[1], args[3], out2, seg2, **kw)
        assert torch.equal(out, out2) and torch.equal(seg, seg2) and torch.equal(dnll, dnll2)
    assert bool((dnll2[dev(bad)] == 0).all())


@pytest.mark.parametrize("mean", list(MEANS))
@pytest.mark.parametrize("by_seg", [False, True])
def test_no_counted_token(mean, by_seg):
    n = 300
    rng, old, nll, ref, adv = data(n, 4, 9)
    off = offsets(n, 4, rng)
    nll[:] = np.nan
    for o, m in ((off, np.zeros(n, dtype=bool)), (np.zeros(5, dtype=np.int64), None)):
        kw = dict(seg_offsets=dev(o), nll_ref=dev(ref), mask=dev(m), mean=MEANS[mean], kl=0.1,
                  level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN)
        out, seg = jq.policy_loss(dev(nll), dev(old), dev(adv), **kw)
        dnll = jq.policy_loss_bwd(dev(nll), dev(old), dev(adv), out, seg, **kw)
        assert bool((out == 0).all()) and bool((seg == 0).all()) and bool((dnll == 0).all())
    e = torch.empty(0, device=DEV)
    out, seg = jq.policy_loss(e, e, dev(adv), seg_offsets=torch.zeros(5, dtype=torch.int64, device=DEV))
    assert bool((out == 0).all()) and bool((seg == 0).all())
    assert jq.policy_loss_bwd(e, e, dev(adv), out, seg,
                              seg_offsets=torch.zeros(5, dtype=torch.int64, device=DEV)).numel() == 0


@pytest.mark.parametrize("by_seg", [False, True])
def test_ratios_that_overflow(by_seg):
    """exp(200) is infinite: bounded for A >= 0 (A = 0 too), and for A < 0 by clip_dual; exp(-200) is zero."""
    old = np.float32([200, 200, 200, -200, -200, 200, 0, 0])
    adv = np.float32([1, 0, -1, 1, -1, -2, 3, -3])
    off = np.arange(9, dtype=np.int64)
    check(np.zeros(8, dtype=np.float32), old, adv, off, dual=3.0, by_seg=by_seg, mean="sum", per_token=True)
    out, seg = jq.policy_loss(torch.zeros(8, device=DEV), dev(old), dev(adv), seg_offsets=dev(off),
                              mean=jq.POLICY_SUM, level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN)
    assert float(out[0]) == math.inf  # without it


def test_which_side_of_the_border():
    """Log ratios a few ulp around each border, split over two numbers whose difference is not an FP32 number."""
    low, high, dual = 0.2, 0.28, 3.0
    rows = []
    for A, border in ((1.0, 1.0 + float(np.float32(high))), (-1.0, 1.0 - float(np.float32(low))), (-1.0, dual)):
        for base in (0.0, 1.7, 11.3):
            t = np.float32(math.log(border))
            for step in range(-4, 5):
                nll = np.float32(base)
                old = np.float32(np.float64(nll) + np.float64(t))
                for _ in range(abs(step)):
                    old = np.nextafter(old, np.float32(np.inf if step > 0 else -np.inf), dtype=np.float32)
                rows.append((nll, old, A))
    nll, old, adv = (np.array(c, dtype=np.float32) for c in zip(*rows))
    check(nll, old, adv, low=low, high=high, dual=dual, mean="sum")
    off = np.arange(nll.size + 1, dtype=np.int64)
    check(nll, old, adv, off, low=low, high=high, dual=dual, mean="sum", by_seg=True, per_token=True)


@pytest.mark.parametrize("by_seg", [False, True])
def test_gradient_against_differences(by_seg):
    """(loss(nll + h v) - loss(nll - h v)) / 2h.  h = 2^-6: the third derivative of each term is at most its size,
    so h^2 / 6 of the terms, and the two losses' errors over 2h; borders are far (clip 0.9 and 9)."""
    n, nseg, h = 2000, 11, 2.0 ** -6
    rng, old, nll, ref, adv = data(n, nseg, 21)
    off = offsets(n, nseg, rng, 5)
    kw = dict(seg_offsets=dev(off), nll_ref=dev(ref), clip_low=0.9, clip_high=9.0, kl=0.2, mean=jq.POLICY_SUM,
              level=jq.POLICY_SEGMENT if by_seg else jq.POLICY_TOKEN)
    v = rng.choice(np.float32([-1, 1]), n)
    out, seg = jq.policy_loss(dev(nll), dev(old), dev(adv), **kw)
    slope = float((jq.policy_loss_bwd(dev(nll), dev(old), dev(adv), out, seg, **kw).double() * dev(v).double()).sum())
    ends = [np.float32(nll + s * h * v) for s in (1, -1)]
    up, down = (float(jq.policy_loss(dev(e), dev(old), dev(adv), **kw)[0][0]) for e in ends)
    _, _, size, sums = reference(nll, old, adv, off, ref, None, 0.9, 9.0, 0.0, 0.2, by_seg, "sum", 1.0, False)
    bound = (h * h / 6 * 2 + 2.0 ** -20 / h) * (size.sum() + sums[0]) + 2 * n * 2.0 ** -22 * size.max()
    assert abs((up - down) / (2 * h) - slope) <= bound


def test_repeatable_captured_and_on_another_stream():
    n, nseg = 20000, 100
    rng, old, nll, ref, adv = data(n, nseg, 30)
    out, seg, dnll, args, kw = check(nll, old, adv, offsets(n, nseg, rng), ref, rng.random(n) < 0.9, kl=0.03)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, s1 = jq.policy_loss(*args, stream=side, **kw)
    d1 = jq.policy_loss_bwd(*args, o1, s1, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, out) and torch.equal(s1, seg) and torch.equal(d1, dnll)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2, s2 = jq.policy_loss(*args, **kw)
        d2 = jq.policy_loss_bwd(*args, o2, s2, **kw)
    for t in (o2, s2, d2):
        t.fill_(7)
    for _ in range(3):
        g.replay()
    assert torch.equal(o2, out) and torch.equal(s2, seg) and torch.equal(d2, dnll)
    args[0].add_(0.01)  # new data under the same graph
    g.replay()
    o3, s3 = jq.policy_loss(*args, **kw)
    assert torch.equal(o2, o3) and torch.equal(d2, jq.policy_loss_bwd(*args, o3, s3, **kw))


def test_a_workspace_that_holds_anything():
    n, nseg = 9000, 600
    rng, old, nll, ref, adv = data(n, nseg, 31)
    off = dev(offsets(n, nseg, rng))
    need = jq.jetq_policy_loss_workspace_bytes(n, nseg)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    a = jq.policy_loss(dev(nll), dev(old), dev(adv), off, workspace=ws)
    b = jq.policy_loss(dev(nll), dev(old), dev(adv), off)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
