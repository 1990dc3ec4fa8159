"""ar_policy_loss against its formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.norm_ref import policy as reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def inputs(T, S, seed=1, masked=True, token=False, spare=0):
    """Ragged sequences, some empty, over tokens 0 .. T - spare; the rest belong to none."""
    rng = np.random.Generator(np.random.PCG64(seed))
    offsets = np.concatenate([[0], np.sort(rng.integers(0, T - spare + 1, max(S - 1, 0))), [T - spare]])[:S + 1].astype(np.int64)
    nll = -np.log(rng.random(T) + 1e-7)
    old = nll + rng.standard_normal(T) * np.where(rng.random(T) < 0.1, 1.0, 0.1)
    ref = nll + rng.standard_normal(T) * np.where(rng.random(T) < 0.1, 1.5, 0.2)
    adv = rng.standard_normal(T if token else S)
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    f = lambda x: x.astype(np.float32)  # noqa: E731
    return f(nll), offsets, f(adv), f(old), f(ref), mask


def run(nll, offsets, adv, old=None, ref=None, mask=None, low=0.2, high=0.28, beta=0.04, scale=1.0, mean="tokens",
        token=False, stream=None, lead=0, gradient=True, in_place=False):
    T = len(nll)
    tps.ar_init(1, max(1, T))

    def dev(x):
        if x is None:
            return None
        t = torch.zeros(len(x) + lead, dtype=torch.from_numpy(np.asarray(x)[:0]).dtype, device="cuda")[lead:]
        t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        return t
    n, o, a, ol, r, m = (dev(x) for x in (nll, offsets, adv, old, ref, mask))
    totals = torch.full((6,), 7.0, device="cuda")
    grad = torch.full((T + lead + 2,), 7.0, device="cuda")
    d = None if not gradient else n if in_place else grad[lead + 1:lead + 1 + T] if lead else torch.full((T,), 7.0, device="cuda")
    tps.ar_policy_loss(n, o, a, totals[1:5], d, ol, r, m, low, high, beta, scale, mean, token, stream=stream)
    torch.cuda.synchronize()
    want, dw, t_off, d_off = reference(nll, offsets, adv, old, ref, mask, low, high, beta, scale, mean, token)
    got = totals.cpu().numpy()
    assert got[0] == got[5] == 7
    same = np.abs(got[1:5] - want) <= t_off + 1e-38
    assert (same | (np.isnan(got[1:5]) & np.isnan(want))).all(), (got[1:5], want, t_off)
    if gradient:
        g = d.cpu().numpy().astype(np.float64)
        bad = ~(np.abs(g - dw) <= d_off + 1e-38) & ~(np.isnan(g) & np.isnan(dw)) & ~(g == dw)
        assert not bad.any(), (np.nonzero(bad)[0][:5], g[bad][:5], dw[bad][:5])
        if lead:
            assert (grad[:lead + 1] == 7).all() and grad[-1] == 7
    return totals[1:5], d


@pytest.mark.parametrize("T,S", [(1, 1), (2, 1), (7, 3), (8, 8), (31, 1), (300, 5), (2047, 9), (2048, 1), (2049, 40), (5000, 5000),
                                 (8191, 3), (8193, 700), (40_000, 17), (300_000, 11), (70_001, 9000), (60_001, 50_000)])
@pytest.mark.parametrize("mean", ["sum", "tokens", "sequences"])
@pytest.mark.parametrize("token", [False, True])
def test_sizes(T, S, mean, token):
    nll, offsets, adv, old, ref, mask = inputs(T, S, T + S, token=token, spare=T // 9)
    run(nll, offsets, adv, old, ref, mask, mean=mean, token=token)


@pytest.mark.parametrize("mean", ["sum", "tokens", "sequences"])
@pytest.mark.parametrize("T,S", [(500, 7), (30_001, 50)])
@pytest.mark.parametrize("old,ref,masked", [(False, False, False), (True, False, False), (False, True, True), (True, True, False)])
def test_optional_parts(T, S, mean, old, ref, masked):
    nll, offsets, adv, o, r, mask = inputs(T, S, 3, masked)
    run(nll, offsets, adv, o if old else None, r if ref else None, mask, mean=mean)
    run(nll, offsets, adv, o if old else None, r if ref else None, mask, mean=mean, gradient=False)


@pytest.mark.parametrize("lead", [1, 2, 3, 4])
@pytest.mark.parametrize("T", [77, 5003])
def test_starts(lead, T):
    nll, offsets, adv, old, ref, mask = inputs(T, 6, 4, spare=5)
    run(nll, offsets, adv, old, ref, mask, lead=lead, mean="sequences")


@pytest.mark.parametrize("mean", ["sum", "tokens", "sequences"])
def test_sequences_with_nothing(mean):
    T = 6000
    nll, offsets, adv, old, ref, mask = inputs(T, 12, 5)
    mask[offsets[3]:offsets[5]] = 0
    run(nll, offsets, adv, old, ref, mask, mean=mean)
    totals, d = run(nll, offsets, adv, old, ref, np.zeros(T, np.uint8), mean=mean)
    assert (totals == 0).all() and (d == 0).all()
    # every sequence empty, none at all, no tokens at all
    totals, d = run(nll, np.full(13, 100, np.int64), adv, old, ref, mask, mean=mean)
    assert (totals == 0).all() and (d == 0).all()
    totals, d = run(nll, np.zeros(1, np.int64), adv[:0], old, ref, mask, mean=mean)
    assert (totals == 0).all() and (d == 0).all()
    e = np.zeros(0, np.float32)
    totals, _ = run(e, np.zeros(4, np.int64), adv[:3], e, e, np.zeros(0, np.uint8), mean=mean)
    assert (totals == 0).all()


@pytest.mark.parametrize("T", [400, 20_000])
def test_masked_tokens_may_hold_anything(T):
    nll, offsets, adv, old, ref, mask = inputs(T, 5, 6, spare=30)
    clean = run(nll, offsets, adv, old, ref, mask, mean="sequences")
    out = (mask == 0) | (np.arange(T) >= T - 30)
    for x, v in ((nll, np.nan), (old, np.inf), (ref, -np.inf)):
        x[out] = v
    dirty = run(nll, offsets, adv, old, ref, mask, mean="sequences")
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("T", [300, 9000])
def test_ratios_next_to_the_limits(T):
    """Log ratios that float rounds onto the rounded limit: 64 bits decide."""
    low, high = 0.2, 0.28
    rng = np.random.Generator(np.random.PCG64(7))
    limit = np.where(rng.random(T) < 0.5, math.log1p(high), math.log1p(-low))
    # one of the two likelihoods small, so that the difference has bits below a float's at the limit
    small = (rng.random(T) * 0.01).astype(np.float32).astype(np.float64)
    nll = np.where(limit > 0, small, small - limit).astype(np.float32)
    old = (nll.astype(np.float64) + limit).astype(np.float32)
    near = np.where(limit > 0, rng.integers(-2, 3, T), rng.integers(-8, 9, T)).astype(np.int32)
    old = (old.view(np.int32) + near).view(np.float32)
    adv = rng.choice([-1.5, 2.0], T).astype(np.float32)
    x = old.astype(np.float64) - nll.astype(np.float64)
    for bound in (math.log1p(high), math.log1p(-low)):
        rounded_onto = x[x.astype(np.float32) == np.float32(bound)]
        assert bool((rounded_onto > bound).any()) and bool((rounded_onto < bound).any())
    run(nll, np.array([0, T], np.int64), adv, old, token=True, low=low, high=high, mean="sum")


@pytest.mark.parametrize("low,high", [(0.0, 0.0), (1.0, math.inf), (0.1, 5.0)])
def test_limits(low, high):
    nll, offsets, adv, old, ref, mask = inputs(3000, 4, 8)
    run(nll, offsets, adv, old, ref, mask, low=low, high=high)


@pytest.mark.parametrize("beta", [0.0, 1.0, 30.0])
@pytest.mark.parametrize("scale", [1.0, -65536.0, 0.0])
def test_weights(beta, scale):
    nll, offsets, adv, old, ref, mask = inputs(3000, 4, 9)
    adv[1] = 0
    run(nll, offsets, adv, old, ref, mask, beta=beta, scale=scale)


@pytest.mark.parametrize("T", [200, 5000])
def test_far_log_ratios(T):
    """From differences that float hardly sees to exponentials near overflow."""
    nll, offsets, adv, old, ref, mask = inputs(T, 3, 10, False)
    d = np.geomspace(1e-7, 80, T) * np.where(np.arange(T) % 2, 1, -1)
    nll = np.abs(d).astype(np.float32) * (d > 0)
    ref = np.abs(d).astype(np.float32) * (d < 0)
    old = ref[::-1].copy()
    run(nll, offsets, adv, np.minimum(old, 80), ref, None, mean="sum")


def test_overflow_stays_where_it_is():
    """An exponential past float's range is infinite in its token's gradient and leaves the others alone."""
    nll, offsets, adv, old, ref, mask = inputs(2100, 3, 11, False)
    adv[:] = -1
    old[7] = nll[7] + 200
    a, d = run(nll, offsets, adv, None, ref, None)
    tps.ar_init(1, 2100)
    t = [torch.from_numpy(x).cuda() for x in (nll, offsets, adv, old)]
    totals, g = torch.empty(4, device="cuda"), torch.empty(2100, device="cuda")
    tps.ar_policy_loss(*t[:3], totals, g, old_nll=t[3])
    assert g[7] == -math.inf and totals[0] == math.inf and torch.isfinite(torch.cat([g[:7], g[8:]])).all()


@pytest.mark.parametrize("T", [120, 30_000])
def test_numbers_that_are_none_stay_with_their_tokens(T):
    """A NaN in a counted token makes its gradient NaN, wherever it stands, and the totals."""
    tps.ar_init(1, T)
    for which in range(4):
        nll, offsets, adv, old, ref, _ = inputs(T, 3, 19, False, token=True)
        (nll, adv, old, ref)[which][50] = np.nan
        t = [torch.from_numpy(x).cuda() for x in (nll, offsets, adv, old, ref)]
        totals, g = torch.empty(4, device="cuda"), torch.empty(T, device="cuda")
        tps.ar_policy_loss(*t[:3], totals, g, old_nll=t[3], ref_nll=t[4], kl_weight=0.1, token_advantages=True)
        assert g[50].isnan() and totals[0].isnan() and int(g.isnan().sum()) == 1, which


def test_offsets_out_of_order_touch_nothing_else():
    """Offsets that break the rule give unspecified numbers, but no token outside of the arrays is touched."""
    T = 5000
    rng = np.random.Generator(np.random.PCG64(12))
    nll, _, _, old, ref, mask = inputs(T, 2, 12)
    tps.ar_init(1, T)
    back = torch.full((T + 512,), 7.0, device="cuda")
    for S in (1, 3, 70, 4000):
        offsets = rng.integers(-(1 << 40), 1 << 40, S + 1)
        adv = rng.standard_normal(S).astype(np.float32)
        t = [torch.from_numpy(x).cuda() for x in (nll, offsets, adv, old, ref)]
        for mean in ("sum", "tokens", "sequences"):
            tps.ar_policy_loss(*t[:3], torch.empty(4, device="cuda"), back[256:256 + T], t[3], t[4], mean=mean)
    torch.cuda.synchronize()
    assert (back[:256] == 7).all() and (back[-256:] == 7).all()


def test_in_place_and_repeatable():
    args = inputs(50_000, 30, 13, spare=100)
    a = run(*args, mean="sequences")
    b = run(*args, mean="sequences")
    c = run(*args, mean="sequences", in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(*inputs(50_000, 30, 14), mean="sequences", stream=s)


def test_bool_masks():
    nll, offsets, adv, old, ref, mask = inputs(900, 4, 15)
    tps.ar_init(1, 900)
    t = [torch.from_numpy(x).cuda() for x in (nll, offsets, adv, mask)]
    out = [(torch.empty(4, device="cuda"), torch.empty(900, device="cuda")) for _ in range(2)]
    for m, (totals, d) in zip((t[3], t[3].bool()), out):
        tps.ar_policy_loss(*t[:3], totals, d, mask=m)
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("mean", ["sum", "tokens", "sequences"])
def test_matches_autograd_and_differences(mean):
    T = 600
    nll, offsets, adv, old, ref, mask = inputs(T, 5, 16)
    totals, d = run(nll, offsets, adv, old, ref, mask, mean=mean)
    seq = torch.repeat_interleave(torch.arange(5), torch.from_numpy(np.diff(offsets)))
    x = torch.from_numpy(nll).double().requires_grad_()
    m, a = torch.from_numpy(mask).double(), torch.from_numpy(adv).double()[seq]

    def loss(x):
        ratio = torch.exp(torch.from_numpy(old).double() - x)
        gain = torch.minimum(ratio * a, ratio.clamp(0.8, 1.28) * a)
        diff = x - torch.from_numpy(ref).double()
        each = (-gain + 0.04 * (torch.exp(diff) - diff - 1)) * m
        if mean == "sum":
            return each.sum()
        if mean == "tokens":
            return each.sum() / m.sum()
        rows = [each[seq == s].sum() / m[seq == s].sum() for s in range(5) if m[seq == s].sum() > 0]
        return torch.stack(rows).mean()
    value = loss(x)
    value.backward()
    want = x.grad.numpy()
    assert np.abs(d.cpu().numpy() - want).max() <= 1e-6 * np.abs(want).max()  # a dozen float roundings
    # the loss is piecewise smooth: central differences away from the limits
    step = 1e-4
    for t in np.nonzero((mask != 0) & (np.abs(old - nll - math.log(1.28)) > 0.01) & (np.abs(old - nll - math.log(0.8)) > 0.01))[0][:5]:
        up, down = x.detach().clone(), x.detach().clone()
        up[t] += step
        down[t] -= step
        diff = ((loss(up) - loss(down)) / (2 * step)).item()
        assert abs(diff - d[t].item()) <= 1e-6 * max(1.0, abs(want).max())  # step^2 / 6 of the third derivative


@pytest.mark.parametrize("T,S", [(500, 4), (30_000, 60)])
def test_in_a_graph(T, S):
    nll, offsets, adv, old, ref, mask = inputs(T, S, 17)
    tps.ar_init(1, T)
    n, o, a, ol, r, m = (torch.from_numpy(x).cuda() for x in (nll, offsets, adv, old, ref, mask))
    outs = [(torch.empty(4, device="cuda"), torch.empty(T, device="cuda")) for _ in range(3)]

    def step(out):
        tps.ar_policy_loss(n, o, a, out[0], out[1], ol, r, m, kl_weight=0.1, mean="sequences")
    step(outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs[0])
        step(outs[1])
    for shift in (0.0, 0.05):
        ol += shift
        g.replay()
        step(outs[2])
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k][0], outs[2][0]) and torch.equal(outs[k][1], outs[2][1])


def test_refusals_leave_the_outputs_alone():
    T = 100
    nll, offsets, adv, old, ref, mask = inputs(T, 3, 18)
    tps.ar_init(1, T)
    n, o, a, ol = (torch.from_numpy(x).cuda() for x in (nll, offsets, adv, old))
    totals, d = torch.full((4,), 5.0, device="cuda"), torch.full((T,), 5.0, device="cuda")
    for kw in (dict(clip_low=2.0), dict(kl_weight=-1.0), dict(scale=math.nan), dict(old_nll=d),
               dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        if "old_nll" in kw:  # part of it: an overlap that is not exact
            buf = torch.full((T + 4,), 5.0, device="cuda")
            kw, out = dict(old_nll=buf[4:]), buf[:T]
        else:
            out = d
        with pytest.raises(tps.ARError):
            tps.ar_policy_loss(n, o, a, totals, out, **kw)
    for bad in (dict(dnll=d[:-1]), dict(old_nll=ol[:-1]), dict(ref_nll=ol.double()), dict(mask=ol), dict(token_advantages=True),
                dict(old_nll=ol.cpu())):
        with pytest.raises((TypeError, ValueError)):
            tps.ar_policy_loss(n, o, a, totals, **{"dnll": d, **bad})
    torch.cuda.synchronize()
    assert (totals == 5).all() and (d == 5).all()
