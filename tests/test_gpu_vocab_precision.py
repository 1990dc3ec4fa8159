"""Precision of the vocabulary calls where a float computation is exact enough
to tell: nearly sure tokens, long sums of one sign, unequal token weights."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.test_gpu_vocab import DTYPES, UNIT, grads_of, loss_of, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    tps.ar_init(2, 1 << 26)
    yield
    assert tps.ar_query("device_status") == 0
    tps.ar_free()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_one_infinite_dloss_leaves_other_tokens_alone(dtype, T, bad):
    """A token's hidden gradient depends on its own dloss: another token's
    overflow changes no bit of it."""
    hidden, weights, targets = make(dtype, T, 72, [130, 77], seed=T)
    dloss = torch.linspace(-100, 100, T, device="cuda")
    dloss[7] = 0
    _, lse = loss_of(hidden, weights, targets)
    want, _ = grads_of(hidden, weights, targets, lse, dloss, want=("dhidden",))
    dloss[7] = bad
    got, dw = grads_of(hidden, weights, targets, lse, dloss)
    others = torch.arange(T, device="cuda") != 7
    for a, b in zip(got, want):
        assert torch.isfinite(a[others]).all() and torch.equal(a[others], b[others])
        assert not torch.isfinite(a[7]).all()
    assert not any(torch.isfinite(w).all() for w in dw)


def nearly_sure(dtype, T, D):
    """Tokens whose target has 1 - p of 1e-6 to 1e-3, half of them with a
    positive, half with a negative logit, all products of a logit of one sign.
    Element D - 2 + k of a hidden gradient is the logits' gradient of row k
    (k = 0, 1: the targets), because only that row holds a one there."""
    gen = torch.Generator(device="cuda").manual_seed(D + T)

    def noise(*shape):
        return 1 + 0.2 * (torch.rand(shape, device="cuda", generator=gen) - 0.5)
    V, n = 200, (D - 2) // 2
    w = torch.zeros((V, D), device="cuda")
    w[:, :n], w[:, n:2 * n] = -7 / n * noise(V, n), -20 / n * noise(V, n)
    w[0, :n], w[0, n:2 * n] = 6 / n * noise(n), -20 / n * noise(n)
    w[1, :n], w[1, n:2 * n] = -7 / n * noise(n), -6 / n * noise(n)
    w[0, D - 2] = w[1, D - 1] = 1
    h = torch.zeros((T, D), device="cuda")
    targets = torch.arange(T, device="cuda") % 2
    scale = torch.linspace(1.0, 1.4, T, device="cuda")[:, None]
    h[:, :n] = (targets == 0)[:, None] * scale * noise(T, n)
    h[:, n:2 * n] = (targets == 1)[:, None] * scale * noise(T, n)
    dt = DTYPES[dtype]
    return h.to(dt), w.to(dt), targets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [20, 64, 66, 300])
@pytest.mark.parametrize("D", [8194, 8250])
def test_target_entry_of_nearly_sure_tokens(dtype, T, D):
    """The target's p - 1 to the bits that a float log-sum-exp leaves it: the
    gradient's logits and the loss's drift alike or not at all.

    Off by half a unit of the lse (at most 2^-22 below 16), by a rounding of a
    sum between 1 and 2 for each of the 128 columns of a thread and of a few
    joins (2^-24 each), and, relative to itself, by the logits' own errors in
    the other rows (their drift, below 2^-12) and two roundings to the type."""
    hidden, w, targets = nearly_sure(dtype, T, D)
    _, lse = loss_of(hidden, [w], targets)
    dh, _ = grads_of(hidden, [w], targets, lse, torch.ones(T, device="cuda"), want=("dhidden",))
    z = hidden.double() @ w.double().t()
    rest = z.clone()
    rest.scatter_(1, targets[:, None], float("-inf"))
    picked = z.gather(1, targets[:, None])[:, 0]
    other = torch.logsumexp(rest, 1) - picked            # log of (1 - p) / p
    want = -torch.sigmoid(other)
    assert (picked[targets == 0] > 5).all() and (picked[targets == 1] < -5).all() and picked.abs().max() < 16
    assert want.abs().min() < 1e-5 and want.abs().max() < 2e-3
    got = dh[0][:, D - 2:].double().gather(1, targets[:, None])[:, 0]
    tol = 2.0 ** -22 + 136 * 2.0 ** -24 + want.abs() * (2.0 ** -12 + 2 * UNIT[dtype]) + (2.0 ** -24 if dtype == "f16" else 0)
    err = (got - want).abs()
    assert (err <= tol).all(), f"off by {err.max().item():.3g}, {(err / tol).max().item():.3g} times what is allowed"


def one_sign_bound(z):
    """Of a logit whose products all have one sign: a run's 32 products of 16
    terms are cut off by at most two units in the last place of a running sum
    that is half its end on average, the (up to 16) runs are added with half a
    unit each.  Some 40 times 2^-23 of the logit; the log-sum-exp adds half a
    unit of its own and of the logarithm, and 136 roundings of a sum near 1."""
    return (32 + 8 + 2) * 2.0 ** -23 * z.abs().amax(1) + 136 * 2.0 ** -24


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [5, 64, 66, 300])
def test_log_sum_exp_of_long_sums_of_one_sign(dtype, T):
    """Sums that only grow, where whatever is cut off adds up."""
    hidden, w, targets = nearly_sure(dtype, T, 8194)
    loss, lse = loss_of(hidden, [w], targets)
    z = hidden.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    near_rows = z.gather(1, targets[:, None])
    tol = one_sign_bound(near_rows)
    assert ((lse.double() - want).abs() <= tol).all()
    # the loss is a difference of two sums with the same drift
    tol = 2.0 ** -22 + 136 * 2.0 ** -24 + 2.0 ** -12 * (want - near_rows[:, 0])
    assert ((loss.double() - (want - near_rows[:, 0])).abs() <= tol).all()


@pytest.mark.parametrize("T,D,pieces", [(2, 230, [25929]), (5, 384, [2884] * 8), (12, 187, [51812]), (64, 1024, [9000, 700]),
                                        (65, 640, [20000]), (300, 512, [10000, 5000]), (700, 1031, [4000, 77])])
def test_float_gradients_are_no_worse_than_a_float_computation(T, D, pieces):
    """Errors against 64 bits, relative to the whole gradient: at most twice
    those of elementary float operations, and two roundings (2^-22)."""
    hidden, weights, targets = make("f32", T, D, pieces, seed=D, ignored=0.1)
    gen = torch.Generator(device="cuda").manual_seed(T)
    dloss = torch.rand(T, device="cuda", generator=gen)
    loss, lse = loss_of(hidden, weights, targets)
    dh, dw = grads_of(hidden, weights, targets, lse, dloss)

    def step(dtype):
        h, ws = hidden.to(dtype), [w.to(dtype) for w in weights]
        z = h @ torch.cat(ws).t()
        top = z.amax(1, keepdim=True)
        s = top[:, 0] + (z - top).exp().sum(1).log()
        counted = targets >= 0
        at = torch.where(counted, targets, 0)[:, None]
        ls = torch.where(counted, s - z.gather(1, at)[:, 0], 0.0)
        d = (z - s[:, None]).exp()
        d.scatter_add_(1, at, torch.full_like(at, -1, dtype=dtype))
        d *= torch.where(counted, dloss.to(dtype), 0.0)[:, None]
        parts = d.split([w.shape[0] for w in ws], 1)
        return [ls, s], [p @ w for p, w in zip(parts, ws)] + [p.t() @ h for p in parts]

    allow = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        plain_values, plain = step(torch.float32)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allow
    values, exact = step(torch.float64)
    unit = 2 * 2.0 ** -23 * values[1].abs().max() + 2.0 ** -22
    for got, mine, want in zip((loss, lse), plain_values, values):
        assert (got.double() - want).abs().max() <= 2 * (mine.double() - want).abs().max() + unit
    for got, mine, want in zip(dh + dw, plain, exact):
        assert (got.double() - want).norm() <= 2 * (mine.double() - want).norm() + 2.0 ** -22 * want.norm()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [48, 512])
@pytest.mark.parametrize("V,depth", [(100, 3.1), (1000, 6.3), (20000, 9.1), (100000, 11.3), (100000, 15.7)])
def test_many_small_terms_next_to_a_large_one(dtype, T, V, depth):
    """Row 0 has the logit 0, all others have one far below it, and together
    they weigh as much: the sum keeps them as well as a float computation does.

    At most twice its error in the mean over the tokens, and half a unit."""
    dt = DTYPES[dtype]
    h, w = torch.zeros((T, 8), device="cuda", dtype=dt), torch.zeros((V, 8), device="cuda", dtype=dt)
    h[:, 0] = torch.linspace(1, 1.05, T, device="cuda").to(dt)
    w[1:, 0] = -depth
    _, lse = loss_of(h, [w], torch.zeros(T, dtype=torch.int64, device="cuda"))
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    plain = z.float().exp().sum(1).log()                    # the logits are exact, the largest is 0

    def off(x):
        return (x.double() - want).square().mean().sqrt().item()
    assert off(lse) <= 2 * off(plain) + 2.0 ** -24 * (want.abs().max().item() + 1)
