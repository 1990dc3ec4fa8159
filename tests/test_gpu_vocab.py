"""ar_vocab_loss and its gradient against the formulas in 64 bits.

Tolerances, element by element, from the formulas: a float sum of K terms is
taken to be off by at most 4 sqrt(K) 2^-23 of the sum of its terms' sizes (each
addition off by one unit in the last place at most, signs mixed); a logit error
moves a probability by that much relative to itself; a value held in a 16-bit
type is off by the type's unit roundoff (2^-8 bf16, 2^-11 f16), once for the
logits' gradient and once for the output."""
import math

import pytest
import torch

import tensor_partial_sum_gb300 as tps

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 1e-30, "f16": 2.0 ** -25, "bf16": 1e-30}  # half the smallest step
IGNORE = -100
POISON = -7.0


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


def rows(n, d, pad, dtype, lead=0):
    """[n, d] with `pad` poisoned elements between rows and `lead` before the first."""
    t = torch.full((lead + n * (d + pad),), POISON, dtype=dtype, device="cuda")
    return t[lead:].view(n, d + pad)[:, :d], t


def make(dtype, T, D, pieces, seed=0, ignored=0.0, pad=0, lead=0, gain=2.0, lean=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[dtype]
    V = sum(pieces)
    weights = []
    for n in pieces:
        w, _ = rows(n, D, pad, dt, lead)
        w.copy_(torch.randn((n, D), device="cuda", generator=gen) * (gain / math.sqrt(D)))
        weights.append(w)
    targets = torch.randint(0, V, (T,), device="cuda", generator=gen)
    full = torch.cat([w.float() for w in weights])
    hidden, _ = rows(T, D, pad, dt, lead)
    hidden.copy_(torch.randn((T, D), device="cuda", generator=gen)
                 + torch.rand((T, 1), device="cuda", generator=gen) * lean * full[targets])
    if ignored:
        targets[torch.rand(T, device="cuda", generator=gen) < ignored] = IGNORE
    return hidden, weights, targets


def formula(hidden, weights, targets, dloss=None, dtype="f32"):
    """Loss, lse and gradients in 64 bits, with the size of each sum's terms."""
    live = (targets >= 0) & (targets < sum(w.shape[0] for w in weights))
    h = torch.where(live[:, None], hidden.double(), 0) if dloss is not None else hidden.double()
    W = torch.cat([w.double() for w in weights])
    z = h @ W.t()
    D = h.shape[1]
    size = (h.abs() @ W.abs().t())
    ez = 4 * math.sqrt(D) * 2.0 ** -23 * size.amax(1)
    lse = torch.logsumexp(z, 1)
    at = torch.where(live, targets, 0)[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
    # the exponentials' sum has V positive terms; the logarithm turns its relative error into an absolute one
    el = ez + 4 * math.sqrt(W.shape[0]) * 2.0 ** -23 + 2.0 ** -22 * (lse.abs() + 1)
    out = {"lse": (lse, el), "loss": (loss, torch.where(live, ez + el + 2.0 ** -22 * z.gather(1, at)[:, 0].abs(), 0.0))}
    if dloss is None:
        return out
    q = torch.exp(z - lse[:, None])
    e_q = q * (ez + el + 2.0 ** -21)[:, None]
    q.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    g = torch.where(live, dloss.double(), 0.0)[:, None]
    d, e_d = q * g, e_q * g.abs()
    # the logits' gradient is held in the type, relative to the largest |dloss|
    e_d = e_d + (0 if dtype == "f32" else UNIT[dtype]) * d.abs() + (
        2.0 ** -30 * g.abs().max() if dtype == "f16" else 0) + 2.0 ** -23 * d.abs()
    out["dhidden"], out["dweights"], first = [], [], 0
    for w in weights:
        n = w.shape[0]
        dp, ep, wd = d[:, first:first + n], e_d[:, first:first + n], w.double()
        first += n
        for name, x, err, a in (
                ("dhidden", dp @ wd, ep @ wd.abs() + 4 * math.sqrt(max(n, 1)) * 2.0 ** -23 * (dp.abs() @ wd.abs()), n),
                ("dweights", dp.t() @ h, ep.t() @ h.abs()
                 + 4 * math.sqrt(max(len(h), 1)) * 2.0 ** -23 * (dp.abs().t() @ h.abs()), n)):
            out[name].append((x, err + UNIT[dtype] * x.abs() * 1.01 + TINY[dtype]))
    return out


def near(got, want, what):
    value, tol = want
    err = (got.double() - value).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert worst <= 0, f"{what}: off by {err.max().item():.3g}, {worst:.3g} more than allowed"


def loss_of(hidden, weights, targets, **kw):
    T = hidden.shape[0]
    loss, lse = (torch.full((T,), POISON, device="cuda") for _ in range(2))
    tps.ar_vocab_loss(hidden, weights, targets, loss, lse, ignore_index=IGNORE, **kw)
    return loss, lse


def grads_of(hidden, weights, targets, lse, dloss, pad=0, lead=0, want=("dhidden", "dweights"), **kw):
    T, D = hidden.shape
    dt = hidden.dtype
    dh = [rows(T, D, pad, dt, lead) for _ in weights] if "dhidden" in want else None
    dw = [rows(w.shape[0], D, pad, dt, lead) for w in weights] if "dweights" in want else None
    tps.ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dhidden=dh and [x for x, _ in dh],
                           dweights=dw and [x for x, _ in dw], ignore_index=IGNORE, **kw)
    torch.cuda.synchronize()
    for x, back in (dh or []) + (dw or []):
        keep = torch.ones_like(back, dtype=torch.bool)
        if x.numel():
            keep[lead:].view(x.shape[0], D + pad)[:, :D] = False
        assert (back[keep] == POISON).all(), "an element outside the output was written"
    return dh and [x for x, _ in dh], dw and [x for x, _ in dw]


def check_all(dtype, hidden, weights, targets, dloss, pad=0, lead=0):
    loss, lse = loss_of(hidden, weights, targets)
    plain = formula(hidden, weights, targets)
    near(lse, plain["lse"], "lse")
    near(loss, plain["loss"], "loss")
    dh, dw = grads_of(hidden, weights, targets, lse, dloss, pad, lead)
    want = formula(hidden, weights, targets, dloss, dtype)
    for r in range(len(weights)):
        near(dh[r], want["dhidden"][r], f"dhidden[{r}]")
        near(dw[r], want["dweights"][r], f"dweights[{r}]")


SHAPES = [(1, 1, [1]), (1, 64, [7]), (2, 8, [300]), (5, 33, [100, 0, 28]), (64, 128, [256]), (128, 64, [128, 128]),
          (130, 72, [300, 301]), (257, 200, [1000]), (300, 513, [2049, 77, 1]), (1500, 64, [130]), (3, 1024, [40000]),
          (63, 4096, [511]), (129, 65, [257] * 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,D,pieces", SHAPES)
def test_shapes(dtype, T, D, pieces):
    hidden, weights, targets = make(dtype, T, D, pieces, seed=T + D)
    gen = torch.Generator(device="cuda").manual_seed(1)
    check_all(dtype, hidden, weights, targets, torch.randn(T, device="cuda", generator=gen))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,lead", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("D", [128, 200, 77])
def test_strides_and_starts(dtype, pad, lead, D):
    hidden, weights, targets = make(dtype, 150, D, [270, 131], seed=D, ignored=0.3, pad=pad, lead=lead)
    check_all(dtype, hidden, weights, targets, torch.full((150,), 1 / 150, device="cuda"), pad, lead)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ignored", [0.05, 0.5, 0.97, 1.0])
def test_ignored_tokens(dtype, ignored):
    hidden, weights, targets = make(dtype, 400, 96, [500, 333], seed=4, ignored=ignored)
    check_all(dtype, hidden, weights, targets, torch.full((400,), 0.01, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ignored_tokens_may_hold_anything(dtype):
    """Infinities and NaN in the hidden states of ignored tokens (and in their
    dloss) reach neither another token's loss nor any gradient."""
    hidden, weights, targets = make(dtype, 300, 128, [256, 100], seed=6)
    dloss = torch.full((300,), 0.01, device="cuda")
    clean = hidden.clone()
    for at, bad in ((0, float("nan")), (17, float("inf")), (130, float("-inf")), (299, torch.finfo(hidden.dtype).min)):
        hidden[at] = bad
        targets[at] = IGNORE
        dloss[at] = float("nan")
    loss, lse = loss_of(hidden, weights, targets)
    live = targets != IGNORE
    plain = formula(clean, weights, targets)
    near(loss, plain["loss"], "loss")
    near(lse[live], [x[live] for x in plain["lse"]], "lse")
    dh, dw = grads_of(hidden, weights, targets, lse, dloss)
    want = formula(clean, weights, targets, torch.where(live, dloss, 0), dtype)
    for r in range(2):
        near(dh[r], want["dhidden"][r], f"dhidden[{r}]")
        near(dw[r], want["dweights"][r], f"dweights[{r}]")
        assert (dh[r][~live] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_target_outside_the_vocabulary(dtype):
    hidden, weights, targets = make(dtype, 40, 64, [100, 50], seed=8)
    targets[3], targets[20], targets[39] = 150, -1, 2 ** 62
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 20, 39]] = True
    loss, lse = loss_of(hidden, weights, targets)
    assert torch.isnan(loss[bad]).all()
    plain = formula(hidden, weights, targets)
    near(loss[~bad], [x[~bad] for x in plain["loss"]], "loss")
    near(lse, plain["lse"], "lse")
    dloss = torch.full((40,), 0.1, device="cuda")
    dh, dw = grads_of(hidden, weights, targets, lse, dloss)
    want = formula(hidden, weights, targets, dloss, dtype)
    for r in range(2):
        near(dh[r], want["dhidden"][r], f"dhidden[{r}]")
        near(dw[r], want["dweights"][r], f"dweights[{r}]")


@pytest.mark.parametrize("dtype", DTYPES)
def test_sharp_and_flat_distributions(dtype):
    """Logits of several hundred (one row takes all) and logits of zero."""
    hidden, weights, targets = make(dtype, 70, 256, [400, 11], seed=9, gain=30.0, lean=1.0)
    hidden[5:9] = 0
    check_all(dtype, hidden, weights, targets, torch.ones(70, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1e-8, 1.0, 3e3])
def test_gradients_of_very_different_tokens(dtype, scale):
    hidden, weights, targets = make(dtype, 90, 64, [333], seed=10)
    dloss = torch.linspace(-1, 1, 90, device="cuda") ** 3 * scale
    dloss[4] = 0
    check_all(dtype, hidden, weights, targets, dloss)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_logits(dtype):
    """A row whose logits are all -infinity, and one with a +infinity, as the
    formula has them."""
    w = torch.zeros((300, 8), dtype=DTYPES[dtype], device="cuda")
    w[:, 0] = -1
    w[7, 0] = 1
    h = torch.zeros((2, 8), dtype=DTYPES[dtype], device="cuda")
    targets = torch.tensor([3, 3], device="cuda")
    big = torch.finfo(DTYPES[dtype]).max
    w[:, 1] = -big
    w[7, 1] = big
    h[0, 1] = -big      # row 7: -infinity, all others +infinity
    h[1, 1] = 1         # row 7: the type's largest value, all others its lowest
    loss, lse = loss_of(h, [w], targets)
    assert lse[0] == float("inf") and not torch.isfinite(loss[0])
    assert lse[1] == big and (loss[1] == float("inf") or loss[1] >= big)
    w[:, 1] = -big
    h[0, 1] = big       # every logit -infinity
    _, lse = loss_of(h, [w], targets)
    assert lse[0] == float("-inf")


def test_parts_of_the_gradient():
    hidden, weights, targets = make("bf16", 200, 128, [256, 200], seed=11, ignored=0.2)
    dloss = torch.full((200,), 0.005, device="cuda")
    _, lse = loss_of(hidden, weights, targets)
    dh, dw = grads_of(hidden, weights, targets, lse, dloss)
    only_h, none = grads_of(hidden, weights, targets, lse, dloss, want=("dhidden",))
    assert none is None and all(torch.equal(a, b) for a, b in zip(dh, only_h))
    none, only_w = grads_of(hidden, weights, targets, lse, dloss, want=("dweights",))
    assert none is None and all(torch.equal(a, b) for a, b in zip(dw, only_w))
    grads_of(hidden, weights, targets, lse, dloss, want=())


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_same_call_gives_the_same_bits(dtype):
    hidden, weights, targets = make(dtype, 700, 192, [1111, 1000], seed=12, ignored=0.1)
    dloss = torch.rand(700, device="cuda")
    runs = []
    for _ in range(3):
        loss, lse = loss_of(hidden, weights, targets)
        dh, dw = grads_of(hidden, weights, targets, lse, dloss)
        runs.append([loss, lse, *dh, *dw])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_chunks_of_the_vocabulary(dtype):
    """More tokens and vocabulary rows than one chunk of the logits' gradient holds."""
    hidden, weights, targets = make(dtype, 4096, 64, [70000, 300], seed=13, ignored=0.2)
    check_all(dtype, hidden, weights, targets, torch.full((4096,), 1 / 4096, device="cuda"))


def test_no_tokens():
    hidden, weights, targets = make("bf16", 4, 64, [100], seed=14)
    none = hidden[:0], weights, targets[:0]
    loss, lse = loss_of(*none)
    dh, dw = grads_of(*none, lse, torch.zeros(0, device="cuda"))
    assert (dw[0] == 0).all() and dh[0].numel() == 0


def test_another_stream_and_a_given_workspace():
    hidden, weights, targets = make("bf16", 300, 256, [1000, 24], seed=15)
    dloss = torch.rand(300, device="cuda")
    v = tps.make_vocab(hidden, weights, targets, IGNORE)
    ws = torch.full((max(tps.ar_vocab_workspace(v, g) for g in (False, True)),), 0xFF, dtype=torch.uint8, device="cuda")
    _, lse0 = loss_of(hidden, weights, targets)
    dh0, dw0 = grads_of(hidden, weights, targets, lse0, dloss)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for kw in ({"stream": s}, {"stream": s, "workspace": ws}):
        with torch.cuda.stream(s):
            loss, lse = loss_of(hidden, weights, targets, **kw)
            dh, dw = grads_of(hidden, weights, targets, lse, dloss, **kw)
        s.synchronize()
        assert torch.equal(lse, lse0) and all(torch.equal(a, b) for a, b in zip(dh + dw, dh0 + dw0))


def test_in_a_graph():
    hidden, weights, targets = make("bf16", 128, 128, [512], seed=16)
    dloss = torch.rand(128, device="cuda")
    loss, lse = (torch.zeros(128, device="cuda") for _ in range(2))
    dh, dw = [torch.empty_like(hidden)], [torch.empty_like(weights[0])]

    def step():
        tps.ar_vocab_loss(hidden, weights, targets, loss, lse, ignore_index=IGNORE)
        tps.ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dh, dw, ignore_index=IGNORE)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    fresh, _, _ = make("bf16", 128, 128, [512], seed=17)
    hidden.copy_(fresh)
    g.replay()
    want = formula(hidden, weights, targets, dloss, "bf16")
    near(loss, formula(hidden, weights, targets)["loss"], "loss")
    near(dh[0], want["dhidden"][0], "dhidden")
    near(dw[0], want["dweights"][0], "dweights")


def test_gradient_matches_differences():
    """Central differences of the summed loss in single elements (f32)."""
    hidden, weights, targets = make("f32", 12, 24, [40, 9], seed=18, ignored=0.2)
    c = torch.linspace(0.5, 1.5, 12, device="cuda")
    _, lse = loss_of(hidden, weights, targets)
    dh, dw = grads_of(hidden, weights, targets, lse, c)
    total = sum(d.double() for d in dh)
    h = 2.0 ** -5

    def value():
        return (loss_of(hidden, weights, targets)[0].double() * c.double()).sum().item()

    def difference(t, at):
        keep = t[at].item()
        t[at] = keep + h
        up = value()
        t[at] = keep - h
        down = value()
        t[at] = keep
        return (up - down) / (2 * h)
    # third derivative of the loss along one direction x: at most max|x|^3, times h^2 / 6; plus twelve
    # losses below 32 rounded at 2^-20 of themselves, twice, over 2 h
    rounding = 12 * 1.5 * 2 * 32 * 2.0 ** -20 / (2 * h)
    for j, i in ((0, 0), (5, 7), (11, 23)):
        x = max(w.abs().max().item() for w in weights)
        assert abs(difference(hidden, (j, i)) - total[j, i].item()) <= rounding + c[j].item() * x ** 3 * h * h / 6 + 1e-5
        x3 = (hidden[:, i].abs() ** 3 * c).sum().item()
        for w, d in zip(weights, dw):
            at = (j % w.shape[0], i)
            assert abs(difference(w, at) - d[at].item()) <= rounding + x3 * h * h / 6 + 1e-5


def test_refusals_leave_the_outputs_alone():
    hidden, weights, targets = make("bf16", 16, 64, [100, 28], seed=19)
    loss = torch.full((16,), 5.0, device="cuda")
    lse = torch.full((16,), 5.0, device="cuda")
    dloss = torch.ones(16, device="cuda")
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(tps.ARError):
        tps.ar_vocab_loss(hidden, weights, targets, loss, lse, workspace=small)
    with pytest.raises(tps.ARError):
        tps.ar_vocab_loss(hidden, weights, targets, loss, loss)
    with pytest.raises(tps.ARError):
        tps.ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dhidden=[hidden, torch.empty_like(hidden)])
    with pytest.raises(tps.ARError):
        tps.ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dweights=weights)
    for bad in (lambda: tps.ar_vocab_loss(hidden, weights, targets.int(), loss, lse),
                lambda: tps.ar_vocab_loss(hidden, weights, targets[:15], loss, lse),
                lambda: tps.ar_vocab_loss(hidden, weights, targets, loss[:15], lse),
                lambda: tps.ar_vocab_loss(hidden, [w.t().contiguous().t() for w in weights], targets, loss, lse),
                lambda: tps.ar_vocab_loss(hidden[:1].expand(16, 64), weights, targets, loss, lse),
                lambda: tps.ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dhidden=[torch.empty_like(hidden)])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        tps.ar_vocab_loss(hidden, [w.float() for w in weights], targets, loss, lse)
    torch.cuda.synchronize()
    assert (loss == 5).all() and (lse == 5).all()
    for inject in (1, 0):
        tps.ar_set_option("fault_inject", inject)
        if inject:
            with pytest.raises(tps.ARError):
                tps.ar_vocab_loss(hidden, weights, targets, loss, lse)
    tps.ar_vocab_loss(hidden, weights, targets, loss, lse)
    torch.cuda.synchronize()
    assert not (loss == 5).any()


# ---- shapes of the tiling ---------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [127, 128, 129, 255, 256, 257, 383, 385])
def test_token_counts_around_the_tiles(dtype, T):
    hidden, weights, targets = make(dtype, T, 72, [130, 515], seed=T, ignored=0.1)
    check_all(dtype, hidden, weights, targets, torch.rand(T, device="cuda", generator=torch.Generator("cuda").manual_seed(T)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [1, 8, 63, 65, 127, 129, 191, 255, 257, 320, 640, 1031])
def test_dims_around_the_tiles(dtype, D):
    hidden, weights, targets = make(dtype, 70, D, [300], seed=D)
    check_all(dtype, hidden, weights, targets, torch.full((70,), 1 / 70, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 15, 16, 17, 63, 65, 127, 129, 255, 257, 2000])
def test_vocabularies_around_the_tiles(dtype, V):
    hidden, weights, targets = make(dtype, 33, 128, [V, 3], seed=V)
    check_all(dtype, hidden, weights, targets, torch.full((33,), 1 / 33, device="cuda"))


@pytest.mark.parametrize("T,D,V", [(1, 4096, 20000), (20, 1248, 30000), (700, 2048, 9000), (2, 8192, 600)])
def test_long_reductions_keep_float_precision(T, D, V):
    """lse of 16-bit inputs within a few float roundings of 64 bits: the sums
    of thousands of products do not drift.  (A rounding each of a logit's 32 or
    fewer partial sums and of 32 products in a run, at most 2^-23 of the logit
    each, signs mixed: 4 sqrt(64) 2^-23 of the largest logit.)"""
    hidden, weights, targets = make("bf16", T, D, [V], seed=D)
    loss, lse = loss_of(hidden, weights, targets)
    z = hidden.double() @ weights[0].double().t()
    tol = 4 * 8 * 2.0 ** -23 * z.abs().amax(1) + 2.0 ** -22 * (torch.logsumexp(z, 1).abs() + 1)
    assert ((lse.double() - torch.logsumexp(z, 1)).abs() <= tol).all()
    picked = z.gather(1, targets[:, None])[:, 0]
    assert ((loss.double() - (torch.logsumexp(z, 1) - picked)).abs() <= 2 * tol).all()


def test_few_tokens_large_vocabulary():
    """Reductions over the vocabulary cut into slices."""
    for T, D, pieces in ((1, 512, [30000]), (20, 640, [16192, 9000]), (300, 128, [50000])):
        hidden, weights, targets = make("bf16", T, D, pieces, seed=T)
        check_all("bf16", hidden, weights, targets, torch.full((T,), 1 / T, device="cuda"))


def test_rows_past_32_bit_offsets():
    """Weights, their gradients and the hidden states as narrow views of
    buffers of several GB."""
    T, D, V, wide = 300, 64, 70000, 32768
    hidden, weights, targets = make("bf16", T, D, [V], seed=21)
    big_w = torch.empty((V, wide), dtype=torch.bfloat16, device="cuda")
    big_w[:, 7 * D:8 * D] = weights[0]
    big_h = torch.empty((T, 1 << 23), dtype=torch.bfloat16, device="cuda")
    big_h[:, :D] = hidden
    big_d = torch.empty((V, wide), dtype=torch.bfloat16, device="cuda")
    h, w, d = big_h[:, :D], [big_w[:, 7 * D:8 * D]], [big_d[:, D:2 * D]]
    assert (V - 1) * wide * 2 > 1 << 32 and (T - 1) * (1 << 23) * 2 > 1 << 32
    dloss = torch.full((T,), 1 / T, device="cuda")
    loss, lse = loss_of(h, w, targets)
    plain = formula(hidden, weights, targets)
    near(lse, plain["lse"], "lse")
    near(loss, plain["loss"], "loss")
    tps.ar_vocab_loss_grad(h, w, targets, lse, dloss, dhidden=None, dweights=d, ignore_index=IGNORE)
    want = formula(hidden, weights, targets, dloss, "bf16")
    near(d[0], want["dweights"][0], "dweights")
    out = torch.empty_like(big_h)[:, 2 * D:3 * D]
    tps.ar_vocab_loss_grad(h, w, targets, lse, dloss, dhidden=[out], ignore_index=IGNORE)
    near(out, want["dhidden"][0], "dhidden")


def test_many_pieces_some_empty():
    hidden, weights, targets = make("bf16", 90, 96, [0, 5, 300, 0, 1, 64, 257, 0, 12, 700, 3, 0, 90, 256, 2, 40], seed=22, ignored=0.2)
    check_all("bf16", hidden, weights, targets, torch.full((90,), 1 / 90, device="cuda"))


@pytest.mark.parametrize("T", [4095, 4097, 20000])
def test_long_token_lists(T):
    hidden, weights, targets = make("bf16", T, 64, [200, 60], seed=T, ignored=0.5)
    check_all("bf16", hidden, weights, targets, torch.full((T,), 1 / T, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 4, 5, 16, 17])
@pytest.mark.parametrize("pad,lead,D", [(3, 0, 77), (5, 1, 333), (0, 0, 1023), (0, 3, 64)])
def test_few_tokens_against_rows_off_boundaries(dtype, T, pad, lead, D):
    hidden, weights, targets = make(dtype, T, D, [333, 0, 1, 2050], seed=T + D, ignored=0.2, pad=pad, lead=lead)
    check_all(dtype, hidden, weights, targets, torch.full((T,), 1 / T, device="cuda"), pad, lead)


def test_few_float_tokens_with_infinite_and_nan_logits():
    h = torch.zeros((3, 40), device="cuda")
    w = torch.zeros((100, 40), device="cuda")
    w[:, 0] = torch.linspace(-1, 1, 100, device="cuda")
    w[7, 1], w[9, 2] = float("inf"), float("nan")
    h[:, 0] = 2
    h[1, 1] = 1
    targets = torch.tensor([3, 3, IGNORE], device="cuda")
    loss, lse = loss_of(h, [w], targets)
    # row 7 meets a zero times infinity, row 9 a zero times NaN, in every token
    assert torch.isnan(lse).all() and torch.isnan(loss[:2]).all() and loss[2] == 0
    w[9, 2] = 0
    w[7, 1] = 0
    _, lse = loss_of(h, [w], targets)
    assert torch.allclose(lse, torch.logsumexp(h @ w.t(), 1), rtol=1e-6)
