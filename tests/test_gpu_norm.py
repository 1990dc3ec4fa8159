"""ar_reduce_norm and its gradient against plain implementations: the sums bit
for bit, the rest against 64 bits within what float steps and one rounding leave."""
import itertools

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.gpu_util import TORCH_DTYPE
from tests.norm_ref import HALF_STEP, adds, checkpoint_values, norm_backward, norm_forward

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]
PAIRS = list(itertools.product(TYPES, TYPES))
EPS = 1e-5
POISON = 0x5A


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


class Rows:
    """ne1 rows of ne0 elements `pad` apart, `lead` elements into a poisoned buffer."""

    def __init__(self, ne0, ne1, dst, pad=0, lead=0, fill=None):
        self.dtype = TORCH_DTYPE[dst]
        es = self.dtype.itemsize
        n = lead + (ne1 - 1) * (ne0 + pad) + ne0
        self.back = torch.full((n * es + 64,), POISON, dtype=torch.uint8, device="cuda")
        flat = self.back[:n * es].view(self.dtype)
        self.t = flat[lead:].as_strided((ne1, ne0), (ne0 + pad, 1))
        self.bytes = (ne0 + pad) * es
        self.shape = (ne0, ne1, pad, lead, es)
        if fill is not None:
            self.t.copy_(fill)

    def check_padding(self):
        ne0, ne1, pad, lead, es = self.shape
        b = self.back.clone()
        inner = b[lead * es:lead * es + ((ne1 - 1) * (ne0 + pad) + ne0) * es]
        inner.as_strided((ne1, ne0 * es), ((ne0 + pad) * es, 1), lead * es).fill_(POISON)
        assert (b == POISON).all(), "bytes around the rows were written"


def normal(shape, seed, outliers=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, device="cuda", generator=g)
    if outliers:
        x = torch.where(torch.rand(shape, device="cuda", generator=g) < 0.003, x * 50, x)
    return x


def float_sum(srcs, wire, dst, bias, res):
    """h in the stated order of float steps."""
    acc = None
    for s in srcs:
        x = torch.zeros_like(acc if acc is not None else srcs[-1].t, dtype=torch.float32) if s is None else \
            s.t.to(TORCH_DTYPE[wire]).float()
        acc = x if acc is None else acc + x
    if bias is not None:
        acc = acc + bias.float()
    if res is not None:
        acc = acc + res.float()
    return acc.to(TORCH_DTYPE[dst])


def close(got, want, slack, dtype, what):
    err = (got.double() - want).abs()
    bound = HALF_STEP[dtype] * (want.abs() + slack) + slack + (2.0 ** -25 if dtype == torch.float16 else 1e-40)
    bad = ~((err <= bound) | (got.isnan() & want.isnan()) | (got.double() == want))
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(err / bound).nan_to_num().max().item():.2f} times the bound"


def forward(R, ne0, ne1, dst="f32", wire="bf16", kind="layer", n_dsts=1, n_sums=1, pads=(0,), lead=0, bias=False,
            residual="", affine="both", inactive=(), in_place="", eps=EPS, keep="", seed=3, stream=None, data=None):
    tps.ar_init(R, max(1, ne0 * ne1))
    pad = itertools.cycle(pads)
    shape = (ne1, ne0)
    srcs = [None if r in inactive else Rows(ne0, ne1, dst, next(pad), lead, normal(shape, seed + r) if data is None else data)
            for r in range(R)]
    ys = [Rows(ne0, ne1, dst, next(pad), lead) for _ in range(n_dsts)]
    sums = [Rows(ne0, ne1, dst, next(pad), lead) for _ in range(n_sums)]
    row = lambda k: Rows(ne0, 1, dst, 0, lead, normal((1, ne0), seed + 20 + k, False)).t[0]  # noqa: E731
    weight = row(0) if affine else None
    shift = row(1) if affine == "both" else None
    bias_t = row(2) if bias else None
    res = res_bytes = None
    if residual:
        res = Rows(ne0, 1 if residual == "row" else ne1, dst, next(pad), lead, normal((1 if residual == "row" else ne1, ne0), seed + 30))
        res_bytes = 0 if residual == "row" else res.bytes
    h = float_sum(srcs, wire, dst, bias_t, None if res is None else res.t)
    outs = ys + sums
    if in_place == "source":
        ys[0] = srcs[0]
    if in_place == "residual":
        sums[0] = res
    if in_place == "both":
        ys[0], sums[0] = srcs[0], res
    mean, rstd = (torch.full((ne1 + 2,), 7.0, device="cuda") for _ in range(2))
    ck = tps.empty_checkpoint(ne0, ne1, keep) if keep else None
    lay = tps.make_layout(ne0, ne1, [ne0 * 4 if s is None else s.bytes for s in srcs], [y.bytes for y in ys],
                          None if res is None else res.t, res_bytes, inactive)
    tps.ar_reduce_norm([None if s is None else s.t for s in srcs], [y.t for y in ys], lay,
                       tps.make_norm(eps, weight, shift, bias_t, kind), dst, wire, sums=[s.t for s in sums],
                       sum_row_bytes=[s.bytes for s in sums] or None, mean=mean[1:-1], rstd=rstd[1:-1], checkpoint=ck,
                       stream=stream)
    torch.cuda.synchronize()
    y, m, r, slack = norm_forward(h.double(), weight, shift, eps, kind == "rms")
    for s in sums:
        assert torch.equal(s.t, h) or torch.equal(s.t.isnan(), h.isnan()) and torch.equal(s.t[~h.isnan()], h[~h.isnan()])
    for k, out in enumerate(ys):
        close(out.t, y, slack, h.dtype, f"y {k}")
    close(mean[1:-1], m, adds(ne0) * 2.0 ** -24 * h.double().abs().mean(1), torch.float32, "mean")
    close(rstd[1:-1], r, adds(ne0) * 2.0 ** -24 * r, torch.float32, "rstd")
    assert mean[0] == mean[-1] == rstd[0] == rstd[-1] == 7
    if kind == "rms":
        assert (mean[1:-1] == 0).all()
    for o in outs:
        o.check_padding()
    return ys, sums, mean[1:-1], rstd[1:-1], ck, h


SHAPES = [(1, 1), (3, 5), (8, 3), (9, 300), (31, 7), (33, 77), (64, 33), (255, 40), (257, 9), (1000, 3), (2049, 2), (4096, 5),
          (4099, 1), (8192, 3), (8200, 2), (16384, 2), (20001, 2)]


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("ne0,ne1", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_shapes(dst, ne0, ne1, kind):
    forward(3, ne0, ne1, dst, "bf16", kind, n_dsts=2, bias=True, residual="row")


@pytest.mark.parametrize("ne0", [70001, 131080, 300007])
@pytest.mark.parametrize("dst", ["f32", "bf16"])
def test_very_long_rows(ne0, dst):
    forward(2, ne0, 2, dst, "bf16", residual="full", keep="int8")


@pytest.mark.parametrize("dst,wire", PAIRS)
@pytest.mark.parametrize("R", [1, 2, 5])
@pytest.mark.parametrize("ne0", [1029, 96, 2112])
def test_type_pairs(dst, wire, R, ne0):
    forward(R, ne0, 5, dst, wire, n_dsts=2, bias=True, residual="full")


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("pads,lead", [((0,), 0), ((0,), 1), ((8,), 0), ((8,), 3), ((3,), 0), ((3,), 1), ((1, 2, 5), 0),
                                       ((0, 8, 3), 2), ((13,), 0), ((4,), 4)])
@pytest.mark.parametrize("ne0", [40, 777, 1024, 5001])
def test_strides_and_starts(dst, pads, lead, ne0):
    forward(3, ne0, 9, dst, "bf16", pads=pads, lead=lead, n_dsts=3, n_sums=2, bias=True, residual="full")


@pytest.mark.parametrize("affine", ["", "weight", "both"])
@pytest.mark.parametrize("n_sums", [0, 2])
def test_optional_parts(affine, n_sums):
    forward(2, 520, 17, "bf16", affine=affine, n_sums=n_sums, residual="full")


@pytest.mark.parametrize("R", [8, 16])
@pytest.mark.parametrize("dst", TYPES)
def test_many_ranks_and_destinations(dst, R):
    forward(R, 515, 4, dst, "f16", n_dsts=R, n_sums=R, bias=True)


@pytest.mark.parametrize("inactive", [(0,), (1, 2)])
@pytest.mark.parametrize("ne0", [260, 2048])
def test_inactive_ranks(inactive, ne0):
    forward(3, ne0, 6, "bf16", "bf16", inactive=inactive, bias=True, residual="row")


@pytest.mark.parametrize("ne0", [96, 2048])
def test_no_active_rank_normalises_the_residual(ne0):
    """The norm of a tensor that is there already, and of nothing at all."""
    tps.ar_init(2, 5 * ne0)
    x, y = normal((5, ne0), 4), torch.empty((5, ne0), device="cuda")
    for res in (x, None):
        lay = tps.make_layout(ne0, 5, residual=res, inactive=(0, 1))
        tps.ar_reduce_norm([None, None], [y], lay, tps.make_norm(EPS), "f32", "f32")
        want, _, _, slack = norm_forward((x if res is x else torch.zeros_like(x)).double(), None, None, EPS, False)
        close(y, want, slack, torch.float32, "y")


@pytest.mark.parametrize("pads,lead", [((0,), 0), ((3,), 1)])
@pytest.mark.parametrize("which", ["source", "residual", "both"])
@pytest.mark.parametrize("ne0", [100, 4100, 140001])
def test_in_place(pads, lead, which, ne0):
    forward(2, ne0, 5, "f32", "f16", pads=pads, lead=lead, n_dsts=2, residual="full", in_place=which)


@pytest.mark.parametrize("ne1", [1, 151, 153, 700, 70_001])
def test_row_counts(ne1):
    forward(2, 72, ne1, "bf16", n_dsts=2, residual="full")


def test_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        forward(2, 4096, 64, "f32", "bf16", n_dsts=2, residual="full", stream=s)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("ne0", [64, 1000, 9000])
def test_rows_far_from_zero_and_constant_rows(ne0, kind):
    x = normal((6, ne0), 5, False)
    x[0] += 1000
    x[1] -= 30000
    x[2] = 0
    x[3] = 1000.1
    x[4] *= 1e-6
    x[5] *= 1e15
    forward(1, ne0, 6, "f32", "f32", kind, data=x)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_with_no_norm_leaves_the_others(bad):
    x = normal((5, 600), 6)
    x[2, 17] = bad
    ys, sums, mean, rstd, ck, h = forward(1, 600, 5, "f32", "f32", data=x, keep="e4m3")
    assert ys[0].t[2].isnan().all() and not ys[0].t[[0, 1, 3, 4]].isnan().any() and rstd[2].isnan()


def test_nothing_to_do_and_refusals():
    tps.ar_init(2, 64)
    x = torch.zeros(64, device="cuda")
    y = torch.full((64,), 5.0, device="cuda")
    for ne0, ne1 in ((0, 4), (4, 0)):
        tps.ar_reduce_norm([x, x], [x], tps.make_layout(ne0, ne1), tps.make_norm(), "f32")
    lay, f = tps.make_layout(16, 4), lambda n: torch.empty(n, device="cuda")  # noqa: E731
    stat = f(4)
    grad = lambda **kw: tps.ar_reduce_norm_grad(x, kw.pop("h", x), [y], kw.pop("lay", lay), tps.make_norm(),  # noqa: E731
                                                kw.pop("mean", stat), kw.pop("rstd", stat), "f32", **kw)
    for call in (lambda: tps.ar_reduce_norm([x, None], [y], lay, tps.make_norm(), "f32"),
                 lambda: tps.ar_reduce_norm([x, x], [y], lay, tps.make_norm(-1.0), "f32"),
                 lambda: tps.ar_reduce_norm([x, x], [y], lay, tps.make_norm(), "f32", checkpoint=tps.empty_checkpoint(16, 3)),
                 lambda: grad(lay=tps.make_layout(16, 4, inactive=(0,))),
                 lambda: grad(mean=None), lambda: grad(rstd=None),
                 lambda: grad(h=tps.empty_checkpoint(17, 4)),
                 lambda: grad(dweight=y[:16]), lambda: grad(dbias=x[:16]),
                 lambda: grad(dshift=f(16), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(tps.ARError):
            call()
    torch.cuda.synchronize()
    assert (y == 5).all()
    with pytest.raises(ValueError):
        grad(dweight=f(15))
    with pytest.raises(ValueError):
        tps.ar_reduce_norm([x, x], [y], lay, tps.make_norm(), "f32", mean=f(3))


# ---- gradient -----------------------------------------------------------------------

def backward(ne0, ne1, dst="f32", kind="layer", n_dxs=1, pads=(0,), lead=0, dsum=False, weight=True, keep="",
             sums=("dweight", "dshift", "dbias"), in_place="", seed=5, stream=None):
    tps.ar_init(2, max(1, ne0 * ne1))
    pad = itertools.cycle(pads)
    shape = (ne1, ne0)
    dy = Rows(ne0, ne1, dst, next(pad), lead, normal(shape, seed, False))
    h = Rows(ne0, ne1, dst, next(pad), lead, normal(shape, seed + 1) + 0.5)
    ds = Rows(ne0, 1 if dsum == "row" else ne1, dst, next(pad), lead, normal((1 if dsum == "row" else ne1, ne0), seed + 2, False)) if dsum else None
    dxs = [Rows(ne0, ne1, dst, next(pad), lead) for _ in range(n_dxs)]
    w = Rows(ne0, 1, dst, 0, lead, normal((1, ne0), seed + 3, False) + 1).t[0] if weight else None
    x = h.t.double()
    mean = x.mean(1)
    base = 0 if kind == "rms" else mean[:, None]
    rstd = (1 / torch.sqrt(((x - base) ** 2).mean(1) + EPS)).float()
    mean = mean.float()
    ck = None
    if keep:
        ck = tps.empty_checkpoint(ne0, ne1, keep)
        tps.ar_checkpoint_pack(h.t, ck)
        if ne0 * ne1 < 50_000:
            x = torch.from_numpy(checkpoint_values(x.cpu().numpy(), keep)[0]).cuda()
        else:  # the tables take too long; the values that are read back are tested against them elsewhere
            back = torch.empty(shape, device="cuda")
            tps.ar_checkpoint_unpack(ck, back)
            x = back.double()
    want = norm_backward(dy.t.double(), x, mean.double(), rstd.double(), w, None if ds is None else ds.t.double(), kind == "rms")
    outs = list(dxs)
    given = {"dy": dy, "h": h, "dsum": ds}
    if in_place:
        dxs[0] = given[in_place]
    got = {k: torch.full((ne0 + 2,), 7.0, device="cuda") if k in sums else None for k in ("dweight", "dshift", "dbias")}
    lay = tps.make_layout(ne0, ne1, [dy.bytes] if keep else [dy.bytes, h.bytes], [d.bytes for d in dxs],
                          None if ds is None else ds.t, None if ds is None else 0 if dsum == "row" else ds.bytes)
    tps.ar_reduce_norm_grad(dy.t, ck if keep else h.t, [d.t for d in dxs], lay, tps.make_norm(EPS, w, kind=kind),
                            None if kind == "rms" else mean, rstd, dst,
                            **{k: None if v is None else v[1:-1] for k, v in got.items()}, stream=stream)
    torch.cuda.synchronize()
    for k, d in enumerate(dxs):
        close(d.t, *want["dx"], d.dtype, f"dx {k}")
    for k, v in got.items():
        if v is not None:
            close(v[1:-1], *want[k], torch.float32, k)
            assert v[0] == v[-1] == 7
    for o in outs:
        o.check_padding()
    return dxs, got


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("ne0,ne1", SHAPES + [(40, 5000), (520, 2100), (4096, 257)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_shapes(dst, ne0, ne1, kind):
    backward(ne0, ne1, dst, kind, n_dxs=2, dsum=kind == "layer")


@pytest.mark.parametrize("ne0", [70001, 131080, 300007])
@pytest.mark.parametrize("dst", ["f32", "bf16"])
def test_grad_of_very_long_rows(ne0, dst):
    backward(ne0, 3, dst, dsum=True)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("pads,lead", [((0,), 1), ((8,), 0), ((3,), 0), ((1, 2, 5), 0), ((0, 8, 3), 2), ((13,), 1)])
@pytest.mark.parametrize("ne0", [40, 777, 1024, 5001])
def test_grad_strides_and_starts(dst, pads, lead, ne0):
    backward(ne0, 37, dst, pads=pads, lead=lead, n_dxs=3, dsum=True)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("keep", ["e4m3", "int8"])
@pytest.mark.parametrize("ne0,ne1", [(1, 3), (33, 20), (777, 9), (4096, 5), (8200, 2)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_from_a_checkpoint(dst, keep, ne0, ne1, kind):
    backward(ne0, ne1, dst, kind, keep=keep, n_dxs=2, dsum=True)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("keep", ["", "e4m3", "int8"])
@pytest.mark.parametrize("ne0,pad", [(544, 0), (1029, 11), (4099, 13), (4096, 0), (9001, 7), (20001, 15)])
@pytest.mark.parametrize("dsum", [False, True, "row"])
def test_grad_of_many_rows_on_vector_boundaries(dst, keep, ne0, pad, dsum):
    """Rows that are brought by copies of whole vectors, with odd ends, several blocks to a row, and more rows than
    blocks."""
    assert (ne0 + pad) * TORCH_DTYPE[dst].itemsize % 32 == 0
    backward(ne0, 320, dst, "rms" if ne0 == 4099 else "layer", n_dxs=2, pads=(pad,), dsum=dsum, keep=keep,
             sums=("dweight", "dshift") if ne0 == 544 else ("dweight", "dshift", "dbias"))
    assert tps.ar_query("device_status") == 0


@pytest.mark.parametrize("which", ["dy", "h", "dsum"])
def test_grad_of_many_rows_in_place(which):
    backward(2048, 700, "bf16", dsum=True, n_dxs=2, in_place=which)


@pytest.mark.parametrize("sums", [(), ("dweight",), ("dshift",), ("dbias",), ("dweight", "dbias")])
@pytest.mark.parametrize("ne0", [300, 4099])
def test_grad_sums_are_optional(sums, ne0):
    backward(ne0, 70, sums=sums, n_dxs=4, weight=False)


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("which", ["dy", "h", "dsum"])
@pytest.mark.parametrize("ne0", [100, 4100, 140001])
def test_grad_in_place(lead, which, ne0):
    backward(ne0, 33 if ne0 < 9000 else 3, lead=lead, n_dxs=2, dsum=True, in_place=which)


@pytest.mark.parametrize("R", [16])
def test_grad_many_destinations(R):
    backward(515, 20, "bf16", n_dxs=R, dsum=True)


@pytest.mark.parametrize("ne1", [1, 151, 153, 700, 70_001])
def test_grad_row_counts(ne1):
    backward(72, ne1, "bf16", dsum=True)


def test_grad_is_repeatable():
    a = backward(2048, 500, "bf16", dsum=True)
    b = backward(2048, 500, "bf16", dsum=True)
    assert torch.equal(a[0][0].t, b[0][0].t) and all(torch.equal(a[1][k], b[1][k]) for k in a[1])


def test_grad_of_no_rows_is_zero():
    tps.ar_init(1, 64)
    x, outs = torch.zeros(16, device="cuda"), [torch.full((16,), 3.0, device="cuda") for _ in range(3)]
    tps.ar_reduce_norm_grad(x, x, [torch.zeros(16, device="cuda")], tps.make_layout(16, 0), tps.make_norm(), None, None, "f32", *outs)
    assert all((o == 0).all() for o in outs)


def test_grad_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        backward(4096, 300, "f32", n_dxs=2, dsum=True, stream=s)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_grad_matches_autograd(kind):
    """The whole step differentiated in 64 bits."""
    ne0, ne1 = 300, 21
    tps.ar_init(2, ne0 * ne1)
    srcs = [normal((ne1, ne0), k) for k in range(2)]
    res, dy, ds = (normal((ne1, ne0), 5 + k, False) for k in range(3))
    weight, shift, bias = (normal((ne0,), 9 + k, False) for k in range(3))
    leaves = [t.double().requires_grad_() for t in (srcs[0], res, weight, shift, bias)]
    h = leaves[0] + srcs[1].double() + leaves[4] + leaves[1]
    d = h - h.mean(1, keepdim=True) if kind == "layer" else h
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS) * leaves[2] + leaves[3]
    (y * dy.double()).sum().add((h * ds.double()).sum()).backward()
    out, total, dx = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(dy)
    mean, rstd = torch.empty(ne1, device="cuda"), torch.empty(ne1, device="cuda")
    sums = [torch.empty(ne0, device="cuda") for _ in range(3)]
    norm = tps.make_norm(EPS, weight, shift, bias, kind)
    tps.ar_reduce_norm(srcs, [out], tps.make_layout(ne0, ne1, residual=res), norm, "f32", "f32", sums=[total], mean=mean, rstd=rstd)
    tps.ar_reduce_norm_grad(dy, total, [dx], tps.make_layout(ne0, ne1, residual=ds), norm, mean, rstd, "f32", *sums)
    for got, leaf in ((out, y.detach()), (dx, leaves[0].grad), (dx, leaves[1].grad), (sums[0], leaves[2].grad),
                      (sums[1], leaves[3].grad), (sums[2], leaves[4].grad)):
        leaf = leaf.grad if leaf.requires_grad else leaf
        # sums of at most 300 terms of size about 1: a few hundred roundings of the largest
        assert ((got.double() - leaf).abs() <= 300 * 2.0 ** -24 * leaf.abs().max()).all()


def test_grad_matches_differences():
    """Central differences of the forward pass with a step that leaves a third-order error below the tolerance."""
    ne0, ne1, step = 48, 4, 2.0 ** -6
    tps.ar_init(1, ne0 * ne1)
    x, dy = normal((ne1, ne0), 1, False), normal((ne1, ne0), 2, False)
    weight, shift, bias = (normal((ne0,), 3 + k, False) for k in range(3))
    mean, rstd = torch.empty(ne1, device="cuda"), torch.empty(ne1, device="cuda")
    out, total = torch.empty_like(x), torch.empty_like(x)
    lay = tps.make_layout(ne0, ne1)

    def value():
        tps.ar_reduce_norm([x], [out], lay, tps.make_norm(EPS, weight, shift, bias), "f32", "f32", sums=[total], mean=mean, rstd=rstd)
        return (out.double() * dy.double()).sum().item()
    value()
    dx, sums = torch.empty_like(x), [torch.empty(ne0, device="cuda") for _ in range(3)]
    tps.ar_reduce_norm_grad(dy, total, [dx], lay, tps.make_norm(EPS, weight, shift, bias), mean, rstd, "f32", *sums)
    # 192 outputs below 8, each off by 64 roundings at most, over twice the step; and step^2 / 6 times a third
    # derivative below 32
    tol = ne0 * ne1 * 8 * 2.0 ** -24 * 4 / (2 * step) + step * step / 6 * 32
    for t, grad, at in ((x, dx, (0, 0)), (x, dx, (3, 47)), (weight, sums[0], (5,)), (shift, sums[1], (6,)), (bias, sums[2], (7,))):
        keep = t[at].item()
        t[at] = keep + step
        up, x1 = value(), t[at].item()
        t[at] = keep - step
        down, x0 = value(), t[at].item()
        t[at] = keep
        assert abs((up - down) / (x1 - x0) - grad[at].item()) <= tol


def test_rows_past_32_bit_offsets():
    """Narrow rows of buffers of several GB, forward and backward."""
    ne0, ne1, wide = 72, 2100, 1 << 20
    tps.ar_init(1, ne0 * ne1)
    assert (ne1 - 1) * wide * 4 > 1 << 32
    x, y, h = (torch.empty((ne1, wide), device="cuda")[:, 5:5 + ne0] for _ in range(3))
    x.copy_(normal((ne1, ne0), 3))
    lay = tps.make_layout(ne0, ne1, [wide * 4], [wide * 4])
    mean, rstd = torch.empty(ne1, device="cuda"), torch.empty(ne1, device="cuda")
    tps.ar_reduce_norm([x], [y], lay, tps.make_norm(EPS), "f32", "f32", sums=[h], sum_row_bytes=[wide * 4], mean=mean, rstd=rstd)
    want, m, r, slack = norm_forward(x.double(), None, None, EPS, False)
    assert torch.equal(h, x)
    close(y, want, slack, torch.float32, "y")
    dy = y.contiguous()
    back = norm_backward(dy.double(), x.double(), mean.double(), rstd.double(), None, None, False)
    tps.ar_reduce_norm_grad(dy, h, [y], tps.make_layout(ne0, ne1, [ne0 * 4, wide * 4], [wide * 4]), tps.make_norm(EPS), mean, rstd, "f32")
    close(y, *back["dx"], torch.float32, "dx")


@pytest.mark.parametrize("ne0,ne1", [(512, 64), (4099, 200)])
def test_in_a_graph_with_calls_back_to_back(ne0, ne1):
    """Forward and backward twice in one captured graph, replayed on new inputs, against eager calls."""
    tps.ar_init(2, ne0 * ne1)
    srcs = [normal((ne1, ne0), k).bfloat16() for k in range(2)]
    dy = normal((ne1, ne0), 7, False).bfloat16()
    weight = normal((ne0,), 8, False).bfloat16()
    lay, norm = tps.make_layout(ne0, ne1), tps.make_norm(EPS, weight)
    ck = tps.empty_checkpoint(ne0, ne1, "int8")

    def step(out):
        y, dx, mean, rstd, dw, ds = out
        tps.ar_reduce_norm(srcs, [y], lay, norm, "bf16", "bf16", mean=mean, rstd=rstd, checkpoint=ck)
        tps.ar_reduce_norm_grad(dy, ck, [dx], lay, norm, mean, rstd, "bf16", dw, ds)

    def buffers():
        f = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
        return [torch.zeros_like(dy), torch.zeros_like(dy), f(ne1), f(ne1), f(ne0), f(ne0)]
    a, b, c = buffers(), buffers(), buffers()
    step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
        step(b)
    for seed in (40, 50):
        for k, s in enumerate(srcs):
            s.copy_(normal((ne1, ne0), seed + k))
        dy.copy_(normal((ne1, ne0), seed + 9, False))
        g.replay()
        step(c)
        torch.cuda.synchronize()
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, z) and torch.equal(y, z)
