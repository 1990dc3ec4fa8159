"""ar_reduce_dropout and its gradient against plain implementations: values
bit for bit against the stated order of float steps, column sums against 64
bits."""
import itertools

import numpy as np
import pytest
import torch

import oracle
import tensor_partial_sum_gb300 as tps
from tests.gpu_util import to_device
from tests.libcasts import assert_same
from tests.philox import keep_mask, scale_of
from tests.test_gpu_ex import ES, rows_of, srcs_for, strided_device

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]
PAIRS = list(itertools.product(TYPES, TYPES))
SEED, OFFSET = 0x0123456789ABCDEF, (5 << 32) | 9


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def wide(name, a):
    return np.asarray(oracle.widen(name, a), np.float32)


def expected(srcs, wire, dst, ne0, ne1, p, bias=None, res=None, res_row=False, inactive=(), seed=SEED, offset=OFFSET):
    """The operator in numpy float32 steps."""
    acc = None
    with np.errstate(all="ignore"):
        for r, s in enumerate(srcs):
            x = np.zeros(ne0 * ne1, np.float32) if r in inactive else wide(wire, oracle.round_to(wire, wide(dst, s)))
            acc = x if acc is None else acc + x
        acc = acc.reshape(ne1, ne0)
        if bias is not None:
            acc = acc + wide(dst, bias)[None]
        acc = np.where(keep_mask(ne0, ne1, p, seed, offset), acc * scale_of(p), np.float32(0))
        if res is not None:
            acc = acc + (wide(dst, res)[None] if res_row else wide(dst, res).reshape(ne1, ne0))
        return oracle.round_to(dst, np.ascontiguousarray(acc, np.float32).ravel())


def run_forward(R, ne0, ne1, dst, wire, p=0.25, pads=(0,), lead=0, n_dsts=1, bias=False, residual="", inactive=(),
                seed=3, in_place=False, stream=None):
    """One call on rows `pads[k % len]` elements apart starting `lead` elements
    into their buffers, checked in every destination and in the padding."""
    es = ES[dst]
    tps.ar_init(R, max(1, ne0 * ne1))
    pad = itertools.cycle(pads)
    srcs = srcs_for(seed, R, ne0 * ne1, dst)
    s_pad = [next(pad) for _ in range(R)]
    s_t = [None if r in inactive else strided_device(srcs[r], ne0, ne1, ne0 + s_pad[r], dst, lead)[0] for r in range(R)]
    d_pad = [next(pad) for _ in range(n_dsts)]
    d_t = [strided_device(None, ne0, ne1, ne0 + d_pad[d], dst, lead) for d in range(n_dsts)]
    if in_place:
        d_pad[0], d_t[0] = s_pad[0], (s_t[0], None)
    bias_np = srcs_for(seed + 1, 1, ne0, dst)[0] if bias else None
    bias_t = strided_device(bias_np, ne0, 1, ne0, dst, lead)[0][:ne0] if bias else None
    res_np = res_t = res_bytes = None
    if residual:
        row = residual == "row"
        res_np = srcs_for(seed + 2, 1, ne0 if row else ne0 * ne1, dst)[0]
        r_pad = next(pad)
        res_t = strided_device(res_np, ne0, 1 if row else ne1, ne0 + (0 if row else r_pad), dst, lead)[0]
        res_bytes = 0 if row else (ne0 + r_pad) * es
    lay = tps.make_layout(ne0, ne1, [(ne0 + k) * es for k in s_pad], [(ne0 + k) * es for k in d_pad], res_t, res_bytes,
                          inactive)
    tps.ar_reduce_dropout(s_t, [t for t, _ in d_t], lay, tps.make_dropout(p, SEED, OFFSET, bias_t), dst, wire, stream)
    torch.cuda.synchronize()
    exp = expected(srcs, wire, dst, ne0, ne1, p, bias_np, res_np, residual == "row", inactive)
    for d, (t, back) in enumerate(d_t):
        assert_same(rows_of(t, ne0, ne1, ne0 + d_pad[d], dst), exp, dst, f"{R} {ne0}x{ne1} pads={pads} d={d}")
        if back is not None:
            b = back.cpu().numpy()
            assert (b[:lead * es] == 0x5A).all(), "bytes before the first row were written"
            for j in range(ne1):
                end = (lead + j * (ne0 + d_pad[d]) + ne0) * es
                assert (b[end:end + d_pad[d] * es] == 0x5A).all(), "padding written"


@pytest.mark.parametrize("dst,wire", PAIRS)
@pytest.mark.parametrize("R", [1, 2, 5])
def test_type_pairs(dst, wire, R):
    run_forward(R, 1029, 5, dst, wire, n_dsts=2, bias=True, residual="full")


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("ne0,ne1", [(1, 1), (3, 5), (8, 3), (9, 300), (33, 77), (256, 9), (1000, 3), (2049, 2),
                                     (4099, 1), (50_001, 2)])
@pytest.mark.parametrize("residual", ["", "row"])
def test_shapes(dst, ne0, ne1, residual):
    run_forward(3, ne0, ne1, dst, "bf16", n_dsts=2, bias=True, residual=residual)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("pads,lead", [((0,), 0), ((0,), 1), ((8,), 0), ((8,), 3), ((3,), 0), ((3,), 1), ((1, 2, 5), 0),
                                       ((0, 8, 3), 2), ((13,), 0), ((4,), 4)])
@pytest.mark.parametrize("ne0", [777, 1024])
def test_strides_and_starts(dst, pads, lead, ne0):
    run_forward(3, ne0, 9, dst, "bf16", pads=pads, lead=lead, n_dsts=3, bias=True, residual="full")


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_probabilities(p):
    run_forward(2, 520, 17, "f32", "bf16", p=p, bias=True, residual="full")


@pytest.mark.parametrize("R", [8, 16])
@pytest.mark.parametrize("dst", TYPES)
def test_many_ranks_and_destinations(dst, R):
    run_forward(R, 515, 4, dst, "f16", n_dsts=R, bias=True)


@pytest.mark.parametrize("inactive", [(0,), (1, 2), (0, 1, 2)])
def test_inactive_ranks(inactive):
    run_forward(3, 260, 6, "bf16", "bf16", inactive=inactive, bias=True, residual="row")


@pytest.mark.parametrize("pads,lead", [((0,), 0), ((3,), 1)])
def test_in_place(pads, lead):
    run_forward(2, 1000, 6, "f32", "f16", pads=pads, lead=lead, n_dsts=2, residual="full", in_place=True)


def test_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run_forward(2, 4096, 64, "f32", "bf16", n_dsts=2, bias=True, residual="full", stream=s)


def test_a_dropped_element_is_zero_whatever_the_sum_holds():
    ne0, ne1 = 512, 8
    tps.ar_init(1, ne0 * ne1)
    x = torch.full((ne1, ne0), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = torch.empty_like(x)
    tps.ar_reduce_dropout([x], [y], tps.make_layout(ne0, ne1), tps.make_dropout(0.5, 7), "f32", "f32")
    keep = keep_mask(ne0, ne1, 0.5, 7, 0)
    got = y.cpu().numpy()
    assert (got[~keep] == 0).all() and not np.isfinite(got[keep]).any()


def test_nothing_to_do():
    tps.ar_init(2, 64)
    x = torch.zeros(64, device="cuda")
    for ne0, ne1 in ((0, 4), (4, 0)):
        tps.ar_reduce_dropout([x, x], [x], tps.make_layout(ne0, ne1), tps.make_dropout(0.5, 7), "f32")


# ---- gradient ------------------------------------------------------------------

def run_grad(ne0, ne1, dst, p=0.25, pads=(0,), lead=0, n_dxs=1, dbias=True, dres=True, in_place=False, seed=5):
    es = ES[dst]
    tps.ar_init(1, max(1, ne0 * ne1))
    rng = np.random.Generator(np.random.PCG64(seed))
    dy = oracle.round_to(dst, rng.standard_normal(ne0 * ne1, dtype=np.float32))
    pad = itertools.cycle(pads)
    y_pad = next(pad)
    dy_t, _ = strided_device(dy, ne0, ne1, ne0 + y_pad, dst, lead)
    x_pad = [next(pad) for _ in range(n_dxs)]
    dx_t = [strided_device(None, ne0, ne1, ne0 + x_pad[d], dst, lead)[0] for d in range(n_dxs)]
    if in_place:
        x_pad[0], dx_t[0] = y_pad, dy_t
    sums = [torch.full((ne0,), float("nan"), device="cuda") if want else None for want in (dbias, dres)]
    lay = tps.make_layout(ne0, ne1, [(ne0 + y_pad) * es], [(ne0 + k) * es for k in x_pad])
    drop = tps.make_dropout(p, SEED, OFFSET)
    tps.ar_reduce_dropout_grad(dy_t, dx_t, lay, drop, dst, sums[0], sums[1])
    torch.cuda.synchronize()
    g = wide(dst, dy).reshape(ne1, ne0)
    dx = np.where(keep_mask(ne0, ne1, p, SEED, OFFSET), g * scale_of(p), np.float32(0))
    for d in range(n_dxs):
        assert_same(rows_of(dx_t[d], ne0, ne1, ne0 + x_pad[d], dst), oracle.round_to(dst, dx.ravel()), dst, f"dx {d}")
    for got, terms in zip(sums, (dx, g)):
        if got is not None:
            # every add of n float terms is off by at most 2^-24 of a partial sum, in whatever order
            bound = ne1 * 2.0 ** -24 * np.abs(terms.astype(np.float64)).sum(0) + 1e-30
            err = np.abs(got.cpu().numpy().astype(np.float64) - terms.astype(np.float64).sum(0))
            assert (err <= bound).all(), err.max()
    return sums


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("ne0,ne1", [(1, 1), (5, 3), (8, 40), (33, 1000), (777, 65), (4099, 1), (4096, 257), (520, 2100)])
def test_grad_shapes(dst, ne0, ne1):
    run_grad(ne0, ne1, dst, n_dxs=2)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("pads,lead", [((0,), 1), ((8,), 0), ((3,), 0), ((1, 2, 5), 0), ((0, 8, 3), 2), ((13,), 1)])
@pytest.mark.parametrize("ne0", [777, 1024])
def test_grad_strides_and_starts(dst, pads, lead, ne0):
    run_grad(ne0, 37, dst, pads=pads, lead=lead, n_dxs=3)


@pytest.mark.parametrize("dbias,dres", [(False, False), (True, False), (False, True)])
def test_grad_sums_are_optional(dbias, dres):
    run_grad(1000, 70, "f32", dbias=dbias, dres=dres, n_dxs=4)


@pytest.mark.parametrize("p", [0.0, 1.0])
def test_grad_edge_probabilities(p):
    run_grad(300, 40, "bf16", p=p)


@pytest.mark.parametrize("lead", [0, 1])
def test_grad_in_place(lead):
    run_grad(900, 33, "f32", lead=lead, n_dxs=2, in_place=True)


def test_grad_is_repeatable():
    a = run_grad(2048, 500, "f32")
    b = run_grad(2048, 500, "f32")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_grad_of_no_rows_is_zero():
    tps.ar_init(1, 64)
    db = torch.full((16,), 3.0, device="cuda")
    x = torch.zeros(16, device="cuda")
    tps.ar_reduce_dropout_grad(x, [torch.zeros(16, device="cuda")], tps.make_layout(16, 0), tps.make_dropout(0.1, 1), "f32", dbias=db)
    assert (db == 0).all()


def test_grad_matches_differences():
    """A difference of the forward pass in one element of a source, of the
    bias and of a broadcast residual row (wire f32, so every step is linear;
    powers of two keep the differences exact up to float rounding)."""
    ne0, ne1, p = 40, 12, 0.5
    tps.ar_init(1, ne0 * ne1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn((ne1, ne0), device="cuda", generator=gen) for _ in range(2))
    bias, res = (torch.randn(ne0, device="cuda", generator=gen) for _ in range(2))

    def value(x, bias, res):
        y = torch.empty_like(x)
        lay = tps.make_layout(ne0, ne1, residual=res, residual_row_bytes=0)
        tps.ar_reduce_dropout([x], [y], lay, tps.make_dropout(p, SEED, OFFSET, bias), "f32", "f32")
        return (y.double() * w.double()).sum().item()
    dx, db, dr = torch.empty_like(x), torch.empty_like(bias), torch.empty_like(res)
    tps.ar_reduce_dropout_grad(w, [dx], tps.make_layout(ne0, ne1), tps.make_dropout(p, SEED, OFFSET), "f32", db, dr)
    h = 0.25
    # 2 * 480 float roundings of values below 16, divided by the step, bound the difference's error
    tol = 2 * ne0 * ne1 * 16 * 2.0 ** -24 / (2 * h)
    for j, i in ((0, 0), (3, 17), (11, 39)):
        for t, grad, at in ((x, dx, (j, i)), (bias, db, (i,)), (res, dr, (i,))):
            keep = t[at].item()
            t[at] = keep + h
            up = value(x, bias, res)
            t[at] = keep - h
            down = value(x, bias, res)
            t[at] = keep
            assert abs((up - down) / (2 * h) - grad[at].item()) <= tol


def test_refusals_leave_the_outputs_alone():
    tps.ar_init(2, 64)
    x = torch.ones(64, device="cuda")
    y = torch.full((64,), 5.0, device="cuda")
    drop = tps.make_dropout(0.1, 1)
    lay = tps.make_layout(16, 4)
    calls = [
        lambda: tps.ar_reduce_dropout([x, x], [y], lay, tps.make_dropout(2.0, 1), "f32"),
        lambda: tps.ar_reduce_dropout([x, None], [y], lay, drop, "f32"),
        lambda: tps.ar_reduce_dropout_grad(x, [y], tps.make_layout(16, 4, inactive=(0,)), drop, "f32"),
        lambda: tps.ar_reduce_dropout_grad(x, [y], tps.make_layout(16, 4, residual=x), drop, "f32"),
        lambda: tps.ar_reduce_dropout_grad(x, [y], lay, drop, "f32", dbias=y[:16]),
        lambda: tps.ar_reduce_dropout_grad(x, [y], lay, drop, "f32", dbias=torch.empty(16, device="cuda"),
                                           workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
    ]
    for call in calls:
        with pytest.raises(tps.ARError):
            call()
    torch.cuda.synchronize()
    assert (y == 5).all()
    with pytest.raises(ValueError):
        tps.ar_reduce_dropout_grad(x, [y], lay, drop, "f32", dbias=torch.empty(15, device="cuda"))


def test_rows_past_32_bit_offsets():
    """Narrow rows of buffers of several GB, forward and backward."""
    ne0, ne1, wide, p = 72, 2100, 1 << 20, 0.25
    tps.ar_init(1, ne0 * ne1)
    assert (ne1 - 1) * wide * 4 > 1 << 32
    x, y = (torch.empty((ne1, wide), device="cuda")[:, 5:5 + ne0] for _ in range(2))
    x.copy_(torch.randn((ne1, ne0), device="cuda", generator=torch.Generator("cuda").manual_seed(3)))
    lay = tps.make_layout(ne0, ne1, [wide * 4], [wide * 4])
    drop = tps.make_dropout(p, SEED, OFFSET)
    keep = torch.from_numpy(keep_mask(ne0, ne1, p, SEED, OFFSET)).cuda()
    want = torch.where(keep, x * float(scale_of(p)), 0.0)
    tps.ar_reduce_dropout([x], [y], lay, drop, "f32", "f32")
    assert torch.equal(y, want)
    y.zero_()
    db = torch.empty(ne0, device="cuda")
    tps.ar_reduce_dropout_grad(x, [y], lay, drop, "f32", dbias=db)
    assert torch.equal(y, want)
    bound = ne1 * 2.0 ** -24 * want.double().abs().sum(0)  # as in run_grad
    assert ((db.double() - want.double().sum(0)).abs() <= bound).all()
