"""The element-wise forms of the norm and checkpoint calls: rows past what a cluster holds, and strides past 32 bits.
That these sizes take them is tested on the host's plan."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.gpu_util import TORCH_DTYPE
from tests.norm_ref import HALF_STEP, norm_backward, norm_forward
from tests.test_gpu_norm import EPS, backward, close, forward, normal

pytestmark = pytest.mark.gpu

LONG = [("f32", 458_760), ("f32", 1_000_003), ("f16", 1_000_001), ("bf16", 917_520), ("bf16", 1_000_001)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def same_as_pack(ck, h):
    """The checkpoint that a forward pass wrote is what ar_checkpoint_pack writes of the kept sum."""
    again = tps.empty_checkpoint(h.shape[1], h.shape[0], "e4m3" if ck.format == 0 else "int8")
    tps.ar_checkpoint_pack(h, again)
    n = h.shape[1]
    assert torch.equal(ck._keep[0][:, :n], again._keep[0][:, :n]) and torch.equal(ck._keep[1], again._keep[1])


@pytest.mark.parametrize("dst,ne0", LONG)
@pytest.mark.parametrize("kind,keep,in_place", [("layer", "e4m3", ""), ("rms", "int8", ""), ("layer", "", "source"),
                                                ("rms", "", "residual"), ("layer", "int8", "both")])
def test_forward(dst, ne0, kind, keep, in_place):
    ys, sums, mean, rstd, ck, h = forward(3, ne0, 2, dst, "bf16", kind, n_dsts=2, bias=True, residual="full", keep=keep,
                                          in_place=in_place, inactive=(1,) if keep else ())
    if keep:
        same_as_pack(ck, h)


@pytest.mark.parametrize("dst,ne0", LONG)
def test_forward_of_odd_starts(dst, ne0):
    forward(2, ne0, 3, dst, "f16", pads=(1, 2, 5), lead=1, n_dsts=2, residual="row", keep="e4m3")


@pytest.mark.parametrize("ne0", [72, 4100])
def test_strides_past_32_bits(ne0):
    """Two rows more than 4 GiB apart, forward, backward and as a checkpoint."""
    ne1, gap = 2, (1 << 30) + 32
    tps.ar_init(1, ne0 * ne1)
    x = torch.empty(gap + ne0 + 5, device="cuda")[5:].as_strided((ne1, ne0), (gap, 1))
    x.copy_(normal((ne1, ne0), 3))
    want_h = x.clone()
    mean, rstd = torch.empty(ne1, device="cuda"), torch.empty(ne1, device="cuda")
    y, h = torch.empty((ne1, ne0), device="cuda"), torch.empty((ne1, ne0), device="cuda")
    lay = tps.make_layout(ne0, ne1, [gap * 4])
    ck = tps.empty_checkpoint(ne0, ne1, "int8")
    tps.ar_reduce_norm([x], [y], lay, tps.make_norm(EPS), "f32", "f32", sums=[h], mean=mean, rstd=rstd, checkpoint=ck)
    want, m, r, slack = norm_forward(want_h.double(), None, None, EPS, False)
    assert torch.equal(h, want_h)
    close(y, want, slack, torch.float32, "y")
    same_as_pack(ck, h)
    grad = norm_backward(y.double(), want_h.double(), mean.double(), rstd.double(), None, None, False)
    dy, out = y.clone(), torch.empty((ne1, ne0), device="cuda")
    tps.ar_reduce_norm_grad(dy, x, [out], tps.make_layout(ne0, ne1, [ne0 * 4, gap * 4]), tps.make_norm(EPS), mean, rstd, "f32")
    close(out, *grad["dx"], torch.float32, "dx")
    wide = tps.empty_checkpoint(ne0, ne1, "int8")
    tps.ar_checkpoint_pack(x, wide)
    assert torch.equal(wide._keep[0][:, :ne0], ck._keep[0][:, :ne0]) and torch.equal(wide._keep[1], ck._keep[1])
    tps.ar_checkpoint_unpack(wide, x)
    tps.ar_checkpoint_unpack(ck, out)
    assert torch.equal(x, out)


@pytest.mark.parametrize("keep", ["", "e4m3", "int8"])
@pytest.mark.parametrize("dst", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward(dst, keep, kind):
    backward(131_080, 70, dst, kind, n_dxs=2, dsum=True, keep=keep)


# ---- long sums ---------------------------------------------------------------------------

@pytest.mark.parametrize("dst,ne0", LONG + [("f32", 30_000_001), ("bf16", 30_000_001)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_long_rows_keep_their_variance(dst, ne0, kind):
    """1 / standard deviation to a few roundings, however many squares are added: each square is rounded twice, its
    sum's losses are added up, and the mean square, its distance from the mean's square, eps and the root follow."""
    x = (normal((2, ne0), 7, False) + torch.tensor([[0.0], [1.5]], device="cuda")).to(TORCH_DTYPE[dst])
    tps.ar_init(1, 2 * ne0)
    y, mean, rstd = torch.empty_like(x), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    tps.ar_reduce_norm([x], [y], tps.make_layout(ne0, 2), tps.make_norm(EPS, kind=kind), dst, dst, mean=mean, rstd=rstd)
    h = x.double()
    d = h - h.mean(1, keepdim=True) if kind == "layer" else h
    want = 1 / torch.sqrt((d * d).mean(1) + EPS)
    assert ((rstd.double() - want).abs() <= 8 * 2.0 ** -24 * want).all(), ((rstd.double() - want).abs() / want / 2.0 ** -24).tolist()


@pytest.mark.parametrize("ne0", [1_000_003, 30_000_001])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_long_rows_keep_their_gradient(kind, ne0):
    """dy of one sign, so that g - mean(g) cancels: off by roundings of g, x and the means, not by their number."""
    tps.ar_init(1, 2 * ne0)
    dy, h = 1 + normal((2, ne0), 8, False) * 2.0 ** -4, normal((2, ne0), 9, False)
    x = h.double()
    mean = x.mean(1) if kind == "layer" else torch.zeros(2, dtype=torch.float64, device="cuda")
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + EPS)
    mean, rstd = mean.float(), rstd.float()
    dx = torch.empty_like(dy)
    tps.ar_reduce_norm_grad(dy, h, [dx], tps.make_layout(ne0, 2), tps.make_norm(EPS, kind=kind), mean, rstd, "f32")
    want, _ = norm_backward(dy.double(), x, mean.double(), rstd.double(), None, None, kind == "rms")["dx"]
    xs = ((x - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    g = dy.double().abs()
    size = rstd.double()[:, None] * (g + g.mean(1, keepdim=True) + xs * (g * xs).mean(1, keepdim=True))
    err = (dx.double() - want).abs()
    bound = 8 * HALF_STEP[torch.float32] * (size + want.abs())
    assert (err <= bound).all(), f"worst {(err / bound).max().item():.2f} times the bound"
