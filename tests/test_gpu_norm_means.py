"""Means of ar_reduce_norm against 64 bits: near zero, far from it and of constant rows, to the last roundings.

The row's sum is carried with what its additions lose.  The additions are exact together with their losses; the losses
are added up in floats.  With d additions behind a term the losses of one level are at most 2^-24 of the sum of
magnitudes, those of all d of them d 2^-24, and their own sum is off by d 2^-24 of that: d^2 2^-48 of the mean
magnitude.  The mean itself is rounded once, and the second of the two numbers that it is added from by less than another
rounding of it.  16-bit elements are added plainly in groups of at most 16, in four levels: 2^-24 of the mean magnitude
each, most of them exact.
"""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.gpu_util import TORCH_DTYPE
from tests.norm_ref import UNIT, adds

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def rows(kind, ne1, ne0, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn():
        return torch.randn((ne1, ne0), device="cuda", generator=g)
    if kind == "normal":  # one element in a thousand 50 times larger; the means are near zero
        x = randn()
        return torch.where(torch.rand((ne1, ne0), device="cuda", generator=g) < 0.001, x * 50, x)
    if kind == "cancelled":  # every element has its negative somewhere, but for a few small ones
        x = randn()
        half = ne0 // 2
        x[:, half:2 * half] = -x[:, :half]
        if ne0 % 2:
            x[:, -1] *= 1e-3
        return x[:, torch.randperm(ne0, device="cuda", generator=g)]
    if kind == "far":
        x = randn()
        at = torch.tensor([1000.0, -30000.0, 3.3, -0.07], device="cuda")
        return x + at[torch.arange(ne1, device="cuda") % 4, None]
    c = torch.rand((ne1, 1), device="cuda", generator=g) * 2000 - 1000  # constant
    return c.expand(ne1, ne0).contiguous()


def check(x, dst, pad=0):
    ne1, ne0 = x.shape
    tps.ar_init(1, ne0 * ne1)
    src, y = (torch.empty((ne1, ne0 + pad), dtype=TORCH_DTYPE[dst], device="cuda")[:, :ne0] for _ in range(2))
    src.copy_(x)
    mean = torch.empty(ne1, device="cuda")
    stride = (ne0 + pad) * src.element_size()
    tps.ar_reduce_norm([src], [y], tps.make_layout(ne0, ne1, [stride], [stride]), tps.make_norm(1e-5), dst, dst, mean=mean)
    h = src.double()
    want = h.mean(1)
    groups = 0 if dst == "f32" else 4
    bound = 2 * UNIT * want.abs() + (adds(ne0) ** 2 * UNIT ** 2 + groups * UNIT) * h.abs().mean(1)
    err = (mean.double() - want).abs()
    assert (err <= bound).all(), f"{int((err > bound).sum())} of {ne1} means off, worst {(err / bound).max().item():.1f} times the bound"


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("kind", ["normal", "cancelled", "far", "constant"])
@pytest.mark.parametrize("ne0,ne1,pad", [(33, 64, 0), (96, 500, 0), (777, 300, 0), (1024, 128, 3), (4096, 300, 0), (4099, 257, 0), (4099, 1, 0),
                                         (4096, 1, 0), (8200, 40, 0), (8192, 3, 0), (20001, 8, 0), (70001, 2, 0), (300007, 2, 0)])
def test_means(dst, kind, ne0, ne1, pad):
    check(rows(kind, ne1, ne0, 11 + ne0), dst, pad)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("kind", ["normal", "cancelled", "far", "constant"])
def test_means_of_rows_past_a_cluster(dst, kind):
    check(rows(kind, 2, 1_000_001, 5), dst)


@pytest.mark.parametrize("seed", range(40))
def test_one_row_on_four_ranks(seed):
    """A token's activation, whose mean may happen to be next to zero."""
    ne0 = 4099
    tps.ar_init(4, ne0)
    parts = [rows("normal", 1, ne0, 100 * seed + r) for r in range(4)]
    res = rows("normal", 1, ne0, 100 * seed + 9)
    ys, sums = ([torch.empty((1, ne0), device="cuda") for _ in range(4)] for _ in range(2))
    mean = torch.empty(1, device="cuda")
    tps.ar_reduce_norm(parts, ys, tps.make_layout(ne0, 1, residual=res), tps.make_norm(1e-5), "f32", "f16", sums=sums, mean=mean)
    h = sums[0].double()
    want = h.mean().item()
    assert abs(mean.item() - want) <= 2 * UNIT * abs(want) + adds(ne0) ** 2 * UNIT ** 2 * h.abs().mean().item()
