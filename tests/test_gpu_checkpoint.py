"""8-bit checkpoints against tables of their codes: scales and values are equal."""
import numpy as np
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.gpu_util import TORCH_DTYPE
from tests.norm_ref import LARGEST, checkpoint_values
from tests.test_gpu_norm import Rows, normal

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]
FORMATS = ["e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def check(x, format, dst, pad=0, lead=0, code_pad=0, scale_pad=0, stream=None):
    """Pack and unpack the matrix x (of any float type) as `dst`; returns what came back."""
    ne1, ne0 = x.shape
    tps.ar_init(1, max(1, ne0 * ne1))
    src, out = Rows(ne0, ne1, dst, pad, lead, x), Rows(ne0, ne1, dst, pad, lead)
    width = -(-ne0 // 16) * 16 + 16 * code_pad
    blocks = -(-ne0 // 32)
    codes = torch.full((ne1 * width + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ne1 * (blocks + scale_pad) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    c2 = codes[:ne1 * width].view(ne1, width)
    s2 = scales[:ne1 * (blocks + scale_pad)].view(ne1, blocks + scale_pad)
    ck = tps.make_checkpoint(c2, s2, ne0, format)
    tps.ar_checkpoint_pack(src.t, ck, stream)
    tps.ar_checkpoint_unpack(ck, out.t, stream)
    torch.cuda.synchronize()
    values, bytes_ = checkpoint_values(src.t.double().cpu().numpy(), format)
    assert np.array_equal(s2[:, :blocks].cpu().numpy(), bytes_)
    most = torch.finfo(src.dtype).max
    want = torch.from_numpy(np.clip(values, -most, most)).to(src.dtype)
    got = out.t.cpu()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
    out.check_padding()
    assert (c2[:, ne0:] == 0xA5).all() and (s2[:, blocks:] == 0xA5).all(), "bytes between rows were written"
    assert (codes[ne1 * width:] == 0xA5).all() and (scales[ne1 * (blocks + scale_pad):] == 0xA5).all()
    return got


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("ne0,ne1", [(1, 1), (7, 3), (31, 2), (32, 5), (33, 4), (40, 3), (100, 20), (513, 3), (4099, 1), (256, 17)])
def test_shapes(dst, format, ne0, ne1):
    check(normal((ne1, ne0), ne0), format, dst)


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("pad,lead,code_pad,scale_pad", [(1, 0, 0, 0), (3, 1, 1, 0), (8, 0, 2, 3), (0, 5, 0, 1), (13, 2, 3, 2)])
def test_strides_and_starts(dst, format, pad, lead, code_pad, scale_pad):
    check(normal((9, 203), 4), format, dst, pad, lead, code_pad, scale_pad)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("dst", TYPES)
def test_scales_next_to_their_borders(dst, format):
    """Blocks whose largest element is the largest code times a power of two, and its neighbours in the type."""
    dtype = TORCH_DTYPE[dst]
    rows = []
    for e in (-8, -3, 0, 3, 7):
        top = torch.tensor([LARGEST[format] * 2.0 ** e], dtype=dtype)
        if not torch.isfinite(top):
            continue
        bits = top.view(torch.int32 if dst == "f32" else torch.int16)
        for step in (-1, 0, 1):
            v = (bits + step).view(dtype).float().item()
            row = normal((1, 32), 3 + e, False).cpu()[0] * 2.0 ** e
            row[5] = -v if step else v
            rows.append(row)
    check(torch.stack([r for r in rows]).cuda(), format, dst)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("dst", TYPES)
def test_extremes(dst, format):
    info = torch.finfo(TORCH_DTYPE[dst])
    x = torch.zeros((10, 32))
    x[1] = info.max
    x[2, ::2] = -info.max
    x[3, 3] = info.smallest_normal
    x[4, 3] = info.smallest_normal * info.eps if dst != "bf16" else 2.0 ** -133  # the smallest subnormal
    x[5] = torch.linspace(-1, 1, 32) * info.max
    x[6, 0], x[6, 1] = info.max, info.smallest_normal
    x[7] = -0.0
    x[8] = torch.arange(32) - 16.0
    x[9] = (torch.arange(32) + 0.5) * 2.0 ** -10  # ties
    got = check(x.cuda(), format, dst)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_block_with_no_number(dst, format, bad):
    x = normal((3, 100), 5)
    x[1, 40] = bad
    x[2, 99] = bad
    got = check(x, format, dst)
    assert got[1, 32:64].isnan().all() and got[2, 96:].isnan().all() and int(got.isnan().sum()) == 32 + 4


@pytest.mark.parametrize("format", FORMATS)
def test_stated_errors(format):
    x = normal((64, 4096), 8)
    tps.ar_init(1, x.numel())
    ck = tps.empty_checkpoint(4096, 64, format)
    back = torch.empty_like(x)
    tps.ar_checkpoint_pack(x, ck)
    tps.ar_checkpoint_unpack(ck, back)
    err = (back.double() - x.double()).abs().view(64, -1, 32)
    v = x.double().abs().view(64, -1, 32)
    unit = torch.exp2(ck._keep[1].double() - 127)[..., None]
    bound = torch.maximum(v * 2.0 ** -4, unit * 2.0 ** -10) if format == "e4m3" else v.amax(2, keepdim=True) / 127
    assert (err <= bound).all()


def test_another_stream_and_nothing_to_do():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        check(normal((40, 333), 2), "e4m3", "bf16", stream=s)
    tps.ar_init(1, 64)
    ck = tps.ArCheckpoint(0, 4, 0, None, 0, None, 0)
    empty = torch.empty((4, 0), device="cuda")
    tps.ar_checkpoint_pack(empty, ck)
    tps.ar_checkpoint_unpack(ck, empty)


def test_rows_past_32_bit_offsets():
    ne0, ne1, wide = 72, 1100, 1 << 20
    tps.ar_init(1, ne0 * ne1)
    x = torch.empty((ne1, wide), device="cuda")[:, 3:3 + ne0]
    x.copy_(normal((ne1, ne0), 3))
    codes = torch.empty((ne1, 4 * wide), dtype=torch.uint8, device="cuda")
    ck = tps.make_checkpoint(codes, torch.empty((ne1, 3), dtype=torch.uint8, device="cuda"), ne0, "int8")
    assert (ne1 - 1) * 4 * wide > 1 << 32
    small, back, again = tps.empty_checkpoint(ne0, ne1, "int8"), torch.empty((ne1, ne0), device="cuda"), torch.empty((ne1, ne0), device="cuda")
    tps.ar_checkpoint_pack(x, ck)
    tps.ar_checkpoint_unpack(ck, back)
    tps.ar_checkpoint_pack(x.contiguous(), small)
    tps.ar_checkpoint_unpack(small, again)
    assert torch.equal(back, again) and (back - x).abs().max() < 2


def test_refusals_leave_the_outputs_alone():
    tps.ar_init(1, 64)
    x, ck = torch.ones((4, 16), device="cuda"), tps.empty_checkpoint(16, 4)
    ck._keep[0].fill_(3)
    big, big_ck = torch.ones((5, 16), device="cuda"), tps.empty_checkpoint(16, 5)
    ck.format = 9
    for call in (lambda: tps.ar_checkpoint_pack(x, ck), lambda: tps.ar_checkpoint_pack(big, big_ck)):
        with pytest.raises(tps.ARError):
            call()
    ck.format = 0
    for bad in (x[:, :15], x[:3], x.t(), x.double(), torch.ones(4, 16)):
        with pytest.raises((TypeError, ValueError, KeyError)):
            tps.ar_checkpoint_pack(bad, ck)
    torch.cuda.synchronize()
    assert (ck._keep[0] == 3).all()
