"""Checkpoints of a flattened tensor: one row whose bytes pass 32 bits."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def kept(x, format):
    """(what a checkpoint of the matrix x stands for, its codes, its scales)"""
    ck = tps.empty_checkpoint(x.shape[1], x.shape[0], format)
    out = torch.full_like(x, 7.0)
    tps.ar_checkpoint_pack(x, ck)
    tps.ar_checkpoint_unpack(ck, out)
    return out, *ck._keep


@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("ne0,lead,dtype", [((1 << 30) + 100, 0, torch.float32), ((1 << 30) + 100, 1, torch.float32),
                                            ((1 << 31) + 100, 0, torch.float32), ((1 << 31) - 28, 0, torch.bfloat16),
                                            ((1 << 31) - 28, 1, torch.float16)])
def test_one_row_past_32_bit_offsets(ne0, lead, dtype, format):
    width = 1 << 14
    tps.ar_init(1, ne0)
    back = torch.empty(ne0 + lead, dtype=dtype, device="cuda")
    x = back[lead:].view(1, ne0)
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    out, codes, scales = kept(x, format)
    # the same blocks as rows of an ordinary length, and the rest as one of its own
    whole = ne0 // width * width
    for at, shape in ((0, (whole // width, width)), (whole, (1, ne0 - whole))):
        n = shape[0] * shape[1]
        part, c, s = kept(x[0, at:at + n].view(shape), format)
        assert torch.equal(out[0, at:at + n].view(shape), part)
        assert torch.equal(codes[0, at:at + n], c[:, :shape[1]].reshape(-1))
        assert torch.equal(scales[0, at // 32:at // 32 + s.numel()], s.reshape(-1))
