"""Failure detection of ar_reduce_norm_grad without a GPU fault: the test hook leaves out one row's copies, the blocks that
wait for them give up after a bound, the host reads it from the status word, and the same context is right again."""
import time

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.test_gpu_norm import backward, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


@pytest.mark.parametrize("ne0,ne1,dtype,keep", [(4096, 320, torch.float32, ""), (4096, 700, torch.bfloat16, "int8"),
                                                (20000, 320, torch.float32, ""), (544, 5000, torch.float16, "e4m3")])
@pytest.mark.parametrize("row", [0, 5, 311, 319])
def test_a_row_that_never_comes(ne0, ne1, dtype, keep, row):
    """Rows of one block and of a cluster, the first of a block, one behind the first turn of its stages, and a block's last."""
    name = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[dtype]
    tps.ar_init(2, ne0 * ne1)
    dy, h = normal((ne1, ne0), 3, False).to(dtype), normal((ne1, ne0), 4, False).to(dtype)
    dx = torch.empty_like(dy)
    mean, rstd = torch.zeros(ne1, device="cuda"), torch.ones(ne1, device="cuda")
    dweight, dbias = torch.empty(ne0, device="cuda"), torch.empty(ne0, device="cuda")
    kept = h
    if keep:
        kept = tps.empty_checkpoint(ne0, ne1, keep)
        tps.ar_checkpoint_pack(h, kept)
    torch.cuda.synchronize()
    tps.ar_set_option("device_status", 0)
    tps.ar_set_option("tma_drop_tile", row)
    try:
        began = time.monotonic()
        tps.ar_reduce_norm_grad(dy, kept, [dx], tps.make_layout(ne0, ne1), tps.make_norm(1e-5), mean, rstd, name, dweight, dbias=dbias)
        torch.cuda.synchronize()  # ends: every wait is bounded
        took = time.monotonic() - began
        assert tps.ar_query("device_status") == 2
        # one bound for the row, one for the copies in flight of each of four stages at most
        assert took < 1.0
    finally:
        tps.ar_set_option("tma_drop_tile", -1)
        tps.ar_set_option("device_status", 0)
    backward(ne0, ne1, name, n_dxs=2, dsum=True, keep=keep)
    assert tps.ar_query("device_status") == 0


def test_no_row_dropped():
    """A row number that the call does not have changes nothing."""
    tps.ar_init(2, 4096 * 320)
    tps.ar_set_option("tma_drop_tile", 320)
    try:
        backward(4096, 320, "f32", n_dxs=2, dsum=True)
        assert tps.ar_query("device_status") == 0
    finally:
        tps.ar_set_option("tma_drop_tile", -1)
