"""Stride lists that are shorter than the tensors they belong to are refused before anything reads past them (CPU only)."""
import pytest

import tensor_partial_sum_gb300 as tps

A = 1 << 20  # addresses far apart, never read


def addr(k):
    return A * (k + 1)


def test_gradient_from_a_kept_tensor_needs_its_stride():
    lay, norm = tps.make_layout(8, 2, src_row_bytes=[32]), tps.make_norm()
    with pytest.raises(ValueError, match="stride"):
        tps.ar_reduce_norm_grad(addr(0), addr(1), [addr(2)], lay, norm, addr(3), addr(4), "f32", workspace=addr(5), stream=0)


def test_too_few_strides():
    norm = tps.make_norm()
    two, three = [addr(0), addr(1)], [addr(2), addr(3), addr(4)]
    for kw in (dict(src_row_bytes=[32]), dict(dst_row_bytes=[32, 32])):
        lay = tps.make_layout(8, 2, **kw)
        with pytest.raises(ValueError, match="stride"):
            tps.ar_reduce_norm(two, three, lay, norm, "f32", stream=0)
        with pytest.raises(ValueError, match="stride"):
            tps.ar_reduce_ex(two, three, lay, "f32", stream=0)
    lay = tps.make_layout(8, 2)
    with pytest.raises(ValueError, match="stride"):
        tps.ar_reduce_norm(two, three, lay, norm, "f32", sums=[addr(5), addr(6)], sum_row_bytes=[32], stream=0)
    with pytest.raises(ValueError, match="stride"):
        tps.ar_check_norm(2, two, three, lay, norm, 64, "f32", "f32", sums=[addr(5), addr(6)], sum_row_bytes=[32])


def test_more_strides_than_tensors():
    """As before: the rest is not looked at."""
    lay = tps.make_layout(8, 2, src_row_bytes=[32] * 4, dst_row_bytes=[32] * 4)
    with pytest.raises(tps.ARError):  # no context
        tps.ar_reduce_norm([addr(0)], [addr(1)], lay, tps.make_norm(), "f32", stream=0)
