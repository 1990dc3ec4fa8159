"""Empty calls touch no buffer, so the binding passes whatever it is given on
to the library (CPU only: the library answers that it has no context)."""
import numpy as np
import pytest
import torch

import tensor_partial_sum_gb300 as tps

NOT_INITIALIZED = 4


@pytest.mark.parametrize("ne0,ne1", [(0, 0), (8, 0), (0, 3)])
@pytest.mark.parametrize("strides", [False, True])
@pytest.mark.parametrize("buffer", [torch.zeros(4), np.zeros(4, np.float32), 4096, None])
def test_empty_extended_reductions_are_not_refused(ne0, ne1, strides, buffer):
    layout = tps.make_layout(ne0, ne1, src_row_bytes=[64] if strides else None, dst_row_bytes=[64] if strides else None,
                             residual=buffer, residual_row_bytes=64)
    with pytest.raises(tps.ARError) as e:
        tps.ar_reduce_ex([buffer], [buffer], layout, "f32", stream=0)
    assert e.value.status == NOT_INITIALIZED
    with pytest.raises(tps.ARError) as e:
        tps.ar_reduce_dropout([buffer], [buffer], layout, tps.make_dropout(0.1, 1), "f32", stream=0)
    assert e.value.status == NOT_INITIALIZED
