"""ar_policy_loss without any sequence, behind calls with thousands of them: nothing counts, and no offset is looked for."""
import ctypes

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tensor_partial_sum_gb300 import ar
from tests.test_gpu_policy import inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


@pytest.mark.parametrize("mean", ["sum", "tokens", "sequences"])
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("T", [1, 300, 9000, 16384, 16385, 40_000])
def test_no_sequence_after_many(T, token, mean):
    nll, offsets, adv, old, ref, mask = inputs(16_000, 9000, T, token=token)
    run(nll, offsets, adv, old, ref, mask, mean=mean, token=token)
    tps.ar_init(1, 40_000)
    n, o, r = (torch.randn(T, device="cuda").abs() for _ in range(3))
    a = torch.randn(T, device="cuda")
    for given in (torch.zeros(1, dtype=torch.int64, device="cuda"), None):
        totals, d = torch.full((4,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
        p = tps.ArPolicy(T, 0, ar._ptr(given), n.data_ptr(), o.data_ptr(), r.data_ptr(), a.data_ptr() if token else None, int(token),
                         None, 0.2, 0.2, 0.1, 1.0, ar.POLICY_MEANS[mean])
        ws = torch.empty(tps.ar_policy_workspace(p), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream or None
        assert ar.lib().ar_policy_loss(ctypes.byref(p), totals.data_ptr(), d.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
        torch.cuda.synchronize()
        assert (totals == 0).all() and (d == 0).all()
