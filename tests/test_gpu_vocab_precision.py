"""Precision of the vocabulary calls where a float computation is exact enough
to tell: nearly sure tokens, long sums of one sign, unequal token weights."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.test_gpu_vocab import DTYPES, UNIT, grads_of, loss_of, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    tps.ar_init(2, 1 << 26)
    yield
    assert tps.ar_query("device_status") == 0
    tps.ar_free()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_one_infinite_dloss_leaves_other_tokens_alone(dtype, T, bad):
    """A token's hidden gradient depends on its own dloss: another token's
    overflow changes no bit of it."""
    hidden, weights, targets = make(dtype, T, 72, [130, 77], seed=T)
    dloss = torch.linspace(-100, 100, T, device="cuda")
    dloss[7] = 0
    _, lse = loss_of(hidden, weights, targets)
    want, _ = grads_of(hidden, weights, targets, lse, dloss, want=("dhidden",))
    dloss[7] = bad
    got, dw = grads_of(hidden, weights, targets, lse, dloss)
    others = torch.arange(T, device="cuda") != 7
    for a, b in zip(got, want):
        assert torch.isfinite(a[others]).all() and torch.equal(a[others], b[others])
        assert not torch.isfinite(a[7]).all()
    assert not any(torch.isfinite(w).all() for w in dw)
