"""The vocabulary calls where the packed weights take more than one launch,
against the formulas in 64 bits (tolerances as derived in test_gpu_vocab)."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.test_gpu_vocab import check_all, formula, loss_of, make, near

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
    torch.cuda.empty_cache()


def test_float_weights_of_a_large_vocabulary():
    """Two launches, the first's last tile a narrow one, for the loss and the gradients."""
    hidden, weights, targets = make("f32", 512, 4096, [128256], seed=1, ignored=0.1)
    check_all("f32", hidden, weights, targets, torch.full((512,), 1 / 512, device="cuda"))


@pytest.mark.parametrize("dtype,T,D,pieces,pad", [
    ("f32", 200, 8192, [65536], 0),
    ("f32", 300, 8192, [47000, 7, 50001], 0),
    ("bf16", 300, 8192, [140000], 1),
    ("f32", 3, 8192, [70001], 0),
])
def test_losses_of_a_cut_vocabulary(dtype, T, D, pieces, pad):
    hidden, weights, targets = make(dtype, T, D, pieces, seed=T, ignored=0.1, pad=pad)
    loss, lse = loss_of(hidden, weights, targets)
    want = formula(hidden, weights, targets)
    near(lse, want["lse"], "lse")
    near(loss, want["loss"], "loss")
    del hidden, weights
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D,pieces,pad", [(20, 64, [300000], 0), (5, 72, [280000, 100, 300001], 0), (1, 40, [530000], 3),
                                            (66, 64, [400000, 33], 0), (600, 64, [120000, 250001], 1)])
def test_gradients_of_a_cut_vocabulary(dtype, T, D, pieces, pad):
    """More vocabulary rows than one chunk of the logits' gradient, from one token on."""
    hidden, weights, targets = make(dtype, T, D, pieces, seed=T, pad=pad)
    check_all(dtype, hidden, weights, targets, torch.linspace(0.5, 1, T, device="cuda"), pad)
