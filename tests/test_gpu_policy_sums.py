"""The totals of ar_policy_loss over very many tokens: off by roundings of the terms, not by their number."""
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.norm_ref import UNIT

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
@pytest.mark.parametrize("T", [300, 16384, 16385, 1 << 22, 1 << 28])
def test_equal_terms(T, mean):
    """Every token has the same gain and the same divergence.  A term is within 16 roundings (the exponentials' series, the
    weight); a chunk's eight tokens, five levels of a warp and the totals are 16 more."""
    tps.ar_init(1, T)
    nll, ref = torch.full((T,), 1.1, device="cuda"), torch.full((T,), 1.0, device="cuda")
    offsets, adv = torch.tensor([0, T], device="cuda"), torch.tensor([0.3], device="cuda")
    totals, d = torch.empty(4, device="cuda"), torch.empty(T, device="cuda")
    tps.ar_policy_loss(nll, offsets, adv, totals, d, ref_nll=ref, kl_weight=0.1, mean=mean)
    x = nll[:1].double() - ref[:1].double()
    n = T if mean == "sum" else 1
    gain, kl = -n * adv.double(), n * (torch.expm1(x) - x)
    want = torch.cat([gain + 0.1 * kl, gain, kl])
    off = (totals[:3].double() - want).abs() / torch.cat([gain.abs() + 0.1 * kl, gain.abs(), kl])
    assert (off <= 32 * UNIT).all(), (off / UNIT).tolist()
    assert (d == d[0]).all()
