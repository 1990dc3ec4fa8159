"""The bound of the precision test tells sums in short runs from one unbroken
sum of a tensor core, modelled on the CPU: products of 16 terms added exactly
to a running sum that keeps 24 bits and drops the rest."""
import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_precision import one_sign_bound


def cut(x):
    """x with its last bits dropped, 24 kept."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24), e - 24)


def summed(terms, run):
    """Products of 16 terms in runs, the runs added rounded to nearest."""
    groups = terms.reshape(-1, 16).sum(1)
    total = np.float32(0)
    for at in range(0, len(groups), run):
        acc = 0.0
        for g in groups[at:at + run]:
            acc = float(cut(acc + g))
        total = np.float32(total + np.float32(acc))
    return float(total)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("seed", range(4))
def test_the_bound_holds_in_runs_and_not_without(sign, seed):
    rng = np.random.default_rng(seed)
    n = 8192
    h = torch.from_numpy((1.2 * (1 + 0.2 * (rng.random(n) - 0.5)))).half().double().numpy()
    w = torch.from_numpy((sign * 6 / n * (1 + 0.2 * (rng.random(n) - 0.5)))).half().double().numpy()
    z = (h * w).sum()
    bound = one_sign_bound(torch.tensor([[z]])).item()
    assert abs(summed(h * w, 32) - z) < bound / 2
    assert abs(summed(h * w, n) - z) > bound
