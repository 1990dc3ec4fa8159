"""The example's training step against autograd in 64 bits, and in a graph."""
import os
import sys

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tests.philox import keep_mask, scale_of

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def reference(s, step):
    """The step in 64 bits from the same inputs; the hidden states are taken
    as the step rounded them, so that the loss and its gradients are compared
    on equal inputs."""
    keep = torch.from_numpy(keep_mask(s.D, s.T, s.p, s.seed, step)).cuda().double() * float(scale_of(s.p))
    total = sum(x.double() for x in s.partials) + s.bias.double()
    y = total * keep + s.residual.double()
    h = s.hidden.double().requires_grad_()
    W = torch.cat([w.double() for w in s.weights]).requires_grad_()
    loss = torch.nn.functional.cross_entropy(h @ W.t(), s.targets, ignore_index=-100)
    loss.backward()
    dx = s.dhidden.double() * keep
    return y, loss, h.grad, W.grad, dx


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("ranks,tokens,dim,vocab", [(2, 96, 256, 1000), (4, 300, 512, 5003), (3, 65, 200, 777)])
def test_step_matches_autograd(ranks, tokens, dim, vocab):
    import training_step
    s = training_step.Step(ranks, tokens, dim, vocab)
    loss = s.run(step=7)
    y, want, dh, dW, dx = reference(s, 7)
    unit = 2.0 ** -8  # bf16
    # hidden: the partials' sum is rounded once (bf16 wire of bf16 values rounds nothing)
    assert relative(s.hidden, y) <= unit
    assert abs(loss.item() - want.item()) <= 1e-5 * want.item()  # float sums of 16-bit products
    # partial gradients: the logits' gradient and each of the R partials rounded once, their sum once more
    assert relative(s.dhidden, dh) <= 3 * unit
    assert relative(torch.cat(s.dweights), dW) <= 2 * unit
    for d in s.dpartials:
        assert relative(d, dx) <= unit
    assert relative(s.dbias, dx.sum(0)) <= 1e-5


def test_step_in_a_graph_and_falling_loss():
    import training_step
    s = training_step.Step(2, 128, 256, 2000)
    s.run(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = s.run(0)
    seen = []
    for _ in range(4):
        g.replay()
        seen.append(loss.item())
        s.update(20.0)
    # a step of 20 moves a target's logit by 20 |h|^2 / tokens, about 46: the loss falls to nothing and stays
    assert seen[0] > 5 and seen[1] < 0.1 and all(b <= a for a, b in zip(seen, seen[1:])), seen
