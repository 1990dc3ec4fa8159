"""The policy example's calls together, against autograd in 64 bits and in a graph."""
import os
import subprocess
import sys

import pytest
import torch

import tensor_partial_sum_gb300 as tps

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_partial_sum_gb300 import build
    build.build()
    yield
    tps.ar_free()


def reference(s):
    """The step in 64 bits; the hidden states are taken as the step rounded them and the kept stream as its
    checkpoint stands for, so that each part is compared on equal inputs."""
    h = (sum(x.double() for x in s.partials) + s.residual.double()).to(s.hidden.dtype).double()
    d = h - h.mean(1, keepdim=True)
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * s.weight.double() + s.shift.double()
    hidden = s.hidden.double().requires_grad_()
    W = torch.cat([w.double() for w in s.weights]).requires_grad_()
    nll = torch.nn.functional.cross_entropy(hidden @ W.t(), s.targets, ignore_index=-100, reduction="none")
    lengths = s.offsets[1:] - s.offsets[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), lengths)
    m = s.mask.double()
    a = s.advantages.double()[seq]
    ratio = torch.exp(s.old_nll.double() - nll)
    kl = torch.exp(nll - s.ref_nll.double()) - (nll - s.ref_nll.double()) - 1
    each = (-torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) + s.kl_weight * kl) * m
    counts = torch.zeros(len(lengths), dtype=torch.float64, device="cuda").index_add_(0, seq, m)
    loss = (each / counts[seq].clamp(min=1)).sum() / (counts > 0).sum()
    loss.backward()
    kept = torch.empty_like(s.hidden)
    tps.ar_checkpoint_unpack(s.checkpoint, kept)
    x = (kept.double() - s.mean.double()[:, None]) * s.rstd.double()[:, None]
    dy = s.dhidden.double()
    g = dy * s.weight.double()
    dx = s.rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - x * (g * x).mean(1, keepdim=True))
    return y, loss, hidden.grad, W.grad, dx, (dy * x).sum(0), dy.sum(0)


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("ranks,tokens,dim,vocab,answers,keep", [(2, 96, 256, 1000, 3, "int8"), (4, 300, 512, 5003, 7, "e4m3"),
                                                                (3, 165, 200, 777, 1, "int8")])
def test_step_matches_autograd(ranks, tokens, dim, vocab, answers, keep):
    import policy_step
    s = policy_step.Step(ranks, tokens, dim, vocab, answers, keep)
    totals = s.run().tolist()
    y, loss, dh, dW, dx, dweight, dshift = reference(s)
    unit = 2.0 ** -8  # bf16
    # the stream and the hidden states are rounded once each; a stream next to a border may round the other way
    assert relative(s.hidden, y) <= 2 * unit
    # losses of tokens within 1e-5 of float sums, whose signed mean may cancel: relative to the terms' size of about one
    assert abs(totals[0] - loss.item()) <= 1e-5
    # partial gradients: the logits' gradient and each of the R partials rounded once, their sum once more
    assert relative(s.dhidden, dh) <= 3 * unit
    assert relative(torch.cat(s.dweights), dW) <= 2 * unit
    for d in s.dpartials:
        assert relative(d, dx) <= unit
    assert relative(s.dweight, dweight) <= 1e-5 and relative(s.dshift, dshift) <= 1e-5


def test_step_in_a_graph():
    import policy_step
    s = policy_step.Step(2, 160, 1024, 2000, 5)
    want = [t.clone() for t in (s.run(), s.dnll, s.dweight, s.dpartials[1])]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for t in (s.totals, s.dnll, s.dweight, s.dpartials[1]):
        t.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    for got, w in zip((s.totals, s.dnll, s.dweight, s.dpartials[1]), want):
        assert torch.equal(got, w)


def test_example_runs():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "policy_step.py"), "--tokens", "128", "--dim", "256",
                          "--vocab", "1000", "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.count("loss") == 2
