"""The tail of one tensor-parallel training step, ranks emulated on one GPU.

R ranks hold partials of a layer's output.  The step sums them with bias,
dropout and residual (ar_reduce_dropout), takes the loss against an output
matrix whose vocabulary is split over the ranks (ar_vocab_loss), and goes back:
the ranks' partial gradients of the hidden states (ar_vocab_loss_grad) are
summed by ar_reduce, and the sum becomes the gradient of the partials, of the
bias and of the residual (ar_reduce_dropout_grad).

    python examples/training_step.py [--ranks 4] [--tokens 512] [--dim 1024] [--vocab 16000] [--steps 5] [--rate 1.0]

Each step moves the bias and the output matrix against their gradients, so the
printed loss falls.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_partial_sum_gb300 as tps  # noqa: E402


class Step:
    """Buffers of one step and its four calls."""

    def __init__(self, ranks, tokens, dim, vocab, p=0.1, seed=1, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.R, self.T, self.D, self.p, self.seed = ranks, tokens, dim, p, seed

        def randn(*shape, scale=1.0):
            return (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)
        self.partials = [randn(tokens, dim, scale=ranks ** -0.5) for _ in range(ranks)]
        self.residual = randn(tokens, dim)
        self.bias = torch.zeros(dim, device="cuda", dtype=dtype)
        per = -(-vocab // ranks)
        self.weights = [randn(min(per, vocab - r * per), dim, scale=dim ** -0.5) for r in range(ranks)]
        self.targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        self.targets[::8] = -100  # tokens that do not count
        self.dloss = torch.full((tokens,), 1.0 / int((self.targets != -100).sum()), device="cuda")
        self.hidden = torch.empty_like(self.residual)
        self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.dhidden_parts = [torch.empty_like(self.hidden) for _ in range(ranks)]
        self.dhidden = torch.empty_like(self.hidden)
        self.dpartials = [torch.empty_like(self.hidden) for _ in range(ranks)]
        self.dweights = [torch.empty_like(w) for w in self.weights]
        self.dbias = torch.empty(dim, device="cuda")
        tps.ar_init(ranks, tokens * dim)
        self.forward_layout = tps.make_layout(dim, tokens, residual=self.residual)
        self.layout = tps.make_layout(dim, tokens)

    def run(self, step=0, wire="bf16"):
        """Forward and backward; the mean loss of the counted tokens, on the device."""
        dt = self.hidden.dtype
        drop = tps.make_dropout(self.p, self.seed, offset=step, bias=self.bias)
        tps.ar_reduce_dropout(self.partials, [self.hidden], self.forward_layout, drop, dt, wire)
        tps.ar_vocab_loss(self.hidden, self.weights, self.targets, self.loss, self.lse)
        tps.ar_vocab_loss_grad(self.hidden, self.weights, self.targets, self.lse, self.dloss,
                               dhidden=self.dhidden_parts, dweights=self.dweights)
        tps.ar_reduce(self.dhidden_parts, [self.dhidden], wire_dtype=wire)
        # the residual's gradient is dhidden itself
        tps.ar_reduce_dropout_grad(self.dhidden, self.dpartials, self.layout, drop, dt, dbias=self.dbias)
        return (self.loss * self.dloss).sum()

    def update(self, rate):
        self.bias -= (rate * self.dbias).to(self.bias.dtype)
        for w, d in zip(self.weights, self.dweights):
            w -= rate * d


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 4), ("tokens", 512), ("dim", 1024), ("vocab", 16000), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--rate", type=float, default=1.0)
    a = ap.parse_args()
    s = Step(a.ranks, a.tokens, a.dim, a.vocab)
    for k in range(a.steps):
        print(f"step {k}: loss {s.run(k).item():.4f}", flush=True)
        s.update(a.rate)
    tps.ar_free()


if __name__ == "__main__":
    main()
