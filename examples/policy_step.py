"""The tail of one policy-optimisation step of a tensor-parallel model, ranks
emulated on one GPU.

R ranks hold partials of the last layer's output.  The step adds their sum to
the residual stream and normalises it (ar_reduce_norm), keeping the stream in
8 bits for the backward pass; takes each token's negative log-likelihood against
an output matrix whose vocabulary is split over the ranks (ar_vocab_loss); forms
the clipped policy loss with its KL term over ragged answers (ar_policy_loss),
whose gradient is the ``dloss`` of ar_vocab_loss_grad; and goes back through the
norm from the checkpoint (ar_reduce, ar_reduce_norm_grad).

    python examples/policy_step.py [--ranks 4] [--tokens 512] [--dim 1024] [--vocab 16000] [--answers 8] [--steps 5] [--rate 1.0]

Each step moves the norm's weight and shift and the output matrix against their
gradients, so that the printed loss falls.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_partial_sum_gb300 as tps  # noqa: E402


class Step:
    """Buffers of one step and its calls."""

    def __init__(self, ranks, tokens, dim, vocab, answers, keep="int8", kl_weight=0.05, seed=1, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.R, self.T, self.D, self.kl_weight = ranks, tokens, dim, kl_weight

        def randn(*shape, scale=1.0):
            return (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)

        def floats(*shape):
            return torch.empty(shape, device="cuda")
        self.partials = [randn(tokens, dim, scale=ranks ** -0.5) for _ in range(ranks)]
        self.residual = randn(tokens, dim)
        self.weight, self.shift = torch.ones(dim, device="cuda", dtype=dtype), torch.zeros(dim, device="cuda", dtype=dtype)
        per = -(-vocab // ranks)
        self.weights = [randn(min(per, vocab - r * per), dim, scale=dim ** -0.5) for r in range(ranks)]
        self.targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        # answers of different lengths, the first quarter of each a prompt
        cuts = torch.sort(torch.randperm(tokens - 1, device="cuda", generator=gen)[:answers - 1] + 1).values
        self.offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), tokens)])
        t = torch.arange(tokens, device="cuda")
        answer = torch.searchsorted(self.offsets, t, right=True) - 1
        length = (self.offsets[1:] - self.offsets[:-1])[answer]
        self.mask = t - self.offsets[answer] >= length // 4
        self.targets[~self.mask] = -100  # what does not count costs the vocabulary calls nothing
        self.advantages = torch.randn(answers, device="cuda", generator=gen)
        self.hidden, self.dhidden = torch.empty_like(self.residual), torch.empty_like(self.residual)
        self.checkpoint = tps.empty_checkpoint(dim, tokens, keep)
        self.mean, self.rstd, self.nll, self.lse, self.dnll = (floats(tokens) for _ in range(5))
        self.totals = floats(4)
        self.dhidden_parts = [torch.empty_like(self.hidden) for _ in range(ranks)]
        self.dpartials = [torch.empty_like(self.hidden) for _ in range(ranks)]
        self.dweights = [torch.empty_like(w) for w in self.weights]
        self.dweight, self.dshift = floats(dim), floats(dim)
        tps.ar_init(ranks, tokens * dim)
        self.forward_layout = tps.make_layout(dim, tokens, residual=self.residual)
        self.layout = tps.make_layout(dim, tokens)
        self.norm = tps.make_norm(1e-5, self.weight, self.shift)
        # the policy that sampled the answers, and the reference: this one, slightly off
        self.likelihoods()
        self.old_nll = self.nll + 0.05 * torch.randn(tokens, device="cuda", generator=gen)
        self.ref_nll = self.nll + 0.1 * torch.randn(tokens, device="cuda", generator=gen)

    def likelihoods(self, wire="bf16"):
        tps.ar_reduce_norm(self.partials, [self.hidden], self.forward_layout, self.norm, self.hidden.dtype, wire,
                           mean=self.mean, rstd=self.rstd, checkpoint=self.checkpoint)
        tps.ar_vocab_loss(self.hidden, self.weights, self.targets, self.nll, self.lse)

    def run(self, wire="bf16"):
        """Forward and backward; the totals of the loss, on the device."""
        self.likelihoods(wire)
        tps.ar_policy_loss(self.nll, self.offsets, self.advantages, self.totals, self.dnll, self.old_nll, self.ref_nll, self.mask,
                           kl_weight=self.kl_weight, mean="sequences")
        tps.ar_vocab_loss_grad(self.hidden, self.weights, self.targets, self.lse, self.dnll, dhidden=self.dhidden_parts,
                               dweights=self.dweights)
        tps.ar_reduce(self.dhidden_parts, [self.dhidden], wire_dtype=wire)
        tps.ar_reduce_norm_grad(self.dhidden, self.checkpoint, self.dpartials, self.layout, self.norm, self.mean, self.rstd,
                                self.hidden.dtype, dweight=self.dweight, dshift=self.dshift)
        return self.totals

    def update(self, rate):
        self.weight -= (rate * self.dweight).to(self.weight.dtype)
        self.shift -= (rate * self.dshift).to(self.shift.dtype)
        for w, d in zip(self.weights, self.dweights):
            w -= rate * d


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 4), ("tokens", 512), ("dim", 1024), ("vocab", 16000), ("answers", 8), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--rate", type=float, default=1.0)
    a = ap.parse_args()
    s = Step(a.ranks, a.tokens, a.dim, a.vocab, a.answers)
    for k in range(a.steps):
        loss, _, kl, clipped = s.run().tolist()
        print(f"step {k}: loss {loss:.4f}  kl {kl:.4f}  clipped {clipped:.3f}", flush=True)
        s.update(a.rate)
    tps.ar_free()


if __name__ == "__main__":
    main()
