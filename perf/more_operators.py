"""Cases that measure the normalisation, checkpoint and policy operators around
the partial-sum reduction.

Five calls or runs of calls are measured, each in a plain form (elementary
torch operations in 32 bits, rounded once at the end) and through the library's
entry points:

``reduce_norm``
    The end of a tensor-parallel layer: R partials are rounded through the wire
    type and summed in rank order, a bias row and the residual are added, the
    sum is rounded to the tensor type (the new residual stream, kept where
    asked for), and every row of it is normalised: layer norm or root-mean-square
    norm with a weight and a shift, written to every destination, with each
    row's mean and 1 / standard deviation in float.
``reduce_norm_grad``
    Its backward pass from the kept sum: the gradient of the sum (one value,
    written to every rank's buffer) with the residual stream's own gradient
    added, and the gradients of weight, shift and bias row.
``norm_step``
    Forward and backward of one such layer with the sum kept in 8 bits: the
    forward call writes the checkpoint, the backward call reads it.
``checkpoint``
    An activation written as an 8-bit checkpoint and read back.  32 adjacent
    elements of a row share a power of two: the smallest 2^e, e >= -127, with
    max |x| <= 448 * 2^e (codes in e4m3) or 127 * 2^e (codes in int8).  A code
    is x * 2^-e rounded to nearest, ties to even; the value read back is
    code * 2^e, at most the type's largest finite one in magnitude.
``policy``
    A clipped policy loss with a KL term over ragged sequences of tokens, and
    its gradient: for a counted token with negative log-likelihoods nll (of the
    policy), old (of the policy that sampled it) and ref (of a reference), and
    the advantage A,
        ratio = exp(old - nll)
        loss  = -min(ratio A, clamp(ratio, 1 - low, 1 + high) A)
                + beta (exp(nll - ref) - (nll - ref) - 1),
    summed, averaged over the counted tokens, or averaged over each sequence's
    counted tokens and then over the sequences that have some.
"""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
BLOCK = 32  # elements that share a scale


# ---- cases ------------------------------------------------------------------

def _norm(name, op, R, n_dsts, dtype, wire, ne1, ne0, kind="layer", residual="full", sums=0, bias=False, affine="both",
          keep="", row_pad=0):
    case = {"op": op, "R": R, "n_dsts": n_dsts, "dtype": dtype, "wire": wire, "ne1": ne1, "ne0": ne0, "kind": kind,
            "residual": residual, "sums": sums, "bias": bias, "affine": affine, "keep": keep, "row_pad": row_pad}
    return dict(case, name=name) if name else case


def _check(name, dtype, keep, ne1, ne0, row_pad=0):
    case = {"op": "checkpoint", "dtype": dtype, "keep": keep, "ne1": ne1, "ne0": ne0, "row_pad": row_pad}
    return dict(case, name=name) if name else case


def _policy(name, T, S, mean, per_token=False, masked=True, old=True, kl=0.04):
    case = {"op": "policy", "T": T, "S": S, "mean": mean, "per_token": per_token, "masked": masked, "old": old, "kl": kl}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token's activation on four ranks, the smallest call: latency counts
        _norm("norm one row", "reduce_norm", 4, 4, "f32", "f16", 1, 4099, sums=4),
        # a prompt's activation on two ranks, the residual stream kept once
        _norm("norm prefill", "reduce_norm", 2, 2, "f32", "bf16", 2048, 4096, sums=1, bias=True),
        # odd rows out of wider buffers, root-mean-square norm, a broadcast residual row
        _norm("norm odd", "reduce_norm", 3, 1, "f16", "f16", 1021, 4099, "rms", "row", 1, False, "weight", row_pad=13),
        # the backward pass of the prompt's layer
        _norm("norm grad prefill", "reduce_norm_grad", 2, 2, "f32", "bf16", 2048, 4096, bias=True),
        # odd rows, sums over few of them
        _norm("norm grad odd", "reduce_norm_grad", 3, 1, "f16", "f16", 1021, 4099, residual="", row_pad=13),
        # a training step of a micro-batch whose sums are kept in int8
        _norm("norm step prefill", "norm_step", 2, 1, "bf16", "bf16", 2048, 4096, bias=True, keep="int8"),
        # a large activation on four ranks, kept in e4m3
        _norm("norm step large", "norm_step", 4, 4, "bf16", "bf16", 4096, 8192, keep="e4m3"),
        # an activation of a micro-batch in full precision, kept in e4m3
        _check("checkpoint prefill", "f32", "e4m3", 2048, 4096),
        # a large 16-bit activation kept in int8
        _check("checkpoint large", "bf16", "int8", 4096, 8192),
        # one short answer: latency counts
        _policy("policy one answer", 300, 1, "tokens"),
        # a batch of groups of answers of very different lengths
        _policy("policy groups", 262_143, 257, "sequences"),
        # a large batch with an advantage for each token
        _policy("policy large", 4_194_304, 2048, "tokens", per_token=True),
    ]


MOST_BYTES = 1_076_000_000  # of a drawn norm, step or checkpoint case, about "norm step large"


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reduce_norm", "reduce_norm_grad", "norm_step", "checkpoint", "policy"])
    if op == "policy":
        T = _log_int(rng, 1, 4_194_304)
        return _policy(None, T, _log_int(rng, 1, min(T, 8192)), rng.choice(["sum", "tokens", "sequences"]),
                       rng.random() < 0.3, rng.random() < 0.7, rng.random() < 0.8, rng.choice([0.0, 0.01, 0.04, 0.2]))
    dtype = rng.choice(["f32", "f16", "bf16"])
    ne0, ne1 = _log_int(rng, 33, 16384), _log_int(rng, 1, 8192)
    if rng.random() < 0.5:
        ne0 = max(32, ne0 // 32 * 32)
    pad = rng.choice([0, 0, 8, rng.randint(1, 64)])
    keep = rng.choice(["e4m3", "int8"])
    if op == "checkpoint":
        case = _check(None, dtype, keep, ne1, ne0, pad)
    else:
        R = rng.randint(1, 8)
        n_dsts = rng.choice([1, R])
        case = _norm(None, op, R, n_dsts, dtype, rng.choice(["f32", "f16", "bf16"]), ne1, ne0,
                     rng.choice(["layer", "layer", "rms"]), rng.choice(["", "full", "row"]),
                     rng.choice([0, 1, n_dsts]) if op == "reduce_norm" else 0, rng.random() < 0.4,
                     rng.choice(["", "weight", "both"]), keep if op == "norm_step" else "", pad)
    over = work(case)["bytes"] / MOST_BYTES
    if over > 1:
        case["ne1"] = max(1, int(ne1 / over))
    return case


def work(case):
    if case["op"] == "policy":
        T, S = case["T"], case["S"]
        arrays = 2 + case["old"] + (case["kl"] > 0) + case["per_token"]  # nll and its gradient, and what is given
        other = (T if case["masked"] else 0) + 8 * (S + 1) + (0 if case["per_token"] else 4 * S) + 16
        return {"bytes": 4 * T * arrays + other, "flops": 24 * T}
    es = BYTES[case["dtype"]]
    ne0, ne1 = case["ne0"], case["ne1"]
    n = ne0 * ne1
    kept = n + ne1 * -(-ne0 // BLOCK)  # bytes of a checkpoint
    if case["op"] == "checkpoint":
        return {"bytes": 2 * n * es + 2 * kept, "flops": 4 * n}
    rows = {"": 0, "weight": 1, "both": 2}[case["affine"]]
    full = case["residual"] == "full"
    forward = (case["R"] + case["n_dsts"] + case["sums"] + full) * n * es + 8 * ne1 + (
        rows + case["bias"] + (case["residual"] == "row")) * ne0 * es
    # dy, the kept sum (unless in 8 bits), the residual stream's gradient; dx
    backward = (1 + (not case["keep"]) + full + case["n_dsts"]) * n * es + (kept if case["keep"] else 0) + 8 * ne1 + (
        rows > 0) * ne0 * es + (rows + (case["bias"] or case["residual"] == "row")) * ne0 * 4
    f_ops, b_ops = (case["R"] + 8) * n, 14 * n
    if case["op"] == "reduce_norm":
        return {"bytes": forward, "flops": f_ops}
    if case["op"] == "reduce_norm_grad":
        return {"bytes": backward, "flops": b_ops}
    return {"bytes": forward + kept + backward, "flops": f_ops + b_ops + 2 * n}


# ---- inputs -----------------------------------------------------------------

def _rows(ne1, ne0, pad, dtype):
    """ne1 rows of ne0 elements, `pad` elements apart."""
    return torch.empty((ne1, ne0 + pad), dtype=dtype, device="cuda")[:, :ne0]


def _normal_rows(ne1, ne0, pad, dtype, gen, outliers):
    """N(0, 1); with `outliers`, one element in a thousand is 50 times larger."""
    x = torch.randn((ne1, ne0), device="cuda", generator=gen)
    if outliers:
        x = torch.where(torch.rand((ne1, ne0), device="cuda", generator=gen) < 0.001, x * 50, x)
    out = _rows(ne1, ne0, pad, dtype)
    out.copy_(x)
    return out


def _codes(case):
    """Buffers of a checkpoint: rows of codes on 16-byte boundaries, rows of scales."""
    ne0, ne1 = case["ne0"], case["ne1"]
    return (_rows(ne1, ne0, -ne0 % 16, torch.uint8),
            torch.empty((ne1, -(-ne0 // BLOCK)), dtype=torch.uint8, device="cuda"))


def _prepare_policy(case, gen):
    T, S = case["T"], case["S"]
    # ragged lengths, some of nothing, and the last tokens of the buffer belong to
    # no sequence
    used = T - T // 50
    cuts = torch.sort(torch.randint(0, used + 1, (S - 1,), device="cuda", generator=gen)).values
    ends = torch.tensor([0, used], device="cuda")
    offsets = torch.cat([ends[:1], cuts, ends[1:]])
    state = dict(case, offsets=offsets, totals=torch.empty(4, device="cuda"), dnll=torch.empty(T, device="cuda"))
    randn = lambda scale, n=T: torch.randn(n, device="cuda", generator=gen) * scale  # noqa: E731
    state["nll"] = -torch.log(torch.rand(T, device="cuda", generator=gen).clamp(min=1e-7))
    # most ratios near one, some far outside of the clip range
    far = torch.rand(T, device="cuda", generator=gen) < 0.02
    state["old_nll"] = state["nll"] + torch.where(far, randn(1.0), randn(0.1)) if case["old"] else None
    state["ref_nll"] = state["nll"] + randn(0.2) if case["kl"] > 0 else None
    state["advantages"] = randn(1.0) if case["per_token"] else randn(1.0, S)
    state["mask"] = None
    if case["masked"]:
        # the first tokens of each sequence are the prompt's; of some sequences nothing counts
        t = torch.arange(T, device="cuda")
        s = torch.searchsorted(offsets, t, right=True).sub_(1).clamp_(0, S - 1)
        prompt = torch.rand(S, device="cuda", generator=gen) * (offsets[1:] - offsets[:-1])
        none = torch.rand(S, device="cuda", generator=gen) < (0.05 if S > 1 else 0.0)
        state["mask"] = ((t - offsets[s] >= prompt[s] * 0.5) & ~none[s]).to(torch.uint8)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "policy":
        return _prepare_policy(case, gen)
    dtype, ne0, ne1, pad = DTYPES[case["dtype"]], case["ne0"], case["ne1"], case["row_pad"]
    state = dict(case)
    if case["op"] == "checkpoint":
        state.update(x=_normal_rows(ne1, ne0, pad, dtype, gen, True), codes=_codes(case), out=_rows(ne1, ne0, pad, dtype))
        return state
    row = lambda at, scale: (at + scale * torch.randn(ne0, device="cuda", generator=gen)).to(dtype)  # noqa: E731
    state["weight"] = row(1.0, 0.1) if case["affine"] else None
    state["shift"] = row(0.0, 0.1) if case["affine"] == "both" else None
    state["bias_row"] = row(0.0, 0.1) if case["bias"] else None
    state["mean"], state["rstd"] = torch.empty(ne1, device="cuda"), torch.empty(ne1, device="cuda")
    res_rows = {"": 0, "full": ne1, "row": 1}[case["residual"]]
    state["res"] = state["dres"] = None
    if case["op"] != "reduce_norm_grad":
        state["srcs"] = [_normal_rows(ne1, ne0, pad, dtype, gen, True) for _ in range(case["R"])]
        state["res"] = _normal_rows(res_rows, ne0, pad, dtype, gen, False) if res_rows else None
        state["ys"] = [_rows(ne1, ne0, pad, dtype) for _ in range(case["n_dsts"])]
        state["sum_bufs"] = [_rows(ne1, ne0, pad, dtype) for _ in range(case["sums"])]
        state["codes"] = _codes(case) if case["keep"] else None
    else:
        # a kept sum with the statistics that its forward pass left
        state["h"] = _normal_rows(ne1, ne0, pad, dtype, gen, True)
        x = state["h"].double()
        mean = x.mean(1) if case["kind"] == "layer" else torch.zeros(ne1, dtype=torch.float64, device="cuda")
        state["mean"].copy_(mean)
        state["rstd"].copy_(((x - mean[:, None]).square().mean(1) + EPS).rsqrt())
    if case["op"] != "reduce_norm":
        state["dy"] = _normal_rows(ne1, ne0, pad, dtype, gen, False)
        state["dres"] = _normal_rows(ne1, ne0, pad, dtype, gen, False) if case["residual"] == "full" else None
        state["dxs"] = [_rows(ne1, ne0, pad, dtype) for _ in range(case["n_dsts"])]
        wanted = {"dweight": bool(case["affine"]), "dshift": case["affine"] == "both",
                  "dbias": case["bias"] or case["residual"] == "row"}
        state.update({k: torch.empty(ne0, device="cuda") if w else None for k, w in wanted.items()})
    return state


# ---- the library's calls ------------------------------------------------------

_context = None


def _library(R, elems):
    """The package with a context for R ranks, made once as a program does at its start."""
    global _context
    import tensor_partial_sum_gb300 as tps
    if _context is None or _context[0] != R or _context[1] < elems:
        tps.ar_init(R, elems)
        _context = (R, elems)
    return tps


def _strides(tensors):
    return [t.stride(0) * t.element_size() for t in tensors]


def _own_forward(tps, s, norm, checkpoint):
    strides = dict(src_row_bytes=_strides(s["srcs"]), dst_row_bytes=_strides(s["ys"])) if s["row_pad"] else {}
    res = s["res"]
    res_bytes = None if res is None else _strides([res])[0] if s["residual"] == "full" else 0
    layout = tps.make_layout(s["ne0"], s["ne1"], residual=res, residual_row_bytes=res_bytes, **strides)
    sum_rows = _strides(s["sum_bufs"]) if s["row_pad"] else None
    tps.ar_reduce_norm(s["srcs"], s["ys"], layout, norm, s["dtype"], s["wire"], sums=s["sum_bufs"],
                       sum_row_bytes=sum_rows, mean=s["mean"], rstd=s["rstd"], checkpoint=checkpoint)
    return {"y": s["ys"], "sum": s["sum_bufs"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_backward(tps, s, norm, kept):
    rows = {}
    if s["row_pad"]:
        given = [s["dy"]] if s["keep"] else [s["dy"], s["h"]]
        rows = dict(src_row_bytes=_strides(given), dst_row_bytes=_strides(s["dxs"]))
    res_bytes = None if s["dres"] is None else _strides([s["dres"]])[0]
    layout = tps.make_layout(s["ne0"], s["ne1"], residual=s["dres"], residual_row_bytes=res_bytes, **rows)
    tps.ar_reduce_norm_grad(s["dy"], kept, s["dxs"], layout, norm, s["mean"], s["rstd"], s["dtype"],
                            dweight=s["dweight"], dshift=s["dshift"], dbias=s["dbias"])
    return {"dx": s["dxs"], "dweight": s["dweight"], "dshift": s["dshift"], "dbias": s["dbias"]}


def _own_norm(s):
    tps = _library(s["R"], s["ne0"] * s["ne1"])
    norm = tps.make_norm(EPS, s["weight"], s["shift"], s["bias_row"], kind=s["kind"])
    if s["op"] == "reduce_norm_grad":
        return _own_backward(tps, s, norm, s["h"])
    checkpoint = tps.make_checkpoint(*s["codes"], s["ne0"], s["keep"]) if s["keep"] else None
    out = _own_forward(tps, s, norm, checkpoint)
    if s["op"] == "norm_step":
        out.update(_own_backward(tps, s, norm, checkpoint))
    return out


def _own_checkpoint(s):
    tps = _library(1, s["ne0"] * s["ne1"])
    checkpoint = tps.make_checkpoint(*s["codes"], s["ne0"], s["keep"])
    tps.ar_checkpoint_pack(s["x"], checkpoint)
    tps.ar_checkpoint_unpack(checkpoint, s["out"])
    return {"x": s["out"]}


def _own_policy(s):
    tps = _library(1, s["T"])
    tps.ar_policy_loss(s["nll"], s["offsets"], s["advantages"], s["totals"], dnll=s["dnll"], old_nll=s["old_nll"],
                       ref_nll=s["ref_nll"], mask=s["mask"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                       kl_weight=s["kl"], mean=s["mean"], token_advantages=s["per_token"])
    return {"totals": s["totals"], "dnll": s["dnll"]}


# ---- plain forms --------------------------------------------------------------

LARGEST = {"e4m3": (0.875, 9), "int8": (0.9921875, 7)}  # of a code, as fraction and exponent


def _plain_kept(x, keep):
    """What an 8-bit checkpoint of the rows of x stands for, in 32 bits."""
    ne1, ne0 = x.shape
    v = torch.zeros((ne1, -(-ne0 // BLOCK) * BLOCK), device="cuda")
    v[:, :ne0] = x.float()
    v = v.reshape(ne1, -1, BLOCK)
    most, bits = LARGEST[keep]
    fraction, exponent = torch.frexp(v.abs().amax(2, keepdim=True))
    e = (exponent - bits + (fraction > most)).clamp(min=-127).long()
    power = lambda k: ((k + 1023) << 52).view(torch.float64)  # noqa: E731  2^k
    scaled = v.double() * power(-e)
    code = scaled.float().to(torch.float8_e4m3fn).double() if keep == "e4m3" else scaled.round()
    return (code * power(e)).float().reshape(ne1, -1)[:, :ne0]


def _plain_forward(s):
    dtype, wire = DTYPES[s["dtype"]], DTYPES[s["wire"]]
    acc = functools.reduce(torch.add, [x.to(wire).float() for x in s["srcs"]])
    acc = acc + s["bias_row"].float() if s["bias_row"] is not None else acc
    acc = acc + s["res"].float() if s["res"] is not None else acc
    h = acc.to(dtype)
    x = h.float()
    mean = x.mean(1) if s["kind"] == "layer" else torch.zeros(s["ne1"], device="cuda")
    x = x - mean[:, None]
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    y = x * rstd[:, None]
    y = y * s["weight"].float() if s["weight"] is not None else y
    y = y + s["shift"].float() if s["shift"] is not None else y
    y = y.to(dtype)
    return h, {"y": [y.clone() for _ in s["ys"]], "sum": [h.clone() for _ in s["sum_bufs"]], "mean": mean, "rstd": rstd}


def _plain_backward(s, h, mean, rstd):
    dy = s["dy"].float()
    x = (h - mean[:, None]) * rstd[:, None]
    g = dy * s["weight"].float() if s["weight"] is not None else dy
    dx = g - x * (g * x).mean(1, keepdim=True)
    dx = dx - g.mean(1, keepdim=True) if s["kind"] == "layer" else dx
    dx = dx * rstd[:, None]
    dx = dx + s["dres"].float() if s["dres"] is not None else dx
    d = dx.to(s["dy"].dtype)
    return {"dx": [d.clone() for _ in s["dxs"]], "dweight": (dy * x).sum(0) if s["dweight"] is not None else None,
            "dshift": dy.sum(0) if s["dshift"] is not None else None,
            "dbias": dx.sum(0) if s["dbias"] is not None else None}


def _plain_norm(s):
    if s["op"] == "reduce_norm_grad":
        return _plain_backward(s, s["h"].float(), s["mean"], s["rstd"])
    h, out = _plain_forward(s)
    if s["op"] == "norm_step":
        out.update(_plain_backward(s, _plain_kept(h, s["keep"]), out["mean"], out["rstd"]))
    return out


def _plain_checkpoint(s):
    most = torch.finfo(s["x"].dtype).max
    return {"x": _plain_kept(s["x"], s["keep"]).clamp(-most, most).to(s["x"].dtype)}


def _plain_policy(s):
    T, S, offsets = s["T"], s["S"], s["offsets"]
    t = torch.arange(T, device="cuda")
    seq = (torch.searchsorted(offsets, t, right=True) - 1).clamp(0, S - 1)
    counted = (t >= offsets[0]) & (t < offsets[S])
    counted = counted & (s["mask"] != 0) if s["mask"] is not None else counted
    a = s["advantages"] if s["per_token"] else s["advantages"][seq]
    # the log ratio in 64 bits, where it is compared with the clip range
    log_ratio = s["old_nll"].double() - s["nll"].double() if s["old_nll"] is not None else torch.zeros_like(s["nll"]).double()
    above, below = log_ratio > math.log1p(CLIP_HIGH), log_ratio < math.log1p(-CLIP_LOW)
    ratio = torch.exp(log_ratio.float())
    clipped = (above & (a > 0)) | (below & (a < 0))
    limit = torch.where(above, 1 + CLIP_HIGH, 1 - CLIP_LOW).float()
    gain = torch.where(clipped, limit, ratio) * a
    grad = torch.where(clipped, 0.0, ratio * a)
    kl = torch.zeros_like(gain)
    if s["ref_nll"] is not None:
        d = s["nll"].double() - s["ref_nll"].double()
        kl = (torch.expm1(d) - d).float()
        grad = grad + s["kl"] * torch.expm1(d).float()
    counts = torch.zeros(S, dtype=torch.int64, device="cuda").index_add_(0, seq, counted.long())
    n = counted.sum()
    if s["mean"] == "sum":
        weight = torch.ones(T, dtype=torch.float64, device="cuda")
    elif s["mean"] == "tokens":
        weight = (1 / n.clamp(min=1).double()).expand(T)
    else:
        weight = 1 / (counts.clamp(min=1)[seq].double() * (counts > 0).sum().clamp(min=1))
    weight = torch.where(counted, weight, 0.0)
    total = lambda x: (torch.where(counted, x, 0.0).double() * weight).sum()  # noqa: E731
    policy, divergence = -total(gain), total(kl)
    share = (clipped & counted).sum() / n.clamp(min=1)
    totals = torch.stack([policy + s["kl"] * divergence, policy, divergence, share.double()]).float()
    return {"totals": totals, "dnll": torch.where(counted, grad * weight.float(), 0.0)}


def run(state):
    if state["op"] == "policy":
        return _own_policy(state) if own else _plain_policy(state)
    if state["op"] == "checkpoint":
        return _own_checkpoint(state) if own else _plain_checkpoint(state)
    return _own_norm(state) if own else _plain_norm(state)


# ---- 64 bits --------------------------------------------------------------------

def _exact_kept(x, keep):
    """The values of a checkpoint of x (64 bits) from the definition of the code grids."""
    ne1, ne0 = x.shape
    top = torch.stack([p.abs().amax(1) for p in x.split(BLOCK, 1)], 1)
    largest = 448.0 if keep == "e4m3" else 127.0
    e = torch.ceil(torch.log2(torch.where(top > 0, top / largest, 2.0 ** -127))).clamp(min=-127)
    # the logarithm may be one off next to a power of two
    e = torch.where(top <= largest * torch.exp2(e - 1), (e - 1).clamp(min=-127), e)
    e = torch.where(top > largest * torch.exp2(e), e + 1, e)
    unit = torch.exp2(e).repeat_interleave(BLOCK, 1)[:, :ne0]
    v = x / unit
    step = 1.0
    if keep == "e4m3":
        # three fraction bits, the smallest exponent -6
        step = torch.exp2((torch.frexp(v).exponent - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step * unit


def _exact_norm(case, s):
    out, dtype = {}, DTYPES[case["dtype"]]
    w = s["weight"].double() if case["affine"] else 1.0
    if case["op"] != "reduce_norm_grad":
        h = sum(x.to(DTYPES[case["wire"]]).double() for x in s["srcs"])
        if case["bias"]:
            h += s["bias_row"].double()
        if case["residual"]:
            h += s["res"].double()
        h = h.to(dtype).double()  # what is normalised is the sum as it is stored
        mean = h.mean(1, keepdim=True) * (case["kind"] == "layer")
        rstd = torch.rsqrt(torch.square(h - mean).mean(1, keepdim=True) + EPS)
        y = (h - mean) * rstd * w + (s["shift"].double() if case["affine"] == "both" else 0.0)
        out = {"y": [y] * case["n_dsts"], "sum": [h] * case["sums"], "mean": mean[:, 0], "rstd": rstd[:, 0]}
    else:
        h, mean, rstd = s["h"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    if case["op"] != "reduce_norm":
        x = ((_exact_kept(h, case["keep"]) if case["keep"] else h) - mean) * rstd
        dy = s["dy"].double()
        back = dy * w * rstd
        dx = back - x * (back * x).sum(1, keepdim=True) / case["ne0"]
        if case["kind"] == "layer":
            dx -= back.sum(1, keepdim=True) / case["ne0"]
        if case["residual"] == "full":
            dx += s["dres"].double()
        out.update(dx=[dx] * case["n_dsts"], dweight=(dy * x).sum(0) if case["affine"] else None,
                   dshift=dy.sum(0) if case["affine"] == "both" else None,
                   dbias=dx.sum(0) if case["bias"] or case["residual"] == "row" else None)
    return out


def _exact_policy(case, s):
    """The loss as it is written down, its gradient by differentiation."""
    T, bounds = case["T"], s["offsets"].tolist()
    seq = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    lengths = s["offsets"][1:] - s["offsets"][:-1]
    seq[bounds[0]:bounds[-1]] = torch.repeat_interleave(torch.arange(case["S"], device="cuda"), lengths)
    valid = seq >= 0
    if case["masked"]:
        valid &= s["mask"] > 0
    at = torch.nonzero(valid)[:, 0]
    nll = s["nll"].double().requires_grad_()
    mine = nll[at]
    old = s["old_nll"].double()[at] if case["old"] else mine.detach()
    a = (s["advantages"][at] if case["per_token"] else s["advantages"][seq[at]]).double()
    ratio = torch.exp(old - mine)
    inside = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    policy = -torch.where(ratio * a <= inside * a, ratio * a, inside * a)
    kl = torch.zeros_like(mine)
    if case["kl"] > 0:
        d = mine - s["ref_nll"].double()[at]
        kl = torch.expm1(d) - d
    if case["mean"] == "sequences":
        counts = torch.bincount(seq[at], minlength=case["S"])
        weight = 1.0 / counts[seq[at]].double() / max(1, int((counts > 0).sum()))
    else:
        weight = torch.full_like(a, 1.0 / max(1, len(at)) if case["mean"] == "tokens" else 1.0)
    parts = torch.stack([(policy * weight).sum(), (kl * weight).sum()])
    loss = parts[0] + case["kl"] * parts[1]
    loss.backward()
    clipped = ((ratio > 1 + CLIP_HIGH) & (a > 0)) | ((ratio < 1 - CLIP_LOW) & (a < 0))
    share = clipped.double().sum() / max(1, len(at))
    return {"totals": torch.stack([loss.detach(), parts[0].detach(), parts[1].detach(), share]), "dnll": nll.grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "policy":
        return _exact_policy(case, s)
    if case["op"] == "checkpoint":
        most = torch.finfo(DTYPES[case["dtype"]]).max
        return {"x": _exact_kept(s["x"].double(), case["keep"]).clamp(-most, most)}
    return _exact_norm(case, s)
