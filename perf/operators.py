"""Cases that measure the training operators around the partial-sum reduction.

Four calls are measured, each in a plain form (elementary torch operations in
32 bits, rounded once at the end) and through the library's entry points:

``reduce_dropout``
    The end of a tensor-parallel layer in training.  R partials are rounded
    through the wire type and summed in rank order, a bias row is added, the
    sum goes through dropout, a residual is added, and the result is written
    to every destination.  The dropout mask is a function of (seed, offset,
    row, column) alone and is never stored.
``reduce_dropout_grad``
    Its backward pass: the gradient of the partials (one value, written to
    every rank's buffer), of the bias row, and of a residual row that was
    broadcast.
``vocab_loss``
    Softmax cross entropy of hidden states against an output matrix whose
    vocabulary rows are split into pieces (one per rank), without keeping the
    logits: a loss and a log-sum-exp for each token.
``vocab_train``
    The same loss and its gradients, as one training step needs them: each
    piece's partial gradient of the hidden states (the partials that
    ``ar_reduce`` sums) and the gradient of each piece's weights.

Random words are an input in the form of a seed and an offset: word w of
Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
2011) under the key (seed low, seed high) and the counter (column // 4, row,
offset low, offset high) belongs to column 4 * (column // 4) + w.  An element
is kept when its word is at least floor(p * 2^32).
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
IGNORED = -100


# ---- cases ------------------------------------------------------------------

def _drop(name, op, R, n_dsts, dtype, wire, ne1, ne0, residual, bias, p, row_pad=0):
    case = {"op": op, "R": R, "n_dsts": n_dsts, "dtype": dtype, "wire": wire, "ne1": ne1, "ne0": ne0,
            "residual": residual, "bias": bias, "p": p, "row_pad": row_pad}
    return dict(case, name=name) if name else case


def _vocab(name, op, R, dtype, T, D, V, ignored=0.0, weighted=False, row_pad=0):
    case = {"op": op, "R": R, "dtype": dtype, "T": T, "D": D, "V": V, "ignored": ignored, "weighted": weighted,
            "row_pad": row_pad}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token's activation, the smallest call: latency counts
        _drop("dropout one row", "reduce_dropout", 4, 4, "f32", "f16", 1, 4099, "full", True, 0.1),
        # a prompt's or a micro-batch's activation on two ranks
        _drop("dropout prefill", "reduce_dropout", 2, 2, "f32", "bf16", 2048, 4096, "full", True, 0.1),
        # a large 16-bit activation on four ranks
        _drop("dropout large", "reduce_dropout", 4, 4, "bf16", "bf16", 4096, 8192, "full", True, 0.1),
        # the backward pass of the same layers
        _drop("dropout grad prefill", "reduce_dropout_grad", 2, 2, "f32", "bf16", 2048, 4096, "full", True, 0.1),
        _drop("dropout grad large", "reduce_dropout_grad", 4, 4, "bf16", "bf16", 4096, 8192, "full", True, 0.1),
        # odd rows out of a wider buffer, a broadcast residual row and its gradient
        _drop("dropout grad odd", "reduce_dropout_grad", 3, 1, "f16", "f16", 1021, 4099, "row", True, 0.25, 13),
        # scoring one token: bound by reading the output matrix
        _vocab("loss one token", "vocab_loss", 1, "bf16", 1, 4096, 32768),
        # scoring a prompt on four vocabulary pieces
        _vocab("loss prompt", "vocab_loss", 4, "bf16", 2048, 4096, 32768),
        # a training step whose sizes fit nothing, a third of the tokens masked
        _vocab("train odd", "vocab_train", 3, "f16", 1021, 1031, 50021, 0.33, True, 3),
        # a training step in full precision
        _vocab("train f32", "vocab_train", 2, "f32", 512, 1024, 16384, 0.1),
        # a micro-batch of a training step
        _vocab("train micro-batch", "vocab_train", 4, "bf16", 2048, 4096, 32768, 0.1),
        # a large vocabulary on eight ranks
        _vocab("train large", "vocab_train", 8, "bf16", 4096, 4096, 131072),
    ]


MOST_BYTES = 600_000_000              # of a dropout case, about "dropout large"
MOST_TVD = 4096 * 4096 * 131072       # of a vocabulary case, "train large"


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reduce_dropout", "reduce_dropout_grad", "vocab_loss", "vocab_train"])
    if op.startswith("reduce"):
        dtype = rng.choice(["f32", "f16", "bf16"])
        R = rng.randint(1, 8)
        n_dsts = rng.choice([1, R])
        residual = rng.choice(["", "full", "row"])
        ne0, ne1 = _log_int(rng, 33, 8192), _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            ne0 = max(32, ne0 // 32 * 32)
        case = _drop(None, op, R, n_dsts, dtype, rng.choice(["f32", "f16", "bf16"]), ne1, ne0, residual,
                     rng.random() < 0.6, rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]),
                     rng.choice([0, 0, 8, rng.randint(1, 64)]))
        over = work(case)["bytes"] / MOST_BYTES
        if over > 1:
            case["ne1"] = max(1, int(ne1 / over))
        return case
    T, D, V = _log_int(rng, 1, 4096), _log_int(rng, 128, 8192), _log_int(rng, 1000, 131072)
    if rng.random() < 0.6:
        D = max(128, D // 64 * 64)
    if T * D * V > MOST_TVD:
        V = max(1000, MOST_TVD // (T * D))
    return _vocab(None, op, rng.randint(1, 8), rng.choice(["bf16", "bf16", "f16", "f32"]), T, D, V,
                  rng.choice([0.0, 0.0, 0.2, 0.6]), rng.random() < 0.4, rng.choice([0, 0, 8, rng.randint(1, 32)]))


def _pieces(case):
    """Vocabulary rows of each piece: equal ones, the last takes what is left."""
    per = -(-case["V"] // case["R"])
    return [min(per, case["V"] - r * per) for r in range(case["R"])]


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"].startswith("reduce"):
        n, rows = case["ne0"] * case["ne1"], case["ne0"]
        if case["op"] == "reduce_dropout":
            tensors = case["R"] + case["n_dsts"] + (case["residual"] == "full")
            extra = ((case["residual"] == "row") + bool(case["bias"])) * rows * es
            adds = case["R"] + bool(case["bias"]) + bool(case["residual"])
        else:
            tensors = 1 + case["n_dsts"]
            extra = ((case["residual"] == "row") + bool(case["bias"])) * rows * 4
            adds = 1 + (case["residual"] == "row") + bool(case["bias"])
        return {"bytes": tensors * n * es + extra, "flops": adds * n}
    T, D, V = case["T"], case["D"], case["V"]
    read = (T * D + V * D) * es + T * 8
    if case["op"] == "vocab_loss":
        return {"bytes": read + T * 8, "flops": 2 * T * V * D}
    # the logits, the hidden states' gradient and the weights' gradient, one product each
    return {"bytes": read + T * 12 + (case["R"] * T * D + V * D) * es, "flops": 6 * T * V * D}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"].startswith("reduce"):
        ne0, ne1, pad = case["ne0"], case["ne1"], case["row_pad"]
        state = dict(case, seed=(seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 64, offset=seed * 1000003 % 2 ** 40,
                     outs=[_rows(ne1, ne0, pad, dtype) for _ in range(case["n_dsts"])])
        if case["op"] == "reduce_dropout":
            state["srcs"] = [_normal_rows(ne1, ne0, pad, dtype, gen, True) for _ in range(case["R"])]
            res_rows = {"": 0, "full": ne1, "row": 1}[case["residual"]]
            state["res"] = _normal_rows(res_rows, ne0, pad, dtype, gen, False) if res_rows else None
            state["bias_row"] = torch.randn(ne0, device="cuda", generator=gen).mul(0.1).to(dtype) if case["bias"] else None
        else:
            state["dy"] = _normal_rows(ne1, ne0, pad, dtype, gen, False)
            state["dbias"] = torch.empty(ne0, device="cuda") if case["bias"] else None
            state["dres"] = torch.empty(ne0, device="cuda") if case["residual"] == "row" else None
        return state
    T, D, V, pad, sizes = case["T"], case["D"], case["V"], case["row_pad"], _pieces(case)
    # weights of about unit rows, so that logits have a spread of two; each
    # token's state leans towards its target's row by an amount of its own,
    # so that target probabilities run from 1/V to nearly one
    weights = [_rows(v, D, pad, dtype) for v in sizes]
    for w in weights:
        w.copy_(torch.randn((w.shape[0], D), device="cuda", generator=gen).mul_(2 / math.sqrt(D)))
    targets = torch.randint(0, V, (T,), device="cuda", generator=gen)
    per = sizes[0]
    lean = torch.rand((T, 1), device="cuda", generator=gen) * 4
    aim = torch.zeros((T, D), device="cuda")
    for r, w in enumerate(weights):
        at = (targets - r * per).clamp(0, w.shape[0] - 1)
        aim += torch.where((targets // per == r)[:, None], w[at].float(), 0.0)
    hidden = _rows(T, D, pad, dtype)
    hidden.copy_(torch.randn((T, D), device="cuda", generator=gen) + lean * aim)
    if case["ignored"]:
        targets = torch.where(torch.rand(T, device="cuda", generator=gen) < case["ignored"], IGNORED, targets)
    state = dict(case, hidden=hidden, weights=weights, targets=targets,
                 loss=torch.empty(T, device="cuda"), lse=torch.empty(T, device="cuda"))
    if case["op"] == "vocab_train":
        # the mean over the counted tokens, or a weighted one
        scale = torch.rand(T, device="cuda", generator=gen) if case["weighted"] else torch.ones(T, device="cuda")
        state["dloss"] = scale / max(1.0, T * (1 - case["ignored"]))
        state["dhidden"] = [_rows(T, D, 0, dtype) for _ in sizes]
        state["dweights"] = [_rows(v, D, pad, dtype) for v in sizes]
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


def _own_dropout(s):
    tps = _library(s["R"], s["ne0"] * s["ne1"])
    drop = tps.make_dropout(s["p"], s["seed"], s["offset"], bias=s.get("bias_row"))
    if s["op"] == "reduce_dropout":
        res = s["res"]
        res_bytes = None if res is None else _strides([res])[0] if s["residual"] == "full" else 0
        layout = tps.make_layout(s["ne0"], s["ne1"], src_row_bytes=_strides(s["srcs"]),
                                 dst_row_bytes=_strides(s["outs"]), residual=res, residual_row_bytes=res_bytes)
        tps.ar_reduce_dropout(s["srcs"], s["outs"], layout, drop, s["dtype"], s["wire"])
        return {"y": s["outs"]}
    layout = tps.make_layout(s["ne0"], s["ne1"], src_row_bytes=_strides([s["dy"]]), dst_row_bytes=_strides(s["outs"]))
    tps.ar_reduce_dropout_grad(s["dy"], s["outs"], layout, drop, s["dtype"], dbias=s["dbias"], dresidual=s["dres"])
    return {"dx": s["outs"], "dbias": s["dbias"], "dresidual": s["dres"]}


def _own_vocab(s):
    tps = _library(s["R"], s["T"] * s["D"])
    tps.ar_vocab_loss(s["hidden"], s["weights"], s["targets"], s["loss"], s["lse"], ignore_index=IGNORED)
    out = {"loss": s["loss"], "lse": s["lse"]}
    if s["op"] == "vocab_train":
        tps.ar_vocab_loss_grad(s["hidden"], s["weights"], s["targets"], s["lse"], s["dloss"], dhidden=s["dhidden"],
                               dweights=s["dweights"], ignore_index=IGNORED)
        out.update(dhidden=s["dhidden"], dweights=s["dweights"])
    return out


# ---- plain forms --------------------------------------------------------------

def _philox_round(state, _):
    c0, c1, c2, c3, k0, k1 = state
    # products of two 32-bit words; the upper word survives 64-bit wrap-around
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    m = 0xFFFFFFFF
    return (((b >> 32) & m) ^ c1 ^ k0, b & m, ((a >> 32) & m) ^ c3 ^ k1, a & m,
            (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m)


def _plain_keep(s):
    """[ne1, ne0] truth values: which elements the dropout keeps."""
    groups = -(-s["ne0"] // 4)
    col = torch.arange(groups, device="cuda")[None, :].expand(s["ne1"], groups)
    row = torch.arange(s["ne1"], device="cuda")[:, None].expand(s["ne1"], groups)
    start = (col, row, torch.full_like(col, s["offset"] & 0xFFFFFFFF), torch.full_like(col, s["offset"] >> 32),
             s["seed"] & 0xFFFFFFFF, s["seed"] >> 32)
    words = functools.reduce(_philox_round, range(10), start)[:4]
    threshold = int(float(np.float32(s["p"])) * 4294967296.0)
    return torch.stack(words, -1).reshape(s["ne1"], groups * 4)[:, :s["ne0"]] >= threshold


def _plain_dropout(s):
    dtype, wire = DTYPES[s["dtype"]], DTYPES[s["wire"]]
    keep, scale = _plain_keep(s), float(np.float32(1) / (np.float32(1) - np.float32(s["p"])))
    if s["op"] == "reduce_dropout":
        acc = functools.reduce(torch.add, [x.to(wire).float() for x in s["srcs"]])
        acc = acc + s["bias_row"].float() if s["bias_row"] is not None else acc
        acc = torch.where(keep, acc * scale, 0.0)
        acc = acc + s["res"].float() if s["res"] is not None else acc
        y = acc.to(dtype)
        return {"y": [y.clone() for _ in s["outs"]]}
    dy = s["dy"].float()
    dx = torch.where(keep, dy * scale, 0.0)
    return {"dx": [dx.to(dtype) for _ in s["outs"]],
            "dbias": dx.sum(0) if s["dbias"] is not None else None,
            "dresidual": dy.sum(0) if s["dres"] is not None else None}


def _plain_vocab(s):
    hidden, weight = s["hidden"].float(), torch.cat(s["weights"]).float()
    logits = hidden @ weight.t()
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + (logits - top).exp().sum(1).log()
    counted = s["targets"] != IGNORED
    at = torch.where(counted, s["targets"], 0)[:, None]
    loss = torch.where(counted, lse - logits.gather(1, at)[:, 0], 0.0)
    out = {"loss": loss, "lse": lse}
    if s["op"] == "vocab_train":
        dtype = s["hidden"].dtype
        d = (logits - lse[:, None]).exp()
        d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        d *= torch.where(counted, s["dloss"], 0.0)[:, None]
        parts = d.split([w.shape[0] for w in s["weights"]], 1)
        out["dhidden"] = [(p @ w.float()).to(dtype) for p, w in zip(parts, s["weights"])]
        out["dweights"] = [(p.t() @ hidden).to(dtype) for p in parts]
    return out


def run(state):
    if state["op"].startswith("reduce"):
        return _own_dropout(state) if own else _plain_dropout(state)
    return _own_vocab(state) if own else _plain_vocab(state)


# ---- 64 bits --------------------------------------------------------------------

def _exact_keep(case, s):
    """The same words from 64-bit unsigned products on the host."""
    groups = -(-case["ne0"] // 4)
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = np.zeros((4, case["ne1"], groups), np.uint64)
    ctr[0] += np.arange(groups, dtype=np.uint64)[None]
    ctr[1] += np.arange(case["ne1"], dtype=np.uint64)[:, None]
    ctr[2] += np.uint64(s["offset"] & 0xFFFFFFFF)
    ctr[3] += np.uint64(s["offset"] >> 32)
    key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
    for _ in range(10):
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = np.stack([(p1 >> sh) ^ ctr[1] ^ np.uint64(key[0]), p1 & low,
                        (p0 >> sh) ^ ctr[3] ^ np.uint64(key[1]), p0 & low])
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.moveaxis(ctr, 0, 2).reshape(case["ne1"], groups * 4)[:, :case["ne0"]]
    return torch.from_numpy(words >= np.uint64(math.floor(float(np.float32(case["p"])) * 2 ** 32))).cuda()


def _exact_dropout(case, s):
    kept = _exact_keep(case, s).double() / (1 - float(np.float32(case["p"])))
    if case["op"] == "reduce_dropout":
        total = torch.zeros((case["ne1"], case["ne0"]), dtype=torch.float64, device="cuda")
        for x in s["srcs"]:
            total += x.to(DTYPES[case["wire"]]).double()
        if case["bias"]:
            total += s["bias_row"].double()
        total *= kept
        if case["residual"]:
            total += s["res"].double()
        return {"y": [total] * case["n_dsts"]}
    dy = s["dy"].double()
    return {"dx": [dy * kept] * case["n_dsts"], "dbias": (dy * kept).sum(0) if case["bias"] else None,
            "dresidual": dy.sum(0) if case["residual"] == "row" else None}


def _exact_vocab(case, s):
    train = case["op"] == "vocab_train"
    if (6 if train else 2) * case["T"] * case["D"] * case["V"] > 8e12:
        return None  # over about ten seconds in 64 bits
    h, weights = s["hidden"].double(), [w.double() for w in s["weights"]]
    logits = torch.cat([h @ w.t() for w in weights], 1)
    lse = torch.logsumexp(logits, 1)
    rows = torch.nonzero(s["targets"] >= 0)[:, 0]
    picked = s["targets"][rows]
    loss = torch.zeros(case["T"], dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - logits[rows, picked]
    out = {"loss": loss, "lse": lse}
    if train:
        g = torch.zeros_like(logits)
        g[rows] = torch.softmax(logits[rows], 1)
        g[rows, picked] -= 1
        g *= s["dloss"].double()[:, None]
        out["dhidden"], out["dweights"], first = [], [], 0
        for w in weights:
            part = g[:, first:first + w.shape[0]]
            first += w.shape[0]
            out["dhidden"].append(part @ w)
            out["dweights"].append(part.t() @ h)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_dropout(case, s) if case["op"].startswith("reduce") else _exact_vocab(case, s)
