"""The normalisation, checkpoint and policy operators in 64 bits, for their tests."""
import numpy as np
import torch

UNIT = 2.0 ** -24  # a float rounding, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def adds(n):
    """Float additions behind a sum of n terms: those of one of 512 threads, ten between threads, a few around them."""
    return max(64, n // 512 + 24)


def norm_forward(h, weight, shift, eps, rms):
    """(y, mean, rstd, how far a float computation may leave y off) of 64-bit rows."""
    n = h.shape[1]
    mean = torch.zeros_like(h[:, :1]) if rms else h.mean(1, keepdim=True)
    d = h - mean
    rstd = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / n + eps)
    w = torch.ones_like(h[0]) if weight is None else weight.double()
    s = torch.zeros_like(h[0]) if shift is None else shift.double()
    x = d * rstd
    # the mean is off by so many roundings of the mean |d|, rstd by as many of itself
    slack = adds(n) * UNIT * (w.abs() * (1 + x.abs()) + s.abs())
    return x * w + s, mean[:, 0], rstd[:, 0], slack


def norm_backward(dy, h, mean, rstd, weight, dsum, rms):
    """{name: (value, slack)} of the gradients, from 64-bit rows and the statistics that the call is given."""
    n, rows = dy.shape[1], dy.shape[0]
    rstd = rstd[:, None]
    x = (h if rms else h - mean[:, None]) * rstd
    g = dy if weight is None else dy * weight.double()
    c1 = torch.zeros_like(rstd) if rms else g.mean(1, keepdim=True)
    c2 = (g * x).mean(1, keepdim=True)
    dh = rstd * (g - c1 - x * c2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * x).abs().mean(1, keepdim=True)
    # means of n terms, and at most eight roundings of each operand
    off = UNIT * rstd.abs() * (adds(n) * (a1 + x.abs() * a2) + 8 * (g.abs() + c1.abs() + (x * c2).abs()))
    if dsum is not None:
        dh = dh + dsum
        off = off + UNIT * (dh.abs() + dsum.abs())
    out = {"dx": (dh, off)}
    for name, terms, each in (("dweight", dy * x, 8 * UNIT * (dy * x).abs()), ("dshift", dy, 0 * dy), ("dbias", dh, off)):
        out[name] = (terms.sum(0), each.sum(0) + (rows + 8) * UNIT * terms.abs().sum(0))
    return out


# ---- checkpoints: from tables of the codes' values --------------------------------

def _e4m3_value(code):
    sign, exponent, fraction = code >> 7, (code >> 3) & 15, code & 7
    if exponent == 15 and fraction == 7:
        return float("nan")
    v = fraction / 8 * 2.0 ** -6 if exponent == 0 else (1 + fraction / 8) * 2.0 ** (exponent - 7)
    return -v if sign else v


VALUES = {"e4m3": np.array([_e4m3_value(c) for c in range(256)]),
          "int8": np.array([float(np.int8(np.uint8(c))) for c in range(256)])}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def block_exponent(top, format):
    """The smallest e >= -127 with top <= largest * 2^e, by trying."""
    e = -127
    while top > LARGEST[format] * 2.0 ** e:
        e += 1
    return e


def nearest_code(v, format):
    """The code nearest to v, ties to the even one."""
    values = VALUES[format]
    d = np.abs(values - v)
    best = np.nanmin(d)
    codes = np.nonzero(d == best)[0]
    even = [c for c in codes if c % 2 == 0]
    return float(values[even[0] if len(codes) > 1 and even else codes[0]])


def checkpoint_values(x, format):
    """(values, scale bytes) that the checkpoint of a 64-bit numpy matrix stands for."""
    ne1, ne0 = x.shape
    out = np.zeros_like(x)
    scales = np.zeros((ne1, -(-ne0 // 32)), np.uint8)
    for j in range(ne1):
        for b in range(scales.shape[1]):
            v = x[j, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[j, b] = 255
                out[j, 32 * b:32 * b + 32] = np.nan
                continue
            e = block_exponent(np.abs(v).max(), format)
            scales[j, b] = e + 127
            out[j, 32 * b:32 * b + 32] = [nearest_code(t / 2.0 ** e, format) * 2.0 ** e for t in v]
    return out, scales


# ---- policy: as it is written down --------------------------------------------------

def policy(nll, offsets, adv, old=None, ref=None, mask=None, low=0.2, high=0.2, beta=0.0, scale=1.0, mean="tokens",
           token_advantages=False):
    """(totals, dnll, totals' slack, dnll's slack) in numpy's 64 bits."""
    T, S = len(nll), len(offsets) - 1
    seq = np.full(T, -1)
    for s in range(S):
        seq[offsets[s]:offsets[s + 1]] = s
    counted = seq >= 0
    if mask is not None:
        counted &= mask != 0
    at = np.nonzero(counted)[0]
    N = len(at)
    per = np.bincount(seq[at], minlength=max(S, 1))
    w = np.zeros(T)
    if N:
        w[at] = {"sum": 1.0, "tokens": 1 / N}.get(mean, 0) or 1 / (per[seq[at]] * (per > 0).sum())
    nll = np.where(counted, nll, 0.0).astype(np.float64)
    x = np.zeros(T) if old is None else np.where(counted, old, 0.0).astype(np.float64) - nll
    d = np.zeros(T) if ref is None else nll - np.where(counted, ref, 0.0).astype(np.float64)
    a = np.zeros(T)
    a[at] = adv[at] if token_advantages else np.asarray(adv)[seq[at]]
    with np.errstate(all="ignore"):
        ratio = np.exp(x)
        clipped = counted & (((x > np.log1p(high)) & (a > 0)) | ((x < np.log1p(-low)) & (a < 0)))
        plain = np.where(a == 0, 0.0, ratio * a)
        gain = np.where(clipped, np.where(a > 0, 1 + high, 1 - low) * a, plain)
        kl = np.expm1(d) - d
        small = np.abs(d) < 1e-3  # where the difference would leave too little of 64 bits
        kl[small] = (d ** 2 / 2 + d ** 3 / 6 + d ** 4 / 24 + d ** 5 / 120)[small]
        dkl = np.expm1(d)
        grad = np.where(clipped, 0.0, plain) + (beta * dkl if beta else 0.0)
        dnll = np.where(counted, scale * w * grad, 0.0)
        policy_part, kl_part = -scale * (w * gain).sum(), scale * (w * kl).sum()
        totals = np.array([policy_part + (beta * kl_part if beta else 0.0), policy_part, kl_part, clipped.sum() / max(N, 1)])
        # the exponential of a rounded argument, and a dozen roundings around it
        g_off = UNIT * np.abs(plain) * (16 + np.abs(x))
        k_off = UNIT * (16 * np.abs(kl) + (2 + np.abs(d)) * np.abs(d) * (np.exp(d) + 1))
        d_off = UNIT * (16 + np.abs(d)) * (np.abs(dkl) + np.abs(d) * np.exp(d))
        slack = np.abs(scale) * w * (np.where(clipped, 0.0, g_off) + 4 * UNIT * np.abs(grad) + beta * d_off)
        sums = np.abs(scale) * np.array([(w * (g_off + 32 * UNIT * np.abs(gain))).sum(), (w * (k_off + 32 * UNIT * kl)).sum()])
    t_off = np.array([sums[0] + beta * sums[1], sums[0], sums[1], 0.0]) + 2 * UNIT * np.abs(totals)
    return totals, dnll, t_off, slack
