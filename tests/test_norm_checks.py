"""Host-side checks of the normalisation, checkpoint and policy calls (CPU only)."""
import ctypes
import os
import subprocess

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tensor_partial_sum_gb300 import ar

OK, INVALID, UNSUPPORTED, TOO_LARGE, NOT_INIT, OVERLAP = range(6)
A = 1 << 20  # addresses far apart, never read
NAN, INF = float("nan"), float("inf")


def addr(k):
    return A * (k + 1)


def codes(ne0=64, ne1=4, format="e4m3", at=20, code_row=0, scale_row=0, scales=None):
    return tps.ArCheckpoint(ne0, ne1, ar.CODES.get(format, format), addr(at), code_row,
                            addr(at + 1) if scales is None else scales, scale_row)


def check(R=2, srcs=None, dsts=None, norm=None, ne0=64, ne1=4, max_elems=1 << 20, dst="f32", wire="bf16", kept=None, **kw):
    layout = tps.make_layout(ne0, ne1, **kw)
    return tps.ar_check_norm(R, srcs or [addr(0), addr(1)], dsts or [addr(2)], layout, norm or tps.make_norm(), max_elems,
                             dst, wire, **(kept or {}))


def test_check_norm_statuses():
    assert check() == OK
    assert check(norm=tps.make_norm(0.0, addr(3), addr(4), addr(5), kind="rms")) == OK
    for eps in (-1e-6, NAN, INF):
        assert check(norm=tps.make_norm(eps)) == INVALID
    assert check(norm=tps.ArNorm(2, 1e-5, None, None, None)) == INVALID
    for k in range(3):
        row = [None] * 3
        row[k] = addr(3) + 2
        assert check(norm=tps.make_norm(1e-5, *row)) == INVALID      # off an f32 boundary
        row[k] = addr(2) + 64 * 4
        assert check(norm=tps.make_norm(1e-5, *row)) == OVERLAP      # inside the destination
        row[k] = addr(0)
        assert check(norm=tps.make_norm(1e-5, *row)) == OK           # a source row may serve
    assert check(max_elems=255) == TOO_LARGE
    assert check(wire=9) == UNSUPPORTED
    assert check(dsts=[addr(0) + 4]) == OVERLAP
    assert check(dsts=[addr(0)]) == OK                               # in place
    assert check(ne1=0) == OK


def test_check_what_is_kept():
    row = 64 * 4
    assert check(kept=dict(sums=[addr(6), addr(7)], mean=addr(8), rstd=addr(9), checkpoint=codes())) == OK
    assert check(kept=dict(sums=[addr(0)])) == OK                     # exactly a source
    assert check(kept=dict(sums=[addr(0) + row])) == OVERLAP
    assert check(kept=dict(sums=[addr(3)]), residual=addr(3), residual_row_bytes=row) == OK
    assert check(kept=dict(sums=[addr(3)]), residual=addr(3), residual_row_bytes=0) == OVERLAP
    assert check(kept=dict(sums=[addr(2)])) == OVERLAP                # a destination
    assert check(kept=dict(sums=[addr(6), addr(6)])) == OVERLAP
    assert check(kept=dict(sums=[addr(6)]), norm=tps.make_norm(1e-5, addr(6))) == OVERLAP
    assert check(kept=dict(sums=[addr(6)] * 17)) == INVALID
    assert check(kept=dict(sums=[addr(6)], sum_row_bytes=[row - 4])) == INVALID
    assert check(kept=dict(mean=addr(8) + 2)) == INVALID
    assert check(kept=dict(mean=addr(8), rstd=addr(8) + 8)) == OVERLAP
    assert check(kept=dict(rstd=addr(1) + 16)) == OVERLAP             # inside a source
    assert check(kept=dict(mean=addr(3)), norm=tps.make_norm(1e-5, addr(3))) == OVERLAP
    assert check(kept=dict(checkpoint=codes(ne0=65))) == INVALID      # another shape
    assert check(kept=dict(checkpoint=codes(format=7))) == UNSUPPORTED
    assert check(kept=dict(checkpoint=codes(scales=addr(2) + 8))) == OVERLAP
    assert check(kept=dict(checkpoint=codes(scales=addr(20)))) == OVERLAP


def test_check_checkpoint_statuses():
    def c(ck, tensor=addr(0), row=0, max_elems=1 << 20, dtype="f32"):
        return tps.ar_check_checkpoint(ck, tensor, row, max_elems, dtype)
    assert c(codes()) == OK and c(codes(ne0=65, code_row=80, scale_row=3)) == OK
    assert c(codes(ne1=0), tensor=None) == OK
    assert c(codes(ne0=65, code_row=65)) == INVALID    # off a 16-byte boundary
    assert c(codes(code_row=48)) == INVALID            # rows over one another
    assert c(codes(scale_row=1)) == INVALID
    assert c(codes(code_row=-64)) == INVALID
    assert c(codes(), row=128) == INVALID and c(codes(), row=257) == INVALID
    assert c(codes(), tensor=None) == INVALID and c(codes(), tensor=addr(0) + 2) == INVALID
    assert c(codes(), max_elems=255) == TOO_LARGE
    assert c(codes(ne0=1 << 40, ne1=1 << 40)) == TOO_LARGE
    assert c(codes(format=2)) == UNSUPPORTED and c(codes(), dtype=5) == UNSUPPORTED
    assert c(codes(), tensor=addr(20)) == OVERLAP and c(codes(), tensor=addr(21) - 16) == OVERLAP
    broken = codes()
    broken.codes = addr(20) + 8
    assert c(broken) == INVALID
    broken.codes = None
    assert c(broken) == INVALID


def policy(**kw):
    p = tps.ArPolicy(100, 3, addr(0), addr(1), addr(2), addr(3), addr(4), 0, addr(5), 0.2, 0.2, 0.1, 1.0, 1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_check_policy_statuses():
    def c(max_elems=1 << 20, **kw):
        return tps.ar_check_policy(policy(**kw), max_elems)
    assert c() == OK
    assert c(old_nll=None, ref_nll=None, mask=None) == OK
    assert c(tokens=0, nll=None) == OK and c(sequences=0, offsets=None, advantages=None) == OK
    assert c(clip_low=1.0, clip_high=INF) == OK
    for bad in (dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=NAN), dict(clip_high=-0.1), dict(clip_high=NAN),
                dict(kl_weight=-1.0), dict(kl_weight=INF), dict(scale=NAN), dict(mean=3), dict(mean=-1),
                dict(token_advantages=2), dict(nll=None), dict(offsets=None), dict(advantages=None),
                dict(offsets=addr(0) + 4), dict(nll=addr(1) + 2), dict(advantages=addr(1) + 1)):
        assert c(**bad) == INVALID, bad
    assert c(max_elems=99) == TOO_LARGE
    assert c(max_elems=1 << 60, tokens=1 << 32) == TOO_LARGE
    assert c(sequences=1 << 31) == TOO_LARGE


def test_calls_need_a_context():
    lay, norm = tps.make_layout(8, 2), tps.make_norm()
    for call in (lambda: tps.ar_reduce_norm([addr(0)], [addr(1)], lay, norm, "f32", stream=0),
                 lambda: tps.ar_reduce_norm_grad(addr(0), addr(1), [addr(2)], lay, norm, addr(3), addr(4), "f32",
                                                 workspace=addr(5), stream=0)):
        with pytest.raises(tps.ARError) as e:
            call()
        assert e.value.status == NOT_INIT
    L = ar.lib()
    ck, p = codes(), policy()
    assert L.ar_checkpoint_pack(addr(0), 0, ctypes.byref(ck), 0, None) == NOT_INIT
    assert L.ar_checkpoint_unpack(ctypes.byref(ck), addr(0), 0, 0, None) == NOT_INIT
    assert L.ar_policy_loss(ctypes.byref(p), addr(8), None, addr(9), 1 << 20, None) == NOT_INIT


def test_workspace_sizes():
    n = tps.ar_reduce_norm_grad_workspace
    lay = tps.make_layout
    sizes = [n(lay(4096, 2048), k) for k in range(4)]
    assert sizes == sorted(sizes) and sizes[3] - sizes[2] == sizes[2] - sizes[1] > 0
    assert sizes[3] < 64 << 20
    assert n(lay(0, 8), 3) == 0
    for bad in (-1, 4):
        with pytest.raises(tps.ARError):
            n(lay(8, 8), bad)
    assert tps.ar_policy_workspace(policy()) > 0
    with pytest.raises(tps.ARError):
        tps.ar_policy_workspace(policy(mean=9))


def test_binding_refuses_wrong_buffers():
    lay, norm, host = tps.make_layout(8, 2), tps.make_norm(), torch.zeros(2, 8)
    for call in (lambda: tps.ar_reduce_norm([host], [host], lay, norm, "f32", stream=0),
                 lambda: tps.ar_reduce_norm([addr(0)], [addr(1)], lay, tps.make_norm(1e-5, host[0]), "f32", stream=0),
                 lambda: tps.ar_reduce_norm([addr(0)], [addr(1)], lay, norm, "f32", mean=host[:, 0], stream=0),
                 lambda: tps.ar_reduce_norm([addr(0)], [addr(1)], lay, norm, "f32", sums=[host], stream=0),
                 lambda: tps.ar_reduce_norm_grad(host, addr(0), [addr(1)], lay, norm, addr(2), addr(3), "f32", stream=0),
                 lambda: tps.ar_reduce_norm_grad(addr(0), addr(1), [addr(1)], lay, norm, addr(2), addr(3), "f32",
                                                 dweight=host[0], stream=0),
                 lambda: tps.ar_checkpoint_pack(host, codes(8, 2), stream=0),
                 lambda: tps.make_checkpoint(host.to(torch.uint8), host.to(torch.uint8), 8),
                 lambda: tps.ar_policy_loss(host[0], torch.zeros(2, dtype=torch.int64), host[1, :1], host[1, :4], stream=0)):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(KeyError):
        tps.make_norm(kind="batch")


def test_layout_of_the_structures(tmp_path):
    """Sizes and field offsets as a C compiler lays them out."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "more_offsets")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.join(os.path.dirname(here), "include"), "-o", exe,
                    os.path.join(here, "c", "more_offsets.c")], check=True)
    got = dict(line.split() for line in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for name, kind in (("ar_checkpoint", tps.ArCheckpoint), ("ar_norm", tps.ArNorm), ("ar_norm_kept", ar.ArNormKept),
                       ("ar_policy", tps.ArPolicy)):
        assert int(got.pop(name)) == ctypes.sizeof(kind)
        for field, _ in kind._fields_:
            assert int(got.pop(f"{name}.{field}")) == getattr(kind, field).offset
    assert not got
