"""Host-side checks of the dropout calls, and the tests' own generator
against the published known answers (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tensor_partial_sum_gb300 import ar
from tests.philox import keep_mask, philox

OK, INVALID, UNSUPPORTED, TOO_LARGE, NOT_INIT, OVERLAP = range(6)
A = 1 << 20  # addresses far apart, never read


def addr(k):
    return A * (k + 1)


@pytest.mark.parametrize("counter,seed,words", [
    ([0, 0, 0, 0], 0, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, 2 ** 64 - 1, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], 0x299F31D0A4093822,
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_known_answers(counter, seed, words):
    assert philox(counter, seed).tolist() == words


def test_mask_keeps_the_stated_share():
    n = 1 << 20
    for p in (0.1, 0.5):
        kept = keep_mask(1024, n // 1024, p, seed=77, offset=3).mean()
        assert abs(kept - (1 - p)) < 6 * np.sqrt(p * (1 - p) / n)  # six standard deviations
    assert keep_mask(64, 4, 0.0, 1, 0).all() and not keep_mask(64, 4, 1.0, 1, 0).any()


def check(R=2, srcs=None, dsts=None, drop=None, ne0=64, ne1=4, max_elems=1 << 20, dst="f32", wire="bf16", **kw):
    layout = tps.make_layout(ne0, ne1, **kw)
    return tps.ar_check_dropout(R, srcs or [addr(0), addr(1)], dsts or [addr(2)], layout,
                                drop or tps.make_dropout(0.1, 1), max_elems, dst, wire)


def test_check_dropout_statuses():
    assert check() == OK
    assert check(drop=tps.make_dropout(0.0, 2 ** 64 - 1, 2 ** 64 - 1, bias=addr(3))) == OK
    assert check(drop=tps.make_dropout(1.0, 0)) == OK
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert check(drop=tps.make_dropout(p, 0)) == INVALID
    assert check(drop=tps.make_dropout(0.1, 0, bias=addr(3) + 2)) == INVALID      # off an f32 boundary
    assert check(drop=tps.make_dropout(0.1, 0, bias=addr(2) + 64 * 4)) == OVERLAP  # inside the destination
    assert check(drop=tps.make_dropout(0.1, 0, bias=addr(0))) == OK               # a source row may serve
    assert check(ne0=1, ne1=1 << 32, max_elems=1 << 40, dsts=[1 << 45]) == TOO_LARGE   # rows past a counter word
    assert check(max_elems=255) == TOO_LARGE
    assert check(dst="f32", wire=9) == UNSUPPORTED
    assert check(ne1=0) == OK
    assert check(dsts=[addr(0) + 4]) == OVERLAP
    lay = tps.make_layout(8, 1)
    L = ar.lib()
    assert L.ar_check_dropout(1, ar._ptrs([addr(0)]), ar._ptrs([addr(1)]), 1, ctypes.byref(lay), None, 8, 0, 0) == INVALID


def test_calls_need_a_context():
    lay, drop = tps.make_layout(8, 2), tps.make_dropout(0.1, 1)
    with pytest.raises(tps.ARError) as e:
        tps.ar_reduce_dropout([addr(0)], [addr(1)], lay, drop, "f32", stream=0)
    assert e.value.status == NOT_INIT
    with pytest.raises(tps.ARError) as e:
        tps.ar_reduce_dropout_grad(addr(0), [addr(1)], lay, drop, "f32", stream=0)
    assert e.value.status == NOT_INIT


def test_workspace_size():
    n = tps.ar_reduce_dropout_grad_workspace
    assert n(tps.make_layout(4096, 2048), 0) == 0
    one = n(tps.make_layout(4096, 2048), 1)
    assert 0 < one <= 128 * 4096 * 4 and n(tps.make_layout(4096, 2048), 2) == 2 * one
    assert n(tps.make_layout(4096, 0), 2) == 0
    for bad in (-1, 3):
        with pytest.raises(tps.ARError):
            n(tps.make_layout(8, 8), bad)


def test_binding_refuses_wrong_buffers():
    lay, drop = tps.make_layout(8, 2), tps.make_dropout(0.1, 1)
    host = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        tps.ar_reduce_dropout([host], [host.clone()], lay, drop, "f32", stream=0)
    with pytest.raises(TypeError):
        tps.ar_reduce_dropout_grad(host, [host.clone()], lay, drop, "f32", stream=0)
    with pytest.raises(TypeError):
        tps.ar_reduce_dropout_grad(addr(0), [addr(1)], lay, drop, "f32", dbias=torch.zeros(8), stream=0)
    with pytest.raises(TypeError):
        tps.ar_reduce_dropout([addr(0)], [addr(1)], lay, tps.make_dropout(0.1, 1, bias=torch.zeros(8)), "f32", stream=0)
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, 1 << 64)):
        with pytest.raises(ValueError):
            tps.make_dropout(0.1, seed, offset)
