"""Host-side checks of the vocabulary loss (CPU only)."""
import ctypes

import pytest
import torch

import tensor_partial_sum_gb300 as tps
from tensor_partial_sum_gb300 import ar

OK, INVALID, UNSUPPORTED, TOO_LARGE, NOT_INIT, OVERLAP = range(6)
A = 1 << 30  # addresses far apart, never read


def vocab(rows=16, dim=64, pieces=(100, 28), hidden=A, weights=None, targets=2 * A, hs=0, ws=None, dtype="bf16"):
    v = ar.ArVocab()
    n = len(pieces)
    v.rows, v.dim, v.hidden, v.hidden_row_bytes, v.n_pieces = rows, dim, hidden, hs, n
    v.piece_rows = (ctypes.c_size_t * n)(*pieces)
    v._p = ar._ptrs(weights if weights is not None else [(3 + r) * A for r in range(n)])
    v.weights = v._p
    if ws:
        v.weight_row_bytes = (ctypes.c_int64 * n)(*ws)
    v.targets, v.ignore_index = targets, -100
    v.dtype = tps.DTYPE_CODES.get(dtype, dtype)
    return v


def status(max_elems=1 << 20, **kw):
    return tps.ar_check_vocab(vocab(**kw), max_elems)


def test_check_vocab_statuses():
    assert status() == OK
    assert status(rows=0, hidden=0, targets=0) == OK
    assert status(pieces=(0, 5)) == OK and status(pieces=(5, 0), weights=[3 * A, 0]) == OK
    assert status(pieces=(0, 0)) == INVALID
    assert status(dim=0) == INVALID
    assert status(dtype=7) == UNSUPPORTED
    assert status(max_elems=16 * 64 - 1) == TOO_LARGE and status(max_elems=16 * 64) == OK
    assert status(pieces=(1 << 31,)) == TOO_LARGE
    assert status(hidden=A + 1) == INVALID and status(hidden=0) == INVALID
    assert status(targets=2 * A + 4) == INVALID
    assert status(hs=127) == INVALID and status(hs=126) == INVALID and status(hs=130) == OK and status(hs=-128) == INVALID
    assert status(ws=(128, 126)) == INVALID and status(ws=(256, 130)) == OK
    assert status(weights=[3 * A, 4 * A + 1]) == INVALID
    assert ar.lib().ar_check_vocab(None, 1) == INVALID
    v = vocab()
    for n in (0, 17):
        v.n_pieces = n
        assert tps.ar_check_vocab(v, 1 << 20) == INVALID


def test_workspace():
    for dtype in ("f32", "f16", "bf16"):
        for kw in ({}, {"dim": 63}, {"hs": 520}, {"pieces": (0, 1)}, {"rows": 1}):
            for grad in (False, True):
                assert tps.ar_vocab_workspace(vocab(dtype=dtype, **kw), grad) > 0
    assert tps.ar_vocab_workspace(vocab(rows=0), True) == 0
    with pytest.raises(tps.ARError):
        tps.ar_vocab_workspace(vocab(dim=0), False)
    # a large vocabulary's gradient does not take the logits' room
    big = vocab(rows=8192, dim=4096, pieces=(131072,), dtype="bf16")
    assert tps.ar_vocab_workspace(big, True) < 8192 * 131072 * 2 / 2


def test_calls_need_a_context():
    L, v = ar.lib(), vocab()
    assert L.ar_vocab_loss(ctypes.byref(v), 9 * A, 10 * A, 11 * A, 1 << 28, None) == NOT_INIT
    assert L.ar_vocab_loss_grad(ctypes.byref(v), 9 * A, 10 * A, None, None, None, None, 11 * A, 1 << 28, None) == NOT_INIT


def test_binding_refuses_host_tensors_and_wrong_shapes():
    h, w, y = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        tps.ar_vocab_loss(h, [w], y, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError):
        tps.make_vocab(h[0], [w], y)
    with pytest.raises(ValueError):
        tps.make_vocab(h, [], y)


def test_struct_layouts_match_the_header(tmp_path):
    """The ctypes mirrors have the header's sizes and offsets."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [("ar_dropout", ar.ArDropout, f) for f, _ in ar.ArDropout._fields_]
    fields += [("ar_vocab", ar.ArVocab, f) for f, _ in ar.ArVocab._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "ar.h"\nint main(void) {\n' + "".join(
        f'printf("%zu %zu\\n", sizeof({s}), offsetof({s}, {f}));\n' for s, _, f in fields) + "return 0; }\n")
    exe = tmp_path / "o"
    subprocess.run(["gcc", "-I" + os.path.join(root, "include"), "-o", str(exe), str(src)], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got == [(ctypes.sizeof(c), getattr(c, f).offset) for _, c, f in fields]
