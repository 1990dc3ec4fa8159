"""The plans of the norm and checkpoint calls: every column has a thread, what is launched fits, and which sizes are
taken element by element (CPU only)."""
import os
import random
import shutil
import subprocess

import pytest

from tensor_partial_sum_gb300 import build as B
from tests.test_gpu_norm_any import LONG

HERE = os.path.dirname(os.path.abspath(__file__))
ES = {"f32": 4, "f16": 2, "bf16": 2}
FIELDS = ("f_U f_bx f_cluster f_threads f_warp f_smem r_U r_bx r_cluster r_threads r_warp r_smem r_stages r_blocks "
          "c_U c_cluster c_threads c_smem c_stages c_blocks parts vectors per_row pack_blocks f_blocks").split()
MOST_SMEM = 224 * 1024  # next to 2 KB and a few words of a kernel's own: 227 KB are possible


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "norm_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", B.CSRC, os.path.join(HERE, "c", "norm_plan.cpp"),
                    "-o", exe], check=True)

    def run(calls):
        text = "".join(" ".join(str(int(x)) for x in c) + "\n" for c in calls)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True, timeout=300).stdout
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]
    return run


def call(ne0, ne1, dst, aligned, kept=True, dsum=True, narrow=True):
    """As ar_reduce_norm_grad plans it: with the kept sum as a tensor or as codes, and with or without dsum."""
    es = ES[dst]
    v = 2 if aligned else es // 2 + 1
    return (ne0, ne1, es, aligned, v + (v if kept else 1) + (v if dsum else 0), es + (es if kept else 1) + (es if dsum else 0), narrow)


@pytest.mark.parametrize("aligned", [False, True])
def test_sizes_that_are_taken_element_by_element(plans, aligned):
    """The lengths that the element-wise forms are tested with reach them, from any start."""
    for dst, ne0 in LONG:
        for ne1 in (2, 3):
            assert plans([call(ne0, ne1, dst, aligned)])[0]["f_U"] == 0, (dst, ne0)
    p = plans([call(131_080, 70, dst, aligned) for dst in ES])
    assert all(q["r_U"] == 0 and q["c_U"] == 0 for q in p)


@pytest.mark.parametrize("dst,aligned,most", [("f32", True, 458_752), ("f32", False, 458_752), ("bf16", True, 917_504),
                                              ("f16", False, 917_504)])
def test_longest_rows_of_the_forward_pass(plans, dst, aligned, most):
    at, behind = plans([call(most, 2, dst, aligned), call(most + 1, 2, dst, aligned)])
    assert at["f_U"] > 0 and behind["f_U"] == 0
    assert most < 1 << 24  # where a length is a float


def calls():
    rng = random.Random(11)

    def size(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    out = []
    for _ in range(4000):
        dst = rng.choice(list(ES))
        out.append((dst, call(size(1, 1_000_000), size(1, 100_000), dst, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)))
    return out


def test_every_column_has_a_thread_and_every_launch_fits(plans):
    some = calls()
    for (dst, c), p in zip(some, plans([c for _, c in some])):
        ne0, ne1, es, aligned = c[:4]
        cols = 32 // es if aligned else 8
        if p["f_U"]:
            assert p["f_cluster"] in (1, 2, 4, 8) and p["f_bx"] * p["f_U"] * cols * p["f_cluster"] >= ne0, c
            assert p["f_smem"] == p["f_threads"] * p["f_U"] * cols * es <= MOST_SMEM, c
            # a block of 32 columns with one scale lies in adjacent lanes of a warp
            assert p["f_bx"] * cols % 32 == 0, c
            # every block takes one turn of rows
            turn = p["f_threads"] // p["f_bx"] if p["f_warp"] else 1
            assert p["f_blocks"] % p["f_cluster"] == 0 and p["f_blocks"] // p["f_cluster"] * turn >= c[1], c
        if p["r_U"]:
            assert p["r_bx"] * p["r_U"] * cols * p["r_cluster"] >= ne0 and p["r_threads"] <= 512, c
            assert p["r_smem"] <= MOST_SMEM and 1 <= p["r_stages"] <= 4, c
            assert p["r_blocks"] % p["r_cluster"] == 0 and p["r_blocks"] > 0, c
        if p["c_U"]:
            assert p["c_threads"] * 16 * p["c_cluster"] >= ne0 and p["c_threads"] <= 512 and p["c_threads"] % 32 == 0, c
            assert p["c_smem"] <= MOST_SMEM and 2 <= p["c_stages"] <= 4, c
            assert p["c_blocks"] % p["c_cluster"] == 0 and p["c_blocks"] > 0, c
        assert p["parts"] >= 1


@pytest.mark.parametrize("dst", list(ES))
@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("ne0", [1, 33, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 1, 1 << 31, 1 << 33])
def test_checkpoints_of_one_row(plans, dst, aligned, ne0):
    """Column numbers of a flattened tensor fit 32 bits where vectors are used; their bytes need not."""
    p, = plans([call(ne0, 1, dst, aligned)])
    assert p["vectors"] == (ne0 < 1 << 31)
    cols = 32 // ES[dst] if aligned else 8
    if p["vectors"]:
        assert p["per_row"] * cols >= ne0 and (p["per_row"] - 1) * cols < 1 << 32 and p["per_row"] * cols % 32 == 0
        assert p["pack_blocks"] * 256 >= p["per_row"] and p["pack_blocks"] < 1 << 31


def test_checkpoints_of_far_rows(plans):
    assert plans([call(72, 2, "f32", True, narrow=False)])[0]["vectors"] == 0
