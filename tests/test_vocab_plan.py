"""The plan of the vocabulary calls: what the launches write has room in the
workspace, however the vocabulary is cut (CPU only)."""
import os
import random
import shutil
import subprocess

import pytest

import tensor_partial_sum_gb300 as tps
from tensor_partial_sum_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
FIELDS = ("stats", "stats_room", "packed", "packed_room", "grad_packed", "grad_packed_room", "d", "d_room", "groups", "whole")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "vocab_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-isystem", os.path.join(CUDA, "include"),
                    "-I", B.INCLUDE, "-I", B.CSRC, os.path.join(HERE, "c", "vocab_plan.cpp"), "-o", exe], check=True)

    def run(calls):
        text = "".join(f"{T} {D} {tps.DTYPE_CODES[t]} {stride} {len(p)} {' '.join(map(str, p))}\n" for T, D, t, stride, p in calls)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True, timeout=300).stdout
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]
    return run


def fits(call, p):
    assert p["whole"] == 1, call
    assert p["stats"] <= p["stats_room"], f"{call}: statistics of {p['stats']} bytes in an area of {p['stats_room']}"
    assert p["packed"] <= p["packed_room"] and p["grad_packed"] <= p["grad_packed_room"], call
    assert p["d"] <= p["d_room"], call


CUT = [  # packed rows of more than 2 GiB: the loss takes several launches
    (512, 4096, "f32", 0, [128256]), (512, 4096, "f32", 0, [152064]), (512, 6144, "f32", 0, [131072]),
    (512, 8192, "f32", 0, [64128, 64128]), (1024, 4096, "f32", 0, [152064]), (512, 8192, "f32", 0, [131072]),
    (65, 8192, "f32", 0, [65536]), (200, 8192, "f32", 0, [65536]), (300, 8192, "bf16", 16386, [140000]),
    (3, 8192, "f32", 0, [131072]), (64, 4096, "f32", 0, [200000, 17]),
]


@pytest.mark.parametrize("call", CUT)
def test_statistics_of_a_cut_vocabulary_have_room(plans, call):
    p, = plans([call])
    assert p["groups"] > 1
    fits(call, p)


def test_any_sizes_have_room(plans):
    rng = random.Random(7)

    def size(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    calls = []
    for _ in range(3000):
        D = size(1, 1 << 15)
        dtype = rng.choice(["f32", "f32", "f16", "bf16"])
        stride = 0 if dtype == "f32" or rng.random() < 0.4 else D * 2 + rng.choice([2, 6, 16])
        pieces = [rng.choice([0, size(1, 400000), size(1, 400000)]) for _ in range(rng.randint(1, 16))]
        if sum(pieces):
            calls.append((size(1, 20000), D, dtype, stride, pieces))
    got = plans(calls)
    assert len(got) == len(calls) and sum(p["groups"] > 1 for p in got) > 300
    for call, p in zip(calls, got):
        fits(call, p)
