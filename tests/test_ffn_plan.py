"""CPU tests of the feed-forward block's planner (csrc/ffn_plan.cpp), built with the host compiler."""
import ctypes
import os
import random
import subprocess

import pytest

from test_gpu_ffn_instances import SIZES

HERE = os.path.dirname(os.path.abspath(__file__))
CONFIG = ("big", "wide", "middle", "deep", "low", "small", "thin")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans(T, D, F, esize): for each product its name, tile, splits, steps of a split and steps in all."""
    so = str(tmp_path_factory.mktemp("plan") / "model.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC",
                    os.path.join(HERE, "ffn_plan_model.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    one, three = (ctypes.c_int * 5)(), (ctypes.c_int * 15)()

    def call(T, D, F, esize):
        piece, ke = 16 // esize, 128 // esize
        D, F = -(-D // piece) * piece, -(-F // piece) * piece
        out = []
        for kind, (name, N, K) in enumerate((("gate_up", F, D), ("down", D, F), ("dh", F, D))):
            lib.ffn_plan_one(kind, T, N, K, esize, one)
            out.append((name, CONFIG[one[0]], one[1], one[2], -(-K // ke)))
        lib.ffn_plan_grads(T, D, F, esize, three)
        for i, (name, K) in enumerate((("dx", 2 * F), ("dw_gate_up", T), ("dw_down", T))):
            cfg, splits, steps = three[5 * i:5 * i + 3]
            out.append((name, CONFIG[cfg], splits, steps, -(-K // ke)))
        return out
    return call


def sizes(seed, n):
    """Sizes over the whole range, their logarithms spread evenly, and widths that programs have."""
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(n):
        D, F = (rng.choice([log(1, 65536), log(1, 8192), rng.choice([64, 512, 1024, 2048, 4096, 5632, 8192, 12288])])
                for _ in range(2))
        yield log(1, min(1 << 24, ((1 << 36) - 1) // (D + 2 * F))), D, F


@pytest.mark.parametrize("esize", [2, 4])
def test_splits_cover_k(plans, esize):
    for s in sizes(esize, 5000):
        for name, _, splits, steps, every in plans(*s, esize):
            assert splits * steps >= every > (splits - 1) * steps, (s, name)


@pytest.mark.parametrize("esize", [2, 4])
def test_instances_are_tested(plans, esize):
    """Whatever the planner takes, whole or in splits, test_gpu_ffn_instances.py has a size that takes it."""
    def taken(s):
        return {(name, cfg, splits > 1) for name, cfg, splits, _, _ in plans(*s, esize)}
    tested = set().union(*(taken(s) for s in SIZES[esize]))
    for s in sizes(10 + esize, 30000):
        assert taken(s) <= tested, (s, taken(s) - tested)


@pytest.mark.parametrize("esize", [2, 4])
def test_sums_over_tokens_are_short(plans, esize):
    """A split of a weight's gradient adds up 4096 matrix instructions at most, of 32 products or (fp32) of 4."""
    long = [(1 << 24, D, F) for D, F in ((4, 4), (64, 64), (1024, 1024), (8, 2000), (4000, 8))]
    for s in [*sizes(20 + esize, 5000), *long]:
        for name, _, splits, steps, _ in plans(*s, esize):
            if name.startswith("dw"):
                assert steps * (128 // esize) <= (4096 * 32 if esize == 2 else 4096 * 4), (s, name, splits, steps)
