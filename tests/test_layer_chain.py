"""CPU tests of the gated linear recurrence's chain of segments: a model of its
workgroups over the kernel's own rules (csrc/glr_chain.hpp), built with the host
compiler.  Waiting ends whatever the order in which workgroups start and run."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("chain") / "model.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC",
                    os.path.join(HERE, "glr_chain_model.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def ends(model, order, slots, polls, seed, begins=(), maps_only=False):
    n = len(order)
    return model.glr_chain_ends(n, (ctypes.c_int * n)(*order), slots, polls, int(maps_only),
                                (ctypes.c_int * len(begins))(*begins), len(begins), seed)


def orders(n, seed):
    """In order, from the end, shuffled, and with the segments that close blocks and groups last."""
    rng = random.Random(seed)
    mixed = list(range(n))
    rng.shuffle(mixed)
    return [list(range(n)), list(range(n - 1, -1, -1)), mixed,
            sorted(range(n), key=lambda j: (j % 64 == 63, j % 8 == 7)), sorted(range(n), key=lambda j: (j % 64 == 63, rng.random()))]


@pytest.mark.parametrize("nseg", [2, 8, 9, 64, 65, 150, 200])
@pytest.mark.parametrize("polls", [1, 3])
def test_waiting_ends(model, nseg, polls):
    for seed, order in enumerate(orders(nseg, nseg)):
        for slots in sorted({1, 5, min(70, nseg), nseg}):
            for begins in ([], [nseg // 3], [3, 70, 71]):
                begins = [b for b in begins if b < nseg]
                assert ends(model, order, slots, polls, seed, begins), (order[:4], slots, begins, seed)


def test_the_map_alone_does_not_tell(model):
    """The model finds the rule wanting that asks for the maps only: a block's state stays unpublished when its
    publisher gives up after the map and the block's own workgroup gets no slot."""
    order = sorted(range(150), key=lambda j: j % 64 == 63)
    assert not all(ends(model, order, 70, 1, seed, maps_only=True) for seed in range(40))
    assert all(ends(model, order, 70, 1, seed) for seed in range(40))


def test_reads_cover_what_enters(model):
    assert model.glr_chain_reads_cover(300) == 1
