"""GPU tests of every instance of the feed-forward block's products that the planner dispatches: each product with each of its
tiles, whole and in splits, in each type, against the formulas in 64 bits.  test_ffn_plan.py holds these sizes to
that: a planner that takes up another instance has to be given a size here.  Widths and tokens end inside steps and
tiles wherever an instance allows."""
import pytest
import torch

from test_gpu_ffn import close, inputs, reference, run

pytestmark = pytest.mark.gpu

SIZES = {   # by the bytes of an element: T, D, F
    2: [(1, 1, 1), (33, 1, 3), (711, 1, 1365), (1629, 2056, 764), (722, 1445, 1), (1731, 1030, 1358), (4242, 3018, 512),
        (5274, 65, 4104), (5, 2914, 3411), (2699, 409, 5640), (72, 3674, 4104), (526, 332, 1000), (1189, 5880, 2056),
        (135, 2437, 1007), (1004, 2056, 5928), (465, 2698, 1030), (390, 5640, 5640), (1036, 5826, 1000)],
    4: [(1, 1, 1), (33, 1, 3), (394, 870, 708), (989, 1030, 136), (1, 329, 322), (973, 1, 1030), (330, 2728, 1443),
        (2975, 1030, 1030), (464, 870, 2095)]}
ACTS = ("silu", "gelu", "sigmoid")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


@pytest.mark.parametrize("dtype,T,D,F", [(t, *s) for t in ("bf16", "f16") for s in SIZES[2]] + [("f32", *s) for s in SIZES[4]])
def test_ffn_instance(B, dtype, T, D, F):
    act = ACTS[(T + D + F) % 3]
    d = {n: t.cuda() for n, t in inputs(T, D, F, dtype).items()}
    ref, tol, norm = reference(**d, act=act, dtype=dtype)
    got = run(B, d, act)
    for k, v in got.items():
        close(k, v, ref[k], tol[k], norm)
    # without what the backward needs the forward is another epilogue; and equal inputs give equal bits
    assert torch.equal(B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], act=act)["y"], got["y"])
    again = run(B, d, act)
    assert all(torch.equal(got[k], again[k]) for k in got)
