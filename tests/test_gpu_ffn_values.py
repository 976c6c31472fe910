"""GPU tests of the gated feed-forward block (include/gdn_ffn.h) at values that ordinary
inputs do not have: NaN, infinities and gates far from zero."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("silu", "gelu", "sigmoid")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


def inputs(T, D, F, dtype, positive=False):
    G = torch.Generator().manual_seed(T + 7 * D + 31 * F)

    def r(*shape, scale=1.0):
        t = torch.randn(shape, generator=G) * scale
        return (t.abs() + 0.1 * scale if positive else t).to(DT[dtype]).cuda()
    return dict(x=r(T, D), wg=r(F, D, scale=1.5 / D ** 0.5), wu=r(F, D, scale=D ** -0.5), wd=r(D, F, scale=F ** -0.5),
                dy=r(T, D))


def run(B, d, act):
    f = B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], act=act, want_saved=True)
    return {"y": f["y"], **B.gated_ffn_bwd(d["x"], d["wg"], d["wu"], d["wd"], f["saved"], d["dy"], act=act)}


# dh's sums in one piece, in splits that are joined, and with padded rows
@pytest.mark.parametrize("T,D,F", [(70, 72, 136), (4, 4096, 64), (37, 21, 45)])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("act", ACTS)
def test_ffn_nan_gate(B, T, D, F, dtype, act):
    """One NaN in w_gate: every gate of its row is NaN, and with it all that the definition forms from them; the other
    rows of the weights' gradients keep their bits."""
    d = inputs(T, D, F, dtype)
    want = run(B, d, act)
    f = F // 3
    d["wg"][f, D // 2] = float("nan")
    got = run(B, d, act)
    for k in ("y", "dx"):
        assert torch.isnan(got[k]).all(), k
    rest = [i for i in range(F) if i != f]
    for k in ("dw_gate", "dw_up"):
        assert torch.isnan(got[k][f]).all(), k
        assert torch.equal(got[k][rest], want[k][rest]), k
    assert torch.isnan(got["dw_down"][:, f]).all() and torch.equal(got["dw_down"][:, rest], want["dw_down"][:, rest])
