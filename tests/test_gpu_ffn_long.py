"""GPU test of the feed-forward block's gradients over many tokens (include/gdn_ffn.h: up to 2^24)."""
import pytest
import torch

from test_gpu_ffn import close, inputs, reference, run

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


def test_ffn_weight_gradients_of_equal_tokens(B):
    """2^24 tokens that are all the same, fp32: each weight's gradient is 2^24 times a token's, and every step of a chain of sums
    rounds the same way for as long as the sum's exponent stays.

    A chain is 2^14 products long at most, of which each may be off by 2 u of the sum so far, and the 2^10 chains are
    joined one after another; what a token adds is off by some 40 roundings of the block itself (sums of 4 products, the activation
    and its slope, as derived in test_gpu_ffn.py: (|g| + 32) 1.5 u of terms, here below 100 u of the value)."""
    T, D, F = 1 << 24, 4, 4
    x1 = torch.tensor([1.1, 0.7, 1.3, 0.9])
    dy1 = torch.tensor([0.6, 1.7, 0.8, 1.2])
    wg, wu, wd = (torch.linspace(a, b, 16).view(4, 4) for a, b in ((0.2, 0.5), (0.3, 0.9), (0.4, 1.1)))
    x, dy = (t.cuda().expand(T, D).contiguous() for t in (x1, dy1))
    f = B.gated_ffn_fwd(x, wg.cuda(), wu.cuda(), wd.cuda(), want_saved=True)
    got = B.gated_ffn_bwd(x, wg.cuda(), wu.cuda(), wd.cuda(), f["saved"], dy)
    x1, dy1, wg, wu, wd = (t.double() for t in (x1, dy1, wg, wu, wd))
    g, u = wg @ x1, wu @ x1
    s = torch.sigmoid(g)
    h, dh = g * s * u, wd.T @ dy1
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    limit = 2 * (2 ** 14 + 2 ** 10 + 100) * U
    worst = {}
    for k, ref in (("dw_gate", torch.outer(dg, x1)), ("dw_up", torch.outer(du, x1)), ("dw_down", torch.outer(dy1, h))):
        worst[k] = float((got[k].double().cpu() / (T * ref) - 1).abs().max())
    assert all(v <= limit for v in worst.values()), (worst, limit)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_ffn_many_splits(B, dtype):
    """Sums over the tokens in many splits, the last one short, operands above zero: every element against 64 bits.  (dy is small
    so that fp16 holds the sums.)"""
    T, D, F = 200001, 40, 72
    d = {n: t.cuda() for n, t in inputs(T, D, F, dtype).items()}
    d = {n: t.abs() * (2.0 ** -10 if n == "dy" else 1) for n, t in d.items()}
    ref, tol, norm = reference(**d, act="silu", dtype=dtype)
    got = run(B, d, "silu")
    for k, v in got.items():
        close(k, v, ref[k], tol[k], norm if dtype != "f16" else None)   # dg and du reach fp16's smallest values
    again = run(B, d, "silu")
    assert all(torch.equal(got[k], again[k]) for k in got)
