"""GPU tests of the feed-forward block and the dropout at the ends of the sizes that their headers allow: weights of 2^32
elements, more than 2^32 rows.  Each needs some tens of GB of the card."""
import pytest
import torch

import test_gpu_dropout as dropout
from test_gpu_ffn import act64, half

pytestmark = pytest.mark.gpu
B = dropout.B


def test_ffn_widest(B):
    """D = F = 65536: offsets beyond 2^31 elements in every weight and gradient.  In 64 bits piece by piece; the 2-norms as in
    test_gpu_ffn.py (two roundings on the way to every output)."""
    T, W, piece = 5, 65536, 4096
    G = torch.Generator(device="cuda").manual_seed(5)

    def r(*s, scale=1.0):
        return torch.randn(s, generator=G, device="cuda", dtype=torch.bfloat16) * scale
    x, dy = r(T, W), r(T, W)
    wg, wu, wd = r(W, W, scale=1.5 / 256), r(W, W, scale=1.0 / 256), r(W, W, scale=1.0 / 256)
    f = B.gated_ffn_fwd(x, wg, wu, wd, want_saved=True)
    got = {"y": f["y"], **B.gated_ffn_bwd(x, wg, wu, wd, f["saved"], dy)}
    x64, dy64 = x.double(), dy.double()
    y, dx = torch.zeros_like(x64), torch.zeros_like(x64)
    limit = 2 * half("bf16")

    def check(name, v, ref):
        rel = float((v.double() - ref).norm() / ref.norm())
        assert rel <= limit, (name, rel, limit)
    for i in range(0, W, piece):
        c = slice(i, i + piece)
        g64, u64, d64 = wg[c].double(), wu[c].double(), wd[:, c].double()
        g, u, dh = x64 @ g64.T, x64 @ u64.T, dy64 @ d64
        a, s = act64(g, "silu")
        dg, du, h = dh * u * s, dh * a, a * u
        y += h @ d64.T
        dx += dg @ g64 + du @ u64
        check(f"dw_gate {i}", got["dw_gate"][c], dg.T @ x64)
        check(f"dw_up {i}", got["dw_up"][c], du.T @ x64)
        check(f"dw_down {i}", got["dw_down"][:, c], dy64.T @ h)
    check("y", got["y"], y)
    check("dx", got["dx"], dx)


def test_dropout_more_than_2_32_rows(B):
    """The generator's counter goes on in its second word."""
    rows, p, rng = (1 << 32) + 1000, 0.4, (1 << 45, 3)
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    B.dropout(x, p, rng, out=x)
    for first in (0, (1 << 32) - 500, rows - 1000):
        m, f = dropout.keep(1000, 1, p, *rng, first=first)
        y = x[first:first + 1000].cpu()
        assert torch.equal(y != 0, m) and float(y.max()) == float(torch.tensor(f).bfloat16())


def test_dropout_add_norm_more_than_2_32_rows(B):
    rows, p, rng = (1 << 32) + 1000, 0.4, (1 << 45, 3)
    G = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=G) for _ in range(2))
    w = torch.full((1,), 1.5, device="cuda")
    ends = [slice(0, 1000), slice((1 << 32) - 500, (1 << 32) + 500), slice(rows - 1000, rows)]
    old = [(x[s].cpu(), res[s].cpu()) for s in ends]
    B.dropout_add_norm_fwd(x, res, w, p, rng, eps=dropout.EPS, out={"y": x, "res": res})
    new = [res[s].cpu() for s in ends]
    for s, (a, b) in zip(ends, old):
        m, f = dropout.keep(1000, 1, p, *rng, first=s.start)
        ref, tol = dropout.norm_ref(a, b, w.cpu(), None, m, f, "bf16", "bf16")
        dropout.close("y", x[s], ref["y"], tol["y"])
        dropout.close("res", res[s], ref["res"], tol["res"])
    x.normal_(generator=G)   # dy, and dx in its place; the residual's gradient in the stored sum's
    dy = [x[s].cpu() for s in ends]
    out = {"dx": x, "dres": res, "dw": torch.empty_like(w)}
    B.dropout_add_norm_bwd(x, None, res, w, p, rng, eps=dropout.EPS, out=out)
    for s, d, r in zip(ends, dy, new):
        m, f = dropout.keep(1000, 1, p, *rng, first=s.start)
        ref, tol = dropout.norm_bwd_ref(d, None, r, w.cpu(), d, None, m, f, "bf16", "bf16")
        dropout.close("dres", res[s], ref["dres"], tol["dres"])
        dropout.close("dx", x[s], ref["dx"], tol["dx"])
