"""GPU tests of the dropout and of the residual add with RMSNorm and dropout (include/gdn_layer.h).

The mask is checked bit by bit against the generator in numpy, which its published test vectors pin.
Tolerances as for the add norm: u = 2^-24, an output in type t is rounded once (eps_t / 2), before that
every fp32 operation is off by at most u of its result, a row sum with its norm by NORM_OPS u; the mask's
factor adds one operation."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM_OPS = 64
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def rnd(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale)


def philox(ctr, key):
    """Philox 4x32-10 on uint64 arrays that hold 32 bits each."""
    m = np.uint64(0xFFFFFFFF)
    c, k = list(ctr), [np.uint64(v) for v in key]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & m, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + np.uint64(0x9E3779B9)) & m, (k[1] + np.uint64(0xBB67AE85)) & m]
    return c


def keep(rows, D, p, seed, offset, first=0):
    """The mask of rows first on, and the factor."""
    G = -(-D // 8)
    n = np.uint64(first) * np.uint64(G) + np.arange(rows * G, dtype=np.uint64)
    m, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    off = np.full_like(n, offset)
    w = philox([n & m, n >> s, off & m, off >> s], [seed & 0xFFFFFFFF, seed >> 32])
    bits = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1).reshape(rows, G * 8)[:, :D]
    t = int(np.floor(p * 65536 + 0.5))
    return torch.from_numpy(bits >= t), 65536 / (65536 - t) if t < 65536 else 0.0


def test_generator_vectors():
    """The published vectors of Philox 4x32-10."""
    for ctr, key, out in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = philox([np.array([v], dtype=np.uint64) for v in ctr], key)
        assert tuple(int(v[0]) for v in got) == out


def close(name, got, ref, tol):
    got = got.double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:3], ref[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 8), (2, 9), (1000, 16), (17, 100), (33, 129), (4, 4096), (3, 20001),
                                    (70000, 24)])
@pytest.mark.parametrize("dtype,p,rng", [("bf16", 0.1, (0, 0)), ("f16", 0.5, (0xDEADBEEFCAFEF00D, (1 << 63) + 12345)),
                                         ("f32", 0.3337, (1 << 40, 0xFFFFFFFF)), ("bf16", 0.999, (7, 1 << 32))])
def test_dropout(B, rows, D, dtype, p, rng):
    x = rnd(1, rows, D).to(DT[dtype])
    m, f = keep(rows, D, p, *rng)
    ref = torch.where(m, x.double() * f, 0.0)
    tol = (half(dtype) + 3 * U) * ref.abs() + TINY[dtype]   # the factor's rounding, the product's, the output's
    for off in (0, 1):
        d = torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")[off:].view(x.shape).copy_(x)
        y = B.dropout(d, p, rng)
        close("y", y, ref, tol)
        assert ((y == 0).cpu() | m).all() and torch.equal((y != 0).cpu(), m & (x != 0))
        assert torch.equal(B.dropout(d, p, torch.tensor([v - (1 << 64) if v >> 63 else v for v in rng], device="cuda")), y)
        assert B.dropout(d, p, rng, out=d) is d and torch.equal(d, y)


def test_dropout_ends(B):
    """p = 0 keeps every bit, p = 1 and infinities or NaN that are dropped give zero; shapes without elements."""
    x = rnd(1, 40, 50).cuda()
    assert torch.equal(B.dropout(x, 0.0, (1, 2)), x) and (B.dropout(x, 1.0, (1, 2)) == 0).all()
    x[::2], x[1::2] = float("inf"), float("nan")
    m, _ = keep(40, 50, 0.5, 1, 2)
    y = B.dropout(x, 0.5, (1, 2)).cpu()
    assert (y[~m] == 0).all() and not torch.isfinite(y[m]).any()
    for s in ((0, 5), (5, 0), (0,)):
        assert B.dropout(torch.empty(s, device="cuda"), 0.5, (1, 2)).shape == s
    assert B.dropout(torch.ones(7, device="cuda"), 0.0, (1, 2)).shape == (7,)


def test_dropout_mask_by_row_and_column(B):
    """A row's mask does not depend on how many rows come after it or on the type; D a multiple of 8: flat order."""
    x = torch.ones(300, 40, device="cuda")
    a = B.dropout(x, 0.4, (3, 4))
    assert torch.equal(B.dropout(x[:7].contiguous(), 0.4, (3, 4)), a[:7])
    assert torch.equal(B.dropout(x.bfloat16(), 0.4, (3, 4)) != 0, a != 0)
    assert torch.equal(B.dropout(x.view(75, 160), 0.4, (3, 4)).view(300, 40), a)
    assert not torch.equal(B.dropout(x, 0.4, (3, 5)), a) and not torch.equal(B.dropout(x, 0.4, (4, 4)), a)


def test_dropout_far_offsets(B):
    """Elements beyond 2^31 and groups beyond 2^32 bytes."""
    rows, D, p, rng = 70001, 32771, 0.25, (11, 22)
    x = torch.ones(rows, D, dtype=torch.bfloat16, device="cuda")
    y = B.dropout(x, p, rng, out=x)
    m, f = keep(3, D, p, *rng, first=rows - 3)
    assert torch.equal((y[-3:] != 0).cpu(), m)
    assert float(y[-1][y[-1] != 0][0]) == float(torch.tensor(f).bfloat16())


def norm_ref(x, res, w, scale, m, f, dtype, rdtype):
    x, res, w = x.double(), res.double(), w.double()
    s = 1.0 if scale is None else scale.double()
    b = torch.where(m, x * f, 0.0) * s
    h = res + b
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = h * r * w
    eh = 5 * U * (res.abs() + b.abs())
    # h's error moves y by its own share and, through r, by the row's
    ey = (eh * r + h.abs() * r * (eh.square().sum(-1, keepdim=True) / h.square().sum(-1, keepdim=True).clamp_min(1e-30)).sqrt()) * w.abs()
    return {"y": y, "res": h}, {"y": ey + (half(dtype) + NORM_OPS * U) * y.abs() + TINY[dtype],
                                "res": eh + half(rdtype) * h.abs() * (1 + U) + TINY[rdtype]}


def norm_bwd_ref(dy, dres, res, w, x, scale, m, f, dtype, rdtype):
    dy, res, w, x = dy.double(), res.double().cpu(), w.double(), x.double()
    dres = 0.0 if dres is None else dres.double()
    r = (res.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n, dn = res * r, dy * w
    mag = r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True)) + (dres.abs() if torch.is_tensor(dres) else 0.0)
    dh = dres + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    e = 2 * NORM_OPS * U * mag
    s = 1.0 if scale is None else scale.double()
    mf = m.double() * f
    ref = {"dres": dh, "dx": dh * mf * s, "dw": (dy * n).sum(0)}
    tol = {"dres": e + half(rdtype) * dh.abs() + TINY[rdtype], "dx": (e + 4 * U * mag) * mf * abs(s) + half(dtype) * ref["dx"].abs() + TINY[dtype],
           "dw": ((NORM_OPS + dy.shape[0]) * U * (dy * n).abs()).sum(0) + 1e-38}
    if scale is not None:
        ref["dscale"] = (dh * mf * x).sum(0)
        tol["dscale"] = ((e + (NORM_OPS + dy.shape[0]) * U * mag) * mf * x.abs()).sum(0) + 1e-38
    return ref, tol


@pytest.mark.parametrize("rows,D", [(1, 1), (5, 3), (700, 7), (50, 20), (17, 64), (64, 128), (7, 257), (130, 500), (5, 2048),
                                    (3, 4096), (2, 5001), (3, 8192), (9001, 40)])
@pytest.mark.parametrize("dtype,rdtype,scaled,p", [("bf16", "f32", True, 0.1), ("f16", "f16", True, 0.5),
                                                   ("f32", "f32", False, 0.3), ("bf16", "bf16", False, 0.9),
                                                   ("f16", "f32", False, 0.2), ("f32", "f32", True, 0.6)])
def test_dropout_add_norm(B, rows, D, dtype, rdtype, scaled, p):
    rng = (987654321987, 5 + rows)
    x, res = rnd(1, rows, D).to(DT[dtype]), rnd(2, rows, D, scale=2.0).to(DT[rdtype])
    w, scale = 1 + 0.1 * rnd(3, D), 0.5 + 0.2 * rnd(4, D) if scaled else None
    dy, dres = rnd(5, rows, D).to(DT[dtype]), rnd(6, rows, D).to(DT[rdtype])
    m, f = keep(rows, D, p, *rng)
    ref, tol = norm_ref(x, res, w, scale, m, f, dtype, rdtype)
    d = {k: None if t is None else t.cuda() for k, t in dict(x=x, res=res, w=w, scale=scale, dy=dy, dres=dres).items()}
    got = B.dropout_add_norm_fwd(d["x"], d["res"], d["w"], p, rng, scale=d["scale"], eps=EPS)
    for k in ref:
        close(k, got[k], ref[k], tol[k])
    for back in (d["dres"], None):
        g = B.dropout_add_norm_bwd(d["dy"], back, got["res"], d["w"], p, rng, x=d["x"] if scaled else None,
                                   scale=d["scale"], eps=EPS)
        bref, btol = norm_bwd_ref(dy, None if back is None else dres, got["res"], w, x, scale, m, f, dtype, rdtype)
        assert (g["dscale"] is None) == (not scaled) and g["dx"].data_ptr() != g["dres"].data_ptr()
        for k in bref:
            close(k, g[k], bref[k], btol[k])
        assert (g["dx"].cpu()[~m] == 0).all()


def test_dropout_add_norm_in_place_no_rows_spoilt(B):
    rows, D, p, rng = 901, 128, 0.3, (1, 9)
    x, res, w, s = rnd(1, rows, D).cuda(), rnd(2, rows, D).cuda(), 1 + 0.1 * rnd(3, D).cuda(), rnd(4, D).cuda()
    dy, dres = rnd(5, rows, D).cuda(), rnd(6, rows, D).cuda()
    f = B.dropout_add_norm_fwd(x, res, w, p, rng, scale=s)
    g = B.dropout_add_norm_bwd(dy, dres, f["res"], w, p, rng, x=x, scale=s)
    a, b = x.clone(), res.clone()
    i = B.dropout_add_norm_fwd(a, b, w, p, rng, scale=s, out={"y": a, "res": b})
    assert torch.equal(a, f["y"]) and torch.equal(b, f["res"])
    c, e = dy.clone(), dres.clone()
    i = B.dropout_add_norm_bwd(c, e, f["res"], w, p, rng, x=x, scale=s,
                               out={"dx": c, "dres": e, "dw": torch.empty_like(w), "dscale": torch.empty_like(s)})
    assert all(torch.equal(i[k], g[k]) for k in g)
    # p = 0: the add norm itself, bit by bit
    f0, a0 = B.dropout_add_norm_fwd(x, res, w, 0.0, rng, scale=s), B.add_norm_fwd(x, res, w, scale=s)
    assert all(torch.equal(f0[k], a0[k]) for k in a0)
    # dropped infinities and NaN leave no trace
    m, _ = keep(rows, D, p, *rng)
    bad = torch.where(m.cuda(), x, float("nan"))
    f2 = B.dropout_add_norm_fwd(bad, res, w, p, rng, scale=s)
    g2 = B.dropout_add_norm_bwd(dy, dres, f["res"], w, p, rng, x=bad, scale=s)
    assert all(torch.equal(f2[k], f[k]) for k in f) and all(torch.equal(g2[k], g[k]) for k in g)
    z = torch.empty(0, D, device="cuda")
    assert B.dropout_add_norm_fwd(z, z, w, p, rng)["y"].shape == z.shape
    n = {"dx": z.clone(), "dres": z.clone(), "dw": torch.ones_like(w), "dscale": torch.ones_like(s)}
    B.dropout_add_norm_bwd(z, z, z, w, p, rng, x=z, scale=s, out=n)
    assert (n["dw"] == 0).all() and (n["dscale"] == 0).all()


def test_dropout_autograd(B):
    """Gradients through autograd are the same mask's; the dropout may be differentiated again, the add norm not."""
    from chunked_gated_delta_08_amd import autograd as A
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    x = rnd(1, 30, 21).cuda().requires_grad_()
    y = A.dropout(x * x, 0.4, rng)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    mf = B.dropout(torch.ones_like(x), 0.4, (5, 6))
    assert torch.allclose(y, mf * x * x, rtol=1e-6) and torch.allclose(g, mf * 2 * x, rtol=1e-6)
    assert torch.allclose(torch.autograd.grad(g.sum(), x)[0], 2 * mf, rtol=1e-6)
    res, w = rnd(2, 30, 21).cuda().requires_grad_(), torch.ones(21, device="cuda", requires_grad=True)
    y, r = A.dropout_add_rms_norm(x, res, w, 0.4, (5, 6))
    d = rnd(3, 30, 21).cuda()
    got = torch.autograd.grad((y, r), (x, res, w), (d, d), create_graph=True)
    b = B.dropout_add_norm_bwd(d, d, r.detach(), w.detach(), 0.4, (5, 6))
    assert all(torch.equal(a.detach(), b[k]) for a, k in zip(got, ("dx", "dres", "dw")))
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(got[0].square().sum(), x)
    g, = torch.autograd.grad(A.dropout_add_rms_norm(x, res, w, 0.4, (5, 6))[0].sum(), x)   # the residual unused
    z = B.dropout_add_norm_bwd(torch.ones_like(d), None, r.detach(), w.detach(), 0.4, (5, 6))
    assert torch.equal(g, z["dx"])


def test_dropout_captured(B):
    """A graph reads the generator's numbers at each replay; another device stream, out given."""
    x = rnd(1, 64, 100).cuda()
    rng = torch.tensor([1, 0], dtype=torch.int64, device="cuda")
    y = torch.empty_like(x)
    B.dropout(x, 0.5, rng, out=y)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            B.dropout(x, 0.5, rng, out=y)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        rng[1] = 1000 + i
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, B.dropout(x, 0.5, (1, 1000 + i)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = B.dropout(x, 0.5, (1, 1003), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, y)
