"""GPU tests of the layer operators (include/gdn_layer.h) against plain fp64
references on the CPU.

Tolerances.  u = 2^-24 is half a step of fp32.  An output in type t is rounded
once, at most eps_t/2 of its value off.  Before that every fp32 operation is off
by at most u of its result, a sum of m terms by at most (m - 1) u of the sum of
their magnitudes in any order, exp / rsqrt / rcp by 2 u, the sigmoid by
(|z| + 4) u.  Each test adds these up over the formula's terms; NORM_OPS is the
count for a row sum as the kernels form it (at most 32 terms in a lane and 9
joining steps, next to some ten single operations, so 64 is above it).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM_OPS = 64
GATE0 = 2.0 ** -126
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}   # half the smallest step of the type


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def f64(t):
    return None if t is None else t.double().cpu()


def close(name, got, ref, tol):
    """|got - ref| <= tol elementwise, NaN and infinities in the same places."""
    got = got.double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), name
    assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)]), name
    bad = ((got - ref).abs() > tol) & fin
    if bad.any():
        i = int(((got - ref).abs() / tol.clamp_min(1e-300))[fin].argmax())
        g, r, t = got[fin][i], ref[fin][i], tol[fin][i]
        raise AssertionError(f"{name}: {int(bad.sum())} of {got.numel()} off, worst {g} vs {r}, allowed {t}")


def rnd(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale)


def misaligned(t):
    """The same values on the GPU, one element past an aligned address."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    return b.copy_(t)


# ------------------------------------------------------------------ norms

def gate64(z, act):
    if z is None:
        return 1.0, None
    s = torch.sigmoid(z)
    return (z * s, s * (1 + z * (1 - s))) if act == "silu" else (s, s * (1 - s))


def gated_ref(x, z, w, dy, act, dtype):
    """y, dx, dz, dw and how far each may be off."""
    x, z, w, dy = f64(x), f64(z), f64(w), f64(dy)
    D = x.shape[-1]
    f, df = gate64(z, act)
    zz = 0.0 if z is None else z.abs()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    y = n * w * f
    ops = (NORM_OPS + zz) * U
    ref = {"y": y}
    tol = {"y": half(dtype) * y.abs() + ops * y.abs() + TINY[dtype]}
    if dy is not None:
        dn = dy * w * f
        zm = zz.amax(-1, keepdim=True) if z is not None else 0.0
        opm = (2 * NORM_OPS + zm) * U
        mean = (dn * n).mean(-1, keepdim=True)
        mag = r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))
        ref["dx"] = r * (dn - n * mean)
        tol["dx"] = half(dtype) * ref["dx"].abs() + opm * mag + TINY[dtype]
        if z is not None:
            ref["dz"] = dy * n * w * df
            # act' = s (1 + z (1 - s)): its terms reach (1 + |z|) while it may vanish
            magz = (dy * n * w).abs() * (1 + zz) * torch.sigmoid(z)
            tol["dz"] = half(dtype) * ref["dz"].abs() + 2 * ops * magz + TINY[dtype]
        t = dy * n * f
        ref["dw"] = t.sum(0)
        tol["dw"] = ((NORM_OPS + x.shape[0]) * U * t.abs() + zz * U * t.abs()).sum(0) + 1e-38
    return ref, tol


NORM_SHAPES = [(1, 1), (5, 3), (700, 7), (300, 8), (77, 16), (50, 20), (17, 64), (33, 100), (64, 128), (7, 257), (9, 512), (130, 500), (3, 1000), (5, 2048),
               (4, 2500), (3, 4096), (2, 5001), (3, 8192)]


@pytest.mark.parametrize("rows,D", NORM_SHAPES)
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "sigmoid"), ("f32", "silu"), ("bf16", None)])
def test_gated_norm(B, rows, D, dtype, act):
    x = (rnd(1, rows, D) * torch.exp(rnd(2, rows, 1))).to(DT[dtype])
    z = None if act is None else rnd(3, rows, D, scale=3.0).to(DT[dtype])
    w, dy = 1 + 0.1 * rnd(4, D), rnd(5, rows, D).to(DT[dtype])
    ref, tol = gated_ref(x, z, w, dy, act, dtype)
    for put in (lambda t: t.cuda(), misaligned):
        d = [None if t is None else put(t) for t in (x, z, w, dy)]
        y = B.gated_norm_fwd(d[0], d[1], d[2], eps=EPS, act=act or "silu")
        g = B.gated_norm_bwd(*d, eps=EPS, act=act or "silu")
        assert y.dtype == DT[dtype] and (g["dz"] is None) == (z is None)
        for k, v in {"y": y, **g}.items():
            if v is not None:
                close(k, v, ref[k], tol[k])


def test_gated_norm_extremes(B):
    """Zero rows, gates that saturate, a row with a NaN and one with an infinity: the others are not touched."""
    x, z, w, dy = rnd(1, 9, 128), rnd(2, 9, 128), torch.ones(128), rnd(3, 9, 128)
    x[1] = 0.0
    z[2], z[3] = 150.0, -60.0
    x[4], x[5] = 1e-18, 1e17
    x[6, 7], x[7, 9] = float("nan"), float("inf")
    ref, tol = gated_ref(x, z, w, dy, "silu", "f32")
    d = [t.cuda() for t in (x, z, w, dy)]
    y = B.gated_norm_fwd(*d[:3], eps=EPS)
    g = B.gated_norm_bwd(*d, eps=EPS)
    ok = [0, 1, 2, 3, 4, 5, 8]
    for k, v in (("y", y), ("dx", g["dx"]), ("dz", g["dz"])):
        close(k, v[ok], ref[k][ok], tol[k][ok])
    assert torch.isnan(y[6].cpu()).all() and torch.isnan(g["dx"][6].cpu()).all()
    # an infinite element: r = 0, so the row's finite elements give zero and the infinite one NaN
    yy = y[7].cpu()
    assert torch.isnan(yy[9]) and (yy[torch.arange(128) != 9] == 0).all()


def test_gated_norm_many_rows(B):
    """More rows than the backward's workgroups hold at once, and a row count that fills none evenly."""
    for rows, D in ((70001, 16), (20011, 128)):
        x, z, w, dy = (t.cuda() for t in (rnd(1, rows, D), rnd(2, rows, D), 1 + 0.1 * rnd(3, D), rnd(4, rows, D)))
        ref, tol = gated_ref(x, z, w, dy, "silu", "f32")
        g = B.gated_norm_bwd(x, z, w, dy, eps=EPS)
        close("y", B.gated_norm_fwd(x, z, w, eps=EPS), ref["y"], tol["y"])
        for k in ("dx", "dz", "dw"):
            close(k, g[k], ref[k], tol[k])
        again = B.gated_norm_bwd(x, z, w, dy, eps=EPS)
        assert all(torch.equal(again[k], g[k]) for k in g)


def test_gated_norm_in_place_and_no_rows(B):
    x, z, w, dy = rnd(1, 65, 128).bfloat16().cuda(), rnd(2, 65, 128).bfloat16().cuda(), torch.ones(128).cuda(), \
        rnd(3, 65, 128).bfloat16().cuda()
    want, grads = B.gated_norm_fwd(x, z, w), B.gated_norm_bwd(x, z, w, dy)
    for i in (0, 1):
        a = [x.clone(), z.clone()]
        assert torch.equal(B.gated_norm_fwd(*a, w, out=a[i]), want)
    a, b, c = x.clone(), z.clone(), dy.clone()
    g = B.gated_norm_bwd(a, b, w, c, out={"dx": c, "dz": b, "dw": torch.empty_like(w)})
    assert all(torch.equal(g[k], grads[k]) for k in g)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert B.gated_norm_fwd(e, e, w).shape == e.shape
    dw = torch.full((128,), 7.0, device="cuda")
    B.gated_norm_bwd(e, e, w, e, out={"dx": e.clone(), "dz": e.clone(), "dw": dw})
    assert (dw == 0).all()
    with pytest.raises(B.GdrError):   # shifted by one row: neither apart nor the same buffer
        big = torch.zeros(66, 128, dtype=torch.bfloat16, device="cuda")
        B.gated_norm_fwd(big[:65], None, w, out=big[1:])


def add_ref(x, res, w, scale, dtype, rdtype):
    x, res, w = f64(x), f64(res), f64(w)
    s = torch.ones_like(w) if scale is None else f64(scale)
    h = res + s * x
    hm = res.abs() + (s * x).abs()
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = h * r * w
    # h is off by 2 u of its terms; so, through r, by the mean of those errors relative to the row's size
    dh = 2 * U * hm
    dr = (h.abs() * dh).mean(-1, keepdim=True) * r * r
    return ({"res": h, "y": y},
            {"res": half(rdtype) * h.abs() + dh + TINY[rdtype],
             "y": half(dtype) * y.abs() + NORM_OPS * U * y.abs() + (dh * r + h.abs() * r * dr) * w.abs() + TINY[dtype]})


def add_bwd_ref(dy, dres, h, w, x, scale, dtype, rdtype):
    dy, dres, h, w, x, scale = (f64(t) for t in (dy, dres, h, w, x, scale))
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n, dn = h * r, dy * w
    back = torch.zeros_like(h) if dres is None else dres
    dh = back + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    err = 2 * NORM_OPS * U * (back.abs() + r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True)))
    s = torch.ones_like(w) if scale is None else scale
    many = (NORM_OPS + h.shape[0]) * U
    ref = {"dres": dh, "dx": s * dh, "dw": (dy * n).sum(0)}
    tol = {"dres": half(rdtype) * dh.abs() + err + TINY[rdtype],
           "dx": (half(dtype) + U) * (s * dh).abs() + s.abs() * err + TINY[dtype],
           "dw": (many * (dy * n).abs()).sum(0) + 1e-38}
    if scale is not None:
        ref["dscale"] = (dh * x).sum(0)
        tol["dscale"] = (many * (dh * x).abs() + err * x.abs()).sum(0) + 1e-38
    return ref, tol


@pytest.mark.parametrize("rows,D", NORM_SHAPES)
@pytest.mark.parametrize("dtype,rdtype,scaled", [("bf16", "f32", True), ("f16", "f16", True), ("f32", "f32", False),
                                                 ("bf16", "bf16", False), ("f16", "f32", False)])
def test_add_norm(B, rows, D, dtype, rdtype, scaled):
    x, res = rnd(1, rows, D).to(DT[dtype]), rnd(2, rows, D, scale=2.0).to(DT[rdtype])
    w, scale = 1 + 0.1 * rnd(3, D), 0.5 + 0.2 * rnd(4, D) if scaled else None
    dy, dres = rnd(5, rows, D).to(DT[dtype]), rnd(6, rows, D).to(DT[rdtype])
    ref, tol = add_ref(x, res, w, scale, dtype, rdtype)
    for put in (lambda t: t.cuda(), misaligned):
        d = {k: None if t is None else put(t) for k, t in dict(x=x, res=res, w=w, scale=scale, dy=dy, dres=dres).items()}
        f = B.add_norm_fwd(d["x"], d["res"], d["w"], scale=d["scale"], eps=EPS)
        for k in ("y", "res"):
            close(k, f[k], ref[k], tol[k])
        for back in (d["dres"], None):
            g = B.add_norm_bwd(d["dy"], back, f["res"], d["w"], x=d["x"] if scaled else None, scale=d["scale"], eps=EPS)
            bref, btol = add_bwd_ref(dy, None if back is None else dres, f["res"], w, x, scale, dtype, rdtype)
            assert (g["dscale"] is None) == (not scaled)
            assert (g["dx"] is g["dres"]) == (not scaled and dtype == rdtype)
            for k in bref:
                close(k, g[k], bref[k], btol[k])


def test_add_norm_many_rows_in_place_no_rows(B):
    rows, D = 9001, 128
    x, res, w, s = rnd(1, rows, D).cuda(), rnd(2, rows, D).cuda(), 1 + 0.1 * rnd(3, D).cuda(), rnd(4, D).cuda()
    dy, dres = rnd(5, rows, D).cuda(), rnd(6, rows, D).cuda()
    f = B.add_norm_fwd(x, res, w, scale=s, eps=EPS)
    g = B.add_norm_bwd(dy, dres, f["res"], w, x=x, scale=s, eps=EPS)
    ref, tol = add_bwd_ref(dy, dres, f["res"], w, x, s, "f32", "f32")
    for k in ref:
        close(k, g[k], ref[k], tol[k])
    a, b = x.clone(), res.clone()
    i = B.add_norm_fwd(a, b, w, scale=s, eps=EPS, out={"y": a, "res": b})
    assert torch.equal(i["y"], f["y"]) and torch.equal(b, f["res"])
    c, e = dy.clone(), dres.clone()
    i = B.add_norm_bwd(c, e, f["res"], w, x=x, scale=s, eps=EPS,
                       out={"dx": c, "dres": e, "dw": torch.empty_like(w), "dscale": torch.empty_like(s)})
    assert all(torch.equal(i[k], g[k]) for k in g)
    z = torch.empty(0, D, device="cuda")
    assert B.add_norm_fwd(z, z, w)["y"].shape == z.shape
    n = {"dx": z.clone(), "dres": z.clone(), "dw": torch.ones_like(w), "dscale": torch.ones_like(s)}
    B.add_norm_bwd(z, z, z, w, x=z, scale=s, out=n)
    assert (n["dw"] == 0).all() and (n["dscale"] == 0).all()


# ------------------------------------------------------- linear recurrence

def glr_ref(x, g, h0, lens, dh=None, dht=None):
    """The recurrence token by token, next to a bound on each value's error.

    Every token adds at most (8 + |g|) u of |a| H + |x|, H the recurrence of the
    magnitudes: |g| + 3 for the gate, 1 each for the product and the sum, the rest for the
    products and sums of the same factors that joining pieces of a sequence takes."""
    x, g, h0, dh, dht = (f64(t) for t in (x, g, h0, dh, dht))
    a = g.exp()
    gm = torch.where(torch.isfinite(g), g.abs(), 0.0)   # an infinite gate is exactly zero
    n, D = len(lens), x.shape[1]
    out = {k: torch.zeros_like(x) for k in ("h", "hp", "H", "Hp", "E", "Ep", "lam", "La", "Le")}
    ht, hte = torch.zeros(n, D, dtype=torch.float64), torch.zeros(n, D, dtype=torch.float64)
    t = 0
    for i, m in enumerate(lens):
        h = torch.zeros(D, dtype=torch.float64) if h0 is None else h0[i].clone()
        H, E = h.abs(), torch.zeros_like(h)
        for t in range(t, t + m):
            out["hp"][t], out["Hp"][t], out["Ep"][t] = h, H, E
            h = a[t] * h + x[t]
            E = a[t] * E + GATE0 * H
            H = a[t] * H + x[t].abs()
            E = E + (8 + gm[t]) * U * H
            out["h"][t], out["H"][t], out["E"][t] = h, H, E
        t = sum(lens[:i + 1])
        ht[i], hte[i] = h, E
    ref = {"h": out["h"], "ht": ht}
    err = {"h": out["E"], "ht": hte + 1e-38}
    if dh is not None:
        dh0, dh0e = torch.zeros_like(ht), torch.zeros_like(ht)
        for i, m in reversed(list(enumerate(lens))):
            mu = torch.zeros(D, dtype=torch.float64) if dht is None else dht[i].clone()
            M, E = mu.abs(), torch.zeros_like(mu)
            e = sum(lens[:i + 1])
            for t in range(e - 1, e - 1 - m, -1):
                lam, LA = dh[t] + mu, dh[t].abs() + M
                le = E + 8 * U * LA
                out["lam"][t], out["La"][t], out["Le"][t] = lam, LA, le
                mu, M, E = a[t] * lam, a[t] * LA, a[t] * le + ((5 + gm[t]) * U * a[t] + GATE0) * LA
            dh0[i], dh0e[i] = mu, E
        ref.update(dx=out["lam"], dg=out["lam"] * a * out["hp"], dh0=dh0)
        err.update(dx=out["Le"], dh0=dh0e + 1e-38,
                   dg=a * (out["La"] * out["Ep"] + out["Hp"] * out["Le"] + (8 + gm) * U * out["La"] * out["Hp"]) +
                   GATE0 * out["La"] * out["Hp"] + 1e-38)
    return ref, err


GLR_LENS = [[1], [4500], [33, 2500, 1, 4100], [2], [15], [16], [17], [63, 1], [127], [128], [129], [300], [1025], [5, 0, 1, 16, 33, 0, 200],
            [0, 0, 40, 0], [1] * 37, [64] * 3, [100] * 5, [0], [0, 0]]


@pytest.mark.parametrize("lens", GLR_LENS, ids=lambda v: "-".join(map(str, v[:8])))
@pytest.mark.parametrize("D,dtype,given", [(1, "f32", True), (3, "bf16", False), (64, "f32", False), (70, "f16", True),
                                           (257, "bf16", True), (515, "f32", True), (256, "bf16", False)])
def test_glr(B, lens, D, dtype, given):
    T, N = sum(lens), len(lens)
    x, dh = rnd(1, T, D).to(DT[dtype]), rnd(2, T, D).to(DT[dtype])
    g = -torch.exp(2 * rnd(3, T, D) - 3)
    g[rnd(4, T, D) > 2.5] = float("-inf")       # a gate that drops the state
    g[:, :1] = torch.where(rnd(5, T, 1) > 0.5, 0.0, g[:, :1])
    h0, dht = (rnd(6, N, D), rnd(7, N, D)) if given else (None, None)
    ref, err = glr_ref(x, g, h0, lens, dh, dht)
    kw = dict(B=N)
    if len(set(lens)) > 1:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    for put in (lambda t: t.cuda(), misaligned):
        d = {k: None if t is None else put(t) for k, t in dict(x=x, g=g, h0=h0, dh=dh, dht=dht).items()}
        f = B.glr_fwd(d["x"], d["g"], h0=d["h0"], want_states=True, **kw)
        b = B.glr_bwd(d["x"], d["g"], d["dh"], f["states"], dht=d["dht"], h0=d["h0"], **kw)
        for k, v in {"h": f["h"], "ht": f["ht"], **b}.items():
            t = dtype if k in ("h", "dx") else "f32"
            close(k, v, ref[k], err[k] + half(t) * ref[k].abs() + TINY[t])


def test_glr_long(B):
    """A long sequence among short ones, slow gates: the state crosses many tiles and segments."""
    lens, D = [3, 9000, 70], 64
    T = sum(lens)
    x, g, dh = rnd(1, T, D), -torch.exp(rnd(2, T, D) - 7), rnd(3, T, D)
    h0, dht = rnd(4, 3, D), rnd(5, 3, D)
    ref, err = glr_ref(x, g, h0, lens, dh, dht)
    cu = torch.tensor([0, 3, 9003, 9073], dtype=torch.int32)
    kw = dict(h0=h0.cuda(), cu_seqlens=cu.cuda())      # no host mirror: it is copied
    f = B.glr_fwd(x.cuda(), g.cuda(), want_states=True, **kw)
    b = B.glr_bwd(x.cuda(), g.cuda(), dh.cuda(), f["states"], dht=dht.cuda(), **kw)
    for k, v in {"h": f["h"], "ht": f["ht"], **b}.items():
        close(k, v, ref[k], err[k] + U * ref[k].abs())
    f2 = B.glr_fwd(x.cuda(), g.cuda(), want_states=True, **kw)
    b2 = B.glr_bwd(x.cuda(), g.cuda(), dh.cuda(), f2["states"], dht=dht.cuda(), **kw)
    assert all(torch.equal(f[k], f2[k]) for k in f) and all(torch.equal(b[k], b2[k]) for k in b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_glr_gates_above_one(B, dtype):
    """Log-gates of both signs whose sum over a sequence reaches some 45: products of gates grow to e^45."""
    lens, D = [9000], 70
    x, dh = rnd(1, 9000, D).to(DT[dtype]), rnd(2, 9000, D).to(DT[dtype])
    g = 0.005 + 0.05 * rnd(3, 9000, D)
    ref, err = glr_ref(x, g, None, lens, dh)
    f = B.glr_fwd(x.cuda(), g.cuda(), want_states=True)
    b = B.glr_bwd(x.cuda(), g.cuda(), dh.cuda(), f["states"])
    for k, v in {"h": f["h"], "ht": f["ht"], **b}.items():
        t = dtype if k in ("h", "dx") else "f32"
        close(k, v, ref[k], err[k] + half(t) * ref[k].abs() + TINY[t])


@pytest.mark.parametrize("lens,D", [([3000], 130), ([700, 1, 0, 1500, 40], 64), ([9000], 2)])
def test_glr_without_patience(B, lens, D):
    """Workgroups that hardly look for the others' results before they compute them themselves give the same bits."""
    T, N = sum(lens), len(lens)
    x, g, dh, h0, dht = (t.cuda() for t in (rnd(1, T, D).bfloat16(), -torch.exp(rnd(2, T, D) - 4), rnd(3, T, D).bfloat16(),
                                            rnd(4, N, D), rnd(5, N, D)))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    kw = dict(h0=h0, cu_seqlens=cu.cuda(), cu_seqlens_host=cu)

    def both(polls):
        f = B.glr_fwd(x, g, want_states=True, polls=polls, **kw)
        return {**f, **B.glr_bwd(x, g, dh, f["states"], dht=dht, polls=polls, **kw)}
    want = both(0)
    for polls in (1, 2, 20):
        got = both(polls)
        assert all(torch.equal(got[k], want[k]) for k in want), polls


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_glr_neighbours_are_not_touched(B, bad):
    """A sequence that is not finite leaves the others as they are, wherever the borders fall."""
    lens, D = [300, 20, 7, 1000], 130
    T = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    x, g, dh, h0, dht = (t.cuda() for t in (rnd(1, T, D), -torch.exp(rnd(2, T, D) - 4), rnd(3, T, D), rnd(4, 4, D),
                                            rnd(5, 4, D)))
    kw = dict(h0=h0, cu_seqlens=cu.cuda(), cu_seqlens_host=cu)

    def both():
        f = B.glr_fwd(x, g, want_states=True, **kw)
        return {**f, **B.glr_bwd(x, g, dh, f["states"], dht=dht, **kw)}
    clean = both()
    x[310], dh[315], h0[1] = bad, bad, bad       # in the second sequence
    spoilt = both()
    keep = torch.ones(T, dtype=torch.bool)
    keep[300:320] = False
    for k in ("h", "dx", "dg"):
        assert torch.equal(clean[k][keep.cuda()], spoilt[k][keep.cuda()]), k
    for k in ("ht", "dh0"):
        assert torch.equal(clean[k][[0, 2, 3]], spoilt[k][[0, 2, 3]]), k
    assert not torch.isfinite(spoilt["ht"][1]).any()


def test_glr_gradient_by_differences(B):
    """The kernel's gradients against central differences of the fp64 recurrence, whose own
    error is (2nd step)^2 / 6 of a third derivative; 1e-6 covers it at a step of 1e-4."""
    lens, D = [19, 4], 2
    T = sum(lens)
    x, g, h0 = rnd(1, T, D), -torch.exp(rnd(2, T, D) - 1), rnd(3, 2, D)
    dh, dht = rnd(4, T, D), rnd(5, 2, D)
    cu = torch.tensor([0, 19, 23], dtype=torch.int32).cuda()
    f = B.glr_fwd(x.cuda(), g.cuda(), h0=h0.cuda(), cu_seqlens=cu, want_states=True)
    b = B.glr_bwd(x.cuda(), g.cuda(), dh.cuda(), f["states"], dht=dht.cuda(), h0=h0.cuda(), cu_seqlens=cu)

    def loss(v):
        r, _ = glr_ref(v["x"], v["g"], v["h0"], lens)
        return float((r["h"] * dh.double()).sum() + (r["ht"] * dht.double()).sum())
    _, err = glr_ref(x, g, h0, lens, dh, dht)
    for name, got, e in (("x", b["dx"], err["dx"]), ("g", b["dg"], err["dg"]), ("h0", b["dh0"], err["dh0"])):
        base = {"x": x.double(), "g": g.double(), "h0": h0.double()}
        for i in range(0, base[name].numel(), 3):
            v = []
            for s in (1e-4, -1e-4):
                p = {k: t.clone() for k, t in base.items()}
                p[name].view(-1)[i] += s
                v.append(loss(p))
            want = (v[0] - v[1]) / 2e-4
            assert abs(float(got.view(-1)[i]) - want) <= float(e.view(-1)[i]) + U * abs(want) + 1e-6, (name, i)


# ------------------------------------------------------------------- steps

def glr_step_ref(x, g, state, slots):
    x, g, st = f64(x), f64(g), f64(state)
    h, err = torch.zeros_like(x), torch.zeros_like(st)
    he = torch.zeros_like(x)
    for n, s in enumerate(slots):
        if 0 <= s < st.shape[0]:
            new = g[n].exp() * st[s] + x[n]
            err[s] = g[n].exp() * err[s] + 8 * U * (g[n].exp() * st[s].abs() + x[n].abs())
            st[s] = h[n] = new
            he[n] = err[s]
    return h, he, st, err


SLOTS = {"own": None, "perm": [4, 0, 7, 2], "pad": [-1, 3, 9, 8, 100, 3 - 4], "twice": [5, 1, 5, 5, -1, 1, 0],
         "all": list(range(9)) * 15}


@pytest.mark.parametrize("which", SLOTS)
@pytest.mark.parametrize("D,dtype", [(1, "f32"), (100, "bf16"), (256, "f16"), (1027, "f32")])
def test_glr_step(B, which, D, dtype):
    slots = SLOTS[which]
    N = 6 if slots is None else len(slots)
    x, g, state = rnd(1, N, D).to(DT[dtype]), -torch.exp(rnd(2, N, D)), rnd(3, 9, D)
    h, he, st, se = glr_step_ref(x, g, state, range(N) if slots is None else slots)
    for put in (lambda t: t.cuda(), misaligned):
        s = put(state)
        got = B.glr_step(put(x), put(g), s, slots=None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda())
        close("h", got, h, he + half(dtype) * h.abs() + TINY[dtype])
        close("state", s, st, se + 1e-38)
        untouched = [i for i in range(9) if i not in (range(N) if slots is None else slots)]
        assert torch.equal(s.cpu()[untouched], state[untouched])
        xx = put(x)
        assert torch.equal(B.glr_step(xx, put(g), put(state), out=xx, slots=None if slots is None else
                                      torch.tensor(slots, dtype=torch.int32).cuda()), got)


def gdr_step_ref(q, k, v, g, beta, state, slots, scale):
    """The rule token by token; the state's error: K + 16 operations on the magnitudes of its terms."""
    q, k, v, g, beta, st = (f64(t) for t in (q, k, v, g, beta, state))
    N, HK, K = k.shape
    HV = v.shape[1]
    o, oe, se = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(st)
    head = torch.arange(HV) // (HV // HK)
    for n in range(N):
        s = slots[n]
        if not 0 <= s < st.shape[0]:
            continue
        S, E = st[s], se[s]
        al, kk, qq, b = g[n].exp()[:, None, None], k[n][head], q[n][head], beta[n][:, None]
        u = (al * S * kk[:, :, None]).sum(1)
        um = (al * S.abs() * kk.abs()[:, :, None]).sum(1)
        ue = (al * E * kk.abs()[:, :, None]).sum(1)
        d, dm, de = b * (v[n] - u), b * (v[n].abs() + um), b * (ue + (K + 16) * U * (v[n].abs() + um))
        new = al * S + kk[:, :, None] * d[:, None, :]
        E = al * E + kk.abs()[:, :, None] * de[:, None, :] + 8 * U * (al * S.abs() + kk.abs()[:, :, None] * dm[:, None, :])
        st[s], se[s] = new, E
        o[n] = scale * (new * qq[:, :, None]).sum(1)
        # o is formed as scale (al S^T q + (q.k) d): its terms' magnitudes bound it
        om = (al * S.abs() * qq.abs()[:, :, None]).sum(1) + (qq.abs() * kk.abs()).sum(1, keepdim=True) * dm
        oe[n] = scale * ((2 * K + 16) * U * om + (E * qq.abs()[:, :, None]).sum(1) +
                         (qq.abs() * kk.abs()).sum(1, keepdim=True) * de)
    return o, oe, st, se


def step_inputs(seed, N, HK, HV, K, dtype, S=9):
    q, k = rnd(seed, N, HK, K), rnd(seed + 1, N, HK, K)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    return dict(q=q.to(DT[dtype]), k=k.to(DT[dtype]), v=rnd(seed + 2, N, HV, K).to(DT[dtype]),
                g=torch.nn.functional.logsigmoid(rnd(seed + 3, N, HV)), beta=torch.sigmoid(rnd(seed + 4, N, HV)).to(DT[dtype]),
                state=rnd(seed + 5, S, HV, K, K))


@pytest.mark.parametrize("which", SLOTS)
@pytest.mark.parametrize("HK,HV,K,dtype", [(1, 1, 64, "f32"), (2, 2, 128, "bf16"), (1, 3, 128, "f32"), (2, 4, 64, "f16")])
def test_gdr_step(B, which, HK, HV, K, dtype):
    slots = SLOTS[which]
    N = 6 if slots is None else len(slots)
    i = step_inputs(10, N, HK, HV, K, dtype)
    for scale in (None, 0.5):
        o, oe, st, se = gdr_step_ref(*(i[k] for k in ("q", "k", "v", "g", "beta", "state")),
                                     range(N) if slots is None else slots, scale or K ** -0.5)
        for put in (lambda t: t.cuda(), misaligned):
            d = {k: put(t) for k, t in i.items()}
            sl = None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda()
            got = B.gdr_step(**d, slots=sl, scale=scale)
            close("o", got, o, oe + half(dtype) * o.abs() + TINY[dtype])
            close("state", d["state"], st, se + 1e-38)
            untouched = [j for j in range(9) if j not in (range(N) if slots is None else slots)]
            assert torch.equal(d["state"].cpu()[untouched], i["state"][untouched])
            d2 = {k: put(t) for k, t in i.items()}
            assert torch.equal(B.gdr_step(**d2, slots=sl, scale=scale, out=d2["v"]), got)


def test_gdr_step_spoilt_slot(B):
    """A state that is not finite spoils its own rows only; padding writes zeros and no state."""
    i = step_inputs(3, 4, 1, 2, 64, "f32")
    d = {k: t.cuda() for k, t in i.items()}
    d["state"][2] = float("nan")
    o = B.gdr_step(**d, slots=torch.tensor([0, 2, -5, 1], dtype=torch.int32).cuda())
    assert torch.isnan(o[1]).all() and torch.isfinite(o[[0, 2, 3]]).all() and (o[2] == 0).all()
    assert torch.isfinite(d["state"][[0, 1]]).all() and torch.equal(d["state"][3:].cpu(), i["state"][3:])


def test_steps_empty(B):
    i = {k: t.cuda() for k, t in step_inputs(3, 0, 1, 2, 64, "bf16").items()}
    assert B.gdr_step(**i).shape == (0, 2, 64)
    assert B.glr_step(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"),
                      torch.ones(3, 8, device="cuda")).shape == (0, 8)
    x = torch.ones(2, 8, device="cuda")      # an empty pool: every row is padding
    h = B.glr_step(x, x, torch.empty(0, 8, device="cuda"), slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert (h == 0).all()


# ------------------------------------------------------------- used together

def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


def test_prefill_then_decode(B):
    """gdr_chunk_fwd over a prompt, then gdr_step token by token on its final states, against gdr_chunk_fwd
    over the whole text (rel-L2 2e-2, the 16-bit bar of the chunked calls)."""
    from chunked_gated_delta_08_amd import workloads as W
    T, P = 150, 130
    inp = W.gdr_inputs(2, T, 2, 4, 128, 128, dtype="bf16", seed=5, gate_scale=1 / 8)
    q, k, v, beta, graw = (inp[n].cuda().view(2, T, *inp[n].shape[1:]) for n in ("q", "k", "v", "beta", "graw"))
    flat = lambda t: t.reshape(-1, *t.shape[2:]).contiguous()  # noqa: E731
    whole = B.gdr_chunk_fwd(*(flat(t) for t in (q, k, v)), B.gdr_gate_cumsum(flat(graw), B=2), flat(beta), B=2)
    head = [t[:, :P] for t in (q, k, v, graw, beta)]
    pre = B.gdr_chunk_fwd(*(flat(t) for t in head[:3]), B.gdr_gate_cumsum(flat(head[3]), B=2), flat(head[4]), B=2)
    pool = torch.full((5, 4, 128, 128), float("nan"), device="cuda")
    pool[[3, 1]] = pre["ht"]
    slots = torch.tensor([3, 1, -1], dtype=torch.int32, device="cuda")
    outs = []
    for t in range(P, T):
        row = [torch.cat([a[:, t], torch.zeros_like(a[:1, t])]).contiguous() for a in (q, k, v, graw, beta)]
        o = B.gdr_step(*row, pool, slots=slots)
        assert (o[2] == 0).all()
        outs.append(o[:2])
    assert rel(torch.stack(outs, 1), whole["o"].view(2, T, 4, 128)[:, P:]) <= 2e-2
    assert rel(pool[[3, 1]], whole["ht"]) <= 2e-2 and torch.isnan(pool[[0, 2, 4]]).all()
    # the same tokens as successive rows of one call
    pool[[3, 1]] = pre["ht"]
    rows = [a[:, P:].transpose(0, 1).reshape(-1, *a.shape[2:]).contiguous() for a in (q, k, v, graw, beta)]
    o = B.gdr_step(*rows, pool, slots=slots[:2].repeat(T - P))
    assert torch.equal(o.view(T - P, 2, 4, 128).transpose(0, 1), torch.stack(outs, 1))


def test_glr_steps_follow_the_scan(B):
    """glr_fwd over a prompt and glr_step after it give the bits of one another's recurrence up to its bound."""
    T, P, D = 80, 61, 96
    x, g = rnd(1, T, D), -torch.exp(rnd(2, T, D) - 2)
    ref, err = glr_ref(x, g, None, [T])
    pre = B.glr_fwd(x[:P].cuda(), g[:P].cuda())
    st = pre["ht"].clone()
    for t in range(P, T):
        h = B.glr_step(x[t:t + 1].cuda(), g[t:t + 1].cuda(), st)
        close("h", h, ref["h"][t:t + 1], err["h"][t:t + 1] + U * ref["h"][t:t + 1].abs())
    close("state", st, ref["ht"], err["ht"] + U * ref["ht"].abs())


def _layer(A, p, x, res, lens):
    """A block as a user writes it: norm of the residual stream, the gated delta rule, its gated norm and
    projection; then the next norm, the linear recurrence and the add that ends the block."""
    T = x.shape[0]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    y, res = A.add_rms_norm(x, res, p["w1"], p["s1"])
    q, k, v, z = (y @ p[n] for n in ("wq", "wk", "wv", "wz"))
    l2 = lambda t: torch.nn.functional.normalize(t.view(T, 2, 64).float(), dim=-1).to(t.dtype)  # noqa: E731
    g = torch.nn.functional.logsigmoid((y @ p["wg"]).float())
    beta = torch.sigmoid(y @ p["wb"])
    o, _ = A.chunk_gated_delta_rule(l2(q), l2(k), v.view(T, 2, 64), g, beta, cu_seqlens=cu.cuda())
    o = A.gated_rms_norm(o, z.view(T, 2, 64), p["wn"])
    y, res = A.add_rms_norm(o.reshape(T, 128) @ p["wo"], res, p["w2"], p["s2"])
    gate = -torch.nn.functional.softplus((y @ p["wa"]).float())
    h, _ = A.gated_linear_recurrence(y @ p["wi"], gate, cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    y, res = A.add_rms_norm(h, res, p["w1"])
    return y, res


class _Plain:
    """The same operators in torch, fp64."""
    @staticmethod
    def gated_rms_norm(x, z, w, eps=1e-5):
        return x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w * z * torch.sigmoid(z)

    @staticmethod
    def add_rms_norm(x, res, w, scale=1.0, eps=1e-5):
        res = res + scale * x
        return res * (res.square().mean(-1, keepdim=True) + eps).rsqrt() * w, res

    @staticmethod
    def gated_linear_recurrence(x, g, cu_seqlens, cu_seqlens_host=None):
        out = []
        for a, b in zip(cu_seqlens.tolist()[:-1], cu_seqlens.tolist()[1:]):
            h = torch.zeros_like(x[0])
            for t in range(a, b):
                h = g[t].exp() * h + x[t]
                out.append(h)
        return torch.stack(out), None

    @staticmethod
    def chunk_gated_delta_rule(q, k, v, g, beta, cu_seqlens):
        out = []
        for a, b in zip(cu_seqlens.tolist()[:-1], cu_seqlens.tolist()[1:]):
            S = torch.zeros(q.shape[1], q.shape[2], v.shape[2], dtype=q.dtype)
            for t in range(a, b):
                S = S * g[t].exp()[:, None, None]
                d = beta[t][:, None] * (v[t] - (S * k[t][:, :, None]).sum(1))
                S = S + k[t][:, :, None] * d[:, None, :]
                out.append((S * q[t][:, :, None]).sum(1) * q.shape[2] ** -0.5)
        return torch.stack(out), None


def test_layer_forward_and_gradients(B, monkeypatch):
    """The operators in a block, forward and through autograd, against the block in fp64.  The block runs in fp32,
    so 1e-4 relative (the fp32 bar of the chunked calls) holds for outputs and gradients."""
    from chunked_gated_delta_08_amd import autograd as A
    lens = [70, 1, 0, 29]
    T, D = sum(lens), 128
    shapes = dict(wq=(D, D), wk=(D, D), wv=(D, D), wz=(D, D), wo=(D, D), wa=(D, D), wi=(D, D), wg=(D, 2), wb=(D, 2))
    p = {n: rnd(i, *s, scale=D ** -0.5) for i, (n, s) in enumerate(shapes.items())}
    p.update(w1=1 + 0.1 * rnd(20, D), w2=1 + 0.1 * rnd(21, D), wn=1 + 0.1 * rnd(22, 64), s1=0.5 + 0.1 * rnd(23, D),
             s2=0.5 + 0.1 * rnd(24, D))
    x, res, dy, dr = rnd(30, T, D), rnd(31, T, D), rnd(32, T, D), rnd(33, T, D)

    def grads(ops, move, *tensors):
        q = {n: move(t).requires_grad_() for n, t in p.items()}
        a, b = move(x).requires_grad_(), move(res).requires_grad_()
        y, r = _layer(ops, q, a, b, lens)
        ((y * move(dy)).sum() + (r * move(dr)).sum()).backward()
        return {"y": y.detach(), "res": r.detach(), "dx": a.grad, "dres": b.grad, **{"d" + n: t.grad for n, t in q.items()}}
    got = grads(A, lambda t: t.cuda())
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    monkeypatch.setattr(torch.Tensor, "float", lambda t: t.double())
    want = grads(_Plain, lambda t: t.double())
    monkeypatch.undo()
    for n in want:
        assert rel(got[n], want[n]) <= 1e-4, (n, rel(got[n], want[n]))


def test_unused_outputs_have_no_gradient(B):
    """One of two outputs used: the other's gradient is taken as zero."""
    from chunked_gated_delta_08_amd import autograd as A
    x, res, g = rnd(1, 40, 32).cuda(), rnd(2, 40, 32).cuda(), -torch.exp(rnd(3, 40, 32)).cuda()
    w, d = 1 + 0.1 * rnd(4, 32).cuda(), rnd(5, 40, 32).cuda()
    for pick in (0, 1):
        a, b = x.clone().requires_grad_(), res.clone().requires_grad_()
        (A.add_rms_norm(a, b, w)[pick] * d).sum().backward()
        zero = torch.zeros_like(d)
        f = B.add_norm_fwd(x, res, w)
        r = B.add_norm_bwd(d if pick == 0 else zero, zero if pick == 0 else d, f["res"], w)
        assert torch.equal(a.grad, r["dx"]) and torch.equal(b.grad, r["dres"])
        a = x.clone().requires_grad_()
        out = A.gated_linear_recurrence(a, g)[pick]
        dd = d if pick == 0 else d[:1]
        (out * dd).sum().backward()
        f = B.glr_fwd(x, g, want_states=True)
        r = B.glr_bwd(x, g, d if pick == 0 else zero, f["states"], dht=None if pick == 0 else dd.contiguous())
        assert torch.equal(a.grad, r["dx"])


# --------------------------------------------------------------- far offsets

def test_far_offsets_norms(B):
    """Rows beyond 2^32 bytes and 2^31 elements: the last ones are the ones a short call gives."""
    D = 128
    rows = (1 << 31) // D + 1000
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[-500:] = rnd(1, 500, D).bfloat16().cuda()
    w = 1 + 0.1 * rnd(2, D).cuda()
    y = B.gated_norm_fwd(x, x, w)
    assert torch.equal(y[-500:], B.gated_norm_fwd(x[-500:].clone(), x[-500:].clone(), w))
    del y
    g = B.gated_norm_bwd(x, None, w, x)
    assert torch.equal(g["dx"][-500:], B.gated_norm_bwd(x[-500:].clone(), None, w, x[-500:].clone())["dx"])
    del g
    f = B.add_norm_fwd(x, x, w)
    assert torch.equal(f["y"][-500:], B.add_norm_fwd(x[-500:].clone(), x[-500:].clone(), w)["y"])
    r = B.add_norm_bwd(x, x, f["res"], w)["dres"]
    t = x[-500:].clone()
    assert torch.equal(r[-500:], B.add_norm_bwd(t, t, f["res"][-500:].clone(), w)["dres"])


def test_far_offsets_steps(B):
    """Pools beyond 2^32 bytes and 2^31 elements."""
    i = step_inputs(7, 3, 1, 2, 128, "f32", S=1)
    S = (1 << 31) // (2 * 128 * 128) + 9
    d = {k: t.cuda() for k, t in i.items()}
    pool = torch.empty(S, 2, 128, 128, device="cuda")
    slots = torch.tensor([S - 1, 0, S - 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = d["state"]
    small = d["state"].expand(3, -1, -1, -1).contiguous()
    args = [d[k] for k in ("q", "k", "v", "g", "beta")]
    assert torch.equal(B.gdr_step(*args, pool, slots=slots), B.gdr_step(*args, small))
    assert torch.equal(pool[slots.long()], small)
    x, g = rnd(1, 3, 4099).cuda(), -torch.exp(rnd(2, 3, 4099)).cuda()
    S = (1 << 31) // 4099 + 9
    pool = pool.view(-1)[:S * 4099].view(S, 4099) if pool.numel() >= S * 4099 else torch.empty(S, 4099, device="cuda")
    slots = torch.tensor([S - 1, 0, S - 3], dtype=torch.int32, device="cuda")
    small = rnd(3, 3, 4099).cuda()
    pool[slots.long()] = small
    assert torch.equal(B.glr_step(x, g, pool, slots=slots), B.glr_step(x, g, small))
    assert torch.equal(pool[slots.long()], small)


def test_far_offsets_glr(B):
    """Tokens times channels beyond 2^32 elements: the last tokens of a slab of channels, whose gates forget the rest,
    are the ones that the slab alone gives.  The two calls cut the tokens into tiles differently: with gates of 0.4 and
    |x| of 1 the states' magnitudes stay below 10, so they differ by less than 10 * 16 u * 5 tokens < 1e-4, and two
    roundings to bf16 of such values by a step of 2^-8; dg is a product of two."""
    T, D, n = 66000, 1 << 16, 300
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    g = torch.empty(T, D, device="cuda").fill_(-0.5)
    xs, gs = rnd(1, n, 200).bfloat16().cuda(), -torch.exp(rnd(2, n, 200)).cuda()
    gs[0] = float("-inf")      # nothing from before reaches past here
    x[-n:, -200:], g[-n:, -200:] = xs, gs
    f = B.glr_fwd(x, g, want_states=True)
    want = B.glr_fwd(xs, gs, want_states=True)
    close("h", f["h"][-n:, -200:], f64(want["h"]), f64(want["h"]).abs() * 2.0 ** -8 + 1e-4)
    close("ht", f["ht"][:, -200:], f64(want["ht"]), f64(want["ht"]).abs() * 1e-4 + 1e-5)
    b = B.glr_bwd(x, g, x, f["states"], want_dh0=False)
    bw = B.glr_bwd(xs, gs, xs, want["states"], want_dh0=False)
    close("dx", b["dx"][-n:, -200:], f64(bw["dx"]), f64(bw["dx"]).abs() * 2.0 ** -8 + 1e-4)
    close("dg", b["dg"][-n:, -200:], f64(bw["dg"]), f64(bw["dg"]).abs() * 1e-3 + 1e-4)


# ------------------------------------------------- streams, graphs, workspaces

def _everything(B, d, ws):
    """One call of every operator on preallocated buffers and the given workspaces."""
    B.gated_norm_fwd(d["x"], d["z"], d["w"], out=d["y"])
    B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"], out=d["gn"], workspace=ws[0])
    B.add_norm_fwd(d["x"], d["res"], d["w"], scale=d["w"], out=d["an"])
    B.add_norm_bwd(d["dy"], d["res"], d["an"]["res"], d["w"], x=d["x"], scale=d["w"], out=d["ab"], workspace=ws[1])
    B.glr_fwd(d["x"], d["g"], cu_seqlens=d["cu"], cu_seqlens_host=d["cuh"], out=d["gf"], workspace=ws[2])
    B.glr_bwd(d["x"], d["g"], d["dy"], d["gf"]["states"], cu_seqlens=d["cu"], cu_seqlens_host=d["cuh"], out=d["gb"],
              workspace=ws[3])
    B.glr_step(d["x"][:4], d["g"][:4], d["pool"], slots=d["slots"], out=d["hs"])
    B.gdr_step(*d["rule"], slots=d["slots"], out=d["o"])


def _state(B, T=3000, D=256):
    dev = dict(device="cuda")
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, **dev)  # noqa: E731
    bf = torch.bfloat16
    cuh = torch.tensor([0, 1000, 1001, T], dtype=torch.int32)
    i = {k: t.cuda() for k, t in step_inputs(50, 4, 1, 2, 64, "bf16").items()}
    d = dict(x=rnd(1, T, D).to(bf).cuda(), z=rnd(2, T, D).to(bf).cuda(), dy=rnd(3, T, D).to(bf).cuda(),
             res=rnd(4, T, D).to(bf).cuda(), g=-torch.exp(rnd(5, T, D) - 3).cuda(), w=1 + 0.1 * rnd(6, D).cuda(),
             cu=cuh.cuda(), cuh=cuh, pool=rnd(7, 9, D).cuda(), slots=torch.tensor([2, 0, 2, -1], dtype=torch.int32).cuda(),
             rule=[i[k] for k in ("q", "k", "v", "g", "beta", "state")], y=e(T, D, t=bf), hs=e(4, D, t=bf),
             o=e(4, 2, 64, t=bf),
             gn=dict(dx=e(T, D, t=bf), dz=e(T, D, t=bf), dw=e(D)), an=dict(y=e(T, D, t=bf), res=e(T, D, t=bf)),
             ab=dict(dx=e(T, D, t=bf), dres=e(T, D, t=bf), dw=e(D), dscale=e(D)),
             gf=dict(h=e(T, D, t=bf), ht=e(3, D), states=e(B.glr_num_states(T), D)),
             gb=dict(dx=e(T, D, t=bf), dg=e(T, D), dh0=e(3, D)))
    n = B.norm_workspace_size(T, D, bf)
    m = B.glr_workspace_size(T, D, bf, cu_seqlens_host=cuh)
    ws = [e(n, t=torch.uint8), e(n, t=torch.uint8), e(m, t=torch.uint8), e(m, t=torch.uint8)]
    return d, ws


def _results(d):
    return [t.clone() for t in (d["y"], *d["gn"].values(), *d["an"].values(), *d["ab"].values(), *d["gf"].values(),
                                *d["gb"].values(), d["pool"], d["hs"], d["o"], d["rule"][5])]


def test_captured_and_replayed(B):
    """Every operator captured into one graph, replayed with other work between: the eager bits each time."""
    d, ws = _state(B)
    start = [d["pool"].clone(), d["rule"][5].clone()]

    def reset():
        d["pool"].copy_(start[0])
        d["rule"][5].copy_(start[1])
        for t in (d["y"], d["gn"]["dw"], d["ab"]["dscale"], d["gf"]["h"], d["gb"]["dg"], d["o"]):
            t.fill_(float("nan"))
    reset()
    _everything(B, d, ws)
    want = _results(d)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            _everything(B, d, ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        reset()
        for w in ws:
            w.fill_(255)                 # whatever the workspace held
        torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_results(d), want))
        B.gated_norm_fwd(d["x"], None, d["w"])
        torch.cuda.synchronize()


def test_two_streams_at_once(B):
    """Two users, each with its own workspaces, on two streams at the same time."""
    states = [_state(B), _state(B)]
    keep = [(d["pool"].clone(), d["rule"][5].clone()) for d, _ in states]
    _everything(B, *states[0])
    want = _results(states[0][0])
    for (d, _), (a, b) in zip(states, keep):
        d["pool"].copy_(a)
        d["rule"][5].copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (d, ws), s, (a, b) in zip(states, streams, keep):
            with torch.cuda.stream(s):
                d["pool"].copy_(a)
                d["rule"][5].copy_(b)
                _everything(B, d, ws)
    torch.cuda.synchronize()
    for d, _ in states:
        assert all(torch.equal(a, b) for a, b in zip(_results(d), want))


def test_given_stream(B):
    """A stream that is not the current one: temporaries allocated for the call live until it is done."""
    d, _ = _state(B)
    want = B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"])
    f = B.glr_fwd(d["x"], d["g"], want_states=True)
    wantb = B.glr_bwd(d["x"], d["g"], d["dy"], f["states"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"], stream=s)
        gotb = B.glr_bwd(d["x"], d["g"], d["dy"], f["states"], stream=s)
        junk = [torch.full((1 << 18,), 3.0, device="cuda") for _ in range(8)]
        s.synchronize()
        del junk
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert all(torch.equal(gotb[k], wantb[k]) for k in wantb)


def test_given_stream_waits_for_what_it_allocates(B):
    """What the call allocates was just freed on the current stream, which still writes there."""
    d, _ = _state(B, T=20000, D=512)
    want = B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(d["x"]) for _ in range(4)]
        for _ in range(100):
            for t in old:
                t.fill_(7.0)
        del old, t
        got = B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"], stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
        del got


def _capture(run):
    """run() warmed up on a side stream and captured there; returns the graph and what run() gave."""
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        with torch.cuda.graph(graph, stream=side):
            out = run()
    torch.cuda.current_stream().wait_stream(side)
    return graph, out


def test_captured_training_step(B):
    """Forward and backward through autograd in one graph: on new inputs the eager bits each time."""
    from chunked_gated_delta_08_amd import autograd as A
    T, D = 700, 130
    cu = torch.tensor([0, 1, 1, 400, T], dtype=torch.int32)
    dev = cu.cuda()
    rows = {n: rnd(i, T, D).cuda().requires_grad_() for i, n in enumerate("xrgz")}
    vecs = {n: (1 + 0.1 * rnd(9 + i, D)).cuda().requires_grad_() for i, n in enumerate("wsv")}
    dy, dr = rnd(20, T, D).cuda(), rnd(21, T, D).cuda()

    def run():
        y, res = A.add_rms_norm(rows["x"], rows["r"], vecs["w"], vecs["s"])
        h, _ = A.gated_linear_recurrence(y, -torch.exp(rows["g"]), cu_seqlens=dev, cu_seqlens_host=cu)
        o = A.gated_rms_norm(h, rows["z"], vecs["v"])
        grads = torch.autograd.grad((o, res), [*rows.values(), *vecs.values()], (dy, dr))
        return (o.detach(), res.detach()) + grads   # no autograd graph outlives its pass
    graph, out = _capture(run)
    for i in range(4):
        with torch.no_grad():
            for n, t in enumerate(rows.values()):
                t.copy_(rnd(100 + 10 * i + n, T, D))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_decoding(B):
    """A decode step of a layer in one graph, replayed token by token while sequences come and go: states and
    outputs as eager steps give them."""
    N, H, K, D = 5, 2, 64, 128
    t = dict(x=torch.zeros(N, D), q=torch.zeros(N, H, K), k=torch.zeros(N, H, K), g=torch.zeros(N, H),
             beta=torch.zeros(N, H), a=torch.zeros(N, D))
    t = {n: v.cuda() for n, v in t.items()}
    slots = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    w, wn = (1 + 0.1 * rnd(1, D)).cuda(), (1 + 0.1 * rnd(2, K)).cuda()
    pool, diag = torch.zeros(7, H, K, K, device="cuda"), torch.zeros(7, D, device="cuda")

    def run():
        f = B.add_norm_fwd(t["x"], t["a"], w)
        o = B.gdr_step(t["q"], t["k"], f["y"].view(N, H, K), t["g"], t["beta"], pool, slots)
        o = B.gated_norm_fwd(o, f["y"].view(N, H, K), wn)
        return o, B.glr_step(o.view(N, D), -f["res"].abs(), diag, slots)
    graph, out = _capture(run)
    want_pool, want_diag = rnd(3, 7, H, K, K).cuda(), rnd(4, 7, D).cuda()
    pool.copy_(want_pool)
    diag.copy_(want_diag)
    for i, s in enumerate(([0, 1, 2, -1, -1], [0, 2, 6, 5, 3], [6, 0, 0, 1, 7], [-1] * 5, [4, 3, 2, 1, 0])):
        for n, (name, v) in enumerate(t.items()):
            v.copy_(rnd(50 + 10 * i + n, *v.shape) * (-1 if name == "g" else 1))
        t["g"].copy_(-t["g"].abs())
        t["k"].copy_(torch.nn.functional.normalize(t["k"], dim=-1))
        t["beta"].sigmoid_()
        slots.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got, have = [v.clone() for v in out], (pool.clone(), diag.clone())
        pool.copy_(want_pool)
        diag.copy_(want_diag)
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(have[0], pool) and torch.equal(have[1], diag)
        want_pool, want_diag = pool.clone(), diag.clone()


@pytest.mark.parametrize("rows,D,dtype,rdtype", [(600, 8192, "bf16", "bf16"), (1100, 4100, "f16", "f32"), (530, 8192, "f32", "f32"),
                                                 (1030, 1500, "f32", "f32"), (300, 4500, "f16", "f16")])
def test_norms_many_wide_rows(B, rows, D, dtype, rdtype):
    """Rows of many lanes, several to a workgroup of the backward; in place too."""
    x, z, res = rnd(1, rows, D).to(DT[dtype]), rnd(2, rows, D).to(DT[dtype]), rnd(3, rows, D, scale=2.0).to(DT[rdtype])
    w, s = 1 + 0.1 * rnd(4, D), 0.5 + 0.2 * rnd(5, D)
    dy, dres = rnd(6, rows, D).to(DT[dtype]), rnd(7, rows, D).to(DT[rdtype])
    d = {k: t.cuda() for k, t in dict(x=x, z=z, res=res, w=w, s=s, dy=dy, dres=dres).items()}
    ref, tol = gated_ref(x, z, w, dy, "silu", dtype)
    g = B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"], eps=EPS)
    for k, v in {"y": B.gated_norm_fwd(d["x"], d["z"], d["w"], eps=EPS), **g}.items():
        close(k, v, ref[k], tol[k])
    f = B.add_norm_fwd(d["x"], d["res"], d["w"], scale=d["s"], eps=EPS)
    ref, tol = add_ref(x, res, w, s, dtype, rdtype)
    for k in ("y", "res"):
        close(k, f[k], ref[k], tol[k])
    a = B.add_norm_bwd(d["dy"], d["dres"], f["res"], d["w"], x=d["x"], scale=d["s"], eps=EPS)
    ref, tol = add_bwd_ref(dy, dres, f["res"], w, x, s, dtype, rdtype)
    for k in ref:
        close(k, a[k], ref[k], tol[k])
    b = {"dx": d["dy"].clone(), "dres": d["dres"].clone(), "dw": torch.empty_like(a["dw"]), "dscale": torch.empty_like(a["dw"])}
    B.add_norm_bwd(b["dx"], b["dres"], f["res"], d["w"], x=d["x"], scale=d["s"], eps=EPS, out=b)
    assert all(torch.equal(a[k], b[k]) for k in a)
    c = {"dx": d["x"], "dz": d["z"], "dw": b["dw"]}
    B.gated_norm_bwd(d["x"], d["z"], d["w"], d["dy"], eps=EPS, out=c)
    assert all(torch.equal(g[k], c[k]) for k in g)


# ------------------------------------------- the recurrence over many segments

def chain_inputs(lens, D, dtype):
    """Every even channel has gates of 1 and small whole numbers, so each of its sums is exact in fp32 (below 2^24
    throughout) and a state that is lost or taken twice anywhere shows; the odd ones have time constants of some
    thousand tokens."""
    T, N = sum(lens), len(lens)
    x, dh, h0, dht = rnd(1, T, D), rnd(2, T, D), rnd(3, N, D), rnd(4, N, D)
    g = -torch.exp(0.5 * rnd(5, T, D) - 8)
    for t in (x, dh, h0, dht):
        t[:, ::2] = (t[:, ::2] * 2).round().clamp(-6, 6)
    g[:, ::2] = 0.0
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    d = {k: t.cuda() for k, t in dict(x=x.to(DT[dtype]), g=g, dh=dh.to(DT[dtype]), h0=h0, dht=dht).items()}
    return d, dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu) if N > 1 else {}


def chain_run(B, d, kw, polls=0):
    f = B.glr_fwd(d["x"], d["g"], h0=d["h0"], want_states=True, polls=polls, **kw)
    return {**f, **B.glr_bwd(d["x"], d["g"], d["dh"], f["states"], dht=d["dht"], h0=d["h0"], polls=polls, **kw)}


@pytest.mark.parametrize("lens,D,dtype", [([27000], 66, "bf16"), ([27000], 3, "f16"), ([17500], 70, "f32")])
def test_glr_many_blocks_without_patience(B, lens, D, dtype):
    """Chains of more than two blocks of 64 segments (192 tokens each in the 16-bit forward, else 128) whose
    workgroups take up one another's segments: the same bits."""
    d, kw = chain_inputs(lens, D, dtype)
    want = chain_run(B, d, kw)
    for polls in (1, 2, 9):
        got = chain_run(B, d, kw, polls)
        assert all(torch.equal(got[k], want[k]) for k in want), polls


def test_second_derivatives_raise(B):
    """create_graph leaves the gradients as they are; differentiating them again raises instead of leaving the
    operators' terms out."""
    from chunked_gated_delta_08_amd import autograd as A
    x, z, g = (rnd(i, 40, 32).cuda().requires_grad_() for i in range(3))
    w = (1 + 0.1 * rnd(4, 32)).cuda().requires_grad_()
    q, k, v = (rnd(i, 40, 1, 64).cuda().requires_grad_() for i in range(5, 8))
    a, b = (-torch.rand(40, 1, device="cuda")).requires_grad_(), torch.rand(40, 1, device="cuda", requires_grad=True)
    for run, args in ((lambda: A.gated_rms_norm(x, z, w), (x, z, w)), (lambda: A.add_rms_norm(x, z, w)[1], (x, z)),
                      (lambda: A.add_rms_norm(x, z, w, w)[0], (x, z, w)),
                      (lambda: A.gated_linear_recurrence(x, -g.exp())[0], (x, g)),
                      (lambda: A.chunk_gated_delta_rule(q, k, v, a, b)[0], (q, k, v, a, b))):
        plain = torch.autograd.grad(run().sum(), args)
        grads = torch.autograd.grad(run().sum(), args, create_graph=True)
        assert all(torch.equal(s, t) for s, t in zip(plain, grads))
        for t, arg in zip(grads, args):
            with pytest.raises(RuntimeError, match="no second derivative"):
                torch.autograd.grad(t.sum() + arg.square().sum(), arg, retain_graph=True)


def test_glr_gate_error(B):
    """exp(g) as both directions form it: (|g| + 3) u over the range of fp32, |g| u of it the rounding of the
    exponent's argument, zero below 2^-126.  One token from the state 1 shows it unrounded."""
    D = 1 << 20
    g = -torch.from_numpy(np.exp(np.random.default_rng(1).uniform(-9, np.log(89), (1, D))).astype(np.float32))
    g[0, :4] = torch.tensor([0.0, -0.0, float("-inf"), 70.0])
    zero, one = torch.zeros(1, D, device="cuda"), torch.ones(1, D, device="cuda")
    ref = f64(g).exp()
    tol = torch.where(torch.isfinite(g), (g.abs() + 3) * U * ref, 0.0) + GATE0
    f = B.glr_fwd(zero, g.cuda(), h0=one, want_states=True)
    b = B.glr_bwd(zero, g.cuda(), zero, f["states"], dht=one, h0=one)
    close("ht", f["ht"], ref, tol)
    close("dh0", b["dh0"], ref, tol)
    assert f["ht"][0, 0] == 1 and f["ht"][0, 2] == 0


def test_sigmoid_error(B):
    """The gate's sigmoid over its range: (|z| + 5) u, |z| u of it the rounding of the exponent's argument.  Rows of
    ones show it: their mean of squares is 1 exactly, its rsqrt is off by 2 u and the product by u; the sigmoid is
    zero below 2^-126."""
    z = torch.from_numpy(np.random.default_rng(1).uniform(-90, 30, (1 << 13, 128)).astype(np.float32))
    z[0, :4] = torch.tensor([0.0, -0.0, 200.0, -200.0])
    one = torch.ones_like(z).cuda()
    s = 1 / (1 + (-f64(z)).exp())
    y = B.gated_norm_fwd(one, z.cuda(), one[0].contiguous(), eps=0.0, act="sigmoid")
    close("y", y, s, (z.abs().double() + 8) * U * s + 2.0 ** -126)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_slope_of_open_and_shut_gates(B, act, dtype):
    """dz where the gate is nearly open or shut: its slope s c (1 + z c for silu) falls like exp(-|z|), and every digit
    of it counts.  s and c = 1 - s are each off by (|z| + 6) u (the sigmoid's |z| + 5, or that of the smaller one
    and one subtraction), the rest of dz by NORM_OPS operations; below 2^-126 they are zero."""
    rows, D = 400, 128
    x, dy, w = rnd(1, rows, D).to(DT[dtype]), rnd(2, rows, D).to(DT[dtype]), 1 + 0.1 * rnd(3, D)
    z = torch.from_numpy(np.random.default_rng(4).uniform(-80, 80, (rows, D)).astype(np.float32)).to(DT[dtype])
    g = B.gated_norm_bwd(*(t.cuda() for t in (x, z, w, dy)), eps=EPS, act=act)
    x, z, w, dy = f64(x), f64(z), f64(w), f64(dy)
    s, c = 1 / (1 + (-z).exp()), 1 / (1 + z.exp())
    t = dy * w * x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    one = (NORM_OPS + z.abs() + 6) * U
    ref, err = (t * s * c, 2 * one * s * c) if act == "sigmoid" else (t * s * (1 + z * c), 2 * one * s * (1 + z.abs() * c))
    close("dz", g["dz"], ref, half(dtype) * ref.abs() + t.abs() * (err + 2.0 ** -126) + TINY[dtype])


def test_steps_of_many_rows(B):
    """2^20 heads in one rule step, 2^22 workgroups in one step of the recurrence: the last rows as a short call gives them."""
    N, H, K, n = 65536, 16, 64, 40
    i = {k: t.cuda() for k, t in step_inputs(7, n, 2, H, K, "bf16", S=n).items()}
    big = {}
    for k, t in i.items():
        big[k] = torch.zeros(N, *t.shape[1:], dtype=t.dtype, device="cuda")
        big[k][-n:] = t
    assert torch.equal(B.gdr_step(**big)[-n:], B.gdr_step(**i))
    assert torch.equal(big["state"][-n:], i["state"]) and not big["state"][:-n].any()
    del big
    D = 32768
    x, g, st = rnd(1, n, D).bfloat16().cuda(), -torch.exp(rnd(2, n, D)).cuda(), rnd(3, n, D).cuda()
    bx, bg, bs = (torch.zeros(N, D, dtype=t.dtype, device="cuda") for t in (x, g, st))
    bx[-n:], bg[-n:], bs[-n:] = x, g, st
    assert torch.equal(B.glr_step(bx, bg, bs)[-n:], B.glr_step(x, g, st))
    assert torch.equal(bs[-n:], st) and not bs[:-n].any()


def test_given_stream_writes_cu_seqlens(B):
    """Without a host mirror cu_seqlens is copied once the given stream has written it."""
    T, D = 300, 64
    right = torch.tensor([0, 100, T], dtype=torch.int32).cuda()
    x, g, dh = rnd(1, T, D).cuda(), -torch.exp(rnd(2, T, D)).cuda(), rnd(3, T, D).cuda()
    want = B.glr_fwd(x, g, cu_seqlens=right, want_states=True)
    wantb = B.glr_bwd(x, g, dh, want["states"], cu_seqlens=right)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for bwd in (False, True):
        cu = torch.zeros_like(right)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)
            cu.copy_(right)
        if bwd:
            got, ref = B.glr_bwd(x, g, dh, want["states"], cu_seqlens=cu, stream=s), wantb
        else:
            got, ref = B.glr_fwd(x, g, cu_seqlens=cu, want_states=True, stream=s), want
        s.synchronize()
        assert all(torch.equal(got[k], ref[k]) for k in ref)


def test_out_without_what_is_skipped(B):
    """Outputs that a call may skip need not be in `out`; one that it needs is named."""
    T, D = 300, 64
    x, z, r, g = (rnd(i, T, D).cuda() for i in range(4))
    w, g = 1 + 0.1 * rnd(5, D).cuda(), -torch.exp(g)
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    for args, call, keys in (((x, None, w, z), B.gated_norm_bwd, ("dx", "dw")), ((z, r, x, w), B.add_norm_bwd, ("dres", "dw")),
                             ((z, r, x, w), B.add_norm_bwd, ("dres", "dw", "dx")), ((x, r, w), B.add_norm_fwd, ("y", "res")),
                             ((x, g), B.glr_fwd, ("h",)), ((x, g), B.glr_fwd, ("h", "ht")),
                             ((x, g, z, B.glr_fwd(x, g, want_states=True)["states"]), B.glr_bwd, ("dx", "dg"))):
        want = call(*args)
        out = {k: torch.empty_like(want[k]) for k in keys}
        got = call(*args, out=out)
        assert got is out and set(out) == set(keys) and all(torch.equal(got[k], want[k]) for k in keys)
        with pytest.raises(ValueError, match="required"):
            call(*args, out={k: out[k] for k in keys[1:]})
    half_x = x.bfloat16()       # x's gradient skipped where it has a type of its own
    got = B.add_norm_bwd(half_x, r, x, w, out={"dres": e(T, D), "dw": e(D)})
    assert torch.equal(got["dres"], B.add_norm_bwd(half_x, r, x, w)["dres"])


@pytest.mark.parametrize("lens,D,dtype", [([27000], 3, "bf16"), ([27000], 66, "f16"), ([17500], 2, "f32"), ([17500], 70, "f32"),
                                          ([13000, 1, 0, 30000, 77], 66, "bf16"), ([5000, 21000], 3, "f32")])
def test_glr_many_blocks(B, lens, D, dtype):
    """Every value of chains of more than two blocks of 64 segments (192 tokens each in the 16-bit forward, else 128),
    from the start of a block or its middle on.  Channels with gates of 1 are exact: equal but for an output's rounding."""
    d, kw = chain_inputs(lens, D, dtype)
    got = chain_run(B, d, kw)
    ref, err = glr_ref(*(d[k] for k in ("x", "g", "h0")), lens, d["dh"], d["dht"])
    assert max(float(r[:, ::2].abs().max()) for r in ref.values()) < 2.0 ** 24
    for k in ref:
        t = dtype if k in ("h", "dx") else "f32"
        close(k, got[k], ref[k], err[k] + half(t) * ref[k].abs())
        assert torch.equal(got[k][:, ::2].cpu(), ref[k][:, ::2].to(DT[t])), k
        if k in ("h", "dx"):   # what a lost state would change is far above what may be off
            assert float((err[k][:, 1::2] / ref[k][:, 1::2].abs().mean()).median()) < 0.2, k


@pytest.mark.parametrize("dtype,base", [("bf16", 512), ("bf16", 1024), ("f32", 256), ("f32", 1024)])
def test_odd_wide_rows_in_place(B, dtype, base):
    """A row whose last vector begins a wave's columns is read from columns of the wave before, which may be writing
    them already when an output replaces that input: what is read of those is dropped."""
    vec = 8 if dtype == "bf16" else 4
    for D in range(base + 1, base + vec):
        rows = 1300
        t = {k: rnd(i, rows, D).to(DT[dtype]).cuda() for i, k in enumerate(("x", "z", "dy", "res", "dres"))}
        w, s = 1 + 0.1 * rnd(7, D).cuda(), 0.5 + 0.2 * rnd(8, D).cuda()
        new = lambda: {k: v.clone() for k, v in t.items()}  # noqa: E731
        y = B.gated_norm_fwd(t["x"], t["z"], w)
        for k in ("x", "z"):
            c = new()
            assert torch.equal(B.gated_norm_fwd(c["x"], c["z"], w, out=c[k]), y), (D, k)
        g = B.gated_norm_bwd(t["x"], t["z"], w, t["dy"])
        for dx, dz in (("x", "z"), ("dy", "z"), ("x", "dy")):
            c = new()
            o = B.gated_norm_bwd(c["x"], c["z"], w, c["dy"], out={"dx": c[dx], "dz": c[dz], "dw": torch.empty_like(w)})
            assert all(torch.equal(o[k], g[k]) for k in g), (D, dx, dz)
        f = B.add_norm_fwd(t["x"], t["res"], w, scale=s)
        c = new()
        o = B.add_norm_fwd(c["x"], c["res"], w, scale=s, out={"y": c["x"], "res": c["res"]})
        assert all(torch.equal(o[k], f[k]) for k in f), D
        a = B.add_norm_bwd(t["dy"], t["dres"], t["res"], w, x=t["x"], scale=s)
        for dx, dres in (("dy", "dres"), ("x", "res"), ("dy", "res"), ("x", "dres")):
            c = new()
            o = B.add_norm_bwd(c["dy"], c["dres"], c["res"], w, x=c["x"], scale=s,
                               out={"dx": c[dx], "dres": c[dres], "dw": torch.empty_like(w), "dscale": torch.empty_like(w)})
            assert all(torch.equal(o[k], a[k]) for k in a), (D, dx, dres)
