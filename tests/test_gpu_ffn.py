"""GPU tests of the gated feed-forward block (include/gdn_ffn.h) against its formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32, h = eps / 2 of the type.  A sum of m products
of exact operands is off by at most 2 (m + 20) u of the sum of their magnitudes: a step
of the matrix unit may cut off instead of rounding (2 u), the 20 are the joins of splits and
the waves' order.  An element's bound adds up what its terms can be off by, with h for
every rounding to the type (h, dg, du, the output).  That bound grows with the terms' number
where the roundings' signs would cancel, so the 2-norm of an output's error is held as well:
roundings are independent, each adds at most h of the norm, and there are two of them on the way to
every output (an operand and the output itself); in fp32 2 sqrt(m) u + 16 u, m the longest sum.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}   # half the smallest step of the type
NAMES = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from chunked_gated_delta_08_amd import binding
    return binding


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2 if dtype != "f32" else U


def rnd(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale)


def inputs(T, D, F, dtype, seed=0):
    t = DT[dtype]
    return dict(x=rnd(seed + 1, T, D).to(t), wg=rnd(seed + 2, F, D, scale=1.5 / D ** 0.5).to(t),
                wu=rnd(seed + 3, F, D, scale=D ** -0.5).to(t), wd=rnd(seed + 4, D, F, scale=F ** -0.5).to(t),
                dy=rnd(seed + 5, T, D).to(t))


def act64(g, act):
    """act(g), its slope."""
    if act == "gelu":
        phi = 0.5 * torch.erfc(-g / 2 ** 0.5)
        return g * phi, phi + g * torch.exp(-g * g / 2) / (2 * np.pi) ** 0.5
    s = torch.sigmoid(g)
    return (g * s, s * (1 + g * (1 - s))) if act == "silu" else (s, s * (1 - s))


def reference(x, wg, wu, wd, dy, act, dtype):
    """Outputs by the formulas and how far each element may be off."""
    h_, tiny = half(dtype), TINY[dtype]
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))

    def M(k):
        return 2 * (k + 20) * U
    T, D, F = x.shape[0], x.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = M(D) * (x.abs() @ wg.abs().T), M(D) * (x.abs() @ wu.abs().T)
    a, s = act64(g, act)
    # slopes of act are at most 1.13, of its slope 0.8; the functions themselves lose up to (|g| + 16) u of
    # their terms, which reach 1.5
    ea = 1.13 * eg + (g.abs() + 16) * U * a.abs() + 4 * U
    es = 0.8 * eg + 1.5 * (g.abs() + 32) * U
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu + 3 * U * h.abs()
    eh = eh * (1 + h_) + h_ * h.abs() + tiny
    y = h @ wd.T
    out = {"y": y}
    err = {"y": eh @ wd.abs().T + M(F) * ((h.abs() + eh) @ wd.abs().T)}
    dh = dy @ wd
    edh = M(D) * (dy.abs() @ wd.abs())
    du, dg = dh * a, dh * u * s

    def rounded(v, e):
        e = e + 3 * U * (v.abs() + e)
        return e * (1 + h_) + h_ * v.abs() + tiny
    edu = rounded(du, edh * (a.abs() + ea) + dh.abs() * ea)
    edg = rounded(dg, edh * (u.abs() + eu) * (s.abs() + es) + dh.abs() * (eu * (s.abs() + es) + u.abs() * es))
    out["dx"] = dg @ wg + du @ wu
    err["dx"] = edg @ wg.abs() + edu @ wu.abs() + M(2 * F) * ((dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs())
    for k, d, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        out[k] = d.T @ x
        err[k] = e.T @ x.abs() + M(T) * ((d.abs() + e).T @ x.abs())
    out["dw_down"] = dy.T @ h
    err["dw_down"] = dy.abs().T @ eh + M(T) * (dy.abs().T @ (h.abs() + eh))
    tol = {k: e * (1 + h_) + h_ * out[k].abs() + tiny for k, e in err.items()}
    m = max(T, D, 2 * F)
    norm = 2 * h_ if dtype != "f32" else 2 * m ** 0.5 * U + 16 * U
    return out, tol, norm


def close(name, got, ref, tol, norm=None):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(((got - ref).abs() / tol).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {got.numel()} off, worst {got.flatten()[i]} vs "
                             f"{ref.flatten()[i]}, allowed {tol.flatten()[i]}")
    if norm is not None and got.numel() >= 64:
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= norm, f"{name}: {rel:.3g} of the norm off, allowed {norm:.3g}"


def run(B, d, act, **kw):
    f = B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], act=act, want_saved=True)
    b = B.gated_ffn_bwd(d["x"], d["wg"], d["wu"], d["wd"], f["saved"], d["dy"], act=act, **kw)
    return {"y": f["y"], **b}


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 8, 8), (1, 64, 264), (5, 16, 24), (16, 64, 72), (31, 72, 136), (32, 520, 264),
          (33, 128, 256), (61, 256, 96), (64, 64, 64), (65, 264, 520), (127, 100, 260), (129, 515, 133), (130, 7, 1030),
          (200, 1024, 24), (257, 64, 2056), (300, 520, 1032), (1000, 40, 200)]


@pytest.mark.parametrize("T,D,F", SHAPES)
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu"), ("f32", "sigmoid"), ("f32", "gelu"),
                                       ("bf16", "sigmoid"), ("f16", "silu")])
def test_ffn(B, T, D, F, dtype, act):
    d = inputs(T, D, F, dtype)
    ref, tol, norm = reference(**d, act=act, dtype=dtype)
    for k, v in run(B, {n: t.cuda() for n, t in d.items()}, act).items():
        assert v.dtype == DT[dtype]
        close(k, v, ref[k], tol[k], norm)


@pytest.mark.parametrize("T,D,F,dtype,act", [
    (2048, 1024, 2048, "bf16", "silu"), (4100, 512, 4096, "f16", "gelu"), (1200, 2048, 5632, "bf16", "sigmoid"),
    (5000, 2048, 2056, "bf16", "gelu"), (700, 1030, 2815, "bf16", "silu"), (1100, 768, 1536, "f32", "silu"),
    (48, 4096, 8192, "bf16", "silu"), (1, 2048, 8192, "f16", "silu"), (128, 2048, 8192, "bf16", "silu")])
def test_ffn_large(B, T, D, F, dtype, act):
    """Every tile and the splits along k, checked on the GPU in 64 bits."""
    d = {n: t.cuda() for n, t in inputs(T, D, F, dtype).items()}
    ref, tol, norm = reference(**d, act=act, dtype=dtype)
    got = run(B, d, act)
    for k, v in got.items():
        close(k, v, ref[k], tol[k], norm)
    again = run(B, d, act)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("T,D,F,dtype", [
    (1, 64, 12288, "bf16"), (17, 8192, 64, "bf16"), (40, 8192, 96, "f16"), (64, 136, 12296, "bf16"), (60, 8200, 1000, "f32"),
    (3, 4096, 5632, "f32"), (50, 4096, 5632, "f32"), (64, 1024, 2816, "bf16"), (32, 512, 1408, "f16")])
def test_ffn_few_tokens(B, T, D, F, dtype):
    """Many splits of either product, few, and none."""
    d = {n: t.cuda() for n, t in inputs(T, D, F, dtype).items()}
    ref, tol, norm = reference(**d, act="silu", dtype=dtype)
    y = B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"])["y"]
    close("y", y, ref["y"], tol["y"], norm)
    assert torch.equal(run(B, d, "silu")["y"], y)


def test_ffn_misaligned_odd_rows(B):
    """Odd widths may begin at any element."""
    for dtype in DT:
        d = inputs(37, 21, 45, dtype)
        want = run(B, {n: t.cuda() for n, t in d.items()}, "silu")
        off = {n: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) for n, t in d.items()}
        got = run(B, off, "silu")
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("D,F", [(64, 45), (21, 64), (64, 1), (1, 64)])
@pytest.mark.parametrize("dtype", DT)
def test_ffn_one_width_odd(B, D, F, dtype):
    """Only rows that need it are copied: the others are read where they lie, with NaN behind the last, or from any element."""
    T = 37
    d = inputs(T, D, F, dtype)
    ref, tol, norm = reference(**d, act="gelu", dtype=dtype)
    for shift in (0, 1):
        big = {n: torch.full((t.numel() + 4096,), float("nan"), dtype=t.dtype, device="cuda") for n, t in d.items()}
        at = {n: big[n][shift:shift + t.numel()].view(t.shape).copy_(t) for n, t in d.items()}
        got = run(B, at, "gelu")
        for k, v in got.items():
            close(k, v, ref[k], tol[k], norm)
        assert torch.equal(B.gated_ffn_fwd(at["x"], at["wg"], at["wu"], at["wd"], act="gelu")["y"], got["y"])


@pytest.mark.parametrize("T,D,F,dtype", [(70, 72, 136, "bf16"), (37, 21, 45, "f16"), (300, 64, 200, "f32")])
def test_ffn_spoilt_tokens(B, T, D, F, dtype):
    """A token with an infinity and one with a NaN: the other tokens' rows keep their bits (no sum
    takes in a row beside it, also where D, F or T end inside a step)."""
    d = {n: t.cuda() for n, t in inputs(T, D, F, dtype).items()}
    want = run(B, d, "silu")
    x, dy = d["x"].clone(), d["dy"].clone()
    x[T // 2, 0], x[T - 1, D - 1] = float("inf"), float("nan")
    dy[1, 0] = float("nan")
    got = run(B, {**d, "x": x, "dy": dy}, "silu")
    ok = [i for i in range(T) if i not in (T // 2, T - 1)]
    assert torch.equal(got["y"][ok], want["y"][ok])
    ok.remove(1)
    assert torch.equal(got["dx"][ok], want["dx"][ok])
    assert torch.isnan(got["y"][T - 1]).all() and torch.isnan(got["dx"][1]).all()


def test_ffn_extreme_gates(B):
    """Gates far from zero on both sides: the functions and their slopes saturate, none gives a NaN."""
    T, D, F = 40, 16, 32
    for dtype in ("f32", "bf16"):
        for act in ("silu", "gelu", "sigmoid"):
            d = inputs(T, D, F, dtype)
            d["wg"] = (d["wg"].float() * 60.0).to(DT[dtype])
            ref, tol, _ = reference(**d, act=act, dtype=dtype)
            for k, v in run(B, {n: t.cuda() for n, t in d.items()}, act).items():
                assert torch.isfinite(v).all()
                close(k, v, ref[k], tol[k])


def test_ffn_no_tokens(B):
    d = {n: t.cuda() for n, t in inputs(3, 40, 72, "bf16").items()}
    e = {**d, "x": d["x"][:0], "dy": d["dy"][:0]}
    f = B.gated_ffn_fwd(e["x"], e["wg"], e["wu"], e["wd"], want_saved=True)
    assert f["y"].shape == (0, 40) and f["saved"].shape == (0, 180)
    out = {k: torch.ones_like(v) for k, v in zip(NAMES, (e["x"], e["wg"], e["wu"], e["wd"]))}
    B.gated_ffn_bwd(e["x"], e["wg"], e["wu"], e["wd"], f["saved"], e["dy"], out=out)
    assert all((out[k] == 0).all() for k in NAMES[1:])


@pytest.mark.parametrize("T,D,F", [(70, 72, 136), (19, 21, 45), (1, 256, 512)])
def test_ffn_writes_only_its_outputs(B, T, D, F):
    """Outputs, saved rows and workspaces of the stated sizes in the middle of larger buffers; skipped gradients."""
    bf = torch.bfloat16
    d = {n: t.cuda() for n, t in inputs(T, D, F, "bf16").items()}
    want = run(B, d, "gelu")
    held = []

    def room(shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        big = torch.full((n + 512 - n % 256,), 0xA5, dtype=torch.uint8, device="cuda")
        held.append((big, n))
        return big[256:256 + n].view(dtype).view(shape)

    def untouched():
        return all((b[:256] == 0xA5).all() and (b[256 + n:] == 0xA5).all() for b, n in held)
    ws = [room((B.ffn_workspace_size(T, D, F, bf, bwd=b),), torch.uint8) for b in (0, 1)]
    f = {"y": room((T, D), bf), "saved": room((T, B.ffn_saved_width(F, bf)), torch.float32)}
    B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], act="gelu", out=f, workspace=ws[0])
    shapes = {"dx": (T, D), "dw_gate": (F, D), "dw_up": (F, D), "dw_down": (D, F)}
    g = {k: room(s, bf) for k, s in shapes.items()}
    B.gated_ffn_bwd(d["x"], d["wg"], d["wu"], d["wd"], f["saved"], d["dy"], act="gelu", out=g, workspace=ws[1])
    assert torch.equal(f["y"], want["y"]) and all(torch.equal(g[k], want[k]) for k in g) and untouched()
    for some in (("dx",), ("dw_down",), ("dw_gate", "dw_up"), ("dx", "dw_down")):
        g = {k: room(shapes[k], bf) for k in some}
        B.gated_ffn_bwd(d["x"], d["wg"], d["wu"], d["wd"], f["saved"], d["dy"], act="gelu", out=g, workspace=ws[1])
        assert all(torch.equal(g[k], want[k]) for k in some) and untouched()
    r = run(B, d, "gelu", want_dw=False)
    assert torch.equal(r["dx"], want["dx"]) and r["dw_gate"] is r["dw_up"] is r["dw_down"] is None


def test_ffn_inference_is_the_same(B):
    """Without the saved rows the output keeps its bits."""
    d = {n: t.cuda() for n, t in inputs(77, 136, 264, "f16").items()}
    a = B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"])
    assert a["saved"] is None
    assert torch.equal(a["y"], B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], want_saved=True)["y"])


def test_ffn_halves_of_one_weight(B):
    """Gate and up as halves of one tensor, x of more dimensions."""
    d = {n: t.cuda() for n, t in inputs(60, 64, 128, "bf16").items()}
    w = torch.cat([d["wg"], d["wu"]])
    y = B.gated_ffn_fwd(d["x"].view(3, 20, 64), w[:128], w[128:], d["wd"])["y"]
    assert torch.equal(y.view(60, 64), B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"])["y"])


def test_ffn_far_offsets(B):
    """Rows beyond 2^32 bytes of the saved gate and up rows (4.6 GB, h behind them) and of dgu."""
    T, D, F = 70000, 64, 8192
    G = torch.Generator(device="cuda").manual_seed(3)

    def r(*s, scale=1.0):
        return (torch.randn(s, generator=G, device="cuda") * scale).bfloat16()
    d = dict(x=r(T, D), wg=r(F, D, scale=0.2), wu=r(F, D, scale=0.125), wd=r(D, F, scale=F ** -0.5), dy=r(T, D))
    got = run(B, d, "silu")
    last = {**d, "x": d["x"][-100:], "dy": d["dy"][-100:]}
    ref, tol, norm = reference(**last, act="silu", dtype="bf16")
    for k in ("y", "dx"):
        close(k, got[k][-100:], ref[k], tol[k], norm)
    want = {k: torch.zeros(got[k].shape, dtype=torch.float64, device="cuda") for k in NAMES[1:]}
    for i in range(0, T, 10000):
        ref, _, _ = reference(**{**d, "x": d["x"][i:i + 10000], "dy": d["dy"][i:i + 10000]}, act="silu", dtype="bf16")
        for k in want:
            want[k] += ref[k]
    for k in want:
        rel = float((got[k].double() - want[k]).norm() / want[k].norm())
        assert rel <= norm, (k, rel)


def test_ffn_gradient_by_differences(B):
    """Each gradient along a direction against central differences of the forward, in fp32.

    The difference over 2 e is off by e^2 / 6 times a third derivative (of order 10 for these inputs, allowed: 200) and by
    the forward's rounding over e: its error bound's share, at most 2 (m + 20) u of the sums' magnitudes, here
    below 300 u of sum |dy y|, on both sides."""
    from chunked_gated_delta_08_amd import autograd as A
    T, D, F = 9, 12, 20
    for act in ("silu", "gelu", "sigmoid"):
        d = {n: t.cuda() for n, t in inputs(T, D, F, "f32", seed=7).items()}
        names = ("x", "wg", "wu", "wd")
        leaves = [d[n].clone().requires_grad_() for n in names]
        y = A.gated_ffn(*leaves, act=act)
        grads = torch.autograd.grad(y, leaves, d["dy"])
        e = 2.0 ** -7
        for i, n in enumerate(names):
            v = rnd(50 + i, *d[n].shape).cuda()
            v = v / v.norm()

            def f(s):
                a = [d[m] + (s * v if m == n else 0) for m in names]
                return float((B.gated_ffn_fwd(*a, act=act)["y"].double() * d["dy"].double()).sum())
            diff = (f(e) - f(-e)) / (2 * e)
            mag = float((y.detach().double() * d["dy"].double()).abs().sum())
            want = float((grads[i].double() * v.double()).sum())
            assert abs(diff - want) <= 200 * e * e / 6 + 300 * U * mag / e + 1e-5 * abs(want), (act, n, diff, want)


def test_ffn_streams(B):
    """A given stream, and two calls at once with workspaces of their own."""
    d = {n: t.cuda() for n, t in inputs(300, 256, 512, "bf16").items()}
    want = run(B, d, "silu")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for st in s:
            f = B.gated_ffn_fwd(d["x"], d["wg"], d["wu"], d["wd"], want_saved=True, stream=st)
            outs.append({"y": f["y"], **B.gated_ffn_bwd(d["x"], d["wg"], d["wu"], d["wd"], f["saved"], d["dy"], stream=st)})
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], want[k]) for k in want)


def _capture(fn):
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
        with torch.cuda.graph(graph, stream=side):
            out = fn()
    torch.cuda.current_stream().wait_stream(side)
    return graph, out


def test_second_half_of_a_layer(B):
    """Norm, feed-forward block and dropped-out residual add as a layer has them, forward and backward, against the
    same in 64 bits with the roundings between the operators."""
    from chunked_gated_delta_08_amd import autograd as A
    T, D, F = 130, 64, 136
    rng = (1234567, 89)
    res, x = rnd(1, T, D).cuda(), rnd(2, T, D).cuda()
    w1, w2 = (1 + 0.1 * rnd(3, D)).cuda(), (1 + 0.1 * rnd(4, D)).cuda()
    wg, wu, wd = (t.cuda() for t in (rnd(5, F, D, scale=0.2), rnd(6, F, D, scale=0.125), rnd(7, D, F, scale=0.1)))
    leaves = [t.clone().requires_grad_() for t in (res, x, w1, w2, wg, wu, wd)]
    dy, dr = rnd(8, T, D).cuda(), rnd(9, T, D).cuda()

    def layer(res, x, w1, w2, wg, wu, wd):
        y, r = A.add_rms_norm(x, res, w1)
        return A.dropout_add_rms_norm(A.gated_ffn(y, wg, wu, wd), r, w2, 0.25, rng)
    y, r = layer(*leaves)
    grads = torch.autograd.grad((y, r), leaves, (dy, dr))
    mask = B.dropout(torch.ones(T, D, device="cuda"), 0.25, rng).double()
    l64 = [t.detach().double().requires_grad_() for t in leaves]

    def norm(h, w):
        return h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w
    r1 = l64[0] + l64[1]
    n1 = norm(r1, l64[2])
    a, _ = act64(n1 @ l64[4].T, "silu")
    r2 = r1 + mask * ((a * (n1 @ l64[5].T)) @ l64[6].T)
    y2 = norm(r2, l64[3])
    g64 = torch.autograd.grad((y2, r2), l64, (dy.double(), dr.double()))
    # fp32 throughout: some five operators of sums of up to 272 terms, each off by at most 2 sqrt(m) u + 16 u of the norm
    lim = 5 * (2 * 272 ** 0.5 + 16) * U
    for name, got, ref in (("y", y, y2), ("res", r, r2), *((str(i), g, h) for i, (g, h) in enumerate(zip(grads, g64)))):
        ref = ref.detach()
        rel = float((got.detach().double() - ref).norm() / ref.norm())
        assert rel <= lim, (name, rel, lim)


def test_captured_training_step_of_the_second_half(B):
    """The same captured: every replay takes the inputs and the generator's numbers that it finds."""
    from chunked_gated_delta_08_amd import autograd as A
    T, D, F = 70, 64, 136
    bf = torch.bfloat16
    leaves = [t.cuda().to(bf if i not in (2,) else torch.float32).requires_grad_() for i, t in enumerate(
        (rnd(1, T, D), rnd(2, T, D), 1 + 0.1 * rnd(3, D), rnd(5, F, D, scale=0.2), rnd(6, F, D, scale=0.125),
         rnd(7, D, F, scale=0.1)))]
    dy = rnd(8, T, D).cuda().to(bf)
    rng = torch.tensor([77, 5], dtype=torch.int64, device="cuda")

    def step():
        y, r = A.dropout_add_rms_norm(A.gated_ffn(leaves[0], *leaves[3:], act="gelu"), leaves[1], leaves[2], 0.3, rng)
        return (y.detach(), r.detach()) + torch.autograd.grad((y, r), leaves, (dy, dy))
    graph, out = _capture(step)
    seen = []
    for i in range(4):
        with torch.no_grad():
            leaves[0].copy_(rnd(30 + i, T, D))
            rng[1] = 100 + i
        torch.randn(500, 500, device="cuda") @ torch.randn(500, 500, device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del want
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_ffn_autograd(B):
    """Gradients for what needs them only, none kept without gradients, second derivatives refused."""
    from chunked_gated_delta_08_amd import autograd as A
    d = {n: t.cuda() for n, t in inputs(20, 24, 40, "f32").items()}
    want = run(B, d, "silu")
    x, wg, wu, wd = (d[n].clone() for n in ("x", "wg", "wu", "wd"))
    wd.requires_grad_()
    y = A.gated_ffn(x, wg, wu, wd)
    y.backward(d["dy"])
    assert torch.equal(y, want["y"]) and torch.equal(wd.grad, want["dw_down"]) and x.grad is None
    with torch.no_grad():
        assert not A.gated_ffn(x, wg, wu, wd).requires_grad
    assert torch.equal(A.gated_ffn(x.t().contiguous().t(), wg, wu, wd).detach(), want["y"])   # any strides
    off = torch.empty(x.numel() + 1, device="cuda")[1:].view(x.shape).copy_(x)   # or place
    with pytest.raises(ValueError, match="x must be aligned"):
        B.gated_ffn_fwd(off, wg, wu, d["wd"])
    assert torch.equal(A.gated_ffn(off, wg, wu, wd).detach(), want["y"])
    x.requires_grad_()
    g, = torch.autograd.grad(A.gated_ffn(x, wg, wu, wd).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.square().sum(), x)
