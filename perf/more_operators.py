"""Cases of the operators that follow the gated delta rule in a layer: the gated
feed-forward block (forward, and a whole training pass), dropout from a
counter-based generator, and the residual add with RMSNorm whose branch is
dropped out (forward, backward).

A case names its operator and sizes; `run` computes it in plain torch operations
(32 bits, rounded once at the end) or, with `own`, with this repository's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one sequence decoding, the width of 16 heads of 128 (latency; the weights are read once)
        dict(name="ffn_decode_t1", op="ffn_fwd", T=1, D=2048, F=8192, dtype="bf16", act="silu"),
        # a serving batch of odd size at the widest model (32 heads of 128)
        dict(name="ffn_decode_t61", op="ffn_fwd", T=61, D=4096, F=12288, dtype="bf16", act="silu"),
        # prefill at the widest model
        dict(name="ffn_prefill_t8k", op="ffn_fwd", T=8192, D=4096, F=12288, dtype="bf16", act="silu"),
        # a training step's forward and backward, the width of the dense workload
        dict(name="ffn_train_t16k", op="ffn_train", T=16384, D=2048, F=8192, dtype="bf16", act="silu"),
        # few tokens, odd sizes of everything, fp16
        dict(name="ffn_train_odd", op="ffn_train", T=1531, D=515, F=1373, dtype="f16", act="gelu"),
        # full precision
        dict(name="ffn_train_f32", op="ffn_train", T=1000, D=1024, F=2816, dtype="f32", act="sigmoid"),
        # a short training micro-batch with an fp32 residual stream (latency)
        dict(name="drop_add_norm_n300", op="drop_add_norm_fwd", rows=300, D=2048, dtype="bf16", res="f32", scale=False, p=0.1),
        # the dense training workload's tokens and width
        dict(name="drop_add_norm_t32k", op="drop_add_norm_fwd", rows=32768, D=2048, dtype="bf16", res="bf16", scale=True, p=0.1),
        # odd rows, backward, fp32
        dict(name="drop_add_norm_bwd_odd", op="drop_add_norm_bwd", rows=1531, D=515, dtype="f32", res="f32", scale=False, p=0.5),
        # training backward at the widest model, fp16
        dict(name="drop_add_norm_bwd_t16k", op="drop_add_norm_bwd", rows=16384, D=4096, dtype="f16", res="f16", scale=True, p=0.1),
        # embeddings of a short batch, odd rows (latency)
        dict(name="dropout_odd", op="dropout", rows=97, D=1029, dtype="f32", p=0.2),
        # embeddings of the dense training workload
        dict(name="dropout_t32k", op="dropout", rows=32768, D=2048, dtype="bf16", p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_train", "ffn_train", "drop_add_norm_fwd", "drop_add_norm_bwd", "dropout"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("ffn"):
        D = rng.choice([512, 1024, 2048, 4096, _log(rng, 8, 4096)])
        F = rng.choice([1408, 2816, 5632, 8192, _log(rng, 8, 12288)])
        most = (1 << 38 if op == "ffn_train" else 1 << 39) >> (3 if dt == "f32" else 0)
        return dict(op=op, T=_log(rng, 1, max(1, min(16384, most // (D * F)))), D=D, F=F, dtype=dt,
                    act=rng.choice(["silu", "silu", "gelu", "sigmoid"]))
    p = rng.choice([0.1, 0.1, 0.5, round(rng.random(), 3)])
    if op == "dropout":
        D = rng.choice([1024, 2048, 4096, _log(rng, 1, 20000)])
        return dict(op=op, rows=_log(rng, 1, (1 << 26) // D), D=D, dtype=dt, p=p)
    D = rng.choice([1024, 2048, 4096, _log(rng, 5, 8192)])
    return dict(op=op, rows=_log(rng, 1, (1 << 26) // D), D=D, dtype=dt, res=rng.choice([dt, "f32"]),
                scale=rng.random() < 0.5, p=p)


def work(c):
    e = SIZE[c["dtype"]]
    if c["op"].startswith("ffn"):
        T, D, F = c["T"], c["D"], c["F"]
        w = 3 * D * F
        if c["op"] == "ffn_fwd":     # x, y and the three weights
            return {"bytes": e * (2 * T * D + w), "flops": 6 * T * D * F}
        return {"bytes": e * (4 * T * D + 2 * w), "flops": 18 * T * D * F}   # x, dy; y, dx; weights and their gradients
    n = c["rows"] * c["D"]
    if c["op"] == "dropout":
        return {"bytes": 2 * e * n, "flops": 2 * n}
    r, s = SIZE[c["res"]], 1 if c["scale"] else 0
    if c["op"] == "drop_add_norm_fwd":   # reads x, res; writes res, y
        return {"bytes": n * (2 * e + 2 * r) + 4 * c["D"] * (1 + s), "flops": 8 * n}
    # reads dy, dres, res (and x for the scale's gradient); writes dres, dx
    return {"bytes": n * ((2 + s) * e + 3 * r) + 8 * c["D"] * (1 + s), "flops": 16 * n}


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    G = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=G, device="cuda", dtype=torch.float32)

    s = {"c": c}
    if c["op"].startswith("ffn"):
        T, D, F = c["T"], c["D"], c["F"]
        s["x"] = randn(T, D).to(dt)          # normed activations
        s["wg"] = (randn(F, D) * (1.5 / math.sqrt(D))).to(dt)
        s["wu"] = (randn(F, D) / math.sqrt(D)).to(dt)
        s["wd"] = (randn(D, F) / math.sqrt(F)).to(dt)
        if c["op"] == "ffn_train":
            s["dy"] = randn(T, D).to(dt)
        return s
    R, D = c["rows"], c["D"]
    s["x"] = randn(R, D).to(dt)
    # the generator's seed and the call's own offset, as a program that counts its calls keeps them
    s["rng"] = (0x9E3779B97F4A7C15 ^ (seed * 0x2545F491), 7 * seed + (1 << 33))
    if c["op"] != "dropout":
        rt = DT[c["res"]]
        s["res"] = (2.0 * randn(R, D)).to(rt)
        s["w"] = 1.0 + 0.1 * randn(D)
        s["scale"] = 0.5 + 0.1 * randn(D) if c["scale"] else None
        if c["op"].endswith("bwd"):
            s["dy"] = randn(R, D).to(dt)
            s["dres"] = randn(R, D).to(rt)
    return s


# ------------------------------------------------------------- plain forms

def _act(g, act):
    """act(g) and its derivative."""
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    sg = torch.sigmoid(g)
    if act == "silu":
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    return sg, sg * (1.0 - sg)


def _ffn_fwd(s):
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    a, _ = _act(x @ wg.t(), s["c"]["act"])
    return ((a * (x @ wu.t())) @ wd.t()).to(s["x"].dtype)


def _ffn_train(s):
    dt = s["x"].dtype
    x, wg, wu, wd, dy = (s[k].float() for k in ("x", "wg", "wu", "wd", "dy"))
    u = x @ wu.t()
    a, da = _act(x @ wg.t(), s["c"]["act"])
    h = a * u
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"y": (h @ wd.t()).to(dt), "dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt),
            "dw_up": (du.t() @ x).to(dt), "dw_down": (dy.t() @ h).to(dt)}


def _keep(shape, p, rng):
    """The elements that stay, and what they are multiplied by: 10 rounds of Philox 4x32 (Salmon et
    al. 2011) for every 8 elements of a row, 16 bits an element."""
    R, D = shape
    M = 0xFFFFFFFF
    n = R * -(-D // 8)
    i = torch.arange(n, device="cuda")
    k0, k1 = rng[0] & M, rng[0] >> 32 & M
    c0, c1 = i & M, i >> 32
    c2 = torch.full_like(i, rng[1] & M)
    c3 = torch.full_like(i, rng[1] >> 32 & M)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # 64 bits, modulo 2^64
        c0, c1, c2, c3 = (b >> 32 & M) ^ c1 ^ k0, b & M, (a >> 32 & M) ^ c3 ^ k1, a & M
        k0, k1 = k0 + 0x9E3779B9 & M, k1 + 0xBB67AE85 & M
    w = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1)
    t = math.floor(p * 65536 + 0.5)
    return w.view(R, -1)[:, :D] >= t, 65536 / (65536 - t) if t < 65536 else 0.0


def _dropout(s):
    keep, m = _keep(s["x"].shape, s["c"]["p"], s["rng"])
    return torch.where(keep, s["x"].float() * m, 0.0).to(s["x"].dtype)


def _drop_add_norm_fwd(s):
    keep, m = _keep(s["x"].shape, s["c"]["p"], s["rng"])
    x = torch.where(keep, s["x"].float() * m, 0.0)
    h = s["res"].float() + (x if s["scale"] is None else x * s["scale"])
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    return {"y": y.to(s["x"].dtype), "res": h.to(s["res"].dtype)}


def _drop_add_norm_bwd(s):
    keep, m = _keep(s["res"].shape, s["c"]["p"], s["rng"])
    h, dy = s["res"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    dn = dy * s["w"]
    dh = s["dres"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    out = {"dw": (dy * n).sum(0), "dres": dh.to(s["res"].dtype), "dscale": None}
    dx = torch.where(keep, dh * m, 0.0)
    if s["scale"] is not None:
        out["dscale"] = (dx * s["x"].float()).sum(0)
        dx = dx * s["scale"]
    out["dx"] = dx.to(s["x"].dtype)
    return out


# ------------------------------------------------------------------- a pass

def _own(s):
    from chunked_gated_delta_08_amd import binding as L
    c = s["c"]
    op = c["op"]
    if op == "ffn_fwd":
        return L.gated_ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], act=c["act"])["y"]
    if op == "ffn_train":
        f = L.gated_ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], act=c["act"], want_saved=True)
        b = L.gated_ffn_bwd(s["x"], s["wg"], s["wu"], s["wd"], f["saved"], s["dy"], act=c["act"])
        return {"y": f["y"], **{k: b[k] for k in ("dx", "dw_gate", "dw_up", "dw_down")}}
    if op == "dropout":
        return L.dropout(s["x"], c["p"], s["rng"])
    if op == "drop_add_norm_fwd":
        r = L.dropout_add_norm_fwd(s["x"], s["res"], s["w"], c["p"], s["rng"], scale=s["scale"], eps=EPS)
        return {"y": r["y"], "res": r["res"]}
    r = L.dropout_add_norm_bwd(s["dy"], s["dres"], s["res"], s["w"], c["p"], s["rng"],
                               x=None if s["scale"] is None else s["x"], scale=s["scale"], eps=EPS)
    return {k: r[k] for k in ("dw", "dres", "dscale", "dx")}


PLAIN = {"ffn_fwd": _ffn_fwd, "ffn_train": _ffn_train, "dropout": _dropout, "drop_add_norm_fwd": _drop_add_norm_fwd,
         "drop_add_norm_bwd": _drop_add_norm_bwd}


def run(s):
    return _own(s) if own else PLAIN[s["c"]["op"]](s)


# ------------------------------------------- the definitions, in 64 bits

def _act64(g, act):
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    return (g if act == "silu" else 1.0) / (1.0 + torch.exp(-g))


def _mask64(R, D, p, rng):
    """The mask times 1 / (1 - p), p in steps of 2^-16; the products of 32 bits from halves of 16."""
    groups = -(-D // 8)
    m32 = (1 << 32) - 1

    def times(k, v):
        """High and low 32 bits of k v."""
        lo, hi = (k & 0xFFFF) * (v & 0xFFFF), (k >> 16) * (v >> 16)
        mid1, mid2 = (k & 0xFFFF) * (v >> 16), (k >> 16) * (v & 0xFFFF)
        mid = (lo >> 16) + (mid1 & 0xFFFF) + (mid2 & 0xFFFF)
        return hi + (mid1 >> 16) + (mid2 >> 16) + (mid >> 16), (mid & 0xFFFF) << 16 | lo & 0xFFFF

    index = (torch.arange(R, device="cuda")[:, None] * groups + torch.arange(groups, device="cuda")[None]).reshape(-1)
    ctr = [index % (1 << 32), index // (1 << 32), torch.tensor(rng[1] % (1 << 32), device="cuda"),
           torch.tensor(rng[1] // (1 << 32) % (1 << 32), device="cuda")]
    for i in range(10):
        key = [(rng[0] + i * 0x9E3779B9) & m32, ((rng[0] >> 32) + i * 0xBB67AE85) & m32]
        h0, l0 = times(0xD2511F53, ctr[0])
        h1, l1 = times(0xCD9E8D57, ctr[2])
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    bits = torch.empty(R, groups, 8, device="cuda", dtype=torch.int64)
    for e in range(8):
        bits[..., e] = (ctr[e // 2] // (1 << 16 * (e % 2)) % (1 << 16)).view(R, groups)
    drop = int(p * 65536 + 0.5)
    keep = (bits.view(R, groups * 8)[:, :D] >= drop).double()
    return keep / (1.0 - drop / 65536.0) if drop < 65536 else keep


def exact(c, seed):
    s = prepare(c, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if c["op"].startswith("ffn"):
        leaves = [f[k].requires_grad_(c["op"] == "ffn_train") for k in ("x", "wg", "wu", "wd")]
        x, wg, wu, wd = leaves
        y = torch.matmul(_act64(torch.matmul(x, wg.T), c["act"]) * torch.matmul(x, wu.T), wd.T)
        if c["op"] == "ffn_fwd":
            return y
        g = torch.autograd.grad(y, leaves, f["dy"])
        return {"y": y.detach(), "dx": g[0], "dw_gate": g[1], "dw_up": g[2], "dw_down": g[3]}
    m = _mask64(c["rows"], c["D"], c["p"], s["rng"])
    if c["op"] == "dropout":
        return f["x"] * m
    x, w = f["x"].requires_grad_(), f["w"].requires_grad_()
    sc = f.get("scale", torch.ones_like(w)).detach().requires_grad_()
    b = x * m * sc
    # the backward is taken at the stored sum
    h = f["res"] + (b if c["op"].endswith("fwd") else b - b.detach())
    y = h / torch.sqrt(torch.sum(h * h, -1, keepdim=True) / c["D"] + EPS) * w
    if c["op"].endswith("fwd"):
        return {"y": y.detach(), "res": h.detach()}
    h.retain_grad()
    ((y * f["dy"]).sum() + (h * f["dres"]).sum()).backward()
    return {"dw": w.grad, "dres": h.grad, "dscale": sc.grad if c["scale"] else None, "dx": x.grad}
