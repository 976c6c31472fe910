"""Cases of the operators around the gated delta rule in a layer: the gated RMSNorm
after the mixer, the residual add with the RMSNorm before the next block, the
gated linear recurrence, and the single-token steps of serving.

A case names its operator and sizes; `run` computes it in plain torch operations
(32 bits, rounded once at the end) or, with `own`, with this repository's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5

# the twelve sequences of the repository's varlen workload (65536 tokens)
VARLEN12 = "7497,540,4615,9439,6283,861,8476,8109,9326,2340,1441,6609"


def listed():
    return [
        # the output norm of a decode step: 8 tokens, 16 heads (latency)
        dict(name="gated_norm_decode", op="gated_norm_fwd", rows=8 * 16, D=128, dtype="bf16", act="silu"),
        # the output norm of the dense training and prefill workload
        dict(name="gated_norm_t32k", op="gated_norm_fwd", rows=32768 * 16, D=128, dtype="bf16", act="silu"),
        # its backward at the varlen grouped-head workload, 32 value heads
        dict(name="gated_norm_bwd_t64k", op="gated_norm_bwd", rows=65536 * 32, D=128, dtype="bf16", act="silu"),
        # residual add and pre-norm of a decode step, odd token count, fp32 residual stream (latency)
        dict(name="add_norm_decode", op="add_norm_fwd", rows=5, D=2048, dtype="bf16", res="f32", scale=True),
        # the same for a prefill of the dense workload's width (16 heads x 128)
        dict(name="add_norm_t32k", op="add_norm_fwd", rows=32768, D=2048, dtype="bf16", res="bf16", scale=True),
        # training backward at the widest model (32 heads x 128), fp16
        dict(name="add_norm_bwd_t16k", op="add_norm_bwd", rows=16384, D=4096, dtype="f16", res="f16", scale=True),
        # one long sequence, 2048 channels: prefill
        dict(name="glr_t32k", op="glr_fwd", lens="32768", D=2048, dtype="bf16", h0=False),
        # a training step over ragged sequences packed without padding
        dict(name="glr_train_varlen", op="glr_train", lens=VARLEN12, D=2048, dtype="bf16", h0=True),
        # odd sizes, fp32, a batch that goes on from given states
        dict(name="glr_odd", op="glr_fwd", lens="1531,1531,1531", D=515, dtype="f32", h0=True),
        # one token for each of 64 sequences, states in a pool (latency)
        dict(name="glr_step_n64", op="glr_step", N=61, pad=3, slots=96, D=2048, dtype="bf16"),
        # one sequence decoding (latency)
        dict(name="gdr_step_n1", op="gdr_step", N=1, pad=0, slots=4, HK=16, HV=16, K=128, dtype="bf16"),
        # a full serving batch, grouped heads, three padding rows
        dict(name="gdr_step_n256", op="gdr_step", N=253, pad=3, slots=288, HK=16, HV=32, K=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_norm_fwd", "gated_norm_bwd", "add_norm_fwd", "add_norm_bwd", "glr_fwd", "glr_train",
                     "glr_step", "gdr_step"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("gated_norm"):
        D = rng.choice([64, 128, 128, 256, _log(rng, 3, 512)])
        return dict(op=op, rows=_log(rng, 1, (1 << 27) // D), D=D, dtype=dt, act=rng.choice(["silu", "sigmoid", "none"]))
    if op.startswith("add_norm"):
        D = rng.choice([1024, 2048, 4096, _log(rng, 5, 8192)])
        return dict(op=op, rows=_log(rng, 1, (1 << 26) // D), D=D, dtype=dt, res=rng.choice([dt, "f32"]),
                    scale=rng.random() < 0.5)
    if op in ("glr_fwd", "glr_train"):
        D = rng.choice([512, 1024, 2048, _log(rng, 1, 4096)])
        n = rng.choice([1, 1, 2, _log(rng, 1, 40)])
        top = max(1, min(32768, (1 << 26) // (D * n)))
        if rng.random() < 0.5:
            lens = [_log(rng, 1, top)] * n
        else:   # packed sequences, an empty one among them now and then
            lens = [0 if n > 2 and rng.random() < 0.1 else _log(rng, 1, top) for _ in range(n - 1)] + [_log(rng, 1, top)]
        return dict(op=op, lens=",".join(map(str, lens)), D=D, dtype=dt, h0=rng.random() < 0.5)
    N, pad = _log(rng, 1, 300), rng.choice([0, 0, 1, 5])
    slots = N + rng.randint(0, 40)
    if op == "glr_step":
        return dict(op=op, N=N, pad=pad, slots=slots, D=rng.choice([512, 2048, 4096, _log(rng, 1, 8192)]), dtype=dt)
    K, HK = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16])
    return dict(op=op, N=min(N, 200), pad=pad, slots=slots, HK=HK, HV=HK * rng.choice([1, 2]), K=K, dtype=dt)


def work(c):
    op, e = c["op"], SIZE[c["dtype"]]
    if op.startswith("gated_norm"):
        n, z = c["rows"] * c["D"], 0 if c["act"] == "none" else 1
        if op.endswith("fwd"):
            return {"bytes": n * e * (2 + z) + 4 * c["D"], "flops": n * (4 + 4 * z)}
        return {"bytes": n * e * (3 + 2 * z) + 8 * c["D"], "flops": n * (10 + 10 * z)}
    if op.startswith("add_norm"):
        n, r, s = c["rows"] * c["D"], SIZE[c["res"]], 1 if c["scale"] else 0
        if op.endswith("fwd"):   # reads x, res; writes res, y
            return {"bytes": n * (2 * e + 2 * r) + 4 * c["D"] * (1 + s), "flops": 6 * n}
        # reads dy, dres, res (and x for the scale's gradient); writes dres, and dx where it is not dres itself
        dx = 0 if (not s and e == r) else e
        return {"bytes": n * (e + 3 * r + s * e + dx) + 8 * c["D"] * (1 + s), "flops": 14 * n}
    if op in ("glr_fwd", "glr_train"):
        lens = [int(v) for v in c["lens"].split(",")]
        n, st = sum(lens) * c["D"], len(lens) * c["D"] * 4
        fwd = n * (2 * e + 4) + st * (2 if c["h0"] else 1)
        if op == "glr_fwd":
            return {"bytes": fwd, "flops": 3 * n}
        return {"bytes": fwd + n * (3 * e + 8) + st * (3 if c["h0"] else 2), "flops": 10 * n}
    if op == "glr_step":
        return {"bytes": c["N"] * c["D"] * (8 + 2 * e + 4), "flops": 3 * c["N"] * c["D"]}
    s = c["N"] * c["HV"] * c["K"] * c["K"]
    io = c["N"] * (2 * c["HK"] * c["K"] + 2 * c["HV"] * c["K"]) * e
    return {"bytes": 8 * s + io, "flops": 8 * s}


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    G = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DT[c["dtype"]], c["op"]

    def randn(*shape):
        return torch.randn(shape, generator=G, device="cuda", dtype=torch.float32)

    s = {"c": c}
    if op.startswith("gated_norm"):
        R, D = c["rows"], c["D"]
        # the mixer's outputs: rows of very different sizes
        s["x"] = (randn(R, D) * torch.exp(randn(R, 1) - 1.0)).to(dt)
        s["z"] = None if c["act"] == "none" else randn(R, D).to(dt)
        s["w"] = 1.0 + 0.1 * randn(D)
        s["dy"] = randn(R, D).to(dt) if op.endswith("bwd") else None
    elif op.startswith("add_norm"):
        R, D, rt = c["rows"], c["D"], DT[c["res"]]
        s["x"] = randn(R, D).to(dt)
        s["res"] = (2.0 * randn(R, D)).to(rt)
        s["w"] = 1.0 + 0.1 * randn(D)
        s["scale"] = 0.5 + 0.1 * randn(D) if c["scale"] else None
        if op.endswith("bwd"):
            s["dy"] = randn(R, D).to(dt)
            s["dres"] = randn(R, D).to(rt)
    elif op in ("glr_fwd", "glr_train"):
        lens = [int(v) for v in c["lens"].split(",")]
        T, N, D = sum(lens), len(lens), c["D"]
        s["x"] = randn(T, D).to(dt)
        # time constants from a few to a thousand tokens, each token's gate its own
        rate = torch.exp(torch.rand(D, generator=G, device="cuda") * 5.5 - 6.5)
        s["g"] = -rate * 2.0 * torch.sigmoid(randn(T, D))
        s["h0"] = randn(N, D) if c["h0"] else None
        s["B"], s["cu"], s["cu_host"] = N, None, None
        if len(set(lens)) > 1:
            s["B"] = 1
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu_host"] = torch.tensor(cu, dtype=torch.int32)
            s["cu"] = s["cu_host"].cuda()
        s["lens"] = lens
        if op == "glr_train":
            s["dh"] = randn(T, D).to(dt)
            s["dht"] = randn(N, D)
    else:
        N, pad, S = c["N"], c["pad"], c["slots"]
        order = torch.randperm(S, generator=G, device="cuda")[:N].to(torch.int32)
        s["slots"] = torch.cat([order, torch.full((pad,), -1, dtype=torch.int32, device="cuda")])
        if op == "glr_step":
            D = c["D"]
            s["x"] = randn(N + pad, D).to(dt)
            s["g"] = -torch.sigmoid(randn(N + pad, D))
            s["state"] = randn(S, D)
        else:
            HK, HV, K = c["HK"], c["HV"], c["K"]
            q, k = randn(N + pad, HK, K), randn(N + pad, HK, K)
            s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)
            s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
            s["v"] = randn(N + pad, HV, K).to(dt)
            s["g"] = torch.nn.functional.logsigmoid(randn(N + pad, HV))
            s["beta"] = torch.sigmoid(randn(N + pad, HV)).to(dt)
            s["state"] = randn(S, HV, K, K)
    return s


# ------------------------------------------------------------- plain forms

def _gated_norm_fwd(s):
    x = s["x"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        y = y * (z * sg if s["c"]["act"] == "silu" else sg)
    return y.to(s["x"].dtype)


def _gated_norm_bwd(s):
    x, dy, w, dt = s["x"].float(), s["dy"].float(), s["w"], s["x"].dtype
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        if s["c"]["act"] == "silu":
            act, der = z * sg, sg * (1.0 + z * (1.0 - sg))
        else:
            act, der = sg, sg * (1.0 - sg)
        dz = (dy * n * w * der).to(dt)
        dy = dy * act
    dw = (dy * n).sum(0)
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": dx.to(dt), "dz": dz, "dw": dw}


def _add_norm_fwd(s):
    x = s["x"].float()
    h = s["res"].float() + (x if s["scale"] is None else x * s["scale"])
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    return {"y": y.to(s["x"].dtype), "res": h.to(s["res"].dtype)}


def _add_norm_bwd(s):
    h, dy = s["res"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    dn = dy * s["w"]
    dh = s["dres"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    out = {"dw": (dy * n).sum(0), "dres": dh.to(s["res"].dtype)}
    if s["scale"] is None:
        out["dx"], out["dscale"] = dh.to(s["x"].dtype), None
    else:
        out["dx"] = (dh * s["scale"]).to(s["x"].dtype)
        out["dscale"] = (dh * s["x"].float()).sum(0)
    return out


def _bounds(s):
    """First and last token of every sequence that has one, and its index."""
    ends = torch.tensor(s["lens"]).cumsum(0)
    some = torch.tensor(s["lens"]) > 0
    first, last = (ends - torch.tensor(s["lens"]))[some], (ends - 1)[some]
    return first.cuda(), last.cuda(), some.nonzero()[:, 0].cuda()


def _scan(a, b, steps):
    """h_t = a_t h_(t-1) + b_t down the first axis, by doubling (a_t = 0 where a sequence begins)."""
    d = 1
    while d < steps:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _glr_parts(s):
    first, last, which = _bounds(s)
    a, b = torch.exp(s["g"]), s["x"].float()
    if s["h0"] is not None:
        b = b.index_add(0, first, a[first] * s["h0"][which])
    a0 = a.index_fill(0, first, 0.0)
    h = _scan(a0, b, max(s["lens"]))
    ht = torch.zeros(len(s["lens"]), h.shape[1], device=h.device) if s["h0"] is None else s["h0"].clone()
    ht[which] = h[last]
    return first, last, which, a, a0, h, ht


def _glr_fwd(s):
    _, _, _, _, _, h, ht = _glr_parts(s)
    return {"h": h.to(s["x"].dtype), "ht": ht}


def _glr_train(s):
    first, last, which, a, a0, h, ht = _glr_parts(s)
    b = s["dh"].float().index_add(0, last, s["dht"][which])
    after = torch.cat([a0[1:], torch.zeros_like(a0[:1])])     # the gate that the next token puts on this one's state
    dx = _scan(after.flip(0), b.flip(0), max(s["lens"])).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0.0 if s["h0"] is None else s["h0"][which]
    dh0 = s["dht"].clone()
    dh0[which] = a[first] * dx[first]
    return {"h": h.to(s["x"].dtype), "ht": ht, "dx": dx.to(s["x"].dtype), "dg": dx * a * before,
            "dh0": None if s["h0"] is None else dh0}


def _glr_step(s):
    live = (s["slots"] >= 0)[:, None]
    at = s["slots"].clamp(min=0).long()
    h = torch.exp(s["g"]) * s["state"][at] + s["x"].float()
    n = s["c"]["N"]
    s["state"].index_copy_(0, at[:n], h[:n])
    return {"h": torch.where(live, h, 0.0).to(s["x"].dtype), "state": s["state"]}


def _gdr_step(s):
    c = s["c"]
    n, G = c["N"], c["HV"] // c["HK"]
    at = s["slots"][:n].long()
    q, k = (s[i][:n].float().repeat_interleave(G, dim=1) for i in ("q", "k"))
    S = s["state"][at] * torch.exp(s["g"][:n])[:, :, None, None]
    u = (S * k[..., None]).sum(2)
    d = s["beta"][:n].float()[..., None] * (s["v"][:n].float() - u)
    S = S + k[..., None] * d[:, :, None, :]
    o = torch.zeros(s["v"].shape, device="cuda")
    o[:n] = (S * q[..., None]).sum(2) / math.sqrt(c["K"])
    s["state"].index_copy_(0, at, S)
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


# ------------------------------------------------------------------- a pass

def _own(s):
    from chunked_gated_delta_08_amd import binding as L
    c = s["c"]
    op = c["op"]
    if op.startswith("gated_norm"):
        act = "silu" if c["act"] == "none" else c["act"]
        if op.endswith("fwd"):
            return L.gated_norm_fwd(s["x"], s["z"], s["w"], eps=EPS, act=act)
        return L.gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], eps=EPS, act=act)
    if op == "add_norm_fwd":
        return L.add_norm_fwd(s["x"], s["res"], s["w"], scale=s["scale"], eps=EPS)
    if op == "add_norm_bwd":
        return L.add_norm_bwd(s["dy"], s["dres"], s["res"], s["w"], x=None if s["scale"] is None else s["x"],
                              scale=s["scale"], eps=EPS)
    if op == "glr_step":
        return {"h": L.glr_step(s["x"], s["g"], s["state"], slots=s["slots"]), "state": s["state"]}
    if op == "gdr_step":
        return {"o": L.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"]),
                "state": s["state"]}
    seq = dict(h0=s["h0"], cu_seqlens=s["cu"], cu_seqlens_host=s["cu_host"], B=s["B"])
    if op == "glr_fwd":
        r = L.glr_fwd(s["x"], s["g"], **seq)
        return {"h": r["h"], "ht": r["ht"]}
    f = L.glr_fwd(s["x"], s["g"], want_states=True, **seq)
    b = L.glr_bwd(s["x"], s["g"], s["dh"], f["states"], dht=s["dht"], want_dh0=s["h0"] is not None, **seq)
    return {"h": f["h"], "ht": f["ht"], "dx": b["dx"], "dg": b["dg"], "dh0": b["dh0"]}


PLAIN = {"gated_norm_fwd": _gated_norm_fwd, "gated_norm_bwd": _gated_norm_bwd, "add_norm_fwd": _add_norm_fwd,
         "add_norm_bwd": _add_norm_bwd, "glr_fwd": _glr_fwd, "glr_train": _glr_train, "glr_step": _glr_step,
         "gdr_step": _gdr_step}


def run(s):
    return _own(s) if own else PLAIN[s["c"]["op"]](s)


# ------------------------------------------- the definitions, in 64 bits

def _act64(z, act):
    return {"silu": lambda: z / (1.0 + torch.exp(-z)), "sigmoid": lambda: 1.0 / (1.0 + torch.exp(-z)),
            "none": lambda: 1.0}[act]()


def _norm64(x, w):
    return x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS) * w


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()
         and op not in ("glr_fwd", "glr_train")}
    if op == "gated_norm_fwd":
        return _norm64(f["x"], f["w"]) * _act64(f.get("z"), c["act"])
    if op == "gated_norm_bwd":   # by differentiation, a slab of rows at a time
        w, out = f["w"].requires_grad_(), {"dx": [], "dz": [], "dw": torch.zeros_like(f["w"])}
        for i in range(0, c["rows"], 1 << 18):
            x = f["x"][i:i + (1 << 18)].requires_grad_()
            z = None if c["act"] == "none" else f["z"][i:i + (1 << 18)].requires_grad_()
            y = (_norm64(x, w) * _act64(z, c["act"]) * f["dy"][i:i + (1 << 18)]).sum()
            g = torch.autograd.grad(y, [x, w] + ([] if z is None else [z]))
            out["dx"].append(g[0])
            out["dw"] += g[1]
            out["dz"] += list(g[2:])
        return {"dx": torch.cat(out["dx"]), "dz": torch.cat(out["dz"]) if out["dz"] else None, "dw": out["dw"]}
    if op == "add_norm_fwd":
        h = f["res"] + f["x"] * f.get("scale", 1.0)
        return {"y": _norm64(h, f["w"]), "res": h}
    if op == "add_norm_bwd":     # the stored sum is res = base + scale x: differentiate through it
        x, w = f["x"].requires_grad_(), f["w"].requires_grad_()
        sc = f.get("scale", torch.ones_like(w)).requires_grad_()
        h = f["res"] + (x * sc - (x * sc).detach())
        h.retain_grad()
        ((_norm64(h, w) * f["dy"]).sum() + (h * f["dres"]).sum()).backward()
        return {"dw": w.grad, "dres": h.grad, "dx": x.grad, "dscale": sc.grad if c["scale"] else None}
    if op == "glr_step":
        h, st = torch.zeros_like(f["x"]), f["state"]
        at = s["slots"].tolist()
        for i in range(c["N"]):
            st[at[i]] = h[i] = st[at[i]] * torch.exp(f["g"][i]) + f["x"][i]
        return {"h": h, "state": st}
    if op == "gdr_step":
        o, st = torch.zeros_like(f["v"]), f["state"]
        eye = torch.eye(c["K"], device="cuda", dtype=torch.float64)
        at, G = s["slots"].tolist(), c["HV"] // c["HK"]
        head = torch.arange(c["HV"], device="cuda") // G
        for i in range(c["N"]):
            k, q, b = f["k"][i][head], f["q"][i][head], f["beta"][i][:, None, None]
            kk = k[:, :, None] * k[:, None, :]
            S = torch.exp(f["g"][i])[:, None, None] * torch.matmul(eye - b * kk, st[at[i]])
            S = S + b * k[:, :, None] * f["v"][i][:, None, :]
            st[at[i]] = S
            o[i] = torch.matmul(q[:, None, :], S)[:, 0] * c["K"] ** -0.5
        return {"o": o, "state": st}
    # the recurrence, token after token; about 15 microseconds for each and pass
    lens, D = s["lens"], c["D"]
    x, a = s["x"].double(), torch.exp(s["g"].double())
    h, ht = torch.empty_like(x), torch.zeros(len(lens), D, device="cuda", dtype=torch.float64)
    before = torch.empty_like(x)
    t = 0
    for n, m in enumerate(lens):
        cur = torch.zeros_like(ht[0]) if s["h0"] is None else s["h0"][n].double()
        for t in range(t, t + m):
            before[t] = cur
            cur = torch.addcmul(x[t], a[t], cur, out=h[t])
        t += 1 if m else 0
        ht[n] = cur
    if op == "glr_fwd":
        return {"h": h, "ht": ht}
    dx, dh0 = s["dh"].double(), torch.empty_like(ht)
    end = sum(lens)
    for n in range(len(lens) - 1, -1, -1):
        lam = s["dht"][n].double()
        for t in range(end - 1, end - 1 - lens[n], -1):
            lam = dx[t].add_(lam) * a[t]
        end -= lens[n]
        dh0[n] = lam
    return {"h": h, "ht": ht, "dx": dx, "dg": dx * a * before, "dh0": None if s["h0"] is None else dh0}
