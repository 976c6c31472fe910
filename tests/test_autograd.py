"""CPU tests of the autograd wrappers: second derivatives raise, first ones are what
the binding gives, whether or not create_graph is set.  The binding's calls are
replaced by stand-ins that return constants of the right shapes."""
import pytest
import torch

Z = torch.zeros


@pytest.fixture
def A(monkeypatch):
    from chunked_gated_delta_08_amd import autograd, binding

    def need(*tensors):
        assert all(t is None or t.is_contiguous() for t in tensors)

    def gated_bwd(x, z, w, dy, **kw):
        need(x, z, w, dy)
        return {"dx": 2.0 * torch.ones_like(x), "dz": None if z is None else torch.ones_like(z), "dw": torch.ones_like(w)}

    def add_bwd(dy, dres, res, w, x=None, scale=None, **kw):
        need(dy, dres, res, w, x, scale)
        d = 2.0 * torch.ones_like(res)
        return {"dx": d if scale is None else d.clone(), "dres": d, "dw": torch.ones_like(w),
                "dscale": None if scale is None else torch.ones_like(scale)}

    def glr_bwd(x, g, dh, states, h0=None, **kw):
        need(x, g, dh, states, h0)
        return {"dx": 2.0 * torch.ones_like(x), "dg": torch.ones_like(g), "dh0": None if h0 is None else torch.ones_like(h0)}

    def rule_bwd(q, k, v, g_cum, beta, do, h0=None, **kw):
        need(q, k, v, g_cum, beta, do, h0)
        return {"dq": 2.0 * torch.ones_like(q), "dk": torch.ones_like(k), "dv": torch.ones_like(v), "dg": torch.ones_like(g_cum),
                "dbeta": torch.ones_like(beta), "dh0": None if h0 is None else torch.ones_like(h0)}
    for name, f in dict(
            gated_norm_fwd=lambda x, z, w, **kw: torch.ones_like(x), gated_norm_bwd=gated_bwd,
            add_norm_fwd=lambda x, res, w, **kw: {"y": torch.ones_like(x), "res": torch.ones_like(res)}, add_norm_bwd=add_bwd,
            glr_fwd=lambda x, g, **kw: {"h": torch.ones_like(x), "ht": Z(1, x.shape[1]), "states": Z(1, x.shape[1])},
            glr_bwd=glr_bwd, gdr_gate_cumsum=lambda g, **kw: g.clone(),
            gdr_chunk_fwd=lambda q, k, v, *a, **kw: {"o": torch.ones_like(v), "ht": Z(1, 1, 4, 4)}, gdr_chunk_bwd=rule_bwd).items():
        monkeypatch.setattr(binding, name, f)
    return autograd


def leaf(*shape, strided=False):
    """A leaf; the operator is given every second of its columns where `strided`, which is not contiguous."""
    return torch.ones(*shape[:-1], 2 * shape[-1] if strided else shape[-1])


CALLS = {"gated": (lambda A, a: A.gated_rms_norm(*a), [(3, 4), (3, 4), (4,)], 1),
         "ungated": (lambda A, a: A.gated_rms_norm(a[0], None, a[1]), [(3, 4), (4,)], 1),
         "add": (lambda A, a: A.add_rms_norm(*a), [(3, 4), (3, 4), (4,)], 2),
         "add scaled": (lambda A, a: A.add_rms_norm(*a), [(3, 4), (3, 4), (4,), (4,)], 2),
         "recurrence": (lambda A, a: A.gated_linear_recurrence(*a), [(3, 4), (3, 4), (1, 4)], 2),
         "rule": (lambda A, a: A.chunk_gated_delta_rule(*a[:5], initial_state=a[5]),
                  [(3, 1, 4)] * 3 + [(3, 1)] * 2 + [(1, 1, 4, 4)], 2)}


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("linear", [True, False], ids=["linear", "square"])
@pytest.mark.parametrize("which", CALLS)
def test_second_derivatives_raise(A, which, linear, strided):
    call, shapes, outs = CALLS[which]
    for only in range(len(shapes)):          # each input in turn is the one that is differentiated
        for pick in range(outs):
            leaves = [leaf(*s, strided=strided) for s in shapes]
            for i, t in enumerate(leaves):
                t.requires_grad_(i == only)
            args = [t[..., ::2] if strided else t for t in leaves]
            out = call(A, args)
            out = out[pick] if outs > 1 else out
            loss = out.sum() if linear else out.square().sum()
            plain, = torch.autograd.grad(loss, leaves[only], retain_graph=True)
            assert plain.grad_fn is None
            g, = torch.autograd.grad(loss, leaves[only], create_graph=True)
            assert torch.equal(g, plain)
            other = leaves[only].square().sum()       # a term that has a second derivative of its own
            with pytest.raises(RuntimeError, match="no second derivative"):
                torch.autograd.grad(g.sum() + other, leaves[only])


def test_create_graph_for_other_terms(A):
    """A second derivative that does not go through the operator is not in the way."""
    x, z, w = (torch.ones(*s, requires_grad=True) for s in ((3, 4), (3, 4), (4,)))
    p = torch.full((3, 4), 3.0, requires_grad=True)
    loss = A.gated_rms_norm(x, z, w).sum() + p.pow(3).sum()
    gx, gp = torch.autograd.grad(loss, (x, p), create_graph=True)
    assert (gx == 2).all()
    h, = torch.autograd.grad(gp.sum(), p)
    assert torch.equal(h, torch.full((3, 4), 18.0))
