"""torch.autograd wrappers around the library's chunked forward and backward, and
around the operators that stand beside it in a layer (gated RMSNorm, residual add
with RMSNorm, dropout, gated feed-forward block, gated linear recurrence).

FlashQLA backward explainer §一: the chunked gated delta rule is exposed to
training code as one autograd function; its forward saves the gate as the
in-chunk cumulative sum and its backward consumes that saved form.  Here the
forward is gdr_gate_cumsum + gdr_chunk_fwd and the backward is gdr_chunk_bwd
(states recomputed, not stored).  Argument marshalling only: every arithmetic
step runs in the library's kernels.

Layouts follow the C ABI (token axis flattened over the batch):
  q, k [B*T, HK, K]   v [B*T, HV, V]   g (raw log-gate) [B*T, HV] fp32
  beta [B*T, HV]      initial_state [N, HV, K, V] fp32

A training step may be captured into a graph (give cu_seqlens_host, so that nothing
is copied to the host).  Let go of the outputs of earlier eager passes over the same
leaves first: torch ties a leaf's gradient to the stream of the graph that is alive.

The operators have first derivatives only: gradients taken with create_graph=True are
the same, and differentiating them again raises.
"""
import torch

from . import binding


class _FirstOrder(torch.autograd.Function):
    """Hands the gradients t[n:] on; they depend on t[:n], and to differentiate them raises."""
    @staticmethod
    def forward(ctx, op, n, *t):
        ctx.op = op
        return t[n:]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.op} has no second derivative (its gradients were differentiated)")


def _first_order(op, ctx, incoming, grads):
    """A backward's results.  The kernels that made them are unknown to torch, so under
    create_graph=True they would count as constants and second derivatives lack their terms."""
    if not torch.is_grad_enabled():
        return grads
    needs = [t for t in (*ctx.saved_tensors, *incoming) if t is not None and t.requires_grad]
    out = iter(_FirstOrder.apply(op, len(needs), *needs, *(g for g in grads if g is not None)))
    return tuple(None if g is None else next(out) for g in grads)


def _contiguous(*tensors):
    """Outside the functions, so that what they save is connected to what they are given."""
    return [None if t is None else t.contiguous() for t in tensors]


class ChunkGatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, scale, cu_seqlens, B, BT, seg_chunks):
        q, k, v, g, beta = (t.contiguous() for t in (q, k, v, g, beta))
        h0 = None if h0 is None else h0.contiguous()
        g_cum = binding.gdr_gate_cumsum(g, cu_seqlens=cu_seqlens, B=B, BT=BT)
        out = binding.gdr_chunk_fwd(q, k, v, g_cum, beta, h0=h0, cu_seqlens=cu_seqlens, B=B, scale=scale, BT=BT,
                                    seg_chunks=seg_chunks)
        ctx.save_for_backward(q, k, v, g_cum, beta, h0, cu_seqlens)
        ctx.cfg = (scale, B, BT, seg_chunks)
        ctx.g = g   # not read again, and so free to be overwritten; _first_order asks whether it needs a gradient
        return out["o"], out["ht"]

    @staticmethod
    def backward(ctx, do, dht):
        q, k, v, g_cum, beta, h0, cu_seqlens = ctx.saved_tensors
        scale, B, BT, seg_chunks = ctx.cfg
        r = binding.gdr_chunk_bwd(q, k, v, g_cum, beta, do.contiguous(), dht=None if dht is None else dht.contiguous(),
                                  h0=h0, cu_seqlens=cu_seqlens, B=B, scale=scale, BT=BT,
                                  want_dh0=h0 is not None and ctx.needs_input_grad[5], seg_chunks=seg_chunks)
        return _first_order("chunk_gated_delta_rule", ctx, (do, dht, ctx.g),
                            (r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"].to(beta.dtype), r["dh0"]) + (None,) * 5)


def chunk_gated_delta_rule(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, B=1, BT=64,
                           seg_chunks=0):
    """o, final_state = chunked gated delta rule over the raw log-gate `g` (fp32).

    Differentiable in q, k, v, g, beta and initial_state.  cu_seqlens: int32 CUDA
    tensor [N+1] (varlen; then the batch is 1) or None.  The final state is fp32."""
    return ChunkGatedDeltaRule.apply(*_contiguous(q, k, v, g, beta, initial_state), scale, cu_seqlens, B, BT, seg_chunks)


class GatedRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, w, eps, act):
        x, w = x.contiguous(), w.contiguous()
        z = None if z is None else z.contiguous()
        ctx.save_for_backward(x, z, w)
        ctx.cfg = (eps, act)
        return binding.gated_norm_fwd(x, z, w, eps=eps, act=act)

    @staticmethod
    def backward(ctx, dy):
        x, z, w = ctx.saved_tensors
        r = binding.gated_norm_bwd(x, z, w, dy.contiguous(), eps=ctx.cfg[0], act=ctx.cfg[1])
        return _first_order("gated_rms_norm", ctx, (dy,), (r["dx"], r["dz"], r["dw"], None, None))


def gated_rms_norm(x, z, weight, eps=1e-5, act="silu"):
    """RMSNorm of x [..., D] times weight [D] (fp32) times the gate act(z); z None: no gate.

    Differentiable in x, z and weight.  act is "silu" or "sigmoid"."""
    return GatedRMSNorm.apply(*_contiguous(x, z, weight), eps, act)


class AddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, res, w, scale, eps):
        x, res, w = x.contiguous(), res.contiguous(), w.contiguous()
        scale = None if scale is None else scale.contiguous()
        out = binding.add_norm_fwd(x, res, w, scale=scale, eps=eps)
        ctx.save_for_backward(None if scale is None else x, out["res"], w, scale)
        ctx.cfg = (eps, x.dtype)
        ctx.set_materialize_grads(False)   # an unused residual stream has no gradient to read
        return out["y"], out["res"]

    @staticmethod
    def backward(ctx, dy, dres):
        x, res, w, scale = ctx.saved_tensors
        incoming = (dy, dres)
        dy = torch.zeros_like(res, dtype=ctx.cfg[1]) if dy is None else dy.contiguous()
        dres = None if dres is None else dres.contiguous()
        r = binding.add_norm_bwd(dy, dres, res, w, x=x, scale=scale, eps=ctx.cfg[0])
        return _first_order("add_rms_norm", ctx, incoming, (r["dx"], r["dres"], r["dw"], r["dscale"], None))


def add_rms_norm(x, res, weight, scale=None, eps=1e-5):
    """y, res' = the residual stream res' = res + scale x and y = RMSNorm(res') weight.

    Differentiable in x, res, weight and scale ([D] fp32, None: 1).  res is in x's
    type or fp32; the gradients are taken at the stored res'."""
    return AddRMSNorm.apply(*_contiguous(x, res, weight, scale), eps)


class GatedLinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, h0, cu_seqlens, cu_seqlens_host, B):
        x, g = x.contiguous(), g.contiguous()
        h0 = None if h0 is None else h0.contiguous()
        out = binding.glr_fwd(x, g, h0=h0, cu_seqlens=cu_seqlens, cu_seqlens_host=cu_seqlens_host, B=B,
                              want_states=True)
        ctx.save_for_backward(x, g, h0, out["states"], cu_seqlens, cu_seqlens_host)
        ctx.B = B
        ctx.set_materialize_grads(False)   # an unused final state has no gradient to read
        return out["h"], out["ht"]

    @staticmethod
    def backward(ctx, dh, dht):
        x, g, h0, states, cu_seqlens, cu_seqlens_host = ctx.saved_tensors
        incoming = (dh, dht)
        dh = torch.zeros_like(x) if dh is None else dh.contiguous()
        dht = None if dht is None else dht.contiguous()
        r = binding.glr_bwd(x, g, dh, states, dht=dht, h0=h0, cu_seqlens=cu_seqlens,
                            cu_seqlens_host=cu_seqlens_host, B=ctx.B,
                            want_dh0=h0 is not None and ctx.needs_input_grad[2])
        return _first_order("gated_linear_recurrence", ctx, incoming, (r["dx"], r["dg"], r["dh0"], None, None, None))


def gated_linear_recurrence(x, g, initial_state=None, cu_seqlens=None, cu_seqlens_host=None, B=1):
    """h, final_state of h_t = exp(g_t) h_{t-1} + x_t over x [B*T, D], the log-gate g [B*T, D] fp32.

    Differentiable in x, g and initial_state ([N, D] fp32).  cu_seqlens as for
    chunk_gated_delta_rule; cu_seqlens_host, its CPU copy, avoids a copy in each pass.
    The final state is fp32."""
    return GatedLinearRecurrence.apply(*_contiguous(x, g, initial_state), cu_seqlens, cu_seqlens_host, B)


def _rng(rng):
    """(the tensor to save or None, the numbers or None)"""
    return (rng, None) if isinstance(rng, torch.Tensor) else (None, (int(rng[0]), int(rng[1])))


class Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng):
        x = x.contiguous()
        t, ctx.numbers = _rng(rng)
        ctx.save_for_backward(t)
        ctx.p = p
        return binding.dropout(x, p, rng)

    @staticmethod
    def backward(ctx, dy):
        # linear in dy: differentiating it again is the same call
        return Dropout.apply(dy.contiguous(), ctx.p, ctx.numbers or ctx.saved_tensors[0]), None, None


def dropout(x, p, rng):
    """x / (1 - p) where the generator keeps the element, else 0 (p to the nearest 2^-16).

    rng: (seed, offset), or an int64 tensor [2] on the GPU that holds them and must not
    change before the backward.  The mask is a function of rng and of the element's row
    and column in x [..., D]; it is not stored.  Calls that shall differ take another offset.
    Differentiable in x, any number of times."""
    return Dropout.apply(x.contiguous(), p, rng)


class DropoutAddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, res, w, scale, p, rng, eps):
        x, res, w = x.contiguous(), res.contiguous(), w.contiguous()
        scale = None if scale is None else scale.contiguous()
        out = binding.dropout_add_norm_fwd(x, res, w, p, rng, scale=scale, eps=eps)
        t, ctx.numbers = _rng(rng)
        ctx.save_for_backward(None if scale is None else x, out["res"], w, scale, t)
        ctx.cfg = (p, eps, x.dtype)
        ctx.set_materialize_grads(False)   # an unused residual stream has no gradient to read
        return out["y"], out["res"]

    @staticmethod
    def backward(ctx, dy, dres):
        x, res, w, scale, t = ctx.saved_tensors
        p, eps, dtype = ctx.cfg
        incoming = (dy, dres)
        dy = torch.zeros_like(res, dtype=dtype) if dy is None else dy.contiguous()
        dres = None if dres is None else dres.contiguous()
        r = binding.dropout_add_norm_bwd(dy, dres, res, w, p, ctx.numbers or t, x=x, scale=scale, eps=eps)
        return _first_order("dropout_add_rms_norm", ctx, incoming,
                            (r["dx"], r["dres"], r["dw"], r["dscale"], None, None, None))


def dropout_add_rms_norm(x, res, weight, p, rng, scale=None, eps=1e-5):
    """y, res' = the residual stream res' = res + scale dropout(x, p, rng) and y = RMSNorm(res') weight,
    in one pass.  As add_rms_norm; p and rng as for dropout."""
    return DropoutAddRMSNorm.apply(*_contiguous(x, res, weight, scale), p, rng, eps)


def _on_16_bytes(t):
    """Contiguous, and where the feed-forward block's operands have to begin."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, act, keep):
        out = binding.gated_ffn_fwd(x, w_gate, w_up, w_down, act=act, want_saved=keep)
        if keep:
            ctx.save_for_backward(x, w_gate, w_up, w_down, out["saved"])
            ctx.act = act
        return out["y"]

    @staticmethod
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        r = binding.gated_ffn_bwd(x, w_gate, w_up, w_down, saved, _on_16_bytes(dy), act=ctx.act, want_dx=need[0],
                                  want_dw=any(need[1:4]))
        return _first_order("gated_ffn", ctx, (dy,), tuple(
            r[k] if n else None for k, n in zip(("dx", "dw_gate", "dw_up", "dw_down"), need)) + (None, None))


def gated_ffn(x, w_gate, w_up, w_down, act="silu"):
    """(act(x w_gate^T) * (x w_up^T)) w_down^T over x [..., D]; w_gate, w_up [F, D], w_down [D, F], all of
    x's dtype.  act is "silu", "gelu" (exact) or "sigmoid".

    Differentiable in x and the weights; the gradients are in x's dtype.  Between the passes it keeps
    2F floats and F of the type a token, its gate and up rows and their product.  That product and
    the gradients of gate and up are held in the type: in fp16 they overflow beyond 65504."""
    t = [_on_16_bytes(v) for v in (x, w_gate, w_up, w_down)]
    return GatedFFN.apply(*t, act, torch.is_grad_enabled() and any(v.requires_grad for v in t))
