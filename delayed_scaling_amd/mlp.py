"""A two-layer perceptron in FP8 with delayed scaling, its element-wise work in
the products' epilogues (fp8_mm_epilogue):

forward   z = X W1^T + b1 (kept in bf16 for the backward), H = act(z): one launch
          y = H W2^T + b2 + residual: one launch
backward  dz = (dY W2) act'(z): one launch, dW2 = dY^T H, db2 = column sums
          dX = dz W1 and dW1 = dz^T X in one launch, db1 = column sums of dz
          d residual = dY

X, W1, H and W2 are quantized to E4M3, dY and dz to E5M2, each with a scale ring
of its own; the backward multiplies the forward's codes and dequantizes with the
1/scale values the forward applied, as the linear layer does.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, E4M3, E5M2, NN, NT, TN, Fp8dsError, ScaleRing,
               fp8_bias_grad, fp8_mm, fp8_mm_epilogue, fp8_mm_pair, fp8_quantize, fp8_quantize_batch)
from .linear import BiasWorkspaces, _dense, _input

_ACTS = {"relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}


class Fp8MLPState:
    """The six scale rings of one perceptron (x, w1, h, w2: E4M3; gy, gz: E5M2)."""

    def __init__(self, hist_len=16, device="cuda"):
        self.x, self.w1, self.h, self.w2 = (ScaleRing(hist_len, E4M3, device=device) for _ in range(4))
        self.gy, self.gz = (ScaleRing(hist_len, E5M2, device=device) for _ in range(2))
        self.workspaces = BiasWorkspaces()

    def workspace(self, rows, cols, device):
        """A bias-gradient workspace for [rows, cols] (all zero between calls)."""
        return self.workspaces.get(rows, cols, device)


class _Fp8MLPFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w1, b1, w2, b2, residual, act, state):
        dev, n_in, hid, n_out = w1.device, x.shape[-1], w1.shape[0], w2.shape[0]
        if w1.dim() != 2 or w2.dim() != 2 or w1.shape[1] != n_in or w2.shape[1] != hid:
            raise Fp8dsError(f"weights {tuple(w1.shape)} and {tuple(w2.shape)} do not take inputs of {n_in} features")
        x2 = _input(x.reshape(-1, n_in), "x", dev)
        t = x2.shape[0]
        bf = torch.bfloat16
        r2 = None
        if residual is not None:
            if residual.dtype != bf or residual.shape != (*x.shape[:-1], n_out):
                raise Fp8dsError("residual must be bf16, of the output's shape")
            r2 = _input(residual.reshape(t, n_out), "residual", dev)
        s = torch.empty(4, dtype=torch.float32, device=dev)             # applied 1/scale of x, w1, h, w2
        sx, s1, sh, s2 = s.unbind()
        if x2.dtype == w1.dtype == w2.dtype:
            x8, w18, w28 = fp8_quantize_batch([x2, _input(w1, "w1", dev), _input(w2, "w2", dev)], E4M3,
                                              [state.x, state.w1, state.w2], scale_inv_outs=[sx, s1, s2])
        else:
            x8, w18, w28 = (fp8_quantize_batch([_input(v, n, dev)], E4M3, [r], scale_inv_outs=[o])[0]
                            for v, n, r, o in ((x2, "x", state.x, sx), (w1, "w1", state.w1, s1),
                                               (w2, "w2", state.w2, s2)))
        z = torch.empty((t, hid), dtype=bf, device=dev)
        h = torch.empty((t, hid), dtype=bf, device=dev)
        fp8_mm_epilogue(x8, w18, E4M3, E4M3, NT, t, hid, n_in, sx, s1, bias=b1, act=act, preact=z, out=h)
        h8 = fp8_quantize_batch([h], E4M3, [state.h], scale_inv_outs=[sh])[0]
        y = torch.empty((t, n_out), dtype=bf, device=dev)
        fp8_mm_epilogue(h8, w28, E4M3, E4M3, NT, t, n_out, hid, sh, s2, bias=b2, act=ACT_NONE, residual=r2, out=y)
        ctx.save_for_backward(x8, w18, h8, w28, z, s)
        ctx.state, ctx.act, ctx.x_shape = state, act, x.shape
        ctx.biases = (b1 is not None, b2 is not None)
        return y.view(*x.shape[:-1], n_out)

    @staticmethod
    @once_differentiable   # (its outputs are written through addresses: no graph leads on)
    def backward(ctx, gy):
        x8, w18, h8, w28, z, s = ctx.saved_tensors
        sx, s1, sh, s2 = s.unbind()
        state, (t, hid), n_in, n_out, dev = ctx.state, z.shape, x8.shape[1], w28.shape[0], z.device
        bf = torch.bfloat16
        need_x, need_w1, need_b1, need_w2, need_b2, need_r = ctx.needs_input_grad[:6]
        g2 = _dense(gy.reshape(t, n_out).to(bf))
        g8 = fp8_quantize(g2, E5M2, state.gy)
        dx = dw1 = db1 = dw2 = db2 = None
        if need_w2:
            dw2 = torch.empty((n_out, hid), dtype=bf, device=dev)
            fp8_mm(g8, h8, E5M2, E4M3, TN, n_out, hid, t, state.gy, sh, out=dw2)
        if ctx.biases[1] and need_b2:
            db2 = fp8_bias_grad(g2, workspace=state.workspace(t, n_out, dev))
        if need_x or need_w1 or (ctx.biases[0] and need_b1):
            dz = torch.empty((t, hid), dtype=bf, device=dev)
            fp8_mm_epilogue(g8, w28, E5M2, E4M3, NN, t, hid, n_out, state.gy, s2, act=ctx.act, grad_preact=z, out=dz)
            dz8 = fp8_quantize(dz, E5M2, state.gz)
            ax = aw = None
            if need_x:
                dx = torch.empty((t, n_in), dtype=bf, device=dev)
                ax = dict(a=dz8, b=w18, fmt_a=E5M2, fmt_b=E4M3, layout=NN, m=t, n=n_in, k=hid, a_scale_inv=state.gz,
                          b_scale_inv=s1, out=dx)
            if need_w1:
                dw1 = torch.empty((hid, n_in), dtype=bf, device=dev)
                aw = dict(a=dz8, b=x8, fmt_a=E5M2, fmt_b=E4M3, layout=TN, m=hid, n=n_in, k=t, a_scale_inv=state.gz,
                          b_scale_inv=sx, out=dw1)
            if ax and aw:
                fp8_mm_pair(ax, aw)
            elif ax or aw:
                fp8_mm(**(ax or aw))
            if ctx.biases[0] and need_b1:
                db1 = fp8_bias_grad(dz, workspace=state.workspace(t, hid, dev))
            dx = dx if dx is None else dx.view(ctx.x_shape)
        return dx, dw1, db1, dw2, db2, gy if need_r else None, None, None


def fp8_mlp(x, w1, b1, w2, b2, state, act="gelu", residual=None):
    """y = act(x @ w1.T + b1) @ w2.T + b2 + residual through FP8 (bf16 in and
    out; b1, b2 and residual may be None).  act: relu, gelu, gelu_tanh or silu."""
    if act not in _ACTS:
        raise Fp8dsError(f"act {act!r} is not one of {', '.join(_ACTS)}")
    return _Fp8MLPFn.apply(x, w1, b1, w2, b2, residual, _ACTS[act], state)


class Fp8MLP(torch.nn.Module):
    """The module over fp8_mlp (bf16 parameters; features multiples of 16)."""

    def __init__(self, features, hidden, act="gelu", bias=True, hist_len=16, device="cuda"):
        super().__init__()
        new = lambda *s: torch.nn.Parameter(torch.zeros(*s, dtype=torch.bfloat16, device=device))
        self.w1, self.w2 = new(hidden, features), new(features, hidden)
        self.b1, self.b2 = (new(hidden), new(features)) if bias else (None, None)
        torch.nn.init.normal_(self.w1, std=features ** -0.5)
        torch.nn.init.normal_(self.w2, std=hidden ** -0.5)
        self.act, self.state = act, Fp8MLPState(hist_len, device)

    def forward(self, x, residual=None):
        return fp8_mlp(x, self.w1, self.b1, self.w2, self.b2, self.state, self.act, residual)


__all__ = ["Fp8MLP", "Fp8MLPState", "fp8_mlp"]
