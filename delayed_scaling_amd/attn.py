"""Attention and its gradients: the part of a transformer's training step
between the FP8 linears (bf16 or fp16 in and out, fp32 sums).

    attn_forward(q, k, v, ...)                  -> out, lse
    attn_backward(dout, q, k, v, out, lse, ...) -> dq, dk, dv
    attention(q, k, v, ...)                     -> out, differentiable

Tensors are [batch, rows, heads, head_dim], or packed [rows, heads, head_dim]
with cu_seqlens; any strides with a dense last dimension and 16-byte aligned
rows, so slices of a fused QKV projection go in as they are.  include/fp8ds.h
holds the formulas and the masks.
"""
import struct

import torch
from torch.autograd.function import once_differentiable

from . import _F32, IN_BF16, IN_F16, Fp8dsError, _check, _lend, _need, _stream, lib

_ATTN_ARGS = struct.Struct("<32q4Q3q9if")    # fp8ds_attn_args, 352 bytes
_WORKSPACE_AT = 264                          # its workspace field
_NO_GRADS = (0,) * 16                        # the views a forward call leaves out
_TYPES = {torch.bfloat16: IN_BF16, torch.float16: IN_F16}


def _bad_view(t, name, shape, dtype, device):
    """Why a tensor cannot be used (the checks of _view failed)."""
    if not isinstance(t, torch.Tensor):
        return Fp8dsError(f"{name} must be a torch tensor" if t is not None else f"{name} is required")
    if t.dtype != dtype:
        return Fp8dsError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if t.shape != shape:
        return Fp8dsError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    if t.device != device:
        return Fp8dsError(f"{name} is on {t.device}; expected {device}")
    return Fp8dsError(f"{name} must be dense in its last dimension")


def _view(t, name, shape, dtype, device):
    """The fp8ds_attn_view of a tensor (address; batch, row and head strides),
    checked.  A dimension of one entry may carry any stride; none is used."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _bad_view(t, name, shape, dtype, device)
    st = t.stride()
    if st[-1] != 1:
        raise _bad_view(t, name, shape, dtype, device)
    if len(st) == 3:
        return t.data_ptr(), 0, st[0] if shape[0] > 1 else shape[2], st[1] if shape[1] > 1 else 0
    return (t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else shape[3],
            st[2] if shape[2] > 1 else 0)


def _int32(x):
    """A length or window as the 32-bit integer of the arguments.  No row is as far
    as the largest one, so a window past it hides as little, and lengths there
    are refused by the library."""
    return max(-1, min(int(x), 0x7FFFFFFF))


def _tail(q, k, causal, window, scale, cu_q, cu_k, max_q, max_k):
    """The scalar fields of the arguments (after lse and workspace), and the
    shape of lse."""
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES:
            raise Fp8dsError(f"{name} must be a bf16 or fp16 tensor")
    if not q.is_cuda:
        raise Fp8dsError("q must be a CUDA (HIP) device tensor")
    qs, ks = q.shape, k.shape
    packed = cu_q is not None or cu_k is not None
    if len(qs) != (3 if packed else 4) or len(ks) != len(qs):
        raise Fp8dsError("q, k and v are [batch, rows, heads, head_dim], or [rows, heads, head_dim] with cu_seqlens")
    dim, hq, hkv = qs[-1], qs[-2], ks[-2]
    if ks[-1] != dim or (not packed and ks[0] != qs[0]):
        raise Fp8dsError(f"k {tuple(ks)} does not go with q {tuple(qs)}")
    scale = dim ** -0.5 if scale is None else float(scale)
    if not packed:
        batch, tq = qs[0], qs[1]
        return (0, 0, tq, tq, ks[1], _TYPES[q.dtype], batch, hq, hkv, dim, tq, ks[1], 1 if causal else 0, _int32(window),
                scale), (batch, hq, tq)
    for name, cu in (("cu_seqlens_q", cu_q), ("cu_seqlens_k", cu_k)):
        _need(cu, name, (torch.int32,), 4)
        if cu.device != q.device:
            raise Fp8dsError(f"{name} is on {cu.device}; expected {q.device}")
    if cu_q.dim() != 1 or cu_q.shape != cu_k.shape:
        raise Fp8dsError("cu_seqlens_q and cu_seqlens_k hold batch + 1 offsets each")
    if max_q is None or max_k is None:
        raise Fp8dsError("cu_seqlens need max_seqlen_q and max_seqlen_k")
    return (cu_q.data_ptr(), cu_k.data_ptr(), qs[0], qs[0], ks[0], _TYPES[q.dtype], cu_q.shape[0] - 1, hq, hkv, dim,
            _int32(max_q), _int32(max_k), 1 if causal else 0, _int32(window), scale), (hq, qs[0])


def _lse(t, shape, device):
    n = 1
    for x in shape:
        n *= x
    _need(t, "lse", _F32, 4 * n)
    if t.device != device:
        raise Fp8dsError(f"lse is on {t.device}; expected {device}")
    return t


def attn_forward(q, k, v, causal=False, window=0, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
                 max_seqlen_q=None, max_seqlen_k=None, out=None, lse=None, stream=None):
    """Attention of q [B, Tq, Hq, D] over k, v [B, Tk, Hkv, D] (Hq a multiple of
    Hkv; packed: [rows, heads, D] with int32 cu_seqlens of batch + 1 offsets and
    the longest lengths).  causal aligns the last query with the last key;
    window w > 0 (with causal) lets a query see its last w keys only; scale
    defaults to D ** -0.5.  Returns (out like q, lse fp32 [B, Hq, Tq], packed
    [Hq, rows]); a row that sees no key gets 0 and -infinity.  Packed rows of no
    sequence (before the first offset, past the last) are not written."""
    tail, shape = _tail(q, k, causal, window, scale, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k)
    dt, dev, qs, ks = q.dtype, q.device, q.shape, k.shape
    made = []
    if out is None:
        made.append(out := torch.empty_like(q))
    if lse is None:
        made.append(lse := q.new_empty(shape, dtype=torch.float32))
    else:
        _lse(lse, shape, dev)
    args = _ATTN_ARGS.pack(*_view(q, "q", qs, dt, dev), *_view(k, "k", ks, dt, dev), *_view(v, "v", ks, dt, dev),
                           *_view(out, "out", qs, dt, dev), *_NO_GRADS, lse.data_ptr(), 0, *tail)
    if made:
        _lend(stream, *made)
    _check(lib().attn_forward(args, _stream(stream)))
    return out, lse


def attn_workspace_bytes(q, k, causal=False, window=0, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None,
                         max_seqlen_k=None):
    """Bytes of the workspace attn_backward needs for these shapes and options."""
    tail, _ = _tail(q, k, causal, window, None, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k)
    return lib().attn_workspace_bytes(_ATTN_ARGS.pack(*_NO_GRADS, *_NO_GRADS, 0, 0, *tail))


def attn_backward(dout, q, k, v, out, lse, causal=False, window=0, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
                  max_seqlen_q=None, max_seqlen_k=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of attn_forward for the output's gradient dout,
    from its inputs, its outputs out and lse and the same options.  dq, dk, dv
    may be given (slices of one dQKV tensor, say); packed rows of no sequence
    are not written; workspace: a dense fp32
    device tensor of at least attn_workspace_bytes, made per call if not given."""
    tail, shape = _tail(q, k, causal, window, scale, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k)
    dt, dev, qs, ks = q.dtype, q.device, q.shape, k.shape
    made = []
    if dq is None:
        made.append(dq := torch.empty_like(q))
    if dk is None:
        made.append(dk := torch.empty_like(k))
    if dv is None:
        made.append(dv := torch.empty_like(v))
    lse = _lse(lse, shape, dev)
    args = _ATTN_ARGS.pack(*_view(q, "q", qs, dt, dev), *_view(k, "k", ks, dt, dev), *_view(v, "v", ks, dt, dev),
                           *_view(out, "out", qs, dt, dev), *_view(dout, "dout", qs, dt, dev),
                           *_view(dq, "dq", qs, dt, dev), *_view(dk, "dk", ks, dt, dev), *_view(dv, "dv", ks, dt, dev),
                           lse.data_ptr(), 0, *tail)
    nbytes = lib().attn_workspace_bytes(args)
    if workspace is None:
        made.append(workspace := lse.new_empty(nbytes // 4))
    _need(workspace, "workspace", _F32, nbytes)
    if made:
        _lend(stream, *made)
    args = args[:_WORKSPACE_AT] + workspace.data_ptr().to_bytes(8, "little") + args[_WORKSPACE_AT + 8:]
    _check(lib().attn_backward(args, _stream(stream)))
    return dq, dk, dv


def _fits(t, dtype):
    """Whether a gradient that autograd hands over can be read where it stands: the
    library's conditions on a view (a new tensor meets them, a contiguous one
    need not: it can begin anywhere)."""
    st, n = t.stride(), t.shape
    return (t.dtype is dtype and st[-1] == 1 and t.data_ptr() % 16 == 0
            and not any(s % 8 for s, k in zip(st[:-1], n) if k > 1) and (n[-3] < 2 or n[-1] <= st[-3] < 1 << 24))


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, kw):
        # Rows of no sequence are not written: zeros, for what comes after takes
        # every row (an amax, a weight's gradient).
        packed = kw["cu_seqlens_q"] is not None and isinstance(q, torch.Tensor)
        out, lse = attn_forward(q, k, v, out=torch.zeros_like(q) if packed else None, **kw)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.kw = kw
        return out

    @staticmethod
    @once_differentiable   # (its outputs are written through addresses: no graph leads on)
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        if not _fits(dout, q.dtype):
            dout = torch.empty(dout.shape, dtype=q.dtype, device=q.device).copy_(dout)
        grads = [torch.zeros_like(t) for t in (q, k, v)] if ctx.kw["cu_seqlens_q"] is not None else (None,) * 3
        return (*attn_backward(dout, q, k, v, out, lse, **ctx.kw, dq=grads[0], dk=grads[1], dv=grads[2]), None)


def attention(q, k, v, causal=False, window=0, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
              max_seqlen_q=None, max_seqlen_k=None):
    """attn_forward's out, differentiable in q, k and v.  Packed rows of no
    sequence are zero, in out and in the gradients."""
    kw = dict(causal=causal, window=window, scale=scale, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
              max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    return _AttentionFn.apply(q, k, v, kw)


__all__ = ["attention", "attn_backward", "attn_forward", "attn_workspace_bytes"]
