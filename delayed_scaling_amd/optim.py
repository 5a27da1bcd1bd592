"""AdamW over many tensors in one launch, with optimizer states in 32 or in 8
bits (the optimizer step of the training loop the FP8 linears run in).

    adamw_step(params, grads, exp_avg, exp_avg_sq, step=..., lr=...)
    adamw_state_values(codes, exps, signed)      what 8-bit states stand for
    AdamW                                        a torch optimizer over both

The arithmetic runs in the library's kernel; include/fp8ds.h holds the formulas
and the 8-bit format.
"""
import struct

import torch

from . import _IN_TYPE, _U8, Fp8dsError, _addr, _check, _lend, _need, _on_device, _stream, lib

ADAMW_BLOCK = 256                            # FP8DS_ADAMW_BLOCK
_ADAM_TENSOR = struct.Struct("<7Qq")         # fp8ds_adamw_tensor, 64 bytes
_ADAM_ARGS = struct.Struct("<5dq3Q3iI")      # fp8ds_adamw_args, 88 bytes
_F32 = torch.float32


def state_exp_bytes(numel):
    """Exponent bytes of an 8-bit state of numel elements."""
    return -(-int(numel) // ADAMW_BLOCK)


def _bad(name, i, t, dtype, numel, device):
    """Why tensor i of a list cannot be used (the checks of the hot loop failed)."""
    name = f"{name}[{i}]"
    if not isinstance(t, torch.Tensor):
        return Fp8dsError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        return Fp8dsError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if not t.is_contiguous():
        return Fp8dsError(f"{name} must be contiguous")
    if t.numel() != numel:
        return Fp8dsError(f"{name} has {t.numel()} elements; expected {numel}")
    if not t.is_cuda:
        return Fp8dsError(f"{name} must be a CUDA (HIP) device tensor")
    return Fp8dsError(f"{name} is on {t.device}; the other tensors are on {device}")


def _addresses(name, ts, numels, dtype, device, sizes=None):
    """The addresses of a list of dense tensors, checked."""
    if ts is None:
        return [0] * len(numels)
    if len(ts) != len(numels):
        raise Fp8dsError(f"{name} has {len(ts)} tensors; params has {len(numels)}")
    out, index = [], device.index            # (None on the CPU, where get_device gives -1)
    for t, n in zip(ts, sizes or numels):
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.is_contiguous()
                and t.get_device() == index):
            raise _bad(name, len(out), t, dtype, n, device)
        out.append(t.data_ptr())
    return out


def _scalar(x, name, dtype, device):
    """A device scalar the kernel reads: a one-element tensor on the parameters' GPU."""
    _need(x, name, (dtype,), 4, device=False)
    if x.device != device:
        raise Fp8dsError(f"{name} is on {x.device}; the parameters are on {device}")
    return x.data_ptr()


def adamw_step(params, grads, exp_avg, exp_avg_sq, *, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               masters=None, grad_scale=None, exp_avg_exp=None, exp_avg_sq_exp=None, seed=0, stream=None):
    """One AdamW step of every parameter, in place.

    params, grads: lists of dense device tensors (bf16, fp16 or fp32; one dtype
    a list); exp_avg, exp_avg_sq: the states, fp32, or uint8 with exponent
    bytes exp_avg_exp / exp_avg_sq_exp (uint8, state_exp_bytes(numel) each);
    masters: fp32 copies the step is taken on (the parameters then receive
    their rounded values).  step (t >= 1) and lr: numbers, or device scalars
    (int32 and fp32 tensors) read when the kernel runs, so that a captured
    graph can be replayed with new ones; step may also be a list of them, one
    for each parameter.  grad_scale: optional fp32 device
    scalar that multiplies every gradient.  seed: of the 8-bit states'
    stochastic rounding; pass another every step (a device step joins it)."""
    n = len(params)
    if len(grads) != n:
        raise Fp8dsError(f"grads has {len(grads)} tensors; params has {n}")
    if n == 0:
        return
    p0, g0 = params[0], grads[0]
    for name, t in (("params[0]", p0), ("grads[0]", g0)):
        if not isinstance(t, torch.Tensor) or t.dtype not in _IN_TYPE:
            raise Fp8dsError(f"{name} must be a bf16, fp16 or fp32 tensor")
    dev, numels = p0.device, [t.numel() for t in params]
    bits = 32 if exp_avg_exp is None and exp_avg_sq_exp is None else 8
    sdt = _F32 if bits == 32 else torch.uint8
    if bits == 8 and (exp_avg_exp is None or exp_avg_sq_exp is None):
        raise Fp8dsError("8-bit states need both exp_avg_exp and exp_avg_sq_exp")
    exps = [state_exp_bytes(k) for k in numels] if bits == 8 else None
    cols = zip(_addresses("params", params, numels, p0.dtype, dev), _addresses("grads", grads, numels, g0.dtype, dev),
               _addresses("exp_avg", exp_avg, numels, sdt, dev), _addresses("exp_avg_sq", exp_avg_sq, numels, sdt, dev),
               _addresses("masters", masters, numels, _F32, dev),
               _addresses("exp_avg_exp", exp_avg_exp, numels, torch.uint8, dev, exps),
               _addresses("exp_avg_sq_exp", exp_avg_sq_exp, numels, torch.uint8, dev, exps), numels)
    table = b"".join([_ADAM_TENSOR.pack(*c) for c in cols])
    steps = None
    if isinstance(step, (list, tuple)):
        if len(step) != n:
            raise Fp8dsError(f"step has {len(step)} tensors; params has {n}")
        steps = struct.pack(f"<{n}Q", *[_scalar(t, f"step[{i}]", torch.int32, dev) for i, t in enumerate(step)])
        step = 1                             # (not used)
    step_dev = _scalar(step, "step", torch.int32, dev) if isinstance(step, torch.Tensor) else 0
    lr_dev = _scalar(lr, "lr", _F32, dev) if isinstance(lr, torch.Tensor) else 0
    gs = 0 if grad_scale is None else _scalar(grad_scale, "grad_scale", _F32, dev)
    args = _ADAM_ARGS.pack(0.0 if lr_dev else float(lr), float(betas[0]), float(betas[1]), float(eps),
                           float(weight_decay), 1 if step_dev else int(step), lr_dev, step_dev, gs,
                           _IN_TYPE[p0.dtype], _IN_TYPE[g0.dtype], bits, int(seed) & 0xFFFFFFFF)
    if steps is None:
        _check(lib().adamw_step(table, n, args, _stream(stream)))
    else:
        _check(lib().adamw_step_counts(table, steps, n, args, _stream(stream)))


def adamw_state_values(codes, exps, signed, out=None, stream=None):
    """The values an 8-bit state holds, as bf16 (exactly): codes uint8 [...],
    exps uint8 of state_exp_bytes(codes.numel()) elements; signed: True for
    exp_avg, False for exp_avg_sq."""
    _need(codes, "codes", _U8, 0, device=False)
    _need(exps, "exps", _U8, state_exp_bytes(codes.numel()), device=False)
    made = out is None
    if made:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    _need(out, "out", (torch.bfloat16,), 2 * codes.numel(), device=False)
    _on_device(("codes", codes), ("exps", exps), ("out", out))
    if made:
        _lend(stream, out)
    _check(lib().adamw_state_values(_addr(codes), _addr(exps), codes.numel(), int(bool(signed)), _addr(out),
                                    _stream(stream)))
    return out


class AdamW(torch.optim.Optimizer):
    """torch.optim.AdamW's step through adamw_step: all of a group's tensors of
    one dtype in one launch.

    state_bits 8 keeps both moments in 8 bits (2 bytes a parameter instead of
    8); master_weights keeps an fp32 copy of bf16 / fp16 parameters, on which
    the step is taken.  capturable: the step counts (and with lr a tensor, the
    rate) live on the device, so a captured step can be replayed.  seed: of the
    8-bit states' rounding."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                 master_weights=True, capturable=False, seed=0):
        if state_bits not in (8, 32):
            raise Fp8dsError(f"state_bits {state_bits} is neither 8 nor 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        self.state_bits, self.master_weights, self.capturable = state_bits, bool(master_weights), bool(capturable)
        self.seed = int(seed)

    def _init_state(self, p):
        s = self.state[p]
        dt = _F32 if self.state_bits == 32 else torch.uint8
        for key in ("exp_avg", "exp_avg_sq"):
            s[key] = torch.zeros(p.shape, dtype=dt, device=p.device)
            if self.state_bits == 8:
                s[key + "_exp"] = torch.zeros(state_exp_bytes(p.numel()), dtype=torch.uint8, device=p.device)
        if self.master_weights and p.dtype != _F32:
            s["master"] = p.detach().float()
        s["step"] = torch.zeros((), dtype=torch.int32, device=p.device) if self.capturable else 0
        return s

    def load_state_dict(self, state_dict):
        """torch's load casts floating states to the parameter's dtype; the
        states here keep their own."""
        super().load_state_dict(state_dict)
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        for i, p in zip(ids, (p for g in self.param_groups for p in g["params"])):
            for key, value in state_dict["state"].get(i, {}).items():
                self.state[p][key] = value.detach().to(p.device).clone() if isinstance(value, torch.Tensor) else value
            count = self.state.get(p, {}).get("step")    # of the other kind, if such an optimizer saved it
            if count is not None and isinstance(count, torch.Tensor) != self.capturable:
                self.state[p]["step"] = int(count) if not self.capturable else \
                    torch.tensor(count, dtype=torch.int32, device=p.device)

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        """One step; grad_scale: optional fp32 device scalar that multiplies
        the gradients (a clip coefficient)."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        at = -1                              # launches so far, over all groups: each rounds by bits of its own
        for group in self.param_groups:
            batches = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                s = self.state[p] or self._init_state(p)
                key = (p.device, p.dtype, p.grad.dtype, "master" in s, None if self.capturable else s["step"])
                batches.setdefault(key, []).append(p)
            for key, ps in batches.items():
                at += 1
                ss = [self.state[p] for p in ps]
                if self.capturable:
                    torch._foreach_add_([s["step"] for s in ss], 1)
                else:
                    for s in ss:
                        s["step"] += 1
                eight = self.state_bits == 8
                seed = self.seed + at * 0x10001 + (0 if self.capturable else ss[0]["step"])
                with torch.cuda.device(key[0]):
                    adamw_step([p.detach() for p in ps],
                               [p.grad if p.grad.is_contiguous() else p.grad.contiguous() for p in ps],
                               [s["exp_avg"] for s in ss], [s["exp_avg_sq"] for s in ss],
                               step=[s["step"] for s in ss] if self.capturable else ss[0]["step"],
                               lr=group["lr"], betas=group["betas"], eps=group["eps"],
                               weight_decay=group["weight_decay"],
                               masters=[s["master"] for s in ss] if "master" in ss[0] else None,
                               grad_scale=grad_scale,
                               exp_avg_exp=[s["exp_avg_exp"] for s in ss] if eight else None,
                               exp_avg_sq_exp=[s["exp_avg_sq_exp"] for s in ss] if eight else None, seed=seed)
                # (The kernel writes through addresses; a graph that saved a parameter has to know.)
                torch.autograd.graph.increment_version(ps)
        return loss


__all__ = ["ADAMW_BLOCK", "AdamW", "adamw_state_values", "adamw_step", "state_exp_bytes"]
