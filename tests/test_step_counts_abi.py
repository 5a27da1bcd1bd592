"""Refusals of adamw_step_counts and of lists of counts in the binding (CPU only)."""
import ctypes

import pytest
import torch

import delayed_scaling_amd as ds
from test_training_abi import adam

PTR = ctypes.c_void_p


def test_refusals():
    L = ds.lib()
    t, a = adam(step=0)                                        # (args' own count is not used)
    call = lambda steps, n=1: L.adamw_step_counts(ctypes.byref(t), steps, n, ctypes.byref(a), None)
    assert call(None) == -1 and b"steps is NULL" in L.fp8_last_error()
    assert call((PTR * 1)(None)) == -1 and b"step count of tensor 0" in L.fp8_last_error()
    assert call((PTR * 1)(4098)) == -2
    assert call(None, 0) == 0
    e, _ = adam(0)
    assert L.adamw_step_counts(ctypes.byref(e), (PTR * 1)(None), 1, ctypes.byref(a), None) == 0   # an empty tensor
    bad, _ = adam(p=None)
    assert L.adamw_step_counts(ctypes.byref(bad), (PTR * 1)(4096), 1, ctypes.byref(a), None) == -1
    assert L.adamw_step_counts(ctypes.byref(t), (PTR * 1)(4096), 1, None, None) == -1


def test_binding():
    t = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)
    with pytest.raises(ds.Fp8dsError, match="device tensor"):
        ds.adamw_step([t(4)], [t(4)], [t(4)], [t(4)], step=[t(1, torch.int32)], lr=1e-3)
    with pytest.raises(ds.Fp8dsError):
        ds.adamw_step([t(4)], [t(4)], [t(4)], [t(4)], step=[], lr=1e-3)
