"""The autograd functions have first derivatives only: a second one raises, where
without a graph behind the first its terms would be missing from the result."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def attention(ds):
    q, k, v = (torch.randn(1, 40, 2, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(3))
    return ds.attention(q, k, v, causal=True), (q, k, v)


def mlp(ds):
    from delayed_scaling_amd.mlp import Fp8MLP
    m = Fp8MLP(32, 64)
    x = torch.randn(20, 32, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    return m(x, residual=x), (x, m.w1, m.b2)


def linear(ds):
    from delayed_scaling_amd.linear import Fp8Linear
    m = Fp8Linear(32, 48)
    x = torch.randn(20, 32, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    return m(x), (x, m.weight)


@pytest.mark.parametrize("make", [attention, mlp, linear])
def test_a_second_derivative_raises(make):
    ds = require_gpu()
    y, leaves = make(ds)
    first = torch.autograd.grad(y.float().square().sum(), leaves, create_graph=True)
    torch.cuda.synchronize()
    assert all(torch.isfinite(g).all() for g in first)
    for g in first:                                     # a gradient penalty beside a loss
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (y.float().sum() + g.float().square().sum()).backward(retain_graph=True)
