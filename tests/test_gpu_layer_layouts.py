"""The FP8 layers take inputs and gradients wherever they stand in memory."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def off(t):
    """The same values, contiguous from an address that no 16 bytes divide."""
    x = torch.cat([t.detach().reshape(-1)[:1], t.detach().reshape(-1)])[1:].view(t.shape)
    assert x.is_contiguous() and x.data_ptr() % 16
    return x


@pytest.mark.parametrize("move", [off, lambda t: t.t().contiguous().t()])
@pytest.mark.parametrize("kind", ["linear", "mlp"])
def test_inputs_and_gradients_in_any_place(kind, move):
    require_gpu()
    from delayed_scaling_amd.linear import Fp8LinearState, fp8_linear
    from delayed_scaling_amd.mlp import Fp8MLPState, fp8_mlp
    g = torch.Generator().manual_seed(5)
    new = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    x, w1, b1, w2, res, gy = new(40, 64), new(96, 64), new(96), new(64, 96), new(40, 64), new(40, 64)
    gl = new(40, 96)

    def run(f):
        leaf = f(x).requires_grad_()
        if kind == "linear":
            y = fp8_linear(leaf, w1, b1, Fp8LinearState(4))
            return y, torch.autograd.grad(y, leaf, f(gl))[0]
        y = fp8_mlp(leaf, w1, b1, w2, None, Fp8MLPState(4), "silu", f(res))
        return y, torch.autograd.grad(y, leaf, f(gy))[0]

    want, got = run(lambda t: t.clone()), run(move)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
