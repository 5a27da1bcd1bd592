"""Captured layers and the bias-gradient workspaces they were captured with."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def layer(kind):
    from delayed_scaling_amd.linear import Fp8Linear
    from delayed_scaling_amd.mlp import Fp8MLP
    if kind == "linear":
        m = Fp8Linear(64, 256)
        return m, [m.state.ring_x, m.state.ring_w, m.state.ring_g], lambda: [m.weight.grad, m.bias.grad]
    m = Fp8MLP(64, 256)
    s = m.state
    return m, [s.x, s.w1, s.h, s.w2, s.gy, s.gz], lambda: [m.w1.grad, m.b1.grad, m.w2.grad, m.b2.grad]


@pytest.mark.parametrize("kind", ["linear", "mlp"])
@pytest.mark.parametrize("warm", [50, 4])
def test_a_graph_outlives_a_larger_eager_shape(kind, warm):
    """An eager call with more rows makes a larger workspace; what the graph was
    captured with stays its own (memory that is then handed out is overwritten).
    Warmed up at fewer rows, the graph makes its workspace itself, whose zeros
    no eager call may count on."""
    require_gpu()
    torch.manual_seed(0)
    mod, rings, read = layer(kind)
    x = {n: torch.randn(n, 64, device="cuda").bfloat16() for n in (4, 50, 6000)}
    g = {n: torch.randn(*mod(x[n]).shape, device="cuda").bfloat16() for n in x}
    start = [r.buf.clone() for r in rings]

    def step(n):
        for r, b in zip(rings, start):
            r.buf.copy_(b)
        mod.zero_grad(set_to_none=True)
        mod(x[n]).backward(g[n])
        return read()

    def fresh(n):
        mod.state.workspaces.__init__()
        out = [t.clone() for t in step(n)]
        torch.cuda.synchronize()
        mod.state.workspaces.__init__()
        return out

    want = {n: fresh(n) for n in (50, 6000)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(50)
    eager = [t.clone() for t in step(6000)]            # before any replay, too
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, want[6000]))
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (512, 2048, 8192, 32768, 131072) * 40]
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[50]))
        eager = [t.clone() for t in step(6000)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[6000]))
    del junk
