"""The bias-gradient workspaces a layer keeps (CPU only)."""
import delayed_scaling_amd as ds
from delayed_scaling_amd.linear import BiasWorkspaces


def test_a_larger_shape_lets_no_workspace_go():
    """Whatever was handed out stays alive, for a graph may hold its address, and
    all of it together is less than twice the last."""
    w = BiasWorkspaces()
    out = [w.get(rows, cols, "cpu") for rows, cols in ((100, 512), (100, 512), (100, 64), (200, 2048), (3000, 2048),
                                                       (100, 512), (100000, 4096))]
    for x, (rows, cols) in zip(out, ((100, 512), (100, 512), (100, 64), (200, 2048), (3000, 2048), (100, 512),
                                     (100000, 4096))):
        assert x.buf.numel() >= ds.bias_grad_workspace_bytes(rows, cols) and x in w.kept and not x.buf.any()
    assert out[0] is out[1] is out[2]
    sizes = [x.buf.numel() for x in w.kept]
    assert len(sizes) > 1 and sum(sizes[:-1]) <= sizes[-1]


def test_a_small_shape_after_a_large_one_takes_the_large_workspace():
    w = BiasWorkspaces()
    large = w.get(5000, 4096, "cpu")
    assert w.get(10, 64, "cpu") is large and w.get(5000, 4096, "cpu") is large and w.kept == [large]
