"""Attention where a kernel's own structure could let it go wrong: row maxima late
in a tile, masks at the ends of the integers, long causal grids whose workgroups
take two row blocks.  References and tolerances as in test_gpu_attention."""
import pytest
import torch

from gpu_util import require_gpu, say
from test_gpu_attention import check_dense, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [64, 96, 97, 99, 104, 127])
def test_a_maximum_in_the_middle_of_an_unmasked_tile(kind, d, at):
    """One key of the second tile outweighs the keys before it by e^30 = 2^43 (fp16
    ends at 2^16): every row's maximum has to have seen it, whichever register of
    the scores it is in."""
    ds = require_gpu()
    say("attention maximum", kind, d, at)
    q, k, v, do = (randn((1, 192, 2, d), 300 + i, kind, 0.1 if i < 2 else 1.0) for i in range(4))
    q += 1
    k[0, at] = 30 / d ** 0.5
    o, lse = ds.attn_forward(q, k, v)
    grads = ds.attn_backward(do, q, k, v, o, lse)
    torch.cuda.synchronize()
    assert (lse > 20).all()
    check_dense((q, k, v, do), o, lse, grads, kind, False, 0, None)
