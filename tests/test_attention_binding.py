"""Which gradients the attention function takes as they stand (CPU only)."""
import pytest
import torch

from delayed_scaling_amd.attn import _fits

BF = torch.bfloat16


def new(*shape):
    return torch.zeros(*shape, dtype=BF)


@pytest.mark.parametrize("fits,make", [
    (True, lambda: new(2, 30, 4, 64)),
    (True, lambda: new(2, 4, 30, 64).transpose(1, 2)),
    (True, lambda: new(2, 30, 6, 64)[:, :, :4]),
    (True, lambda: new(30, 4, 64)),
    (True, lambda: new(2, 1, 4, 64).as_strided((2, 1, 4, 64), (256, 3, 64, 1))),       # one row: any stride
    (False, lambda: torch.zeros(2, 30, 4, 64)),                                        # type
    (False, lambda: new(1).expand(2, 30, 4, 64)),                                      # of a sum
    (False, lambda: new(2, 1, 4, 64).expand(2, 30, 4, 64)),                            # rows that are one
    (False, lambda: new(2, 30, 64, 4).transpose(2, 3)),
    (False, lambda: new(2, 30, 4, 68)[..., :64]),                                      # strides off 8 elements
    (False, lambda: new(2 * 30 * 4 * 64 + 1)[1:].view(2, 30, 4, 64)),                  # contiguous, off 16 bytes
    (False, lambda: new(30 * 4 * 64 + 4)[4:].view(30, 4, 64))])
def test_what_fits(fits, make):
    assert _fits(make(), BF) is fits
