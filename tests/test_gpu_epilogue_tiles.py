"""The activation epilogue where test_gpu_epilogue does not go: slopes of extreme
pre-activations.  References and tolerances as there."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_bits, require_gpu, say, to_dev_u8
from oracle import epilogue as ep
from test_gpu_epilogue import check, dev_bf16, to_f64
from test_gpu_gemm import scale_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", range(1, 5))
def test_slopes_of_extreme_preactivations(act):
    """A product of one times the slope at every magnitude of bf16's range, those
    included whose squares and exponentials overflow: the slope's limits, 0 and 1,
    with one rounding of the result."""
    ds = require_gpu()
    say("epilogue slopes", act)
    m, n, k = 16, 64, 16
    a, b = np.zeros((m, k), np.uint8), np.zeros((k, n), np.uint8)
    a[:, 0], b[0] = 0x3C, 0x38                         # 1 in E5M2 and in E4M3
    mags = 2.0 ** np.linspace(-130, 127.9, m * n // 2)
    z = torch.from_numpy(np.concatenate([mags, -mags])).bfloat16().cuda()
    out = ds.fp8_mm_epilogue(to_dev_u8(a), to_dev_u8(b), 1, 0, oracle.NN, m, n, k, scale_tensor(1.0), scale_tensor(1.0),
                             act=act, grad_preact=z)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        ref = ep.slope(act, z.double().cpu().numpy())
    check(to_f64(bf16_bits(out)), ref, 2.0 ** -18, "slope")
