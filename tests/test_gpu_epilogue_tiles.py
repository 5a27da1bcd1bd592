"""The activation epilogue where test_gpu_epilogue does not go: the 128x128 and
256x256 tiles of large products with every part of it, padded rows, slopes of
extreme pre-activations.  References and tolerances as there."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_bits, require_gpu, say, to_dev_u8
from oracle import epilogue as ep
from synth import bf16_normal, random_codes
from test_gpu_epilogue import check, dev_bf16, problem, to_f64, up
from test_gpu_gemm import FINITE, scale_tensor, stored_shapes

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


def tile_of(ds, kw):
    """The tile the epilogue product of these arguments runs on: that of fp8_mm with
    a bias, whatever the arguments' own."""
    bias = torch.zeros(kw["n"], dtype=torch.bfloat16, device="cuda")
    args, _ = ds._mm_args(**dict(kw, bias=bias))
    return ds.lib().fp8_mm_tile(args)


# Shapes of the 128x128 and the 256x256 tile with ragged last tiles, the last of each
# with more tiles than workgroups at once.
LARGE = [("128x128u", 2081, 2051, 80), ("128x128u", 2905, 2899, 320), ("256x256w8", 3900, 4003, 528),
         ("256x256w8", 4300, 4090, 1040)]


@pytest.mark.parametrize("tile,m,n,k", LARGE)
@pytest.mark.parametrize("act", [0, 3, 4])
def test_forward_on_large_tiles(tile, m, n, k, act):
    """Bias, activation, Z kept and a residual (which no row or column shares) on the
    tiles that large products take."""
    ds = require_gpu()
    kw, z, tol = problem(oracle.NT, 0, 0, m, n, k, m + act, bias=True)
    assert tile_of(ds, kw) == ds.TILES[tile]
    ld = kw["ldc"]
    say("epilogue forward", tile, m, n, k, act)
    res = bf16_normal((m, ld), 79)
    pre = torch.full((m, ld), 5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((m, ld), 5.0, dtype=torch.bfloat16, device="cuda")
    ds.fp8_mm_epilogue(**kw, act=act, residual=dev_bf16(res), preact=pre, out=out)
    torch.cuda.synchronize()
    ref = ep.act(act, z[0]) + to_f64(res)[:, :n]
    check(to_f64(bf16_bits(out))[:, :n], ref, ep.STEEPEST[act] * tol + 2.0 ** -18 * np.abs(z[0]), "c")
    check(to_f64(bf16_bits(pre))[:, :n], z[0], tol, "z")
    assert (out[:, n:] == 5).all() and (pre[:, n:] == 5).all()
    c = dev_bf16(res)                                  # in place, and without keeping Z
    ds.fp8_mm_epilogue(**kw, act=act, residual=c, out=c)
    torch.cuda.synchronize()
    assert torch.equal(c[:, :n], out[:, :n])


@pytest.mark.parametrize("tile,m,n,k", LARGE)
@pytest.mark.parametrize("layout,act", [(oracle.NN, 3), (oracle.TN, 4), (oracle.NT, 1)])
def test_gradient_on_large_tiles(tile, m, n, k, layout, act):
    ds = require_gpu()
    kw, x, tol = problem(layout, 1, 0, m, n, k, 2 * m + act)
    assert tile_of(ds, kw) == ds.TILES[tile]
    ld = kw["ldc"]
    say("epilogue gradient", tile, m, n, k, layout, act)
    z = bf16_normal((m, ld), 80, 2.0)
    out = torch.full((m, ld), 5.0, dtype=torch.bfloat16, device="cuda")
    ds.fp8_mm_epilogue(**kw, act=act, grad_preact=dev_bf16(z), out=out)
    torch.cuda.synchronize()
    s = ep.slope(act, to_f64(z)[:, :n])
    check(to_f64(bf16_bits(out))[:, :n], x[0] * s, tol * np.abs(s) + 2.0 ** -18 * np.abs(x[0]), "dz")
    assert (out[:, n:] == 5).all()


@pytest.mark.parametrize("act", [2])
def test_gelu_and_its_slope_on_the_128_tile(act):
    ds = require_gpu()
    m, n, k = 2050, 2040, 64
    kw, z, tol = problem(oracle.NT, 0, 0, m, n, k, 90, bias=True)
    assert tile_of(ds, kw) == ds.TILES["128x128u"]
    res = bf16_normal((m, n), 91)
    out = ds.fp8_mm_epilogue(**kw, act=act, residual=dev_bf16(res))
    kw2, x, tol2 = problem(oracle.NN, 1, 0, m, n, k, 92)
    zz = bf16_normal((m, n), 93, 2.0)
    dz = ds.fp8_mm_epilogue(**kw2, act=act, grad_preact=dev_bf16(zz))
    torch.cuda.synchronize()
    check(to_f64(bf16_bits(out)).reshape(m, n), ep.act(act, z[0]) + to_f64(res),
          ep.STEEPEST[act] * tol + 2.0 ** -18 * np.abs(z[0]), "c")
    s = ep.slope(act, to_f64(zz))
    check(to_f64(bf16_bits(dz)).reshape(m, n), x[0] * s, tol2 * np.abs(s) + 2.0 ** -18 * np.abs(x[0]), "dz")


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("tile,m,n,k,batch", [("128x128u", 1250, 1233, 48, 3), ("256x256w8", 2040, 2560, 1040, 3)])
def test_batches_and_broadcast_on_large_tiles(tile, m, n, k, batch, shared):
    ds = require_gpu()
    kw, z, tol = problem(oracle.NT, 0, 0, m, n, k, 95, batch=batch, bias=True)
    assert tile_of(ds, kw) == ds.TILES[tile]
    say("epilogue batches", tile, shared)
    res = bf16_normal((1 if shared else batch, m, kw["ldc"]), 96)
    out = ds.fp8_mm_epilogue(**kw, act=ep.ACT_SILU, residual=dev_bf16(res), stride_extra=0 if shared else None)
    torch.cuda.synchronize()
    got = to_f64(bf16_bits(out)).reshape(batch, m, kw["ldc"])[:, :, :n]
    check(got, ep.act(ep.ACT_SILU, z) + to_f64(res)[:, :, :n], 1.2 * tol + 2.0 ** -18 * np.abs(z), "batch")


@pytest.mark.parametrize("layout,fa,fb", [(oracle.NN, 1, 0), (oracle.TN, 1, 0), (oracle.TN, 0, 1), (oracle.NT, 1, 1)])
@pytest.mark.parametrize("m,n,k", [(200, 264, 320), (129, 136, 4096), (2081, 2051, 80), (3900, 4003, 528)])
def test_plain_epilogue_is_fp8_mm_on_padded_rows(layout, fa, fb, m, n, k):
    """No activation: the bits of fp8_mm (on the same tile: with a bias), where a
    stored row is not a multiple of 16 and so is padded."""
    ds = require_gpu()
    (ar, ac), (br, bc) = stored_shapes(layout, m, n, k)
    lda, ldb, ldc = up(ac, 16), up(bc, 16), up(n, 8)
    a, b = to_dev_u8(random_codes((ar, lda), 5, FINITE[fa])), to_dev_u8(random_codes((br, ldb), 6, FINITE[fb]))
    kw = dict(a=a, b=b, fmt_a=fa, fmt_b=fb, layout=layout, m=m, n=n, k=k, a_scale_inv=scale_tensor(0.01),
              b_scale_inv=scale_tensor(0.02), bias=dev_bf16(bf16_normal((n,), 8)), lda=lda, ldb=ldb, ldc=ldc)
    y, c, pre = (torch.zeros((m, ldc), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ds.fp8_mm(**kw, out=y)
    ds.fp8_mm_epilogue(**kw, preact=pre, out=c)
    torch.cuda.synchronize()
    same = lambda p, q: torch.equal(p.view(torch.int16), q.view(torch.int16))
    assert same(y, c) and same(y, pre)
