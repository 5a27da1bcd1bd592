"""Tensors whose element offsets leave 32 bits: the far end gives the bits of the
same rows or elements by themselves."""
import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

ROWS, HEADS, DIM = 140000, 128, 128                    # 2.3e9 elements


@pytest.fixture(scope="module")
def long():
    """Two tensors of [1, ROWS, HEADS, DIM]."""
    require_gpu()
    g = torch.Generator("cuda").manual_seed(1)
    out = []
    for _ in range(2):
        t = torch.empty(1, ROWS, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        for h in range(0, ROWS, 20000):
            t[:, h:h + 20000] = torch.randn(1, 20000, HEADS, DIM, device="cuda", generator=g)
        out.append(t)
    yield out
    del out, t
    torch.cuda.empty_cache()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def test_queries(long):
    """Many query rows over 64 keys: the last ones' out, lse and dQ."""
    ds = require_gpu()
    q, do = long
    k, v = (torch.randn(1, 64, HEADS, DIM, device="cuda").bfloat16() for _ in range(2))
    say("queries", q.numel())
    o, lse = ds.attn_forward(q, k, v)
    dq, dk, dv = ds.attn_backward(do, q, k, v, o, lse)
    torch.cuda.synchronize()
    parts = []
    for rows in (slice(0, 70016), slice(70016, ROWS)):
        one = [x[:, rows].contiguous() for x in (q, do)]
        oo, ll = ds.attn_forward(one[0], k, v)
        gg = ds.attn_backward(one[1], one[0], k, v, oo, ll)
        torch.cuda.synchronize()
        assert same(o[:, rows], oo) and torch.equal(lse[..., rows], ll) and same(dq[:, rows], gg[0])
        parts.append([x.float() for x in gg[1:]])
    # the sums over all rows: those of the halves, each rounded once (2^-8 of itself)
    for whole, a, b in zip((dk, dv), *parts):
        tol = 2.0 ** -8 * (whole.float().abs() + a.abs() + b.abs()) + 1e-3 * a.abs().max()
        assert ((whole.float() - a - b).abs() <= tol).all()


def test_keys(long):
    """Few queries that see a window at the end of many keys: out, lse and dQ, dK and
    dV of those keys, and zero gradients of all before them."""
    ds = require_gpu()
    k, v = long
    q, do = (torch.randn(1, 100, HEADS, DIM, device="cuda").bfloat16() for _ in range(2))
    say("keys", k.numel())
    tail = slice(ROWS - 1088, ROWS)                    # (whole tiles of 64 and the ragged end as in the whole)
    kt, vt = (x[:, tail].contiguous() for x in (k, v))
    kw = dict(causal=True, window=300)
    o, lse = ds.attn_forward(q, k, v, **kw)
    dq, dk, dv = ds.attn_backward(do, q, k, v, o, lse, **kw)
    oo, ll = ds.attn_forward(q, kt, vt, **kw)
    gg = ds.attn_backward(do, q, kt, vt, oo, ll, **kw)
    torch.cuda.synchronize()
    err = lambda a, b: ((a.float() - b.float()).abs() / (2.0 ** -6 * b.float().abs() + 1e-2)).max().item()
    assert err(o, oo) <= 1 and err(lse, ll) <= 1 and err(dq, gg[0]) <= 1
    assert err(dk[:, tail], gg[1]) <= 1 and err(dv[:, tail], gg[2]) <= 1
    assert (dk[:, :ROWS - 400] == 0).all() and (dv[:, :ROWS - 400] == 0).all() and (dv[:, -200:] != 0).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    """2.2e9 elements: the last ones as a tensor of their own (32 bits; codes of 8 bits
    depend on the element's number, so there the weights, which do not)."""
    ds = require_gpu()
    n, cut = (1 << 31) + 70000, 1 << 31
    say("adamw", bits, n)
    new = lambda m, dt: torch.zeros(m, dtype=dt, device="cuda")
    sdt = torch.float32 if bits == 32 else torch.uint8
    p, g, m, v = new(n, torch.bfloat16), new(n, torch.bfloat16), new(n, sdt), new(n, sdt)
    p[cut:] = torch.randn(n - cut, device="cuda")
    g[cut:] = torch.randn(n - cut, device="cuda")
    g[:5] = 1
    kw, kw2 = {}, {}
    if bits == 8:
        e = [new(-(-n // 256), torch.uint8) for _ in range(2)]
        e2 = [new(-(-(n - cut) // 256), torch.uint8) for _ in range(2)]
        kw, kw2 = (dict(exp_avg_exp=[x[0]], exp_avg_sq_exp=[x[1]]) for x in (e, e2))
    tail = [x[cut:].clone() for x in (p, g, m, v)]
    for t in range(1, 2 if bits == 8 else 4):
        ds.adamw_step([p], [g], [m], [v], step=t, lr=1e-2, **kw)
        ds.adamw_step(*[[x] for x in tail], step=t, lr=1e-2, **kw2)
    torch.cuda.synchronize()
    assert torch.equal(p[cut:], tail[0]) and (p[:5] < 0).all() and (p[5:70000] == 0).all()
    if bits == 32:
        assert torch.equal(m[cut:], tail[2]) and torch.equal(v[cut:], tail[3])
    else:
        assert torch.equal(e[0][cut // 256:], e2[0]) and torch.equal(e[1][cut // 256:], e2[1])
        assert (m[cut:] != 0).float().mean() > 0.9 and (m[5:70000] == 0).all()
