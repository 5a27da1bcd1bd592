"""Attention where a kernel's own structure could let it go wrong: row maxima late
in a tile, masks at the ends of the integers, long causal grids whose workgroups
take two row blocks.  References and tolerances as in test_gpu_attention."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say
from oracle import attention as at
from test_gpu_attention import check, check_dense, f64, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", [64, 96, 97, 99, 104, 127])
def test_a_maximum_in_the_middle_of_an_unmasked_tile(kind, d, where):
    """One key of the second tile outweighs the keys before it by e^30 = 2^43 (fp16
    ends at 2^16): every row's maximum has to have seen it, whichever register of
    the scores it is in."""
    ds = require_gpu()
    say("attention maximum", kind, d, where)
    q, k, v, do = (randn((1, 192, 2, d), 300 + i, kind, 0.1 if i < 2 else 1.0) for i in range(4))
    q += 1
    k[0, where] = 30 / d ** 0.5
    o, lse = ds.attn_forward(q, k, v)
    grads = ds.attn_backward(do, q, k, v, o, lse)
    torch.cuda.synchronize()
    assert (lse > 20).all()
    check_dense((q, k, v, do), o, lse, grads, kind, False, 0, None)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 40])
@pytest.mark.parametrize("tq,tk", [(300, 300), (200, 340), (1100, 600)])
def test_a_window_past_every_row_hides_nothing(window, tq, tk):
    """The largest windows (row numbers added to them leave 32 bits) give the bits
    of no window; the last case's backward is shared by workgroups."""
    ds = require_gpu()
    say("attention window", window, tq, tk)
    q, k, v, do = (randn((1, t, h, 64), 320 + i, "bf16") for i, (t, h) in enumerate(((tq, 4), (tk, 2), (tk, 2), (tq, 4))))
    o, lse = ds.attn_forward(q, k, v, causal=True)
    ref = ds.attn_backward(do, q, k, v, o, lse, causal=True)
    o2, lse2 = ds.attn_forward(q, k, v, causal=True, window=window)
    got = ds.attn_backward(do, q, k, v, o2, lse2, causal=True, window=window)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and (ref[1] != 0).any() and (ref[2] != 0).any()


@pytest.mark.parametrize("tq,hq", [(5, 0), (0, 4), (0, 0)])
def test_no_query_leaves_zero_gradients(tq, hq):
    """Without query heads or rows dk and dv are zero, not what their memory held."""
    ds = require_gpu()
    q, k = randn((2, tq, hq, 64), 330, "bf16"), randn((2, 70, 2, 64), 331, "bf16")
    o, lse = ds.attn_forward(q, k, k)
    out = [torch.full_like(k, 7.0) for _ in range(2)]
    dq, dk, dv = ds.attn_backward(q, q, k, k, o, lse, dk=out[0], dv=out[1])
    torch.cuda.synchronize()
    assert o.shape == q.shape and lse.shape == (2, hq, tq) and dq.shape == q.shape
    assert (dk == 0).all() and (dv == 0).all()


def test_packed_rows_of_no_sequence_are_zero_in_autograd():
    """A buffer longer than its sequences: the rest of the output and of the
    gradients is zero, whatever the memory held (a next layer takes all rows)."""
    ds = require_gpu()
    rows, cu = 512, torch.tensor([7, 130, 130, 301], dtype=torch.int32, device="cuda")
    leaf = [randn((rows, h, 64), 340 + i, "bf16").requires_grad_() for i, h in enumerate((4, 2, 2))]
    do = randn((rows, 4, 64), 350, "bf16")
    kw = dict(causal=True, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=171, max_seqlen_k=171)
    for h in (4, 2, 2, 4, 2, 2):                       # what the call's tensors may get
        torch.full((rows, h, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = ds.attention(*leaf, **kw)
    y.backward(do)
    o, lse = ds.attn_forward(*[x.detach() for x in leaf], **kw)
    ref = ds.attn_backward(do, *[x.detach() for x in leaf], o, lse, **kw)
    torch.cuda.synchronize()
    for got, want in zip((y.detach(), *[x.grad for x in leaf]), (o, *ref)):
        assert torch.equal(got[7:301], want[7:301])
        assert (got[:7] == 0).all() and (got[301:] == 0).all()


def alone(ds, case, b, heads, hk, causal):
    """Forward and backward of one key / value head's group by itself."""
    q, k, v, do = (x[b:b + 1, :, s] for x, s in zip(case, (heads, slice(hk, hk + 1), slice(hk, hk + 1), heads)))
    one = [x.contiguous() for x in (q, k, v, do)]
    o, lse = ds.attn_forward(*one[:3], causal=causal)
    return one, o, lse, ds.attn_backward(one[3], *one[:3], o, lse, causal=causal)


@pytest.mark.parametrize("kind,b,hq,hkv,tq,tk,d", [
    ("bf16", 3, 6, 3, 3662, 3662, 64),                 # 29 blocks of rows: the middle one has no partner
    ("f16", 3, 6, 3, 3790, 3790, 128),                 # 30
    ("bf16", 1, 16, 2, 4200, 3300, 128),               # 33; the first 900 rows see nothing
    ("bf16", 5, 8, 1, 1700, 2500, 64)])                # 14
def test_workgroups_of_two_row_blocks(kind, b, hq, hkv, tq, tk, d):
    """Causal grids of more than 512 row blocks, whose workgroups take a block from
    each end: out, lse and dQ of every head are the bits of its group alone (a grid
    that is not paired), and two groups are checked in full against float64, dK and
    dV too.  (dK and dV of a group alone are summed in other parts.)"""
    ds = require_gpu()
    blocks = -(-tq // 128)
    assert b * hq * blocks > 512 and (hq // hkv) * blocks <= 512
    say("attention in pairs", kind, b, hq, hkv, tq, tk, d)
    case = [randn((b, t, h, d), 360 + i, kind) for i, (t, h) in enumerate(((tq, hq), (tk, hkv), (tk, hkv), (tq, hq)))]
    q, k, v, do = case
    o, lse = ds.attn_forward(q, k, v, causal=True)
    dq, dk, dv = ds.attn_backward(do, q, k, v, o, lse, causal=True)
    torch.cuda.synchronize()
    rep = hq // hkv
    same = lambda x, y: torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    for i in range(b):
        for hk in range(hkv):
            heads = slice(hk * rep, (hk + 1) * rep)
            one, oo, ll, gg = alone(ds, case, i, heads, hk, True)
            torch.cuda.synchronize()
            assert same(o[i:i + 1, :, heads], oo) and torch.equal(lse[i:i + 1, heads], ll), (i, hk)
            assert same(dq[i:i + 1, :, heads], gg[0]), (i, hk)
    for i, hk in {(0, 0), (b - 1, hkv - 1)}:
        say("  in full", i, hk)
        heads = slice(hk * rep, (hk + 1) * rep)
        pick = lambda x, s: x[i:i + 1, :, s]
        check_dense((pick(q, heads), pick(k, slice(hk, hk + 1)), pick(v, slice(hk, hk + 1)), pick(do, heads)),
                    pick(o, heads), lse[i:i + 1, heads],
                    (pick(dq, heads), pick(dk, slice(hk, hk + 1)), pick(dv, slice(hk, hk + 1))), kind, True, 0, None)


def test_long_rows_in_full():
    """5000 causal rows of 128 columns, one head: every row of the output and of
    the three gradients against float64."""
    ds = require_gpu()
    case = [randn((1, 5000, 1, 128), 380 + i, "bf16") for i in range(4)]
    q, k, v, do = case
    o, lse = ds.attn_forward(q, k, v, causal=True)
    grads = ds.attn_backward(do, q, k, v, o, lse, causal=True)
    torch.cuda.synchronize()
    check_dense(case, o, lse, grads, "bf16", True, 0, None)


@pytest.mark.parametrize("big", ["k", "q"])
@pytest.mark.parametrize("sigma", [1e-5, 1e-4, 300.0, 5000.0])
@pytest.mark.parametrize("tq,hq,d,causal", [(1500, 4, 64, True), (700, 1, 128, True), (300, 2, 64, False)])
def test_fp16_gradients_small_and_large(monkeypatch, big, sigma, tq, hq, d, causal):
    """Score gradients of 1e-9 to 1e5, past both ends of fp16.  Inside, P and dS are
    carried times 2^15, or less where that would leave the type: they lose their
    rounding (2^-11) and, of dS, at most 2^-36 of the largest; the outputs lose what
    fp16 loses at their size.  Keys large beside queries (or the other way round)
    bring dQ (dK) into fp16's normal range, or keep it from the upper end."""
    ds = require_gpu()
    say("attention fp16", big, sigma, tq, hq, d, causal)
    up = 2.0 ** 8 if sigma < 1 else 2.0 ** -6
    q, k, v, do = (randn((1, tq, h, d), 400 + i, "f16") for i, h in enumerate((hq, 1, 1, hq)))
    q, k = (q / up, k * up) if big == "k" else (q * up, k / up)
    do = (do.float() * sigma).half()
    o, lse = ds.attn_forward(q, k, v, causal=causal)
    grads = ds.attn_backward(do, q, k, v, o, lse, causal=causal)
    torch.cuda.synchronize()
    qn, kn, vn, gn = (f64(x)[0] for x in (q, k, v, do))
    see = at.visible(tq, tq, causal, 0)
    sums = [0.0] * 4
    for h in range(hq):
        args = qn[:, h], kn[:, 0], vn[:, 0]
        _, _, p, _ = at.forward(*args, d ** -0.5, see)
        top = np.abs(p * (gn[:, h] @ vn[:, 0].T - (gn[:, h] * (p @ vn[:, 0])).sum(1, keepdims=True))).max()
        monkeypatch.setitem(at.TINY, "f16", 2.0 ** -40 + 2.0 ** -36 * top)
        r = at.backward(gn[:, h], *args, d ** -0.5, see)
        t = at.backward_tolerance(gn[:, h], *args, d ** -0.5, see, "f16")
        if big == "k":
            check(f64(grads[0])[0, :, h], r[0], t[0] + 2.0 ** -25, (h, "dq"))
        sums = [a + b for a, b in zip(sums, (r[1], r[2], t[1], t[2]))]
    if big == "q":
        check(f64(grads[1])[0, :, 0], sums[0], sums[2] + 2.0 ** -25, "dk")
    if sigma < 1000:
        check(f64(grads[2])[0, :, 0], sums[1], sums[3] + 2.0 ** -25, "dv")


def test_an_infinite_fp16_gradient_stays_in_its_row():
    """A gradient that overflowed in one row reaches that row's dQ and the keys it
    sees; keys after it (in the same tile) keep their bits, and so do other rows."""
    ds = require_gpu()
    q, k, v, do = (randn((1, 200, 1, 64), 420 + i, "f16") for i in range(4))
    o, lse = ds.attn_forward(q, k, v, causal=True)
    ref = ds.attn_backward(do, q, k, v, o, lse, causal=True)
    do2 = do.clone()
    do2[0, 70, 0, 5] = float("inf")
    got = ds.attn_backward(do2, q, k, v, o, lse, causal=True)
    torch.cuda.synchronize()
    rows = [i for i in range(200) if i != 70]
    assert torch.equal(got[0][0, rows], ref[0][0, rows]) and not torch.isfinite(got[0][0, 70]).any()
    assert not torch.isfinite(got[1][0, :71]).any() and torch.equal(got[1][0, 71:], ref[1][0, 71:])


@pytest.mark.parametrize("make", [
    lambda x: torch.cat([x.reshape(-1)[:1], x.reshape(-1)])[1:].view(x.shape),        # contiguous, off 16 bytes
    lambda x: x.transpose(1, 2).contiguous().transpose(1, 2),
    lambda x: torch.nn.functional.pad(x, (0, 4))[..., :64]])
def test_gradients_in_any_layout(make):
    """The autograd function takes the output's gradient wherever it stands."""
    ds = require_gpu()
    leaf = [randn((2, 60, h, 64), 430 + i, "bf16").requires_grad_() for i, h in enumerate((4, 2, 2))]
    do = randn((2, 60, 4, 64), 440, "bf16")
    o, lse = ds.attn_forward(*[x.detach() for x in leaf], causal=True)
    ref = ds.attn_backward(do, *[x.detach() for x in leaf], o, lse, causal=True)
    y = ds.attention(*leaf, causal=True)
    got = torch.autograd.grad(y, leaf, make(do))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
