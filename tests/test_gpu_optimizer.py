"""AdamW as a torch optimizer where its tensors differ: in the steps they have
taken part in (counts on the host and on the device, in graphs too), in type."""
import copy

import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

LR, WD = 1e-2, 0.1


def grads(t, shapes):
    """Gradients that do not depend on the weights."""
    g = torch.Generator().manual_seed(100 + t)
    return [torch.randn(s, generator=g).cuda() for s in shapes]


SHAPES = [(30, 40), (77,), (5, 9)]


def close(ps, qs, steps):
    """Within what two fp32 evaluations of that many steps may differ by: an update
    is at most lr (1 - b1) / sqrt(1 - b2) = 3.2 lr, its bias corrections and its own
    arithmetic are right to 2e-5, and a step rounds the weight at most 4 times a side."""
    for p, q in zip(ps, qs):
        tol = steps * (2e-5 * 3.2 * LR + 8 * 2.0 ** -24 * max(p.abs().max().item(), 1.0))
        worst = (p.detach().float() - q.detach().float()).abs().max().item()
        assert worst <= tol, (worst, tol)


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_that_join_late_or_miss_steps(capturable, bits):
    """Every tensor is stepped with its own count, as torch's AdamW does.  8-bit
    states round the moments, so their weights are compared with those of the same
    tensors stepped alone, each in an optimizer of its own."""
    ds = require_gpu()
    say("optimizer", capturable, bits)
    torch.manual_seed(1)
    start = [torch.randn(s, device="cuda") for s in SHAPES]
    present = [[0], [0], [0, 2], [0, 1, 2], [0, 1], [1, 2], [0, 1, 2], [1], [0, 1, 2]]
    mine = [torch.nn.Parameter(x.clone()) for x in start]
    opt = ds.AdamW(mine, lr=LR, weight_decay=WD, state_bits=bits, capturable=capturable)
    ref = [torch.nn.Parameter(x.clone()) for x in start]
    if bits == 32:
        opts = [torch.optim.AdamW(ref, lr=LR, weight_decay=WD)]
    else:
        opts = [ds.AdamW([p], lr=LR, weight_decay=WD) for p in ref]
    for t, some in enumerate(present):
        for ps in (mine, ref):
            for i, (p, g) in enumerate(zip(ps, grads(t, SHAPES))):
                p.grad = g if i in some else None
        opt.step()
        for o in opts:
            o.step()
    torch.cuda.synchronize()
    if bits == 32:
        close(mine, ref, len(present))
    else:
        # a moment is off by at most an eighth a step: half an update in all is a wide
        # bound for it, and a wrong first count is off by 2 updates
        for p, q in zip(mine, ref):
            assert (p - q).abs().mean().item() < 0.5 * LR
    assert [int(opt.state[p]["step"]) for p in mine] == [sum(i in s for s in present) for i in range(3)]


def test_a_captured_step_of_tensors_at_different_counts():
    """Replays step each tensor with its own count, also after an eager step that
    only some of them took part in."""
    ds = require_gpu()
    torch.manual_seed(2)
    start = [torch.randn(s, device="cuda") for s in SHAPES]
    mine = [torch.nn.Parameter(x.clone()) for x in start]
    ref = [torch.nn.Parameter(x.clone()) for x in start]
    opt = ds.AdamW(mine, lr=LR, weight_decay=WD, capturable=True)
    opt2 = torch.optim.AdamW(ref, lr=LR, weight_decay=WD)
    static = [torch.zeros(s, device="cuda") for s in SHAPES]
    steps = 0

    def load(t, some):
        for p, q, buf, g, i in zip(mine, ref, static, grads(t, SHAPES), range(3)):
            buf.copy_(g)
            p.grad, q.grad = (buf, g) if i in some else (None, None)

    def eager(t, some):
        load(t, some)
        opt.step()
        opt2.step()

    for t, some in enumerate([[0], [0], [0], [0, 1, 2]]):
        eager(t, some)
        steps += 1
    load(9, [0, 1, 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for t in range(10, 16):
        load(t, [0, 1, 2])
        graph.replay()
        opt2.step()
        steps += 1
        torch.cuda.synchronize()
        close(mine, ref, steps)
        if t == 12:
            eager(20, [1])
            steps += 1
    torch.cuda.synchronize()
    close(mine, ref, steps)
    assert [int(opt.state[p]["step"]) for p in mine] == [10, 8, 7]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_half_precision_parameters_resume(bits, capturable):
    """bf16 and fp16 parameters with masters: a state_dict (whose floating states
    torch's loading casts to the parameter's type) resumes to the same bits."""
    ds = require_gpu()
    torch.manual_seed(3)
    types = [torch.bfloat16, torch.float16, torch.bfloat16]
    mine = [torch.nn.Parameter(torch.randn(s, device="cuda").to(d)) for s, d in zip(SHAPES, types)]
    make = lambda ps: ds.AdamW(ps, lr=LR, weight_decay=WD, state_bits=bits, capturable=capturable)

    def run(opt, ps, ts):
        for t in ts:
            for p, g in zip(ps, grads(t, SHAPES)):
                p.grad = g.to(p.dtype)
            opt.step()

    opt = make(mine)
    run(opt, mine, range(4))
    saved, now = copy.deepcopy(opt.state_dict()), [p.detach().clone() for p in mine]
    run(opt, mine, range(4, 8))
    again = [torch.nn.Parameter(x) for x in now]
    opt2 = make(again)
    opt2.load_state_dict(saved)
    for p in again:
        s = opt2.state[p]
        assert s["master"].dtype == torch.float32
        assert s["exp_avg"].dtype == s["exp_avg_sq"].dtype == (torch.float32 if bits == 32 else torch.uint8)
    run(opt2, again, range(4, 8))
    torch.cuda.synchronize()
    for p, q in zip(mine, again):
        assert torch.equal(p, q) and torch.equal(opt.state[p]["master"], opt2.state[q]["master"])


@pytest.mark.parametrize("capturable", [False, True])
def test_a_state_of_the_other_kind_resumes(capturable):
    """A state saved with counts on the host goes on with counts on the device, and
    the other way round, as if it had been of that kind all along (the bias
    corrections of device counts are fp32: `close`)."""
    ds = require_gpu()
    torch.manual_seed(4)
    mine = [torch.nn.Parameter(torch.randn(s, device="cuda")) for s in SHAPES]

    def run(opt, ps, ts):
        for t in ts:
            for p, g in zip(ps, grads(t, SHAPES)):
                p.grad = g
            opt.step()

    opt = ds.AdamW(mine, lr=LR, weight_decay=WD, capturable=not capturable)
    run(opt, mine, range(4))
    again = [torch.nn.Parameter(p.detach().clone()) for p in mine]
    opt2 = ds.AdamW(again, lr=LR, weight_decay=WD, capturable=capturable)
    opt2.load_state_dict(copy.deepcopy(opt.state_dict()))
    assert all(isinstance(opt2.state[p]["step"], torch.Tensor) == capturable for p in again)
    run(opt, mine, range(4, 8))
    run(opt2, again, range(4, 8))
    torch.cuda.synchronize()
    close(mine, again, 4)
    assert all(int(opt2.state[p]["step"]) == 8 for p in again)


@pytest.mark.parametrize("capturable", [False, True])
def test_groups_round_by_bits_of_their_own(capturable):
    """Equal tensors with equal gradients at the same place of two groups: the same
    moments before rounding, rounded by different bits.  Of 4096 elements about a
    third would differ if the bits were independent; equal bits differ nowhere."""
    ds = require_gpu()
    ps = [torch.nn.Parameter(torch.ones(4096, device="cuda")) for _ in range(3)]
    opt = ds.AdamW([dict(params=ps[:1]), dict(params=ps[1:2], weight_decay=0.0), dict(params=ps[2:])], lr=LR,
                   state_bits=8, capturable=capturable)
    g = grads(0, [(4096,)])[0]
    for _ in range(2):
        for p in ps:
            p.grad = g
        opt.step()
        torch.cuda.synchronize()
        for key in ("exp_avg", "exp_avg_sq"):
            for i in range(3):
                a, b = opt.state[ps[i]][key], opt.state[ps[i - 1]][key]
                assert (a != b).float().mean().item() > 0.05, (key, i)


def test_a_graph_from_before_the_step_raises():
    """A backward pass through parameters that the step has changed since raises, as
    after torch's optimizers, instead of mixing old and new values."""
    ds = require_gpu()
    p = torch.nn.Parameter(torch.ones(64, device="cuda"))
    opt = ds.AdamW([p], lr=LR)
    loss = (p * p).sum()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()
    opt.zero_grad()
    (p * p).sum().backward()
    opt.step()
    torch.cuda.synchronize()
    assert torch.isfinite(p).all() and (p < 1).all()
