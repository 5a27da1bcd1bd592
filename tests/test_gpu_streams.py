"""Calls on a given stream whose outputs and workspaces are made by the call: the
memory may still be in use by work queued on the current stream."""
import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def bf16(*s):
    return torch.randn(*s, generator=torch.Generator().manual_seed(s[0])).bfloat16().cuda()


def attn_forward(ds):
    q, k = bf16(2, 300, 4, 64), bf16(2, 300, 2, 64)
    return lambda st: ds.attn_forward(q, k, k, causal=True, stream=st)


def attn_backward(ds):
    q, k = bf16(1, 1100, 4, 64), bf16(1, 1100, 1, 64)
    o, lse = ds.attn_forward(q, k, k, causal=True)
    assert ds.attn_workspace_bytes(q, k, True) > 16 * lse.numel()          # partial sums too
    return lambda st: ds.attn_backward(q, q, k, k, o, lse, causal=True, stream=st)


def quantize(ds):
    x = bf16(512, 512)

    def call(st):
        ring = ds.ScaleRing(4, ds.E4M3, stream=st)
        return [ds.fp8_quantize(x, ds.E4M3, ring, stream=st),
                *ds.fp8_quantize_batch([x], ds.E4M3, [ring], stream=st),
                *ds.fp8_quantize_2d(x, ds.E4M3, ring, ds.DUAL, stream=st)]
    return call


def mm(ds):
    ring = ds.ScaleRing(4, ds.E4M3)
    a, b = (ds.fp8_quantize(bf16(n, 256), ds.E4M3, ring) for n in (512, 384))
    args = (a, b, 0, 0, ds.NT, 512, 384, 256, ring, ring)
    return lambda st: [ds.fp8_mm(*args, stream=st), ds.fp8_mm_epilogue(*args, act=ds.ACT_GELU, stream=st)]


def bias_grad(ds):
    g = bf16(4000, 768)
    return lambda st: [ds.fp8_bias_grad(g, stream=st)]


def state_values(ds):
    c = (torch.arange(70000) % 251).to(torch.uint8).cuda()
    e = torch.full((274,), 120, dtype=torch.uint8, device="cuda")
    return lambda st: [ds.adamw_state_values(c, e, True, stream=st)]


@pytest.mark.parametrize("make", [attn_forward, attn_backward, quantize, mm, bias_grad, state_values])
def test_memory_made_for_another_stream_is_free_there(make, monkeypatch):
    """The current stream, behind a pause of some milliseconds, still overwrites
    the freed blocks that the call then gets; its results are right all the same."""
    ds = require_gpu()
    say("streams", make.__name__)
    call = make(ds)
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    made = []                                          # everything the call allocates
    real, real_new, real_like, real_zeros = torch.empty, torch.Tensor.new_empty, torch.empty_like, torch.zeros
    for name, f in (("empty", real), ("empty_like", real_like), ("zeros", real_zeros)):
        monkeypatch.setattr(torch, name, lambda *a, f=f, **k: made.append(f(*a, **k)) or made[-1])
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda *a, **k: made.append(real_new(*a, **k)) or made[-1])
    call(None)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in made]
    monkeypatch.undo()
    del made[:]
    dirty = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    blocks = {t.data_ptr() for t in dirty}
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                      # about 10 ms
    for t in dirty:
        t.fill_(0xFF)
    del dirty, t
    got = call(side)
    assert {t.data_ptr() for t in got} & blocks or make is quantize, "the allocator does not hand out what was freed"
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))


def test_given_outputs_make_no_stream_wait():
    """A call that makes nothing runs beside the current stream's work."""
    ds = require_gpu()
    q = bf16(2, 64, 4, 64)
    o, lse = ds.attn_forward(q, q, q)
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                     # about 100 ms
    ds.attn_forward(q, q, q, out=o, lse=lse, stream=side)
    done.record(side)
    done.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
