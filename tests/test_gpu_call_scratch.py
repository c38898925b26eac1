"""Calls that allocate their own scratch, on a stream other than the current one (GPU).

The allocator gives a freed tensor's block to the next request of the stream it
was allocated on, because work queued on that stream comes after whatever
still uses the block. A call on another stream must not get such a block: what
the current stream has queued would overwrite the call's partial sums, or be
overwritten by them. So each call here runs while the current stream still has
work queued on a freed block of exactly the scratch's size, and both that
work's result and the call's are compared bit for bit with undisturbed ones.
"""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests._gpu import dev

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # clock cycles that the current stream is kept waiting: 0.1 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _gated(g):
    T, d = 3000, 896
    f, x, dn, gate = (inputs.randn((T, d), "bf16", g, dev()) for _ in range(4))
    gain = torch.ones(d, device=dev())
    outs = [torch.empty_like(f), torch.empty_like(f), torch.empty_like(f), torch.empty(d, device=dev()),
            torch.empty(d, device=dev())]
    return ar.attnres_gated_residual_bwd_scratch_floats(T, d), outs, lambda s: ar.attnres_gated_residual_bwd(
        f, gain, 1e-6, gate, 1, ar.GATE_SIGMOID, 0.5, x, gain, 1e-6, x, dn, *outs, accumulate=False, stream=s)


def _general(g):
    # Rows off the vector width: the scratch holds the rows' statistics as well.
    T, d = 3000, 99
    x, dy = (inputs.randn((T, d), "f32", g, dev()) for _ in range(2))
    gain = torch.ones(d, device=dev())
    outs = [torch.empty_like(x), torch.empty(d, device=dev())]
    return ar.attnres_rmsnorm_bwd_scratch_floats(T, d), outs, lambda s: ar.attnres_rmsnorm_bwd(
        x, gain, 1e-6, dy, None, outs[0], outs[1], accumulate=False, stream=s)


def _rmsnorm(g):
    T, d = 2000, 1024
    x, dy = (inputs.randn((T, d), "bf16", g, dev()) for _ in range(2))
    gain = torch.ones(d, device=dev())
    outs = [torch.empty_like(x), torch.empty(d, device=dev())]
    return ar.attnres_rmsnorm_bwd_scratch_floats(T, d), outs, lambda s: ar.attnres_rmsnorm_bwd(
        x, gain, 1e-6, dy, None, outs[0], outs[1], accumulate=False, stream=s)


def _norm(g):
    grads = [inputs.randn((n,), "f32", g, dev()) for n in (300_000, 77)]
    outs = [torch.empty(1, device=dev())]
    kept = ar.GradList(grads)
    return kept.scratch_floats, outs, lambda s: ar.attnres_grad_norm(kept, outs[0], stream=s)


def _clip(g):
    grads = [inputs.randn((n,), "f32", g, dev()) for n in (300_000, 77)]
    outs = [torch.empty(1, device=dev())] + [torch.empty_like(t) for t in grads]
    kept = ar.GradList(grads, outs[1:])
    return kept.scratch_floats, outs, lambda s: ar.attnres_grad_clip(kept, 1.0, outs[0], stream=s)


def _block(g):
    N, S, T, d = 2, 3, 200, 256
    Src, F = inputs.randn((N, T, d), "f32", g, dev()), inputs.randn((N * S, T, d), "f32", g, dev())
    W, G = inputs.queries(N * S, d, 0.05, g, dev()), torch.ones(N * S, d, device=dev())
    dOut = inputs.randn((N * S, T, d), "f32", g, dev())
    # (added to: zeroed before each call, on the call's stream)
    outs = [torch.zeros(T, d, device=dev()), torch.zeros(N * S, T, d, device=dev())]

    def run(s):
        with torch.cuda.stream(s):
            for t in outs:
                t.zero_()
        ar.attnres_block_bwd(Src, F, N, S, W, G, 1e-6, dOut, outs[0], outs[1], stream=s)
    return ar.attnres_block_bwd_scratch_floats(N, S, T, d), outs, run


@pytest.mark.parametrize("make", [_gated, _general, _rmsnorm, _norm, _clip, _block])
def test_scratch_of_a_call_on_another_stream(make):
    floats, outs, run = make(inputs.generator(90, dev()))
    here, s = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    run(here)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.fill_(float("nan"))
    total = torch.empty(floats, device=dev())
    s.wait_stream(here)
    s.synchronize()
    # The current stream: wait, read a block, then fill it; the block is free again for its pool as soon as that is queued.
    block = torch.full((floats,), 3.0, device=dev())
    address = block.data_ptr()
    torch.cuda._sleep(BUSY)
    total.copy_(block)
    block.fill_(float("nan"))
    del block
    assert torch.empty(floats, device=dev()).data_ptr() == address  # the pool's next block, while work on it is queued
    run(s)
    torch.cuda.synchronize()
    assert (total == 3.0).all()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_scratch_of_calls_by_handle():
    floats, outs, run = _rmsnorm(inputs.generator(91, dev()))
    run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for handle in (0, torch.cuda.Stream().cuda_stream):  # the default stream, from inside another one
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            run(handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
