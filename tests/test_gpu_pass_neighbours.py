"""A Block pass next to kernels that let the following one start at once, without a wait of the host between (GPU).

The library's kernels start while the one before them still runs and wait for it
inside; some fetch or write what that one does not touch before they wait. What
must hold all the same: the pass reads what the call before it wrote, and the
call after it reads what the pass wrote. Each chain is run as it is and with the
device synchronised after every call, eagerly and in a graph, on sizes that
leave most of the GPU free for the next kernel; the results must be the same
bits.
"""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests._gpu import dev

pytestmark = pytest.mark.gpu
SHAPES = [(1, 2, 1, 512), (2, 3, 8, 1024), (2, 6, 64, 2048), (2, 3, 40, 8192), (2, 4, 1000, 896)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Pass:
    def __init__(self, N, S, T, d):
        g = inputs.generator(95, dev())
        self.shape, self.T, self.d = (N, S), T, d
        self.F = inputs.randn((N * S, T, d), "bf16", g, dev())
        self.W, self.G = inputs.queries(N * S, d, 0.05, g, dev()), torch.ones(N * S, d, device=dev())
        self.Src = torch.empty(N + 1, T, d, device=dev(), dtype=torch.bfloat16)
        self.Src[0].copy_(self.F[0])
        self.O = torch.empty(S - 1, T, d, device=dev(), dtype=torch.bfloat16)
        self.lse, self.P = torch.empty(S, T, device=dev()), torch.empty(T, d, device=dev())
        self.out = torch.empty(N * S, T, d, device=dev(), dtype=torch.bfloat16)
        self.gain = torch.ones(d, device=dev())
        self.f = [inputs.randn((T, d), "bf16", g, dev()) for _ in range(2)]
        self.rows = [torch.empty_like(self.f[0]) for _ in range(2)]

    def source(self, which):
        """The first output f as a gated residual leaves it."""
        ar.attnres_gated_residual(self.f[which], None, self.gain, 1e-6, None, 1, 0, 1.0, self.F[0])

    def run(self, freeze_last=False):
        ar.attnres_block_pass(self.F, *self.shape, self.W, self.G, 1e-6, self.Src, self.O, self.lse, self.P, self.out,
                              freeze_last=freeze_last)

    def reader(self, which):
        """The last read into a gated residual, whose rows the next call overwrites nothing of."""
        ar.attnres_gated_residual(self.out[-1], None, self.gain, 1e-6, None, 1, 0, 1.0, self.rows[which])


def check(calls, results):
    """calls of one chain; results: the tensors it leaves, in a copy."""
    want = []
    for c in calls:
        c()
        torch.cuda.synchronize()
    want = [t.clone() for t in results]

    def poison():
        for t in results:
            t.fill_(float("nan"))

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(results, want))
    for _ in range(40):
        poison()
        for c in calls:
            c()
        assert same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for c in calls:
            c()
    for _ in range(40):
        poison()
        graph.replay()
        assert same()


@pytest.mark.parametrize("N,S,T,d", SHAPES)
def test_the_pass_reads_what_the_call_before_it_wrote(N, S, T, d):
    p = Pass(N, S, T, d)
    keep = torch.empty_like(p.out)
    # Twice with another first output each, so that what was there before is never the right one.
    check([lambda: p.source(0), p.run, lambda: keep.copy_(p.out), lambda: p.source(1), p.run], [keep, p.out])


@pytest.mark.parametrize("N,S,T,d", SHAPES)
def test_the_call_after_a_frozen_pass_reads_what_it_wrote(N, S, T, d):
    p = Pass(N, S, T, d)
    # The last merge writes out[-1], and the freeze after it, which need not wait for the merge, ends the pass.
    check([lambda: p.source(0), lambda: p.run(True), lambda: p.reader(0), lambda: p.source(1), lambda: p.run(True),
           lambda: p.reader(1)], p.rows + [p.out, p.Src[1:]])
