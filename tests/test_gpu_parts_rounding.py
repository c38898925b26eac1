"""Merges with the running sum in parts against the one-step merges, element by element in bf16 (GPU).

Two merges of the same row add the score's sums in another order, so their fp32
results z and z' may differ by ORDER = 1e-6 of the largest output (the bound the
fp32 outputs are held to). Each is then rounded to bf16, which moves it by at most
half a step of its own binade: |bf16(z) - bf16(z')| <= |z - z'| + one step of the
larger. With 8 bits a step at a is 2^-7 2^floor(log2 |a|), between 2^-8 |a| and
2^-7 |a|: a bound of 2^-8 of the largest output does not cover it.
"""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests._gpu import dev
from tests.test_gpu_parts import _one_step_sums, _pass_by_one_step_calls

pytestmark = pytest.mark.gpu
ORDER = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def within_one_step(a, b):
    a, b = a.double(), b.double()
    larger = torch.maximum(a.abs(), b.abs())
    step = 2.0 ** -7 * torch.exp2(torch.floor(torch.log2(larger.clamp(min=2.0 ** -126))))
    assert ((a - b).abs() <= step + ORDER * larger.max()).all()


def _inputs(seed, J, T, d):
    g = inputs.generator(seed, dev())
    F, O = inputs.randn((J, T, d), "bf16", g, dev()), inputs.randn((T, d), "bf16", g, dev())
    w = inputs.queries(1, d, 0.05, g, dev())[0]
    gamma = 1 + 0.3 * inputs.queries(1, d, 1.0, g, dev())[0]
    return F, O, torch.randn(T, device=dev(), generator=g), w, gamma


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("T,d", [(300, 1024), (77, 2048), (45, 640), (13, 100), (9, 3)])
def test_merges_in_parts(T, d, seed):
    J = 6
    F, O, lse, w, gamma = _inputs(200 + seed, J, T, d)
    sums = _one_step_sums(F, J)

    def out():
        return torch.full((T, d), float("nan"), device=dev(), dtype=torch.bfloat16)
    for j in range(1, J + 1):
        ref = out()
        ar.attnres_block_merge(O, lse, sums[j - 1].clone(), None, False, w, gamma, 1e-6, ref)
        for m in range(0, j + 1):
            base = sums[m - 1] if m > 0 else None
            if base is None and m == j:
                continue
            got = out()
            ar.attnres_block_merge_parts(O, lse, base, F[m:], j - m, None, w, gamma, 1e-6, got)
            within_one_step(got, ref)
            if j == J:
                continue
            got, summary = out(), out()
            ar.attnres_block_merge_parts(O, lse, base, F[m:], j - m, None, w, gamma, 1e-6, got, summary_out=summary)
            within_one_step(got, ref)


@pytest.mark.parametrize("N,S,T,d", [(3, 6, 200, 2048), (3, 8, 130, 1024), (2, 16, 33, 256), (3, 5, 21, 100)])
def test_a_block_pass(N, S, T, d):
    g = inputs.generator(210, dev())
    emb, F = inputs.randn((T, d), "bf16", g, dev()), inputs.randn((N * S, T, d), "bf16", g, dev())
    W = inputs.queries(N * S, d, 0.05, g, dev())
    G = 1 + 0.2 * inputs.queries(N * S, d, 1.0, g, dev())
    ref, _ = _pass_by_one_step_calls(F, emb, N, S, W, G)
    Src = torch.empty(N, T, d, device=dev(), dtype=emb.dtype)
    Src[0].copy_(emb)
    O = torch.empty(max(S - 1, 1), T, d, device=dev(), dtype=emb.dtype)
    out = torch.empty(N * S, T, d, device=dev(), dtype=emb.dtype)
    ar.attnres_block_pass(F, N, S, W, G, 1e-6, Src, O, torch.empty(S, T, device=dev()), torch.empty(T, d, device=dev()), out)
    for k in range(N * S):
        within_one_step(out[k], ref[k])
