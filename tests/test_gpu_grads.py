"""The global gradient norm and clipping on the GPU against fp64.

Tolerances: the norm's square is a sum of squares: batches of at most 32 (a chain of at most 16 packed additions
and one more; allowed for: 32), their sum with its rounding carried (4), a warp's and a CTA's trees (10), the CTAs' (13), each
addition within 2^-24 of positive terms: 64 x 2^-24, half of which reaches the norm, with a square root and its
own rounding 2 more. A clipped element is one product with max_norm / norm (the norm's error, a division and the
product: 2 more roundings), then its own rounding.
"""
import math

import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests import _residual as ref
from tests._gpu import dev, dtype_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def norm_bound():
    return (64 / 2 + 2) * U


def make(sizes, kinds, seed=0, shift=0, std=1.0):
    g = inputs.generator(seed, dev())
    out = []
    for i, n in enumerate(sizes):
        t = torch.empty(n + shift, device=dev(), dtype=dtype_of(kinds[i % len(kinds)]))[shift:]
        out.append(t.copy_(inputs.randn((n,), "f32", g, dev(), scale=std / (1 + i % 5))))
    return out


def check_clip(grads, outs_types=None, max_norm=1.0):
    keep = [t.clone() for t in grads]
    want = ref.norm_of(keep)
    e = norm_bound()
    norm = torch.full((1,), -1.0, device=dev())
    ar.attnres_grad_norm(grads, norm)
    assert abs(float(norm) - want) <= e * want
    first = norm.clone()
    by = max_norm / want if want > max_norm else 1.0
    outs = None if outs_types is None else [torch.full(t.shape, float("nan"), device=dev(), dtype=dtype_of(k))
                                            for t, k in zip(grads, outs_types)]
    norm.fill_(-1.0)
    ar.attnres_grad_clip(grads, max_norm, norm, outs)
    assert torch.equal(norm, first)
    for a, b in zip(keep, grads if outs is None else outs):
        value = a.double() * by
        ref.check(b, value, (e + 3 * U) * value.abs(), "clipped")
    if outs is not None:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))


@pytest.mark.parametrize("kinds", [["f32"], ["bf16"], ["bf16", "f32"]])
@pytest.mark.parametrize("sizes", [[1], [7], [2048], [2049], [5000, 1, 0, 3, 2047], [896] * 128, [0, 0, 4],
                                   [1_000_003, 17, 65536, 2], [3] * 300, [100] * 1100 + [70_000]])
def test_norm_and_clip(sizes, kinds):
    check_clip(make(sizes, kinds))


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_out_of_place_and_unaligned(shift, out):
    sizes = [4099, 5, 20_000, 8, 2048 * 9]
    grads = make(sizes, ["bf16", "f32"], shift=shift)
    check_clip(grads, [out] * len(sizes))
    check_clip(grads)


def test_large_lists():
    check_clip(make([40_000_000, 3, 10_000_001], ["bf16", "f32"]), ["bf16", "f32", "bf16"])


def test_small_gradients_behind_large_ones():
    # Most of the norm is in 20 million elements that are each 2^-10 of the first ones: added one by one in fp32
    # to the large ones' squares they would all be lost.
    grads = [torch.full((1 << 16,), 1.0, device=dev()), torch.full((20_000_000,), 2.0 ** -10, device=dev()),
             torch.full((20_000_000,), 2.0 ** -10, device=dev(), dtype=torch.bfloat16)]
    want = math.sqrt((1 << 16) + 40_000_000 * 2.0 ** -20)
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_norm(grads, norm)
    assert abs(float(norm) - want) <= norm_bound() * want
    mixed = make([3_000_000] * 4, ["f32"])
    for i, t in enumerate(mixed):
        t.mul_(10.0 ** -i)
    want = ref.norm_of(mixed)
    ar.attnres_grad_norm(mixed, norm)
    assert abs(float(norm) - want) <= norm_bound() * want


def test_shapes_other_than_vectors():
    g = make([64 * 100], ["f32"])[0].view(64, 100)
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_clip([g, torch.tensor(2.0, device=dev())], 0.5, norm)
    total = ref.norm_of([g])
    assert total <= 0.5


@pytest.mark.parametrize("max_norm", [1e9, float("inf")])
def test_below_the_limit_nothing_changes(max_norm):
    grads = make([5000, 33], ["bf16", "f32"])
    keep = [t.clone() for t in grads]
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_clip(grads, max_norm, norm)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    outs = [torch.empty_like(t) for t in grads]
    ar.attnres_grad_clip(grads, max_norm, norm, outs)
    assert all(torch.equal(a, b) for a, b in zip(keep, outs))


def test_zero_gradients_and_none_at_all():
    grads = [torch.zeros(100, device=dev()), torch.zeros(3, device=dev(), dtype=torch.bfloat16)]
    norm = torch.full((1,), -1.0, device=dev())
    ar.attnres_grad_clip(grads, 0.0, norm)
    assert float(norm) == 0.0 and all((t == 0).all() for t in grads)
    norm.fill_(-1.0)
    ar.attnres_grad_norm([], norm)
    assert float(norm) == 0.0
    norm.fill_(-1.0)
    ar.attnres_grad_clip([torch.empty(0, device=dev())], 1.0, norm)
    assert float(norm) == 0.0
    ones = [torch.ones(10, device=dev())]
    ar.attnres_grad_clip(ones, 0.0, norm)
    assert (ones[0] == 0).all()


@pytest.mark.parametrize("size", [1e-38, 3e-30, 1e-20, 1e-12, 1e12, 3e19, 1e30, 2e36])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_over_the_whole_range(size, kind):
    # Squares of these leave fp32's range at both ends; the norm does not.
    grads = [(inputs.randn((n,), "f32", inputs.generator(n, dev()), dev()).clamp_(-3, 3) * size).to(dtype_of(kind))
             for n in (3000, 11)]
    want = ref.norm_of(grads)
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_norm(grads, norm)
    # Elements under 2^-126 after the scaling (or whose scaled squares are) cost at most a normal minimum each.
    assert abs(float(norm) - want) <= norm_bound() * want + 2.0 ** -140
    ar.attnres_grad_norm(grads + [torch.full((5,), 1.0, device=dev())], norm)
    both = math.hypot(want, math.sqrt(5.0))
    assert abs(float(norm) - both) <= norm_bound() * both


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    grads = make([5000, 33], ["bf16", "f32"])
    grads[1][7] = bad
    keep = [t.clone() for t in grads]
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_clip(grads, 1.0, norm)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    assert all(torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                           b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32)) for a, b in zip(keep, grads))


def test_a_tensor_twice_counts_twice():
    t = make([1000], ["f32"])[0]
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_norm([t, t], norm)
    want = math.sqrt(2) * ref.norm_of([t])
    assert abs(float(norm) - want) <= norm_bound() * want
    with pytest.raises(ar.AttnResError):
        ar.attnres_grad_clip([t, t], 1.0, norm)


def test_nothing_else_is_written():
    pad, sizes = 256, [5, 4099, 64]
    bufs = [torch.full((n + 2 * pad,), 777.0, device=dev(), dtype=dtype_of(k)) for n, k in zip(sizes, ("bf16", "f32", "bf16"))]
    views = [b[pad:pad + n] for b, n in zip(bufs, sizes)]
    for v, s in zip(views, make(sizes, ["f32"])):
        v.copy_(s)
    need = ar.attnres_grad_norm_scratch_floats(3)
    scratch = torch.full((need + 2 * pad,), 777.0, device=dev())
    norm = torch.full((3,), 777.0, device=dev())
    ar.attnres_grad_clip(views, 0.1, norm[1:2], scratch=scratch[pad:pad + need])
    assert float(norm[0]) == float(norm[2]) == 777.0
    for b in bufs + [scratch]:
        assert (b[:pad] == 777.0).all() and (b[-pad:] == 777.0).all()


def test_list_kept_and_replayed_on_new_values():
    grads = make([100_000, 77, 3000], ["f32", "bf16"])
    outs = [torch.empty_like(t) for t in grads]
    kept = ar.GradList(grads, outs)
    norm = torch.empty(1, device=dev())
    scratch = torch.full((kept.scratch_floats,), float("nan"), device=dev())
    other = ar.GradList(make([50_000] * 40, ["bf16"], seed=9))
    norm2 = torch.empty(1, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        ar.attnres_grad_clip(kept, 1.0, norm, scratch=scratch)
        ar.attnres_grad_norm(other, norm2, scratch=scratch)
        torch.cuda.synchronize()
        for call in (lambda: ar.attnres_grad_clip(kept, 1.0, norm, scratch=scratch),
                     lambda: ar.attnres_grad_norm(other, norm2, scratch=scratch)):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                call()
            graphs.append(graph)
        for t, v in zip(grads, make([100_000, 77, 3000], ["f32"], seed=5, std=3.0)):
            t.copy_(v)
        for _ in range(3):
            for graph in graphs:
                graph.replay()
    s.synchronize()
    want = ref.norm_of(grads)
    assert abs(float(norm) - want) <= norm_bound() * want
    for a, b in zip(grads, outs):
        ref.check(b, a.double() / want, (norm_bound() + 3 * U) * a.double().abs() / want)
    want = ref.norm_of(other.grads)
    assert abs(float(norm2) - want) <= norm_bound() * want


def test_another_stream_and_lists_made_for_the_call():
    grads = make([300_000, 5, 4097], ["f32", "bf16"])
    want = ref.norm_of(grads)
    s, norm = torch.cuda.Stream(), torch.full((1,), -1.0, device=dev())
    s.wait_stream(torch.cuda.current_stream())
    ar.attnres_grad_norm(grads, norm, stream=s)
    s.synchronize()
    assert abs(float(norm) - want) <= norm_bound() * want
    torch.cuda.synchronize()
    ar.attnres_grad_clip(tuple(grads), want / 3, norm, stream=s.cuda_stream)
    s.synchronize()
    assert abs(ref.norm_of(grads) - want / 3) <= 2.0 ** -8 * want


def test_refusals():
    norm = torch.empty(1, device=dev())
    g = torch.ones(10, 10, device=dev())
    for bad in ([g.t()[:, :3]], [g.half()], [g.cpu()]):
        with pytest.raises((ValueError, TypeError)):
            ar.attnres_grad_norm(bad, norm)
    for bad in (torch.empty(2, device=dev()), torch.empty(1), torch.empty(1, device=dev(), dtype=torch.float64)):
        with pytest.raises(ValueError):
            ar.attnres_grad_norm([g], bad)
    with pytest.raises(ValueError):
        ar.attnres_grad_clip([g], 1.0, norm, [torch.empty(99, device=dev())])
    with pytest.raises(ValueError):
        ar.attnres_grad_clip(ar.GradList([g]), 1.0, norm, [g])
    with pytest.raises(ValueError):
        ar.attnres_grad_norm([g], norm, scratch=torch.empty(3, device=dev()))
    with pytest.raises(ar.AttnResError):
        ar.attnres_grad_clip([g], -1.0, norm)


def test_a_tensor_past_32_bit_offsets():
    n = (1 << 31) + 12345
    t = torch.zeros(n, device=dev(), dtype=torch.bfloat16)
    t[-3:], t[5] = 2.0, 1.0
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_clip([t], 1.0, norm)
    want = math.sqrt(13.0)
    assert abs(float(norm) - want) <= norm_bound() * want
    ref.check(t[-3:], torch.full((3,), 2.0 / want, dtype=torch.float64, device=dev()),
              torch.full((3,), 40 * U, dtype=torch.float64, device=dev()), "clipped")
    assert int((t != 0).sum()) == 4


@pytest.mark.parametrize("max_norm", [1e-3, 1e-8, 1e-20, 1e-30])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e12, 1e30, 2e36])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_clipping_over_the_whole_range(kind, out, size, max_norm):
    # max_norm / norm goes far below fp32's normal range here; the clipped elements do not. Each is a product of at
    # most three rounded factors (the norm's error, its reciprocal, two products), then its own rounding; a factor
    # or an element below 2^-126 is off by at most half a step of 2^-149, the factor times a max_norm under 4.
    grads = [(inputs.randn((n,), "f32", inputs.generator(n, dev()), dev()).clamp_(-3, 3) * size).to(dtype_of(kind))
             for n in (3000, 11, 8, 2049)]
    want = ref.norm_of(grads)
    by = min(1.0, max_norm / want)
    for outs in (None, [torch.full(t.shape, float("nan"), device=dev(), dtype=dtype_of(out)) for t in grads]):
        if outs is None and kind != out:
            continue
        mine = [t.clone() for t in grads]
        norm = torch.empty(1, device=dev())
        ar.attnres_grad_clip(mine, max_norm, norm, outs)
        for a, b in zip(grads, mine if outs is None else outs):
            value = a.double() * by
            half = ref.HALF[b.dtype]
            tiny = 2.0 ** -134 if b.dtype == torch.bfloat16 else 2.0 ** -150   # half a step below the normal range
            limit = (norm_bound() + 3 * U) * value.abs() + 2.0 ** -148
            limit = limit + torch.clamp(half * (value.abs() + limit), min=tiny)
            assert torch.isfinite(b.float()).all()
            assert ((b.double() - value).abs() <= limit).all()


def test_the_longest_table_captured():
    # More tensors than one launch takes, their addresses as a captured kernel's arguments.
    grads = make([100] * 1100 + [70_000], ["f32", "bf16"])
    outs = [torch.empty_like(t) for t in grads]
    kept, norm = ar.GradList(grads, outs), torch.empty(1, device=dev())
    scratch = torch.empty(kept.scratch_floats, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.attnres_grad_clip(kept, 1.0, norm, scratch=scratch)
    for t in grads:
        t.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    want = ref.norm_of(grads)
    assert abs(float(norm) - want) <= norm_bound() * want
    for a, b in zip(grads, outs):
        ref.check(b, a.double() / want, (norm_bound() + 3 * U) * a.double().abs() / want, "clipped")
