"""The Full read over 8-bit rows whose values come near fp32's range.

A row whose squares add up past fp32's range has the score 0 (its mean square is held as infinite), and z is a weighted
mean, so it is finite wherever the values are: no weight, partial sum or product with the query may leave fp32's range
on the way, whatever the order of the sources.
"""
import math

import pytest
import torch

import depth_wise_attention_attnres_gb300 as ar
from tests import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# Each kernel of the read by tokens and features: shared sources (1 to 3 tokens, clusters), warps of their own, wide rows.
FORMS = [(1, 128), (3, 640), (3, 1160), (2, 2048), (300, 300), (700, 2048), (5003, 100), (5003, 256), (3001, 384),
         (5003, 512), (1500, 640), (1200, 896), (2433, 1000), (2433, 1160), (2433, 2048), (5, 2304), (700, 2304)]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def definition(rows, u, eps):
    """z and its bound in fp64. exp's argument is a score's distance to the maximum the weights are scaled by, which is
    at most max(8, ln n) from the scores' own; each of at most n rescalings and the weight take one exp (2^-22, and
    2^-23 of the argument)."""
    n = rows.n
    v = rows.codes.double() * _q8.power(rows.exponents.long() - 127)[..., torch.arange(rows.d, device=DEV) // 128]
    ms = rows.mean_square.double()
    past = ms.isinf()
    size = torch.where(past, 1.0, (ms + eps).sqrt())
    e = torch.where(past, 0.0, (v * u).sum(-1) / size)
    de = ((rows.d + 4) * _q8.U) * (v * u).abs().sum(-1) / size + e.abs() * ((rows.d / 2 + 8) * _q8.U)
    a = torch.softmax(e, 0)
    gap = (e.amax(0) - e).clamp(max=100)
    err = torch.where(past, 0.0, de) + (n + 2) * 2.0 ** -22 + 2 * (gap + 8 + math.log(n)) * 2.0 ** -23 + (2 * n + 24) * _q8.U
    da = a * (err + (a * err).sum(0))
    return (a.unsqueeze(-1) * v).sum(0), (da.unsqueeze(-1) * v.abs()).sum(0)


def check(x, w, gamma, dtype="f32", eps=1e-6):
    n, T, d = x.shape
    rows = ar.attnres_q8_write(x, ar.Q8Rows(n, T, d, device=DEV))
    out = torch.empty(T, d, device=DEV, dtype=TYPES[dtype])
    ar.attnres_full_fwd_q8(rows, n, w, gamma, eps, out)
    assert ar.attnres_device_status() == 0
    z, dz = definition(rows, w.double() * gamma.double(), eps)
    _q8.assert_within(out, z, dz, f"{n} x {T} x {d}")
    # and a query for each token
    Q = w.expand(T, d).contiguous()
    ar.attnres_full_fwd_q8(rows, n, None, gamma, eps, out, Q=Q)
    _q8.assert_within(out, z, dz, f"{n} x {T} x {d}, queries of tokens")
    return rows


def ordinary(n, T, d, g, level):
    """Sources near a constant, so that a query of c / d in each feature gives scores near c."""
    return 0.3 * torch.randn(n, T, d, generator=g, device=DEV) + level


@pytest.mark.parametrize("T,d", FORMS)
def test_a_large_source_past_a_low_score(T, d):
    """Scores of about -6.7, then a source of up to 2e37 with score 0: first, last and in the middle."""
    g = gen(T + d)
    w, gamma = torch.full((d,), 7.0 / d, device=DEV), torch.ones(d, device=DEV)
    for n, at in ((2, 1), (2, 0), (9, 4), (40, 39)):
        if n * T * d > 1 << 26:
            continue
        x = ordinary(n, T, d, g, -1.0)
        x[at] = 2e37 * (2 * torch.rand(T, d, generator=g, device=DEV) - 1)
        rows = check(x, w, gamma, "bf16" if n == 9 else "f32")
        assert rows.mean_square[at].isinf().all()


@pytest.mark.parametrize("T,d", FORMS)
def test_sources_whose_sum_passes_the_range(T, d):
    """Sources of up to 3e38 of one sign, all with score 0: z is their mean."""
    g = gen(T + d + 1)
    w, gamma = torch.randn(d, generator=g, device=DEV) / d, torch.ones(d, device=DEV)
    for n in (2, 7, 40):
        if n * T * d > 1 << 26:
            continue
        check(3e38 * (0.6 + 0.4 * torch.rand(n, T, d, generator=g, device=DEV)), w, gamma)


@pytest.mark.parametrize("T,d", [(3, 640), (2, 2048), (1500, 640), (2433, 1160), (5003, 256), (5, 2304)])
def test_large_sources_among_high_scores(T, d):
    """Weights of e^-10 to e^-60 on values 1e17 (whose squares are finite) to 1e37 times the others'."""
    g = gen(T + d + 2)
    gamma = torch.ones(d, device=DEV)
    for n, size, score in ((5, 1e37, 60.0), (9, 3e36, 25.0), (9, 1e17, 10.0), (6, 1e18, 3.0)):
        x = ordinary(n, T, d, g, 1.0)
        x[n // 2] *= size
        x[0] *= size
        check(x, torch.full((d,), score / d, device=DEV), gamma)


@pytest.mark.parametrize("T,d", [(2, 300), (300, 1024), (2433, 1160), (2, 2048), (700, 2048), (5, 2304), (700, 4096)])
def test_products_of_large_rows_with_the_query(T, d):
    """Rows of 3e38 of one sign and queries whose magnitudes add up to 2^20: the score is 0, not what is left of an
    infinite product."""
    g = gen(T + d + 3)
    gamma = torch.ones(d, device=DEV)
    x = torch.zeros(3, T, d, device=DEV)
    x[1] = 3e38 * (0.9 + 0.1 * torch.rand(T, d, generator=g, device=DEV))
    for scale in (2.0 ** 20 / d, -(2.0 ** 20) / d):
        check(x, torch.full((d,), scale, device=DEV), gamma)


@pytest.mark.parametrize("T,d", [(2, 640), (2433, 1160), (5, 2304)])
def test_the_pre_norm_of_a_large_result(T, d):
    """A z whose squares add up past fp32's range has the pre-norm 0, beside tokens whose z is ordinary."""
    x = torch.ones(2, T, d, device=DEV)
    x[:, 1] = 3e38
    rows = ar.attnres_q8_write(x, ar.Q8Rows(2, T, d, device=DEV))
    one, out, normed = torch.ones(d, device=DEV), torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    ar.attnres_full_fwd_q8(rows, 2, one / d, one, 1e-6, out, gamma_pre=one, eps_pre=0.0, out_normed=normed)
    back = ar.attnres_q8_read(rows, torch.empty(2, T, d, device=DEV))
    assert ((out.double() / back[0].double() - 1).abs() <= 2.0 ** -20).all()
    ordinary = torch.arange(T, device=DEV) != 1
    assert not normed[1].any() and ((normed[ordinary] - 1).abs() <= 2.0 ** -16).all()


def test_tiny_sources_keep_their_bits():
    """Values of 1e-36 to 1e-37, whose scores are 0 beside eps: the weights lose nothing beside such scales."""
    for T, d in ((3, 640), (1500, 640), (2433, 1160), (5, 2304)):
        g = gen(T)
        x = torch.randn(9, T, d, generator=g, device=DEV) * 3e-37
        check(x, torch.randn(d, generator=g, device=DEV) / d ** 0.5, torch.ones(d, device=DEV))
