"""Histories made for more tokens and sources than a call uses: the rows behind the batch, and the sources behind the
last one, hold NaN codes, scales and mean squares, and nothing of them is read."""
import pytest
import torch

import depth_wise_attention_attnres_gb300 as ar
from tests import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def spare(n, T, d, g, extra):
    """n + 1 sources of T + extra rows, the first n sources' first T rows written, all else 0xFF; and their values."""
    rows = ar.Q8Rows(n + 1, T + extra, d, device=DEV)
    rows.buffer.fill_(0xFF)
    ar.attnres_q8_write(_q8.history(n, T, d, g, DEV), rows)
    e = rows.exponents[:n, :T].long() - 127
    v = rows.codes[:n, :T].double() * _q8.power(e)[..., torch.arange(d, device=DEV) // 128]
    assert v.isfinite().all() and rows.mean_square[:, T:].isnan().all() and rows.codes[n].float().isnan().all()
    return rows, v


@pytest.mark.parametrize("n,T,d", [(9, 1, 640), (40, 19, 640), (20, 2, 2048), (3, 229, 384), (9, 300, 2048), (12, 700, 896),
                                   (5, 5003, 256), (5, 5003, 100), (6, 2433, 1160), (3, 3001, 512), (9, 5, 2304),
                                   (4, 700, 2304)])
@pytest.mark.parametrize("extra", [1, 37])
def test_full_read(n, T, d, extra):
    g = gen(T + d)
    rows, v = spare(n, T, d, g, extra)
    gamma, pre = 1 + 0.2 * torch.randn(d, generator=g, device=DEV), 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    w, Q = torch.randn(d, generator=g, device=DEV) / d ** 0.5, torch.randn(T, d, generator=g, device=DEV) / d ** 0.5
    out, normed = torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    for k in {n, max(1, n // 2)}:  # all the sources there are so far, and fewer
        ar.attnres_full_fwd_q8(rows, k, w, gamma, 1e-6, out)
        z, dz, _, _ = _q8.read(v[:k], w, gamma, 1e-6)
        _q8.assert_within(out, z, dz, f"{k} sources")
        ar.attnres_full_fwd_q8(rows, k, None, gamma, 1e-6, out, Q=Q, gamma_pre=pre, eps_pre=1e-5, out_normed=normed)
        z, dz, zn, dn = _q8.read(v[:k], Q, gamma, 1e-6, pre, 1e-5)
        _q8.assert_within(out, z, dz, f"{k} sources, queries of tokens")
        _q8.assert_within(normed, zn, dn, f"{k} sources, normed")
    assert ar.attnres_device_status() == 0
    back = ar.attnres_q8_read(rows, torch.empty(n, T, d, device=DEV))
    assert torch.equal(back.double(), v)


def project(rows, v, src, W8, wv, T):
    Q = torch.empty(T, W8.m, device=DEV)
    ar.attnres_query_projection_q8(rows, src, W8, Q)
    assert ar.attnres_device_status() == 0
    x, d = v[src, :T], rows.d
    bound = (x.abs() @ wv.abs().t()) * ((d + 2 * _q8.groups(d) + 4) * _q8.U)
    _q8.assert_within(Q, x @ wv.t(), bound, f"{T} tokens, {d} by {W8.m}")
    return Q


def weights(m, d, g):
    W8 = ar.attnres_q8_weight(torch.randn(m, d, generator=g, device=DEV) / d ** 0.5, ar.Q8Weight(m, d, device=DEV))
    return W8, _q8.values(W8.codes, W8.exponents.int() - 127, 128)


# Few tokens by either kernel, one CTA a tile of 64 and of 128 columns, and pairs of CTAs.
@pytest.mark.parametrize("T,d,m", [(1, 128, 128), (8, 1000, 130), (16, 896, 896), (16, 2048, 2048), (17, 640, 640),
                                   (300, 1024, 1000), (2433, 640, 640), (2500, 2200, 2048), (9001, 896, 896)])
@pytest.mark.parametrize("extra", [1, 300])
def test_projection(T, d, m, extra):
    g = gen(T + d + m)
    rows, v = spare(2, T, d, g, extra)
    W8, wv = weights(m, d, g)
    for src in (0, 1):
        project(rows, v, src, W8, wv, T)


def test_tokens_beside_others():
    """A token's results among fewer and more others, which other kernels and shares of the work compute: each within the
    definition's bound (the last bits differ)."""
    n, d, m, T = 12, 640, 640, 9000
    g = gen(3)
    rows, v = spare(n, T, d, g, 5)
    W8, wv = weights(m, d, g)
    w, gamma = torch.randn(d, generator=g, device=DEV) * 0.1, torch.ones(d, device=DEV)
    for few in (T, 4000, 2001, 229, 228, 17, 16, 1):
        out = ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, torch.empty(few, d, device=DEV))
        z, dz, _, _ = _q8.read(v[:, :few], w, gamma, 1e-6)
        _q8.assert_within(out, z, dz, f"{few} tokens")
        project(rows, v, 3, W8, wv, few)
