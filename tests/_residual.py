"""fp64 references of the gated residual, its gradients and the RMSNorm backward, with error bounds (torch, CPU or GPU).

Every reference returns (values, bounds). A bound says how far a correct fp32
evaluation may be off, before the result's own rounding: with u = 2^-24, a sum
of n terms in any tree of depth L is within L u of the sum of the terms'
magnitudes, and a product of k rounded factors within k u. `MEAN` bounds what a
row mean and everything built on it carries: depth at most d/256 + 32 (a thread
adds at most max(24, d/256) terms of its own, then 5 levels of a warp and its
warps' sums), which counts half in r, rsqrtf within 2 ulp (4 u), a sigmoid (20 u,
beside an r of half the depth), and at most 16 further factors. Bounds are
therefore MEAN times the sum of the magnitudes that enter; a difference such as
h - u <h u> is bounded through |h| + |u| <|h u|>.
"""
import math

import torch

U = 2.0 ** -24
# A factor below fp32's normal range (the sigmoid of -100, e^-100 = 27 steps of 2^-149) is rounded to whole steps of
# 2^-149, and so is each product with it: four roundings at most (the gate, the scale, D, the gain), each off by
# half a step and then multiplied by the factors that follow, whose magnitudes are at most those of all of them
# (each taken as at least 1). The relative bounds above do not cover that; `TINY` times those factors does.
TINY = 4 * 2.0 ** -149
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def mean_bound(d):
    return (d / 256 + 32 + 4 + 16) * U


def column_bound(T, d):
    """A sum over tokens: any split into runs (a run's own sum, then the runs'), at most T terms deep."""
    return mean_bound(d) + (min(T, 8 + T / 8) + 256) * U


def unit(v, eps):
    r = ((v * v).mean(1, keepdim=True) + eps).rsqrt()
    return v * r, r


def act(gate, sigmoid):
    if not sigmoid:
        return gate, torch.ones_like(gate)
    s = 1 / (1 + torch.exp(-gate))
    return s, s / (1 + torch.exp(gate))


def rows_of(gate, T, gate_rows):
    return gate[torch.arange(T, device=gate.device) // gate_rows]


def forward(f, x, gpost, eps_post, gate, gate_rows, sigmoid, scale, gpre, eps_pre):
    """x_out and normed (None without gpre), and their bounds."""
    f = f.double()
    T, d = f.shape
    e = mean_bound(d)
    y = f if gpost is None else gpost.double() * unit(f, eps_post)[0]
    a = scale if gate is None else scale * act(rows_of(gate.double(), T, gate_rows), sigmoid)[0]
    m = a * y
    xo = m if x is None else x.double() + m
    mag = m.abs() if x is None else x.double().abs() + m.abs()
    vals, bounds = {"x_out": xo}, {"x_out": e * mag}
    if gpre is not None:
        g = gpre.double()
        un, r = unit(xo, eps_pre)
        # An error of e * mag in the row moves the row's own value and, through the mean, r.
        moved = r * mag + un.abs() * r * (un.abs() * mag).mean(1, keepdim=True)
        vals["normed"], bounds["normed"] = g * un, e * g.abs() * (un.abs() + moved)
    return vals, bounds


def backward(f, gpost, eps_post, gate, gate_rows, sigmoid, scale, xo, gpre, eps_pre, dxo, dn):
    """df, dx, dgate, dgamma_post, dgamma_pre and their bounds (f None: the RMSNorm backward alone)."""
    T, d = (f if f is not None else xo).shape
    e, c = mean_bound(d), column_bound(T, d)
    D = torch.zeros(T, d, dtype=torch.float64, device=(f if f is not None else xo).device)
    mD = D.clone()
    vals, bounds = {}, {}
    if dxo is not None:
        D, mD = D + dxo.double(), mD + dxo.double().abs()
    if dn is not None:
        u, r = unit(xo.double(), eps_pre)
        h = gpre.double() * dn.double()
        D = D + r * (h - u * (h * u).mean(1, keepdim=True))
        mD = mD + r * (h.abs() + u.abs() * (h * u).abs().mean(1, keepdim=True))
        vals["dgamma_pre"], bounds["dgamma_pre"] = (dn.double() * u).sum(0), c * (dn.double() * u).abs().sum(0)
    vals["dx"], bounds["dx"] = D, e * mD
    if f is None:
        return vals, bounds
    f = f.double()
    q, rf = (f, 1.0) if gpost is None else unit(f, eps_post)
    gp = 1.0 if gpost is None else gpost.double()
    if gate is None:
        a, slope = torch.ones(1, 1, dtype=torch.float64, device=f.device), None
    else:
        a, slope = act(rows_of(gate.double(), T, gate_rows), sigmoid)
    dy, mdy = scale * a * D, abs(scale) * a.abs() * mD
    if gpost is None:
        vals["df"], bounds["df"] = dy, e * mdy
    else:
        w, mw = gp * dy, (gp * mdy).abs()
        vals["df"] = rf * (w - q * (w * q).mean(1, keepdim=True))
        bounds["df"] = 2 * e * rf * (mw + q.abs() * (mw * q.abs()).mean(1, keepdim=True))
        bounds["df"] = bounds["df"] + TINY * (1 + rf) * (1 + gp.abs()) * (1 + abs(scale) * mD)
        vals["dgamma_post"], bounds["dgamma_post"] = (dy * q).sum(0), 2 * c * (mdy * q.abs()).sum(0)
    if gate is not None:
        share, mshare = scale * slope * gp * q * D, (scale * slope * gp * q).abs() * mD
        groups = gate.shape[0]
        idx = torch.arange(T, device=f.device) // gate_rows
        zero = torch.zeros(groups, d, dtype=torch.float64, device=f.device)
        vals["dgate"] = zero.index_add(0, idx, share)
        bounds["dgate"] = 2 * c * zero.index_add(0, idx, mshare)
    return vals, bounds


def check(got, value, bound, what=""):
    """got within half a step of its type of the value, plus the bound."""
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    # Rounding a value that is off by `bound` adds half a step of it; below the
    # normal range a step is the smallest one.
    limit = HALF[got.dtype] * (value.abs() + bound) + bound + 2.0 ** -140
    over = (g - value).abs() / limit
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def norm_of(tensors):
    return math.sqrt(sum(float((t.double() * t.double()).sum()) for t in tensors))
