"""fp64 references of the 8-bit rows and of what is computed from them, with error bounds (torch, CPU or GPU).

With u = 2^-24: a sum of n terms in any order is within n u of the sum of the terms' magnitudes, a product of k
rounded factors within k u; exp of x <= 0 taken as 2^(x log2 e) is within 2^-22 + |x| 2^-23 of its value.
"""
import torch

GROUP = 128
U = 2.0 ** -24


def groups(d):
    return -(-d // GROUP)


def power(e):
    """2^e in fp64 from its bits (pow, and so ldexp, is not exact on every device), e from -1022 to 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def round_e4m3(y):
    """fp64 rounded to e4m3, ties to even, by scaling to whole steps: 2^-9 below 2^-6, else an eighth of the leading power."""
    _, e = torch.frexp(y)
    step = power((e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def scale_power(amax):
    """The smallest e >= -126 with amax <= 448 2^e, by trying."""
    e = torch.full(amax.shape, -126, dtype=torch.int32, device=amax.device)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):  # the largest power that is too small, plus one
        small = amax > 448 * power(e + step - 1)
        e = torch.where(small, e + step, e)
    return e


def quantise(x, block_rows=1):
    """(codes fp64, e) of x [rows, d]: groups of 128 features and block_rows rows."""
    x = x.double()
    R, d = x.shape
    G, B = groups(d), -(-R // block_rows)
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs()
    amax = torch.zeros(B, G, dtype=torch.float64, device=x.device)
    for b in range(B if block_rows > 1 else 1):
        rows = slice(b * block_rows, (b + 1) * block_rows) if block_rows > 1 else slice(None)
        for g in range(G):
            part = finite[rows, g * GROUP:(g + 1) * GROUP]
            if block_rows > 1:
                amax[b, g] = part.max()
            else:
                amax[:, g] = part.amax(1)
    e = scale_power(amax)
    per = spread(e, R, d, block_rows)
    top = torch.where(per == 120, 240.0, 448.0).double()
    q = round_e4m3(x / power(per))
    q = torch.where(q.abs() > top, torch.copysign(top, q), q)
    return torch.where(torch.isfinite(x), q, torch.full_like(x, float("nan"))), e


def spread(e, R, d, block_rows=1):
    """Exponents [blocks, G] as one per element [R, d]."""
    rows = torch.arange(R, device=e.device) // block_rows
    return e[rows][:, torch.arange(d, device=e.device) // GROUP]


def values(codes, e, block_rows=1):
    return codes.double() * power(spread(e, *codes.shape, block_rows))


def history(n, T, d, g, device, loud=True):
    """Sources of different size, a few features far larger than the others (fp32 [n, T, d])."""
    x = torch.randn(n, T, d, generator=g, device=device)
    x *= torch.exp(0.7 * torch.randn(n, 1, 1, generator=g, device=device))
    if loud:
        x *= 1 + 20 * (torch.rand(d, generator=g, device=device) < 0.02)
    return x


def read(v, q, gamma, eps, gamma_pre=None, eps_pre=0.0):
    """(z, bound, normed, bound) of the read over v [n, T, d] (fp64) with queries q [d] or [T, d]."""
    n, _, d = v.shape
    u = q.double() * gamma.double()
    size = (v.square().mean(-1) + eps).sqrt()
    e = (v * u).sum(-1) / size
    # the dot (products of two roundings, d terms), the mean square (d terms, halved by the root) and 1/sqrt (4 u)
    de = ((d + 4) * U) * (v * u).abs().sum(-1) / size + e.abs() * ((d / 2 + 8) * U)
    a = torch.softmax(e, 0)
    gap = (e.amax(0) - e).clamp(max=100)
    # weights: both errors of the exponent, exp itself twice (weight and a rescaling), the sum of n weights
    da = a * (de + (a * de).sum(0) + 2 * (2.0 ** -22 + gap * 2.0 ** -23) + (a * 2 * (2.0 ** -22 + gap * 2.0 ** -23)).sum(0) +
              (2 * n + 24) * U)
    z = (a.unsqueeze(-1) * v).sum(0)
    dz = (da.unsqueeze(-1) * v.abs()).sum(0)
    if gamma_pre is None:
        return z, dz, None, None
    r = 1 / (z.square().mean(-1, keepdim=True) + eps_pre).sqrt()
    normed = gamma_pre.double() * z * r
    dn = (gamma_pre.double().abs() * r) * (dz + z.abs() * r * dz.square().mean(-1, keepdim=True).sqrt()) + normed.abs() * (
        (d / 2 + 16) * U)
    return z, dz, normed, dn


def rounding(dtype):
    return torch.finfo(dtype).eps / 2


def assert_within(got, ref, bound, what=""):
    """|got - ref| within the bound and got's own rounding."""
    got64 = got.double()
    room = bound + (ref.abs() + bound) * rounding(got.dtype) + torch.finfo(got.dtype).smallest_normal * rounding(got.dtype) * 2
    bad = ~((got64 - ref).abs() <= room)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got64[tuple(i)]} for "
                             f"{ref[tuple(i)]}, room {room[tuple(i)]}")
