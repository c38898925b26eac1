"""The gated residual's reference gradients against autograd and differences, and the entry points' refusals (no GPU)."""
import ctypes

import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding, build
from tests import _residual as ref

INVALID, CUDA_ERR = 1, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _case(T, d, gate_rows, seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)
    groups = -(-T // gate_rows)
    return r(T, d), r(T, d), 1 + 0.3 * r(d), r(groups, d), 1 + 0.3 * r(d), r(T, d), r(T, d)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,d,gate_rows,post,pre,with_x", [
    (5, 7, 1, True, True, True), (6, 4, 4, True, True, True), (3, 5, 9, True, False, True), (4, 6, 2, False, True, False)])
def test_reference_gradients(T, d, gate_rows, post, pre, with_x, sigmoid):
    f, x, gp, gate, gn, dxo, dn = _case(T, d, gate_rows)
    leaves = [t.clone().requires_grad_() for t in (f, x, gp, gate, gn)]

    def loss(f, x, gp, gate, gn):
        v, _ = ref.forward(f, x if with_x else None, gp if post else None, 1e-3, gate, gate_rows, sigmoid, 0.7,
                           gn if pre else None, 1e-2)
        total = (v["x_out"] * dxo).sum()
        return total + (v["normed"] * dn).sum() if pre else total

    grads = torch.autograd.grad(loss(*leaves), leaves, allow_unused=True)
    xo = ref.forward(f, x if with_x else None, gp if post else None, 1e-3, gate, gate_rows, sigmoid, 0.7, None, 0.0)[0]["x_out"]
    got, _ = ref.backward(f, gp if post else None, 1e-3, gate, gate_rows, sigmoid, 0.7, xo, gn, 1e-2, dxo, dn if pre else None)
    for name, auto in zip(("df", "dx", "dgamma_post", "dgate", "dgamma_pre"), grads):
        if auto is None:
            assert name not in got or name == "dx"
            continue
        assert torch.allclose(got[name], auto, rtol=1e-10, atol=1e-12), name
    # Central differences along random directions: error O(h^2) of a smooth loss.
    h = 1e-5
    for k, name in enumerate(("df", "dx", "dgamma_post", "dgate", "dgamma_pre")):
        if grads[k] is None:
            continue
        direction = torch.randn(leaves[k].shape, generator=torch.Generator().manual_seed(k), dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            args = [t.detach().clone() for t in leaves]
            args[k] = args[k] + sign * h * direction
            ends.append(float(loss(*args)))
        assert abs((ends[0] - ends[1]) / (2 * h) - float((got[name] * direction).sum())) < 1e-6, name


def test_rmsnorm_reference_gradient():
    _, x, _, _, gn, dres, dy = _case(4, 6, 1, seed=3)
    xl, gl = x.clone().requires_grad_(), gn.clone().requires_grad_()
    y = gl * xl / torch.sqrt((xl * xl).mean(1, keepdim=True) + 1e-2)
    dx, dg = torch.autograd.grad((y * dy).sum() + (xl * dres).sum(), (xl, gl))
    got, _ = ref.backward(None, None, 0.0, None, 1, False, 1.0, x, gn, 1e-2, dres, dy)
    assert torch.allclose(got["dx"], dx, rtol=1e-10) and torch.allclose(got["dgamma_pre"], dg, rtol=1e-10)


# ------------------------------------------------------------------ refusals ----

P = 1 << 24  # aligned stand-in pointers, far apart: refused calls never reach them


def _fwd(**kw):
    a = dict(f=P, x=2 * P, gpost=3 * P, eps_post=1e-6, gate=4 * P, gate_rows=2, gate_dtype=1, act=1, scale=0.5, T=4,
             d=16, dtype=1, x_dtype=0, x_out=5 * P, gpre=6 * P, eps_pre=1e-6, normed=7 * P)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(dtype=5), dict(x_dtype=3), dict(eps_post=-1.0), dict(eps_pre=float("nan")),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(act=2), dict(gate_rows=0), dict(gate_dtype=7),
    dict(f=None), dict(x_out=None), dict(gpre=None), dict(normed=None), dict(dtype=0, x_dtype=1),
    dict(x_out=P), dict(x_out=2 * P + 64), dict(normed=5 * P + 32), dict(normed=P), dict(normed=4 * P + 16),
    dict(x_out=6 * P), dict(f=P + 1), dict(x_out=5 * P + 2), dict(gpost=3 * P + 2), dict(gate=4 * P + 1),
    dict(T=1 << 60)])
def test_gated_residual_refusals(lib, kw):
    assert lib.attnres_gated_residual(*_fwd(**kw)) == INVALID


def test_gated_residual_accepts(lib):
    assert lib.attnres_gated_residual(*_fwd(T=0, f=None, x_out=None)) == 0
    for kw in (dict(), dict(x=None), dict(x_out=2 * P), dict(gate=None, gate_rows=0), dict(gpost=None),
               dict(gpre=None, normed=None), dict(dtype=0), dict(x_dtype=1), dict(gate_dtype=0)):
        binding.attnres_test_fail_launch(0)             # valid: reaches the launch
        assert lib.attnres_gated_residual(*_fwd(**kw)) == CUDA_ERR, kw
        assert binding.attnres_test_fail_launch(-1) == -1


def _bwd(**kw):
    a = dict(f=P, gpost=2 * P, eps_post=1e-6, gate=3 * P, gate_rows=2, gate_dtype=1, act=1, scale=0.5, T=4, d=16,
             dtype=1, x_dtype=0, x_out=4 * P, gpre=5 * P, eps_pre=1e-6, dx_out=6 * P, dx_dtype=0, dn=7 * P, df=8 * P,
             dx=9 * P, dgate=10 * P, dgpost=11 * P, dgpre=12 * P, acc=1, scratch=13 * P, floats=1 << 20)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(dtype=5), dict(dx_dtype=2), dict(dtype=0, x_dtype=0, dx_dtype=1), dict(act=-1),
    dict(gate_rows=0), dict(f=None), dict(dx_out=None, dn=None), dict(x_out=None), dict(gpre=None), dict(gate=None),
    dict(scratch=None), dict(floats=0), dict(df=P), dict(dx=8 * P), dict(dx=6 * P + 64), dict(dgate=3 * P),
    dict(dgpost=12 * P + 32), dict(dgpre=5 * P), dict(scratch=7 * P), dict(df=13 * P + 4096), dict(scratch=13 * P + 2),
    dict(dx=9 * P + 2), dict(dn=7 * P + 1)])
def test_gated_residual_bwd_refusals(lib, kw):
    assert lib.attnres_gated_residual_bwd(*_bwd(**kw)) == INVALID


def test_gated_residual_bwd_accepts(lib):
    assert lib.attnres_gated_residual_bwd(*_bwd(T=0, f=None, dx_out=None, dn=None)) == 0
    for kw in (dict(), dict(dx=6 * P), dict(dx_out=None), dict(dn=None, x_out=None, gpre=None), dict(df=None),
               dict(gate=None, dgate=None, gate_rows=0), dict(gpost=None), dict(dx=None, dgate=None), dict(dx_dtype=1),
               dict(T=0, f=None, acc=0)):
        binding.attnres_test_fail_launch(0)
        assert lib.attnres_gated_residual_bwd(*_bwd(**kw)) == CUDA_ERR, kw
        assert binding.attnres_test_fail_launch(-1) == -1


def test_rmsnorm_bwd_refusals(lib):
    # (x, T, d, dtype, gamma, eps, dy, dres, dx_dtype, dx, dgamma, accumulate, scratch, floats)
    ok = [P, 4, 16, 1, 2 * P, 1e-6, 3 * P, 4 * P, 0, 5 * P, 6 * P, 1, 7 * P, 1 << 20]
    for at, v in ((0, None), (1, -1), (2, 0), (3, 2), (4, None), (5, -1.0), (6, None), (8, 3), (9, None), (9, P),
                  (9, 4 * P + 64), (10, 5 * P), (12, None), (13, 1), (6, 3 * P + 1)):
        bad = list(ok)
        bad[at] = v
        assert lib.attnres_rmsnorm_bwd(*bad, None) == INVALID, (at, v)
    assert lib.attnres_rmsnorm_bwd(*(ok[:3] + [0] + ok[4:8] + [1] + ok[9:]), None) == INVALID  # fp32 rows, bf16 dx
    for at, v in ((9, 4 * P), (7, None), (10, None)):
        good = list(ok)
        good[at] = v
        binding.attnres_test_fail_launch(0)
        assert lib.attnres_rmsnorm_bwd(*good, None) == CUDA_ERR, (at, v)
    binding.attnres_test_fail_launch(-1)


def test_scratch_sizes(lib):
    for T, d, rows in ((-1, 16, 1), (4, 0, 1), (4, 16, 0)):
        assert binding.attnres_gated_residual_bwd_scratch_floats(T, d, rows) == -1
    assert binding.attnres_gated_residual_bwd_scratch_floats(0, 16, 1) >= 0
    assert binding.attnres_rmsnorm_bwd_scratch_floats(4, 0) == -1
    assert binding.attnres_grad_norm_scratch_floats(-1) == -1
    assert binding.attnres_grad_norm_scratch_floats(0) > 0
    # One float short is refused.
    need = binding.attnres_gated_residual_bwd_scratch_floats(4, 16, 2)
    assert lib.attnres_gated_residual_bwd(*_bwd(floats=need - 1)) == INVALID


def _list(pointers, counts, codes):
    n = len(counts)
    return (ctypes.c_void_p * n)(*pointers), (ctypes.c_int64 * n)(*counts), (ctypes.c_int32 * n)(*codes)


def _clip(lib, pointers, counts, codes, outs=None, out_codes=None, max_norm=1.0, norm=100 * P, scratch=101 * P,
          floats=1 << 16):
    p, c, k = _list(pointers, counts, codes)
    o = ok = None
    if outs is not None:
        o, _, ok = _list(outs, counts, out_codes)
    return lib.attnres_grad_clip(p, c, k, o, ok, len(counts), max_norm, norm, scratch, floats, None)


@pytest.mark.parametrize("kw", [
    dict(pointers=[None]), dict(counts=[-1]), dict(codes=[2]), dict(pointers=[P + 2]), dict(max_norm=-1.0),
    dict(max_norm=float("nan")), dict(norm=None), dict(scratch=None), dict(floats=8), dict(norm=P + 8),
    dict(scratch=P + 64), dict(norm=101 * P), dict(norm=100 * P + 2), dict(outs=[None], out_codes=[0]),
    dict(outs=[P], out_codes=[1]), dict(outs=[P + 16], out_codes=[0]), dict(outs=[2 * P], out_codes=[5]),
    dict(outs=[100 * P - 16], out_codes=[0]), dict(counts=[1 << 50])])
def test_grad_clip_refusals(lib, kw):
    a = dict(pointers=[P], counts=[100], codes=[0])
    a.update(kw)
    assert _clip(lib, **a) == INVALID


def test_grad_list_overlaps(lib):
    # In place, a tensor listed twice or two that share storage; in address order and not, and a long list.
    assert _clip(lib, [P, P], [10, 10], [0, 0]) == INVALID
    assert _clip(lib, [P + 20, P], [10, 10], [0, 0]) == INVALID
    assert _clip(lib, [3 * P, P, 2 * P, P + 36], [10] * 4, [0] * 4) == INVALID
    many = [P + 64 * i for i in range(1500)]
    assert _clip(lib, many + [P + 64 * 700 + 4], [16] * 1501, [0] * 1501) == INVALID
    # Out of place: two outputs that overlap, an output over another tensor's input.
    assert _clip(lib, [P, 2 * P], [10, 10], [0, 0], [3 * P, 3 * P + 16], [0, 0]) == INVALID
    assert _clip(lib, [P, 2 * P], [10, 10], [0, 0], [2 * P, 3 * P], [0, 0]) == INVALID
    good = [
        dict(pointers=[P + 40, P], counts=[10, 10], codes=[0, 0]),                        # touching, not overlapping
        dict(pointers=[P, P], counts=[10, 0], codes=[0, 0]),                              # an empty one anywhere
        dict(pointers=[P, P], counts=[10, 10], codes=[0, 0], outs=[2 * P, 3 * P], out_codes=[0, 1]),  # read twice
        dict(pointers=[None], counts=[0], codes=[0]),
        dict(pointers=[], counts=[], codes=[]),
        dict(pointers=many, counts=[16] * 1500, codes=[0] * 1500),
    ]
    for kw in good:
        binding.attnres_test_fail_launch(0)
        assert _clip(lib, **kw) == CUDA_ERR, kw
        assert binding.attnres_test_fail_launch(-1) == -1


def test_grad_norm_refusals(lib):
    p, c, k = _list([P], [10], [0])
    assert lib.attnres_grad_norm(p, c, k, -1, 2 * P, 3 * P, 1 << 16, None) == INVALID
    assert lib.attnres_grad_norm(None, c, k, 1, 2 * P, 3 * P, 1 << 16, None) == INVALID
    assert lib.attnres_grad_norm(p, c, k, 1, None, 3 * P, 1 << 16, None) == INVALID
    assert lib.attnres_grad_norm(p, c, k, 1, 2 * P, 3 * P, 1, None) == INVALID
    assert lib.attnres_grad_norm(p, c, k, 1, P + 4, 3 * P, 1 << 16, None) == INVALID
    binding.attnres_test_fail_launch(0)
    assert lib.attnres_grad_norm(p, c, k, 1, 2 * P, 3 * P, 1 << 16, None) == CUDA_ERR
    # The second of its launches fails: nothing after it, and the hook is off again. (The first is a real launch,
    # so only its refusal is looked at here.)
    assert binding.attnres_test_fail_launch(-1) == -1


def test_binding_refuses_cpu_tensors(lib):
    with pytest.raises(ValueError):
        binding.GradList([torch.zeros(4)])


def test_kernel_selection(lib):
    A = 1 << 20
    for op in (5, 6, 7):
        for dt in (0, 1):
            for d in (8, 256, 640, 896, 1024, 2048, 5120):
                assert binding.attnres_kernel_path(op, A, 2 * A, 0, 0, 8192, d, dt) == 1, (op, d, dt)
        assert binding.attnres_kernel_path(op, A, 2 * A, 0, 0, 8192, 8192, 1) == 1
        assert binding.attnres_kernel_path(op, A + 8, 2 * A, 0, 0, 8192, 640, 1) == 0     # unaligned rows
        assert binding.attnres_kernel_path(op, A, 2 * A, 0, 0, 8192, 100, 1) == 0         # d % 8
        assert binding.attnres_kernel_path(op, A, 2 * A, 0, 0, 8192, 8200, 1) == 0        # wider than a CTA's teams
    # Five fp32 arrays of 8192 features, the gains and the team's sums just fit in an SM's shared memory.
    assert binding.attnres_kernel_path(6, A, 2 * A, 0, 0, 8192, 8192, 0) == 1
