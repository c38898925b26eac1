"""8-bit rows on the CPU: sizes, refusals before any launch, and the reference the GPU tests use."""
import ctypes

import pytest
import torch

import __graft_entry__ as graft
from depth_wise_attention_attnres_gb300 import binding
from tests import _q8

P = 1 << 20
INVALID, UNSUPPORTED, CUDA_ERR = 1, 2, 3
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    graft.build()
    return binding.lib()


def launches(lib, fn, *args):
    """Whether the call passes its checks: an armed failure then answers for its first launch."""
    binding.attnres_test_fail_launch(0)
    status = fn(*args)
    fired = binding.attnres_test_fail_launch(-1) == -1
    return status == CUDA_ERR and fired


def test_source_and_weight_bytes(lib):
    for d, tail in ((1, 16), (128, 16), (640, 16), (1536, 16), (1537, 32), (2048, 32), (3584, 32), (3585, 48)):
        G = _q8.groups(d)
        assert tail == -(-(-(-G // 4) * 4 + 4) // 16) * 16
        for cap in (0, 1, 7, 8192):
            assert binding.attnres_q8_source_bytes(cap, d) == cap * 128 * G + -(-cap * tail // 128) * 128
    for cap, d in ((1, 0), (1, (1 << 24) + 1), (-1, 5), (1 << 52, 128)):
        assert binding.attnres_q8_source_bytes(cap, d) == -1
    assert binding.attnres_q8_weight_bytes(200, 300) == 200 * 384 + 2 * 16
    assert binding.attnres_q8_weight_bytes(128, 2176) == 128 * 2176 + 32
    assert binding.attnres_q8_weight_bytes(0, 3) == -1 and binding.attnres_q8_weight_bytes(3, 0) == -1


def test_write_and_read_back_refusals(lib):
    # (x, x_stride, n, T, d, dtype, rows, cap); T = 4, d = 16: 64 elements, and 5 rows of 128 + 16 bytes a source
    ok = (P, 64, 2, 4, 16, 1, 8 * P, 5)
    size = 5 * 128 + 128
    assert launches(lib, lib.attnres_q8_write, *ok, None)
    one = ok[:1] + (0, 1) + ok[3:]
    assert launches(lib, lib.attnres_q8_write, *one, None)  # one source: no stride
    bad = [(0, None), (0, P + 1), (1, 63), (2, 0), (3, -1), (4, 0), (4, 1 << 25), (5, 2), (6, None), (6, 8 * P + 8),
           (7, 3), (7, -1), (6, P + 64), (6, P - 2 * size + 16), (7, 1 << 55), (3, 1 << 55)]
    for at, value in bad:
        args = ok[:at] + (value,) + ok[at + 1:]
        assert lib.attnres_q8_write(*args, None) == INVALID, (at, value)
        a = list(args)
        back = (a[6], a[7], a[2], a[3], a[4], a[0], a[1], a[5])
        assert lib.attnres_q8_read(*back, None) == INVALID, (at, value)
    assert launches(lib, lib.attnres_q8_read, 8 * P, 5, 2, 4, 16, P, 64, 0, None)
    assert lib.attnres_q8_write(None, 0, 1, 0, 16, 1, None, 0, None) == 0  # no tokens
    assert lib.attnres_q8_read(None, 0, 1, 0, 16, None, 0, 1, None) == 0


def test_full_read_refusals(lib):
    # (rows, cap, n, T, d, w, Q, gamma, eps, gamma_pre, eps_pre, out, out_normed, dtype)
    ok = (P, 4, 3, 4, 16, 2 * P, None, 3 * P, F(1e-6), None, F(0), 4 * P, None, 1)
    pre = ok[:9] + (5 * P, F(1e-6), None, 6 * P, 0)
    for good in (ok, pre, ok[:5] + (None, 7 * P) + ok[7:], pre[:11] + (4 * P,) + pre[12:]):
        assert launches(lib, lib.attnres_full_fwd_q8, *good, None), good
    bad = [(0, None), (0, P + 8), (1, 3), (1, -4), (2, 0), (3, -1), (3, 5), (4, 0), (5, None), (6, 7 * P),
           (7, None), (8, F(-1)), (8, F(float("nan"))), (9, 5 * P), (11, None), (11, P + 64), (11, 4 * P + 1), (12, 6 * P),
           (13, 4), (5, 2 * P + 2), (7, 3 * P + 1), (11, 2 * P), (11, 3 * P + 32)]
    for at, value in bad:
        assert lib.attnres_full_fwd_q8(*ok[:at], value, *ok[at + 1:], None) == INVALID, (at, value)
    for at, value in [(9, None), (10, F(-1)), (12, None), (12, P), (12, 5 * P), (11, 6 * P + 32)]:
        assert lib.attnres_full_fwd_q8(*pre[:at], value, *pre[at + 1:], None) == INVALID, (at, value)
    tok = ok[:5] + (None, 4 * P - 128) + ok[7:]
    assert lib.attnres_full_fwd_q8(*tok, None) == INVALID  # out overlaps the queries
    assert lib.attnres_full_fwd_q8(*ok[:3], 0, *ok[4:], None) == 0


def test_wide_rows_past_the_general_kernel(lib):
    T, d = 1, 51200 - 128
    args = lambda n: (P, 1, n, T, d, 4 * P, None, 8 * P, F(0), None, F(0), 16 * P, None, 0, None)  # noqa: E731
    assert lib.attnres_full_fwd_q8(*args(129)) == UNSUPPORTED


def test_weight_and_projection_refusals(lib):
    ok = (P, 16, 24, 1, 8 * P)
    assert launches(lib, lib.attnres_q8_weight, *ok, None)
    for at, value in [(0, None), (0, P + 1), (1, 0), (2, 0), (3, 5), (4, None), (4, 8 * P + 4), (4, P + 16)]:
        assert lib.attnres_q8_weight(*ok[:at], value, *ok[at + 1:], None) == INVALID, (at, value)
    ok = (P, 6, 4, 16, 4 * P, 24, 8 * P)  # rows, cap, T, d, W8, m, Q
    assert launches(lib, lib.attnres_query_projection_q8, *ok, None)
    for at, value in [(0, None), (0, P + 4), (1, 3), (2, -1), (2, 7), (3, 0), (4, None), (4, 4 * P + 8), (5, 0), (6, None),
                      (6, 8 * P + 2), (6, P + 64), (6, 4 * P + 1024)]:
        assert lib.attnres_query_projection_q8(*ok[:at], value, *ok[at + 1:], None) == INVALID, (at, value)
    assert lib.attnres_query_projection_q8(None, 0, 0, 16, None, 24, None, None) == 0


def test_reference_rounding():
    """The reference's e4m3 rounding is torch's, and its powers are the smallest."""
    y = torch.cat([torch.linspace(-460, 460, 20001), torch.linspace(-0.04, 0.04, 20001)]).double().clamp(-448, 448)
    want = y.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(_q8.round_e4m3(y.float().double()), want)
    for amax, e in ((0.0, -126), (448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7),
                    (1.75 * 2.0 ** 127, 119), (1.9 * 2.0 ** 127, 120), (2.0 ** -149, -126)):
        assert int(_q8.scale_power(torch.tensor(amax).double())) == e


def test_q8_rows_arguments(lib):
    for args in ((0, 4, 16), (1, -1, 16), (1, 4, 0), (1, 4, 16)):  # the last is not on a CUDA device
        with pytest.raises(ValueError):
            binding.Q8Rows(*args, device="cpu")
