"""Waits that run out at every place where the gated residual's kernels wait for a row (GPU, by the test hook).

Each team (one or several warps) of a kernel leaves the copies of its row
number `index` unissued: its first row, which is waited for before the loop;
its second, waited for inside it; and one past the ring, when every stage has
been used and the other stages' copies are in flight. The wait is bounded (2 s),
the team stops together, and the status reports the timeout once. Rows written
until then hold their values, the others are left as they were, and the next
call gives the bits of an undisturbed one.
"""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests._gpu import dev

pytestmark = pytest.mark.gpu
TIMEOUT = 4
PAST_THE_RING = 9  # a ring holds at most 8 rows


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _hooks_off():
    assert ar.attnres_device_status() == 0
    yield
    ar.attnres_test_withhold_stage(ar.WITHHOLD_NONE)


def _rand(shape, dt, seed):
    return inputs.randn(shape, dt, inputs.generator(seed, dev()), dev())


def _forward(T, d, dt, xt, gate_rows):
    f, x, gate = _rand((T, d), dt, 1), _rand((T, d), xt, 2), _rand((-(-T // gate_rows), d), dt, 3)
    gain = torch.ones(d, device=dev())
    rows = [torch.empty_like(x), torch.empty_like(f)]
    return rows, [], lambda: ar.attnres_gated_residual(f, x, gain, 1e-6, gate, gate_rows, ar.GATE_SIGMOID, 0.5, rows[0],
                                                       gain, 1e-6, rows[1])


def _backward(T, d, dt, xt, gate_rows):
    f, xo, dn, dxo = _rand((T, d), dt, 1), _rand((T, d), xt, 2), _rand((T, d), dt, 3), _rand((T, d), xt, 4)
    gate = _rand((-(-T // gate_rows), d), dt, 5)
    gain = torch.ones(d, device=dev())
    rows = [torch.empty_like(f), torch.empty_like(dxo)]
    sums = [torch.empty_like(gate), torch.empty(d, device=dev()), torch.empty(d, device=dev())]
    return rows, sums, lambda: ar.attnres_gated_residual_bwd(f, gain, 1e-6, gate, gate_rows, ar.GATE_SIGMOID, 0.5, xo, gain,
                                                             1e-6, dxo, dn, *rows, *sums, accumulate=False)


def _norm_backward(T, d, dt, xt, gate_rows):
    x, dy, dres = _rand((T, d), dt, 1), _rand((T, d), dt, 2), _rand((T, d), xt, 3)
    gain = torch.ones(d, device=dev())
    rows, sums = [torch.empty_like(dres)], [torch.empty(d, device=dev())]
    return rows, sums, lambda: ar.attnres_rmsnorm_bwd(x, gain, 1e-6, dy, dres, rows[0], sums[0], accumulate=False)


# (T is enough for more than PAST_THE_RING rows a team.)
CASES = [
    (_forward, 48000, 256, "bf16", "bf16", 1, 0),                   # single warps
    (_forward, 48000, 256, "bf16", "bf16", 1, PAST_THE_RING),
    (_forward, 20000, 896, "bf16", "f32", 1, 1),                    # several warps, rows in turn over the teams
    (_forward, 20000, 896, "bf16", "f32", 300, PAST_THE_RING),      # runs of shared gate rows, left midway
    (_forward, 4000, 8192, "f32", "f32", 1, 1),                     # one team a CTA
    (_backward, 20000, 640, "bf16", "bf16", 1, 0),                  # single warps
    (_backward, 20000, 640, "bf16", "bf16", 20000, PAST_THE_RING),
    (_backward, 20000, 896, "bf16", "f32", 1, 1),                   # several warps
    (_backward, 20000, 896, "bf16", "f32", 300, PAST_THE_RING),
    (_backward, 4000, 8192, "f32", "f32", 1, 0),                    # a ring of one row
    (_backward, 4000, 8192, "f32", "f32", 1, 1),
    (_backward, 4000, 8192, "f32", "f32", 1, PAST_THE_RING),
    (_backward, 4000, 8192, "bf16", "bf16", 7, 1),
    (_norm_backward, 48000, 256, "bf16", "f32", 1, 0),
    (_norm_backward, 20000, 1024, "bf16", "f32", 1, 1),
    (_norm_backward, 20000, 640, "bf16", "bf16", 1, PAST_THE_RING),
    (_norm_backward, 4000, 8192, "f32", "f32", 1, PAST_THE_RING),
]


@pytest.mark.parametrize("make,T,d,dt,xt,gate_rows,index", CASES)
def test_a_withheld_row_times_out(make, T, d, dt, xt, gate_rows, index):
    rows, sums, run = make(T, d, dt, xt, gate_rows)
    run()
    good = [t.clone() for t in rows + sums]
    for t in rows + sums:
        t.fill_(float("nan"))
    assert ar.attnres_device_status() == 0
    ar.attnres_test_withhold_stage(ar.WITHHOLD_RESIDUAL, index)
    run()
    ar.attnres_test_withhold_stage(ar.WITHHOLD_NONE)
    assert ar.attnres_device_status() == TIMEOUT
    assert ar.attnres_device_status() == 0
    written = [~torch.isnan(t) for t in rows]
    for t, g, w in zip(rows, good, written):
        assert (torch.where(w, t, g) == g).all() and not w.all()
    assert any(bool(w.any()) for w in written) == (index > 0)
    run()
    assert ar.attnres_device_status() == 0
    assert all(torch.equal(t, g) for t, g in zip(rows + sums, good))
