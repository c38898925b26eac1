"""The 8-bit projection's tensor-core kernels when a copy never arrives (withheld on purpose; every wait ends after about
two seconds): the call returns, the timeout is reported once, nothing wrong is written, and the next call is right."""
import pytest
import torch

import depth_wise_attention_attnres_gb300 as ar
from depth_wise_attention_attnres_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = 4

# T, d, m, and stages of a CTA: in the first tile, a ring of them, in all. One CTA a tile of 64 columns (two blocks a
# stage), of 128 (one block; some CTAs have two tiles), and pairs of CTAs (two blocks, the tile's last stage one).
SINGLE, WIDE, PAIRS = (40, 2048, 640), (5120, 2048, 640), (8192, 896, 896)
CASES = [(SINGLE, i) for i in (0, 1, 4, 7, 8)] + [(WIDE, i) for i in (0, 6, 15, 20, 31, 32)] + [(PAIRS, i) for i in (0, 3, 5, 7, 8)]
STAGES = {SINGLE: 8, WIDE: 32, PAIRS: 8}


@pytest.fixture(autouse=True)
def _hook_off():
    assert ar.attnres_device_status() == 0
    yield
    binding.attnres_test_withhold_stage(binding.WITHHOLD_NONE)


@pytest.mark.parametrize("sizes,index", CASES)
def test_a_copy_that_never_arrives(sizes, index):
    T, d, m = sizes
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    rows = ar.attnres_q8_write(torch.randn(T, d, generator=g, device=DEV), ar.Q8Rows(1, T, d, device=DEV))
    W8 = ar.attnres_q8_weight(torch.randn(m, d, generator=g, device=DEV) / d ** 0.5, ar.Q8Weight(m, d, device=DEV))
    want = ar.attnres_query_projection_q8(rows, 0, W8, torch.empty(T, m, device=DEV))
    assert ar.attnres_device_status() == 0
    Q = torch.full((T, m), float("nan"), device=DEV)
    binding.attnres_test_withhold_stage(binding.WITHHOLD_Q8_PROJ, index)
    ar.attnres_query_projection_q8(rows, 0, W8, Q)
    status = ar.attnres_device_status()
    binding.attnres_test_withhold_stage(binding.WITHHOLD_NONE)
    written = ~Q.isnan()
    if index < STAGES[sizes]:
        assert status == TIMEOUT and ar.attnres_device_status() == 0 and not written.all()
    else:
        assert status == 0 and written.all()
    assert torch.equal(Q[written], want[written])
    ar.attnres_query_projection_q8(rows, 0, W8, Q)
    assert ar.attnres_device_status() == 0 and torch.equal(Q, want)
