"""The storage of 8-bit rows and weights replaced: calls and views go to the new one, and what does not fit is refused."""
import copy

import pytest
import torch

import depth_wise_attention_attnres_gb300 as ar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def look(holder):
    names = ("codes", "exponents") + (("tails", "mean_square") if isinstance(holder, ar.Q8Rows) else ())
    return {k: getattr(holder, k) for k in names}


def fill(holder, scale):
    shape = (holder.n, holder.T, holder.d) if isinstance(holder, ar.Q8Rows) else (holder.m, holder.d)
    x = torch.arange(shape[-1], device=DEV).float().add(1).expand(shape) * scale
    (ar.attnres_q8_write if isinstance(holder, ar.Q8Rows) else ar.attnres_q8_weight)(x.contiguous(), holder)
    return x


def same(holder, x):
    """The views show what a holder looked at for the first time shows, and that is x."""
    fresh = ar.Q8Rows(holder.n, holder.T, holder.d, device=DEV) if isinstance(holder, ar.Q8Rows) else \
        ar.Q8Weight(holder.m, holder.d, device=DEV)
    fresh.buffer.copy_(holder.buffer)
    for k, t in look(holder).items():
        want = look(fresh)[k]
        assert t.data_ptr() - holder.pointer == want.data_ptr() - fresh.pointer, k
        if t.dtype == torch.float8_e4m3fn:
            t, want = t.float(), want.float()
        assert torch.equal(t, want), k
    if isinstance(holder, ar.Q8Rows):
        back = ar.attnres_q8_read(holder, torch.empty(holder.n, holder.T, holder.d, device=DEV))
        assert ((back - x).abs() <= x.abs() * 2.0 ** -4).all()


@pytest.mark.parametrize("make", [lambda: ar.Q8Rows(2, 5, 300, device=DEV), lambda: ar.Q8Weight(200, 300, device=DEV)],
                         ids=["rows", "weight"])
def test_views_follow_the_buffer(make):
    holder = make()
    same(holder, fill(holder, 1.0))
    before, old = look(holder), holder.buffer.clone()
    # a copy with storage of its own
    other = copy.copy(holder)
    other.buffer = torch.zeros_like(holder.buffer)
    same(other, fill(other, 64.0))
    assert torch.equal(holder.buffer, old)
    for k, t in look(holder).items():
        assert t.data_ptr() == before[k].data_ptr()  # the first one's views are what they were
    # the same holder, and a buffer whose data is replaced in place
    holder.buffer = torch.zeros_like(old)
    same(holder, fill(holder, 2.0 ** -20))
    holder.buffer.data = torch.zeros_like(old)
    same(holder, fill(holder, 4096.0))
    # through a view into what calls read
    holder.exponents.add_(1)
    if isinstance(holder, ar.Q8Rows):
        back = ar.attnres_q8_read(holder, torch.empty(2, 5, 300, device=DEV))
        assert float(back[1, 4, 7]) == 8 * 8192.0
    # looked at twice, a view is the same tensor
    assert all(a is b for a, b in zip(look(holder).values(), look(holder).values()))
    deep = copy.deepcopy(holder)
    assert deep.pointer != holder.pointer
    same(deep, fill(deep, 1.0))


@pytest.mark.parametrize("make", [lambda: ar.Q8Rows(2, 5, 300, device=DEV), lambda: ar.Q8Weight(200, 300, device=DEV)],
                         ids=["rows", "weight"])
def test_buffers_that_do_not_fit(make):
    holder = make()
    b, at = holder.buffer, holder.pointer
    for other in (torch.zeros_like(b)[..., :-16], b.cpu(), b.char(), torch.zeros(*b.shape[:-1], 2 * b.shape[-1],
                  dtype=torch.uint8, device=DEV)[..., ::2], b.view(-1).float(), b.unsqueeze(0)):
        with pytest.raises(ValueError):
            holder.buffer = other
        assert holder.pointer == at
