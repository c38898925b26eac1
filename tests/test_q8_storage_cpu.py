"""Replacing the storage of 8-bit rows and weights: what is refused before any call."""
import pytest
import torch

import __graft_entry__ as graft
from depth_wise_attention_attnres_gb300 import binding


@pytest.mark.parametrize("kind,sizes,shape", [(binding.Q8Rows, {"n": 2, "T": 5, "d": 300}, (2, 2048)),
                                              (binding.Q8Weight, {"m": 200, "d": 300}, (76832,))])
def test_buffers_that_do_not_fit(kind, sizes, shape):
    graft.build()
    size = binding.attnres_q8_source_bytes(5, 300) if kind is binding.Q8Rows else binding.attnres_q8_weight_bytes(200, 300)
    assert shape[-1] == size
    holder = kind.__new__(kind)  # its own storage would have to be on a GPU
    holder.__dict__.update(sizes, _shape=shape)
    for bad in (torch.zeros(shape, dtype=torch.int8), torch.zeros(*shape[:-1], size - 16, dtype=torch.uint8),
                torch.zeros(*shape[:-1], 2 * size, dtype=torch.uint8)[..., ::2], torch.zeros(shape, dtype=torch.uint8)):
        with pytest.raises(ValueError):  # the last one is on the CPU
            holder.buffer = bad
    with pytest.raises(ValueError):
        kind(*sizes.values(), device="cpu")
