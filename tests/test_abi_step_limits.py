"""Refusals of the serving-step entry points at the limits of 32-bit sizes, without
a GPU."""
import pytest
import torch

import quantized_paged_attention_gb300 as qpa


def _meta(*shape):
    """No memory behind it: the call has to be refused for its sizes."""
    return torch.empty(*shape, dtype=torch.int32, device="meta")


@pytest.mark.parametrize("kw", [dict(max_tokens=(1 << 32) + 8), dict(max_tokens=1 << 31), dict(max_tokens=-1),
                                dict(block_size=(1 << 32) + 16), dict(block_size=-16),
                                dict(free_blocks=_meta(1 << 31)), dict(block_table=_meta(2, 1 << 31))])
def test_slot_map_refuses_sizes_past_32_bits(kw):
    """Each would reach the library cut to 32 bits: 2^32 + 8 rows as 8, the others
    left unwritten."""
    args = dict(new_lens=_meta(2), cached_lens=_meta(2), block_table=_meta(2, 4), free_blocks=_meta(3), block_size=16,
                max_tokens=8)
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.paged_slot_map(**{**args, **kw})


def test_chunk_refuses_a_table_past_32_bits():
    q = torch.empty(1, 1, 64, dtype=torch.bfloat16, device="meta")
    cache = torch.empty(1, 2, 1, 16, 64, dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.chunk_desc(q, cache, _meta(1, (1 << 32) + 4), 1, False)
