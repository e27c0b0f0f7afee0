"""Sizes past 31 bits in every dimension of the 4-bit cache's calls and of reading back: the
binding refuses them (a descriptor's field would be cut to its 32 bits)."""
import pytest
import torch

import quantized_paged_attention_gb300 as qpa

U8, I32, I64, F = torch.uint8, torch.int32, torch.int64, torch.float32
BIG = 1 << 32


def _t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _scales():
    return dict(k_scale=_t(1, dtype=F), v_scale=_t(1, dtype=F))


# (blocks, heads, block size, bytes of a row), one past 2^31 that would be cut to a supported one
CACHES4 = [(BIG + 4, 2, 16, 72), (4, BIG + 2, 16, 72), (4, 2, BIG + 16, 72), (4, 2, 16, 9 * (BIG + 128) // 16)]


@pytest.mark.parametrize("NB,Hk,bs,row", CACHES4)
def test_four_bit_caches(NB, Hk, bs, row):
    D = row // 9 * 16
    cache = _t(NB, 2, Hk, bs, row, dtype=U8)
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.kv_append_nvfp4(_t(3, Hk, D), _t(3, Hk, D), cache, _t(3, dtype=I64), **_scales())
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.kv_gather_nvfp4(cache, _t(2, 4, dtype=I32), _t(3, dtype=I32), _t(2, dtype=I32), **_scales(), num_tokens=5)
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.nvfp4_desc(_t(2, 4 * Hk, D), cache, _t(2, 4, dtype=I32), 4)


@pytest.mark.parametrize("NB,Hk,bs,D", [(BIG + 4, 2, 16, 128), (4, BIG + 2, 16, 128), (4, 2, BIG + 16, 128), (4, 2, 16, BIG + 128)])
def test_fp8_caches(NB, Hk, bs, D):
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.kv_gather_fp8(_t(NB, 2, Hk, bs, D, dtype=U8), _t(2, 4, dtype=I32), _t(3, dtype=I32), _t(2, dtype=I32), **_scales(),
                          num_tokens=5)


def test_requests():
    R = BIG + 2
    cache = _t(4, 2, 2, 16, 72, dtype=U8)
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.kv_gather_nvfp4(cache, _t(R, 4, dtype=I32), _t(R + 1, dtype=I32), _t(R, dtype=I32), **_scales(), num_tokens=5)
    with pytest.raises(ValueError, match="2\\^31"):
        qpa.nvfp4_desc(_t(R, 8, 128), cache, _t(R, 4, dtype=I32), 4)
