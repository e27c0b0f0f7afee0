"""kv_gather_fp8 with scales per token: every code with scales of few and of many bits, next to
midpoints of bf16, negative, infinite and NaN ones, and products down to the smallest normal
number. Values are equal to the exact product rounded once."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import dev
from test_gpu_nvfp4 import done, f32, same_bf16, t32

pytestmark = pytest.mark.gpu


def _scales():
    r = synth.rng(80)
    gs = [(1 + i / 128) * 2.0 ** r.integers(-60, 60) for i in range(128)] + list(np.exp(r.uniform(-60, 60, 60)))
    gs += [np.nextafter(np.float32(m / x), np.float32(d)) for x in (1, 3, 5, 7, 9, 11, 13, 15) for m in (257, 259, 301, 511)
           for d in (0, 1e9)]
    return np.array(gs + [-g for g in gs[:40]] + [0.0, np.inf, -np.inf, np.nan, 3e38, -3e38], dtype=np.float32)


def _check(gs, lowest=0.0):
    """A token per scale, of 256 codes (four heads of 64); products below `lowest` are not looked at."""
    bs = 16
    NB = -(-len(gs) // bs)
    cache = np.empty((NB, 2, 4, bs, 64), dtype=np.uint8)
    cache[:] = np.arange(256, dtype=np.uint8).reshape(4, 1, 64)
    sc = np.zeros((NB, 4, bs), dtype=np.float32)
    t = np.arange(len(gs))
    sc[t // bs, :, t % bs] = gs[:, None]
    d = torch.from_numpy(sc).to(dev())
    args = (torch.from_numpy(cache).to(dev()), t32(np.arange(NB)[None]), t32([0, len(gs)]), t32([len(gs)]))
    with np.errstate(invalid="ignore", over="ignore"):
        want = oracle.decode_e4m3fn(cache[0, 0, :, 0])[None] * gs.astype(np.float64)[:, None, None]
        single = want.astype(np.float32)
    for got, wide in zip(qpa.kv_gather_fp8(*args, d, d, len(gs)), qpa.kv_gather_fp8(*args, d, d, len(gs), out_dtype=torch.float32)):
        assert np.array_equal(wide.cpu().numpy(), single, equal_nan=True)
        # 2^128 - 2^119: halfway between bf16's largest number and the next one
        inf = np.abs(want) >= 2.0 ** 128 - 2.0 ** 119
        g = got.float().cpu().numpy()
        assert np.array_equal(g[inf], np.sign(want[inf]) * np.inf)
        seen = ~inf & ~(np.abs(want) < lowest)
        with np.errstate(invalid="ignore"):
            same_bf16(torch.where(torch.from_numpy(seen).to(dev()), got, 0), np.where(seen, want, 0.0))
    done()


def test_every_code_with_many_scales():
    _check(_scales())


def test_an_infinite_scale_reads_as_it_does_per_tensor():
    cache = torch.arange(256, dtype=torch.uint8, device=dev()).view(1, 1, 1, 1, 256).expand(1, 2, 4, 16, 256)
    cache = cache.reshape(1, 2, 4, 16, 4, 64)[:, :, :, :, 0].contiguous()
    cache += (64 * torch.arange(4, device=dev())).to(torch.uint8).view(1, 1, 4, 1, 1)
    for g in (np.inf, -np.inf, 2.0, -3e38):
        per = torch.full((1, 4, 16), g, device=dev())
        for dtype in (torch.bfloat16, torch.float32):
            a = qpa.kv_gather_fp8(cache, t32([[0]]), t32([0, 16]), t32([16]), per, per, 16, out_dtype=dtype)
            b = qpa.kv_gather_fp8(cache, t32([[0]]), t32([0, 16]), t32([16]), f32(g), f32(g), 16, out_dtype=dtype)
            for x, y in zip(a, b):
                assert torch.equal(torch.isnan(x), torch.isnan(y)) and torch.equal(torch.nan_to_num(x, nan=0.0), torch.nan_to_num(y, nan=0.0))
    done()


def test_products_next_to_the_smallest_normal_number():
    """Products a little above a midpoint of bf16 (7 bits behind the point, then 1, then zeros up to a last bit below 2^-149)
    that are at least 2^-126."""
    gs = []
    for x in (1.125, 1.375, 1.625, 1.875, 9 * 2.0 ** -9, 15 * 2.0 ** -9, 7 * 2.0 ** -9):
        for m in range(257, 512, 2):
            g = np.float32(m * 2.0 ** -134 / x)
            gs += [g, np.nextafter(g, np.float32(1))]
    _check(np.array(gs, dtype=np.float32), lowest=2.0 ** -126)
