"""pa_decode_nvfp4 with logits so large that float32 has steps of 2 to 32 there: where the
running reference is put and when it moves are decided in rounded numbers.

A logit may be off by 2^-21 of itself (of 2^26: 32 and more), so weights of tokens that lie
nearer than that say nothing; the tests give such tokens one and the same value. A weighted
mean of equal values v is off by the rounding of the result, 2^-8, and 2^-18 for the sums of
float32 (p is the same number in both sums). Tokens whose logits are further below than
that weigh 0: their values are others."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import done, f32, rand_table, t32

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


def _pages(lens_max, D, key1, value):
    """(cache, table row) of one head: token t's key is 1 in dim 0, key1[t] (an e2m1 code) in dim 16 and 0 elsewhere;
    its values are the code value[t] everywhere, scale 1."""
    table, NB = rand_table(synth.rng(D + lens_max), [lens_max], 16)
    codes = np.zeros((NB, 2, 1, 16, D // 2), dtype=np.uint8)
    scales = np.full((NB, 2, 1, 16, D // 16), 0x38, dtype=np.uint8)
    t = np.arange(lens_max)
    blk, off = table[0, t // 16], t % 16
    codes[blk, 0, 0, off, 0] = 2
    codes[blk, 0, 0, off, 8] = key1
    codes[blk, 1, 0, off] = (value | value << 4).astype(np.uint8)[:, None]
    return oracle.nvfp4._join(codes, scales), table


def _decode(q, cache, table, lens, G, scale=1 / LOG2E):
    n = q.shape[0]
    out = qpa.pa_decode_nvfp4(bf16_tensor(synth.round_to_bf16_bits(q), dev()), torch.from_numpy(cache).to(dev()),
                              t32(np.repeat(table, n, axis=0)), t32(lens), f32(1.0), f32(1.0), G, softmax_scale=scale)
    done()
    return out.float().cpu().numpy()


@pytest.mark.parametrize("D,G", [(128, 8), (64, 8), (128, 16), (64, 12)])
@pytest.mark.parametrize("L", [1, 40])
@pytest.mark.parametrize("scale", [1.0, 0.37])
def test_one_logit_of_up_to_2_to_the_29(D, G, L, scale):
    """Tokens of one key, logits (base 2) of 2^23 to 2^29 of either sign and of all of float32's bits: steps of 1 to 64."""
    B = 64
    amp = np.exp2(np.linspace(23, 29, B * G)).reshape(B, G) / (scale * LOG2E)
    for sign in (1, -1):
        q = np.zeros((B, G, D))
        q[:, :, 0] = sign * amp
        cache, table = _pages(L, D, np.zeros(L, dtype=np.uint8), np.full(L, 5, dtype=np.uint8))
        out = _decode(q, cache, table, [L] * B, G, scale)
        assert np.all(np.abs(out - 3.0) <= 3.0 * (2.0 ** -8 + 2.0 ** -18)), np.isnan(out).sum()


@pytest.mark.parametrize("D,G", [(128, 8), (64, 8), (128, 16), (64, 12)])
def test_logits_a_few_steps_apart_in_different_tiles(D, G):
    """From tile to tile the logits go up by 0 to 6 of float32's steps, so that the reference moves by as little as it
    can, or just does not; then tokens behind them with logits 2^-7 of themselves below, which weigh nothing."""
    B, tiles = 64, 30
    r = synth.rng(D + G)
    up = np.array([0, 1, 2, 3, 4, 5, 6, 7])                                # codes of 0, .5, 1, 1.5, 2, 3, 4, 6
    pick = np.sort(r.integers(0, 8, (tiles // 3, 3)), axis=0)              # (ascending among the tiles a group of warps takes)
    key1 = np.concatenate([np.repeat(up[pick.reshape(-1)], 128), np.full(100, 9)])
    value = np.concatenate([np.full(128 * tiles, 5), np.full(100, 15)]).astype(np.uint8)   # 3, and -6 behind
    cache, table = _pages(key1.size, D, key1.astype(np.uint8), value)
    for sign in (1, -1):
        q = np.zeros((B, G, D))
        x = np.exp2(r.uniform(24, 29, (B, G)))
        q[:, :, 0] = sign * x
        q[:, :, 16] = np.exp2(np.floor(np.log2(x)) - 23) * 2 ** r.integers(0, 2, (B, G))
        out = _decode(q, cache, table, [128 * tiles] * B, G)
        assert np.all(np.abs(out - 3.0) <= 3.0 * (2.0 ** -8 + 2.0 ** -18)), np.isnan(out).sum()
        q[:, :, 16] = x * 2.0 ** -6
        out = _decode(q, cache, table, [key1.size] * B, G)
        assert np.all(np.abs(out - 3.0) <= 3.0 * (2.0 ** -8 + 2.0 ** -18)), np.isnan(out).sum()


@pytest.mark.parametrize("x", [-3.05e38, -3.3e38, 3.05e38, 3.3e38])
def test_logits_next_to_the_largest_float(x):
    q = np.zeros((2, 4, 64))
    q[:, :, 0] = x
    cache, table = _pages(300, 64, np.zeros(300, dtype=np.uint8), np.full(300, 5, dtype=np.uint8))
    out = _decode(q, cache, table, [300, 7], 4)
    assert np.all(np.abs(out - 3.0) <= 3.0 * (2.0 ** -8 + 2.0 ** -18)), out
