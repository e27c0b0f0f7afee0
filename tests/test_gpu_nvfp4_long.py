"""The longest sequence with values that differ from range to range of the work, so that each
range's piece shows in the result."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import done, f32, rand_cache, t32
from test_gpu_nvfp4_cut import ctas_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(128, 4), (64, 12)])
def test_every_range_of_2_to_the_31_tokens_counts(D, G):
    """Spans of the table, each of one block whose values lie in two dims of its own: leaving out any of the
    152 ranges, or counting one twice, changes some dims of the result by a tenth and more.

    Tolerance: 2^-8 of the result, weights as in the other tests, and for float32 sums of n terms n 2^-23 of the sum of
    their magnitudes: a warp adds 2 sums of 16 tokens per tile, every third (with more than 8 rows every second, with
    heads of 64 and up to 8 every fourth) of its range's tiles."""
    r = synth.rng(D + 1)
    bs, spans = 256, 2 * D
    maxb = (2 ** 31 - 1) // bs
    span = np.minimum(np.arange(maxb) * spans // maxb, spans - 1).astype(np.int32)
    L = maxb * bs - 3
    cache = rand_cache(r, spans, 1, bs, D, smax=48)
    codes, scales = oracle.nvfp4._split(cache)
    codes[:, 1] = 0
    for s in range(spans):
        codes[s, 1, :, :, s % (D // 2)] = 0x57                              # 6 and 3
    scales[:, 1] = 0x38                                                     # 1
    cache = oracle.nvfp4._join(codes, scales)
    q = synth.round_to_bf16_bits(0.3 * r.standard_normal((1, G, D)))
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), torch.from_numpy(span[None]).to(dev()),
                              t32([L]), f32(.2), f32(.2), G)
    done()
    blk, off = np.repeat(np.arange(spans), bs), np.tile(np.arange(bs), spans)
    K = oracle.values_nvfp4(cache, 0, .2, blk, off)[:, 0]
    V = oracle.values_nvfp4(cache, 1, .2, np.arange(spans), np.zeros(spans, dtype=int))[:, 0]    # (one value per block)
    x = oracle.decode_bf16(q)[0] @ K.T / np.sqrt(D)
    e = np.exp(x - x.max(axis=1, keepdims=True)).reshape(G, spans, bs)
    last = e[:, span[-1], -3:].sum(axis=1)                                  # the tokens behind the end
    w = e.sum(axis=2)                                                       # weight of one block of each span
    ctas = ctas_of(1 << 20)

    def attention(count, cut):
        p = w * count
        p[:, span[-1]] -= cut * last
        return p @ V / p.sum(axis=1, keepdims=True)

    count = np.bincount(span, minlength=spans).astype(np.float64)
    want = attention(count, 1)
    adds = 2 * 2 ** 24 / ctas / (3 if D == 128 and G <= 8 else 4 if G <= 8 else 2)
    qq = np.abs(oracle.decode_bf16(q)[0])
    slack = (qq.max(axis=1) * 2.0 ** -16 * np.abs(K).sum(axis=1).max()) / np.sqrt(D) + 2.0 ** -21 * np.abs(x).max(axis=1)
    tol = np.abs(want) * (2.0 ** -8 + 2 * 2.0 ** -11 + 2 * np.expm1(slack)[:, None] + 2 * adds * 2.0 ** -23)
    err = np.abs(out[0].float().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()
    # what the tolerance tells apart
    edge = np.linspace(0, maxb, ctas + 1).astype(int)
    for a, b in zip(edge[:-1], edge[1:]):
        part = np.bincount(span[a:b], minlength=spans)
        for f in (-1, 1):
            assert np.any(np.abs(attention(count + f * part, 1) - want) > 2 * tol)
