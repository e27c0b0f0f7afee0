"""pa_decode_nvfp4 with tensor scales and softmax scales at the ends of float32, where the
logits and the results are ordinary numbers."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import done, f32, rand_cache, rand_table, t32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,bs,lens,cols", [(128, 8, 16, [4000, 300, 1], 1), (64, 16, 32, [9000], 1), (64, 3, 128, [500, 20], 0)])
@pytest.mark.parametrize("g", [1e-36, -3e-35, 2.0 ** -132, 1e33])
def test_value_scales(D, G, bs, lens, cols, g):
    """Results keep bf16's bits however small v_scale is. Tolerance: as the other decodes, and 2^-133 (bf16's smallest step,
    half of it for the rounding of a result below 2^-126, less for float32's before). The last case has a table of 512 tokens."""
    r = synth.rng(D + G)
    table, NB = rand_table(r, lens, bs, cols=cols)
    cache, lens = rand_cache(r, NB, 2, bs, D, smax=127), np.array(lens)
    q = synth.round_to_bf16_bits(0.2 * r.standard_normal((len(lens), 2 * G, D)))
    want, bound, total, slack = oracle.pa_decode_nvfp4(q, cache, table, lens, .02, g, G)
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), t32(table), t32(lens), f32(.02), f32(g), G)
    done()
    tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(slack)[..., None] + 2.0 ** -18)
    tol += 2.0 ** -33 * (total + lens[:, None, None] * np.abs(want)) + 2.0 ** -133
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("k_scale,scale,size,group_scale", [
    (2.0 ** -140, 0.06566, 2.0 ** 126, 0x7E), (2.0 ** -100, 1.37 * 2.0 ** -40, 2.0 ** 126, 0x7E),
    (2.0 ** -149, 1.7 * 2.0 ** 30, 2.0 ** 111, 0x38), (2.0 ** 60, 2.0 ** -148, 2.0 ** 80, 0x38),
    (2.0 ** 127, 1.3 * 2.0 ** 10, 2.0 ** -130, 0x01), (1.9 * 2.0 ** 100, -1.1 * 2.0 ** 30, 2.0 ** -130, 0x01),
    (1.9 * 2.0 ** 100, 1.7 * 2.0 ** -100, 2.0 ** -7, 0x38)])
def test_key_and_softmax_scales(k_scale, scale, size, group_scale):
    """Products of the two scales outside float32's normal range, queries and group scales that bring the logits back.

    Seven tokens, each of one key in all dims; the last query is zeros. Queries and keys enter the product exactly, so a logit is off by 2^-21 of
    itself at most (the factors' and the sums' roundings), and weights as in the other tests."""
    q = np.zeros((1, 5, 64)) + size * np.array([1.0, 1.5, 0.75, -1.0, 0.0])[:, None]
    codes = np.zeros((1, 2, 1, 16, 32), dtype=np.uint8)
    scales = np.full((1, 2, 1, 16, 4), 0x38, dtype=np.uint8)
    codes[0, 0, 0, :7] = np.array([0x77, 0x55, 0xDD, 0xFF, 0x22, 0x00, 0x44], dtype=np.uint8)[:, None]
    scales[0, 0] = group_scale
    codes[0, 1, 0, :7] = synth.rng(3).integers(0, 256, (7, 32), dtype=np.uint8)
    cache = oracle.nvfp4._join(codes, scales)
    bits = synth.round_to_bf16_bits(q)
    assert np.array_equal(oracle.decode_bf16(bits), q)
    got = qpa.pa_decode_nvfp4(bf16_tensor(bits, dev()), torch.from_numpy(cache).to(dev()), t32([[0]]), t32([7]), f32(k_scale),
                              f32(1.0), 5, softmax_scale=scale)
    done()
    got = got.float().cpu().numpy()[0]
    K, V = (oracle.values_nvfp4(cache, i, g, np.zeros(7, dtype=int), np.arange(7))[:, 0] for i, g in ((0, k_scale), (1, 1.0)))
    x = float(np.float32(scale)) * (q[0] @ K.T)
    assert 0.5 < np.abs(x[:4]).max(axis=1).min() and np.abs(x).max() < 400
    w = np.exp(x - x.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    want, bound = w @ V, w @ np.abs(V)
    tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(2.0 ** -21 * np.abs(x).max(axis=1))[:, None] + 2.0 ** -18)
    tol += 2.0 ** -33 * (np.abs(V).sum(axis=0) + 7 * np.abs(want))
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("k_scale,scale", [(np.nan, 0.1), (np.inf, 0.1), (-np.inf, 0.1), (1.0, np.nan), (1.0, np.inf)])
def test_scales_that_are_not_finite(k_scale, scale):
    """Logits are NaN or infinite: every row is NaN, that of a query of zeros (0 times infinity) too."""
    r = synth.rng(4)
    cache = rand_cache(r, 4, 1, 16, 64, smax=60)
    q = r.standard_normal((2, 3, 64))
    q[:, 1] = 0.0
    out = qpa.pa_decode_nvfp4(bf16_tensor(synth.round_to_bf16_bits(q), dev()),
                              torch.from_numpy(cache).to(dev()), t32([[1, 2], [3, 0]]), t32([32, 9]),
                              f32(k_scale), f32(1.0), 3, softmax_scale=scale)
    done()
    assert bool(torch.isnan(out).all())
