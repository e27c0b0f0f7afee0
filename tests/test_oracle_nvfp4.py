"""The 4-bit cache's oracle against exact rational arithmetic and the formats."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
import synth

E2M1 = [Fraction(x).limit_denominator(2) for x in (0, .5, 1, 1.5, 2, 3, 4, 6)]
E4M3 = [Fraction(float(v)) for v in oracle.decode_e4m3fn(np.arange(127, dtype=np.uint8))]


def _pick(x, values):
    """Index of the nearest value, ties to the even index."""
    best = min(range(len(values)), key=lambda i: (abs(values[i] - x), i % 2))
    return best


@pytest.mark.parametrize("g", [1.0, 0.031, 7.3, 2.0 ** -20, 1.0 / 3])
def test_codes_are_the_nearest(g):
    r = synth.rng(int(g * 1000) + 5)
    x = oracle.decode_bf16(synth.round_to_bf16_bits(r.standard_normal((24, 32)) * g * r.choice([1, 30, 0.01], (24, 1))))
    x[0, :16] = 0.0
    codes, scales = oracle.quantise_nvfp4(x, np.float32(g))
    gf = Fraction(float(np.float32(g)))
    for row in range(x.shape[0]):
        nib = oracle.formats.unpack_nibbles(codes[row])
        for b in range(2):
            grp = [Fraction(float(v)) for v in x[row, 16 * b:16 * b + 16]]
            s = max(1, _pick(max(abs(v) for v in grp) / (6 * gf), E4M3))
            assert scales[row, b] == s
            for v, c in zip(grp, nib[16 * b:16 * b + 16]):
                assert c & 7 == _pick(abs(v) / (E4M3[s] * gf), E2M1)
                assert v == 0 or (c >> 3) == (v < 0)


def test_values_that_the_format_holds_come_back():
    """Every code times every scale from 2^-6 on (below, a smaller scale may serve) with the group's largest code 6."""
    e2 = oracle.decode_e2m1(np.arange(16, dtype=np.uint8))
    for s in range(8, 127):
        x = e2 * oracle.decode_e4m3fn(np.uint8(s))
        codes, scales = oracle.quantise_nvfp4(x[None], 1.0)
        assert scales[0, 0] == s
        assert np.array_equal(oracle.formats.unpack_nibbles(codes[0]), np.arange(16))


def test_special_groups():
    x = np.zeros((4, 16))
    x[0, 3], x[1, 3], x[2, 0] = np.nan, np.inf, 1e-30
    codes, scales = oracle.quantise_nvfp4(x, 1.0)
    assert scales[:, 0].tolist() == [0x7F, 0x7E, 0x01, 0x01]
    assert codes[0].tolist() == [0] * 8 and codes[1, 1] == 0x70 and not codes[2:].any()
    for g in (0.0, -1.0, np.nan, np.inf):
        codes, scales = oracle.quantise_nvfp4(np.ones((1, 16)), g)
        assert scales[0, 0] == 0x7F and not codes.any()


def test_pages_read_as_the_scorer_does():
    """One plane, one head, 128 tokens of 128 dims with g = 1: the scorer's page."""
    r = synth.rng(3)
    k = synth.round_to_bf16_bits(r.standard_normal((150, 1, 128)))
    cache = oracle.kv_append_nvfp4(k, None, np.zeros((2, 1, 1, 128, 72), dtype=np.uint8), np.arange(150), 1.0, None)
    q = oracle.round_e4m3(r.standard_normal((1, 1, 128)))
    codes = np.array([[[int(np.argmin(np.abs(oracle.decode_e4m3fn(np.arange(127, dtype=np.uint8)) - abs(v)))) |
                        (0x80 if v < 0 else 0) for v in q[0, 0]]]], dtype=np.uint8)
    dots = oracle.nvfp4_index_score_per_token(codes, cache.reshape(2, 9216), np.array([[0, 1]]), np.array([150]), 1, 150)
    K = oracle.values_nvfp4(cache, 0, 1.0, np.arange(150) // 128, np.arange(150) % 128)[:, 0]
    assert np.allclose(dots[0, 0], K @ q[0, 0], rtol=1e-12, atol=1e-12)


def test_decode_against_a_dense_softmax():
    r = synth.rng(4)
    k, v = (synth.round_to_bf16_bits(r.standard_normal((37, 2, 64))) for _ in range(2))
    table = np.array([[2, 0, 1]])
    slots = table[0, np.arange(37) // 16] * 16 + np.arange(37) % 16
    cache = oracle.kv_append_nvfp4(k, v, np.zeros((3, 2, 2, 16, 36), dtype=np.uint8), slots, 0.1, 0.2)
    q = synth.round_to_bf16_bits(r.standard_normal((1, 6, 64)))
    out, bound, total, slack = oracle.pa_decode_nvfp4(q, cache, table, [37], 0.1, 0.2, 3)
    K, V = (oracle.values_nvfp4(cache, i, g, slots // 16, slots % 16) for i, g in ((0, 0.1), (1, 0.2)))
    assert np.all(np.abs(K - oracle.decode_bf16(k)) <= 0.2 * np.abs(oracle.decode_bf16(k)).max())
    for hq in range(6):
        x = K[:, hq // 3] @ oracle.decode_bf16(q)[0, hq] / 8
        w = np.exp(x) / np.exp(x).sum()
        assert np.allclose(out[0, hq], w @ V[:, hq // 3], rtol=1e-12, atol=1e-12)
        assert np.all(bound[0, hq] >= np.abs(out[0, hq]) - 1e-12) and np.all(total[0, hq] >= bound[0, hq]) and 0 < slack[0, hq] < 1e-2
