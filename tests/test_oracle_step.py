"""Pins of the serving-step oracle (slots, append, chunk attention): values
worked out by hand, closed forms, and agreement with the decode oracle."""
import numpy as np
import torch

import oracle
import synth
from oracle.formats import decode_e4m3fn


def _bits(x):
    return synth.round_to_bf16_bits(np.asarray(x, dtype=np.float32))


def test_slot_map_by_hand():
    # block size 16; request 0 holds 14 tokens in block 7 and brings 3: the
    # third needs a new block; request 1 is new with 17 tokens: two blocks;
    # request 2 brings none
    table = np.array([[7, -1, -1], [-1, -1, -1], [3, -1, -1]])
    start, lens, tab, slots, pos, taken, short = oracle.paged_slot_map([3, 17, 0], [14, 0, 5], table, [20, 21, 22, 23],
                                                                      16, 22)
    assert start.tolist() == [0, 3, 20, 20] and lens.tolist() == [17, 17, 5] and taken == 3 and not short
    assert tab.tolist() == [[7, 20, -1], [21, 22, -1], [3, -1, -1]]
    assert slots.tolist() == [7 * 16 + 14, 7 * 16 + 15, 20 * 16] + [21 * 16 + i for i in range(16)] + [22 * 16, -1, -1]
    assert pos.tolist() == [14, 15, 16] + list(range(17)) + [0, 0]


def test_slot_map_short_of_blocks_and_columns():
    start, lens, tab, slots, pos, taken, short = oracle.paged_slot_map([20, 20], [0, 0], np.full((2, 1), -1), [4, 5], 16, 40)
    assert short and taken == 4 and lens.tolist() == [20, 20]
    # request 0: block 4, then no column for its second block (id 5 is passed
    # over); request 1: no id left
    assert tab.tolist() == [[4], [-1]]
    assert slots.tolist() == [64 + i for i in range(16)] + [-1] * 24


def test_nearest_code_agrees_with_the_cast_where_that_is_exact():
    # scale 1: the cast of a bf16 value to e4m3 is one rounding
    bits = np.arange(0, 65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).float()
    ok = ~torch.isnan(x) & (x.abs() <= 448)
    want = x[ok].to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_nearest(x[ok].numpy(), np.float32(1)), want)
    assert oracle.e4m3_nearest(np.array([np.inf, -np.inf, np.nan, 1e30]), 1.0).tolist() == [0x7E, 0xFE, 0x7F, 0x7E]


def test_nearest_code_is_nearest_and_ties_to_even():
    r = synth.rng(5)
    s = np.exp(r.uniform(-8, 8, size=4000)).astype(np.float32)
    x = decode = torch.from_numpy(r.standard_normal(4000) * 300 * s).to(torch.bfloat16).double().numpy()
    got = decode_e4m3fn(oracle.e4m3_nearest(x, s))
    vals = decode_e4m3fn(np.arange(256, dtype=np.uint8))
    vals = vals[~np.isnan(vals)]
    q = np.clip(decode / s, -448, 448)
    best = np.abs(q[:, None] - vals[None]).min(axis=1)
    # the quotient itself is rounded to 53 bits here
    assert np.all(np.abs(got - q) <= best + 1e-12 * np.abs(q))
    # 3 x 17/16 is the midpoint of codes 3 (1 + 0/8) and 3 (1 + 1/8) at scale 3
    assert oracle.e4m3_nearest(3 * 17 / 16, 3.0) == oracle.e4m3_nearest(3.0, 3.0)
    assert oracle.e4m3_nearest(3 * 19 / 16, 3.0) == oracle.e4m3_nearest(3 * 20 / 16, 3.0)


def test_append_scales_and_untouched_slots():
    r = synth.rng(6)
    k, v = r.standard_normal((3, 2, 64)), r.standard_normal((3, 2, 64))
    k[1, 0] = 0
    cache = np.full((2, 2, 2, 16, 64), 0xAA, dtype=np.uint8)
    ks = np.full((2, 2, 16), 9.0, dtype=np.float32)
    out, ks2, vs2 = oracle.kv_append_fp8(_bits(k), _bits(v), cache, [17, 5, -1], ks, ks)
    touched = np.zeros(cache.shape, bool)
    touched[1, :, :, 1] = touched[0, :, :, 5] = True
    assert np.all(out[~touched] == 0xAA)
    assert ks2[0, 0, 5] == np.float32(2.0 ** -126) and np.all(out[0, 0, 0, 5] == 0)
    # the largest element of a vector takes the largest code
    assert decode_e4m3fn(out[1, 1, 1, 1]).__abs__().max() == 448
    assert ks2[1, 1, 1] != 9 and ks2[1, 1, 2] == 9


def test_chunk_agrees_with_the_multi_token_decode():
    for per_token in (False, True):
        c = synth.make_fp8_ext_case(3, [40, 3, 130], 2, 3, 4, per_token)
        want = oracle.pa_decode_fp8_ext(c.q_bits, c.kv_cache, c.block_table, c.seq_lens, c.k_scale, c.v_scale, 3, 4,
                                        c.softmax_scale)
        q = c.q_bits.reshape(12, 6, 128)
        got, bound = oracle.pa_chunk_fp8(q, c.kv_cache, c.block_table, [0, 4, 8, 12], c.seq_lens, c.k_scale, c.v_scale,
                                         3, c.softmax_scale)
        assert np.allclose(got.reshape(want.shape), want, rtol=1e-12, atol=1e-14)
        assert np.all(bound >= np.abs(got) - 1e-12)


def test_chunk_rows_of_no_request_are_marked():
    c = synth.make_fp8_ext_case(4, [10], 1, 2, 2, False)
    got, _ = oracle.pa_chunk_fp8(np.concatenate([c.q_bits[0]] * 2), c.kv_cache, c.block_table, [0, 2], c.seq_lens,
                                 c.k_scale, c.v_scale, 2)
    assert np.all(np.isfinite(got[:2])) and np.all(np.isnan(got[2:]))
