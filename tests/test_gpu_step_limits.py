"""GPU tests of the serving-step entry points at the limits of what they take:
rows that see no token beside queries that are not finite, weights and scales far
apart, logits far from 0, every significand of a scale, calls from two threads,
two errors at once.

The attention's tolerance, per element, with A = sum_t p_t |v_t| and M the
largest p_t times V scale, times the largest code, all over the tokens that the
row sees:
    2^-8 |ref| + 2^-11 A + 2^-18 A  the bf16 output, p in f16, float32 sums and the
                                    merge of split rows
  + 2^-10 A                         per-token scales: the V scale's rounding to f16
                                    and that of the scaled V, 2^-11 each
  + 2 (dq + da) A                   a logit error e changes p by e^(+-e): dq from the
                                    query's residue (2^-17 of the row's largest |q|
                                    per dim), da from float32 sums of D products, the
                                    scale product and the exponential (2^-24 each step)
  + L 2^-32 M                       p below f16's normals has an error of 2^-25 against
                                    a largest one of at least 2^7
  + L 2^-24 M                       instead, per-token scales: the reference of p times
                                    the scale is at most 2^8 above what the row sees (a
                                    bit to a power of two, `spread` = 7 bits between the
                                    scales of a tile that share one)
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import dev
from oracle.formats import decode_bf16, decode_e4m3fn
from test_gpu_step import Chunk, _check_append, _clean, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _reference(c, spread=7):
    """(ref, tolerance), float64, of the requests' rows."""
    q = decode_bf16(c.q_bits)[:int(c.start[-1])]
    T, Hq, D = q.shape
    Hk = c.cache.shape[2]
    scale = D ** -0.5 if c.scale is None else c.scale
    ref, tol = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    for r, L in enumerate(int(x) for x in c.lens):
        a, b = int(c.start[r]), int(c.start[r + 1])
        pos = np.arange(L)
        blk, off = c.table[r, pos // c.bs].astype(np.int64), pos % c.bs
        seen = pos[None, :] <= (L - (b - a) + np.arange(b - a))[:, None]          # [rows, L]
        for h in range(Hk):
            ks, vs = ((x[blk, h, off].astype(np.float64) if c.per_token else np.full(L, float(x[0])))
                      for x in (c.ks, c.vs))
            k, code = (decode_e4m3fn(c.cache[blk, i, h, off]) for i in (0, 1))
            k, v = k * ks[:, None], code * vs[:, None]
            for g in range(h * c.G, (h + 1) * c.G):
                with np.errstate(all="ignore"):
                    s = np.where(seen, scale * (q[a:b, g] @ k.T), -np.inf)
                    p = np.exp(s - np.where(seen.any(axis=1), s.max(axis=1, initial=-np.inf), 0.0)[:, None])
                    p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
                # (0 times what a row does not see is 0)
                for i in range(b - a):
                    n = int(seen[i].sum())
                    w = p[i, :n]
                    ref[a + i, g] = w @ v[:n]
                    A = w @ np.abs(v[:n])
                    M = (w * np.abs(vs[:n])).max(initial=0.0) * np.nan_to_num(np.abs(code[:n])).max(initial=0.0)
                    qk = np.abs(q[a + i, g]).max() * np.abs(k[:n]).sum(axis=1).max(initial=0.0) * abs(scale)
                    e = 2.0 ** -17 * qk + (D + 4) * 2.0 ** -24 * qk + 2.0 ** -22
                    pv = 2.0 ** -11 + 2.0 ** -18 + (2.0 ** -10 if c.per_token else 0.0)
                    tol[a + i, g] = (2.0 ** -8 * np.abs(ref[a + i, g]) + (pv + 2 * e) * A
                                     + n * (2.0 ** (spread - 31) if c.per_token else 2.0 ** -32) * M)
    return ref, tol


def _run(c):
    """The requests' rows; those behind them are left as they were."""
    t = c.tensors()
    out = torch.full(tuple(t["q"].shape), 77.0, dtype=torch.bfloat16, device=dev())
    qpa.pa_chunk_fp8(out=out, **t)
    _clean()
    n = int(c.start[-1])
    assert bool((out[n:] == 77).all())
    return out[:n].double().cpu().numpy()


def _check(c, spread=7):
    got = _run(c)
    ref, tol = _reference(c, spread)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), "NaN pattern differs"
    err, lim = np.abs(got - ref)[~nan], tol[~nan]
    assert np.all(err <= lim), f"worst {np.max(err / np.maximum(lim, 1e-300)):.3g} of the tolerance"


def _place(c, r, pos):
    return c.table[r, pos // c.bs].astype(np.int64), pos % c.bs


VARIANTS = [(128, False), (64, False), (128, True), (64, True)]


@pytest.mark.parametrize("D,per_token", VARIANTS)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_rows_without_a_token_and_bad_queries(D, per_token, bad):
    """A row that sees no token gives 0 whatever its query holds, in an item that
    the schedule cuts (280 rows over 260 tokens, 2 heads: head 1's first item lies
    in two CTAs) as in one that it does not."""
    c = Chunk(41, [(280, 260)], 2, 1, D, 16, per_token)
    q = decode_bf16(c.q_bits)
    q[3, :, 5] = q[19, 1, 0] = bad
    c.q_bits = synth.round_to_bf16_bits(q)
    out = _run(c)
    assert np.all(out[:20] == 0)
    q[3, :, 5] = q[19, 1, 0] = 0
    c.q_bits = synth.round_to_bf16_bits(q)
    ref, tol = _reference(c)
    assert np.all(np.abs(out - ref) <= tol)


@pytest.mark.parametrize("D,per_token", VARIANTS)
@pytest.mark.parametrize("drop", [13.3, 24.5, 25.01, 27.3])
def test_many_small_probabilities(D, per_token, drop):
    """A token of weight 1 and V = 0 in every page, the others 2^-drop of it: the
    result is the sum of those, whatever f16 makes of each."""
    L = 65536
    c = Chunk(42, [(1, L)], 1, 1, D, 256, per_token)
    c.cache[:, 0] = 0
    c.cache[:, 1] = 0x38                                # 1
    c.cache[:, 0, 0, 0, 0] = 0x38
    c.cache[:, 1, 0, 0] = 0
    c.ks[:], c.vs[:] = 0.25, 0.5
    q = np.zeros((1, 1, D))
    q[..., 0] = 1
    c.q_bits = synth.round_to_bf16_bits(q)
    c.scale = float(drop * np.log(2) / 0.25)
    _check(c, spread=0)


# ------------------------------------------------------------------ V scales
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("factor", [1e3, 1e6, -3e7, 1e8, 1e30])
def test_v_scale_of_a_token_that_a_row_does_not_see(D, factor):
    """The rows before a token with an outlying V scale do not notice it."""
    c = Chunk(43, [(60, 300), (40, 40)], 2, 4, D, 16, True)
    for r, tok in ((0, 290), (0, 250), (1, 17)):
        blk, off = _place(c, r, np.array([tok]))
        c.vs[blk, :, off] *= factor
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("factor", [1e6, 1e8, 1e30])
def test_v_scale_of_a_token_without_weight(D, factor):
    """Tokens that are seen with a weight of 0 (keys far against the query) and
    outlying V scales, in the first, a middle and the last key tile."""
    c = Chunk(44, [(9, 600), (2, 5000)], 2, 4, D, 32, True)
    q = np.abs(decode_bf16(c.q_bits))
    c.q_bits = synth.round_to_bf16_bits(q + 0.25)
    for r, toks in ((0, [3, 200, 590]), (1, [1, 2500, 4990])):
        blk, off = _place(c, r, np.array(toks))
        c.cache[blk, 0, :, off] = 0xFE                  # -448
        c.ks[blk, :, off] = 0.08
        c.vs[blk, :, off] *= factor
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("decades", [1, 4, 15, 33])
def test_v_scales_far_apart(D, decades):
    """Scales over many decades within every key tile, zeros and signs among them."""
    c = Chunk(45, [(150, 500), (1, 3000)], 1, 2, D, 16, True)
    r = synth.rng(46)
    live = ~np.isnan(c.vs)
    x = 10.0 ** r.uniform(-decades, decades, c.vs.shape) * np.where(r.random(c.vs.shape) < 0.5, -1, 1)
    x[r.random(c.vs.shape) < 0.1] = 0
    c.vs[live] = x[live].astype(np.float32)
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("order", [1, -1])
def test_v_scales_that_differ_between_key_tiles(D, order):
    """A tile of large scales and little weight beside one of small scales and all
    the weight, in both orders: neither the values of the first nor the weights of
    the second get lost (10^33 between the scales, e^-18 between the weights)."""
    c = Chunk(47, [(3, 384)], 1, 4, D, 128, True)
    q = np.abs(decode_bf16(c.q_bits)) + 0.25
    q *= 4 / q.sum(axis=-1, keepdims=True)
    c.q_bits = synth.round_to_bf16_bits(q)
    c.scale = 1.0
    blk = c.table[0, :3][::order].astype(np.int64)
    c.cache[blk[0], 0], c.cache[blk[1:], 0] = 0xB8, 0x38          # -1 and 1
    c.ks[blk] = 2.25                                              # logits -9 and 9
    c.vs[blk[0]], c.vs[blk[1]], c.vs[blk[2]] = 1e30, 1e-3, 3e-3
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e33])
def test_v_scales_near_the_ends_of_float32(D, size):
    c = Chunk(48, [(20, 300), (1, 2000)], 2, 4, D, 16, True)
    c.vs *= np.float32(size)
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
def test_v_scales_of_zeros(D):
    """Tokens whose V is 0, with the scale that kv_append_fp8 gives them, beside others
    and alone; scales that small with codes beside others of their size."""
    c = Chunk(54, [(40, 300), (20, 20), (30, 500)], 2, 4, D, 16, True)
    r = synth.rng(55)
    for req in (0, 1):
        zero = np.arange(c.lens[req])[(r.random(c.lens[req]) < 0.5) | (req == 1)]
        blk, off = _place(c, req, zero)
        c.cache[blk, 1, :, off] = 0
        c.vs[blk, :, off] = 2.0 ** -126
    blk, off = _place(c, 2, np.arange(500))
    c.vs[blk, :, off] = (2.0 ** r.uniform(-126, -115, (500, 2))).astype(np.float32)
    _check(c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_v_scale_that_is_not_finite(D, bad):
    """NaN in every dim of the rows that see the token, nothing elsewhere."""
    c = Chunk(49, [(60, 300), (40, 40)], 2, 4, D, 16, True)
    for r, tok, h in ((0, 270, 0), (0, 290, 1), (1, 17, 1)):
        blk, off = _place(c, r, np.array([tok]))
        c.vs[blk, h, off] = bad
    out = _run(c)
    clean = np.nan_to_num(c.vs, nan=1.0, posinf=1.0, neginf=1.0)
    blind = np.zeros(out.shape, bool)
    for r, tok, h in ((0, 270, 0), (0, 290, 1), (1, 17, 1)):
        first = int(c.start[r]) + tok - int(c.lens[r] - (c.start[r + 1] - c.start[r]))
        blind[first:int(c.start[r + 1]), h * 4:(h + 1) * 4] = True
    assert np.array_equal(np.isnan(out), blind)
    c.vs = np.where(np.isfinite(c.vs), c.vs, clean)
    ref, tol = _reference(c)
    assert np.all(np.abs(out - ref)[~blind] <= tol[~blind])


# ------------------------------------------------------------------ logits
@pytest.mark.parametrize("D,per_token", VARIANTS)
@pytest.mark.parametrize("size", [1e4, 3e6, 2e7, 6e7])
def test_logits_far_from_zero(D, per_token, size):
    """Logits of about `size` that differ by as much: each row is the V of its
    largest, whatever float32's steps are there."""
    c = Chunk(50, [(70, 400), (1, 700)], 1, 3, D, 16, per_token)
    q = np.abs(decode_bf16(c.q_bits)) + 0.25
    c.q_bits = synth.round_to_bf16_bits(q)
    c.scale = float(size / 0.02 / q.sum(axis=-1).max())
    c.ks[:] = 0.01
    c.cache[:, 0] = 0x38
    for r, tok in ((0, 40), (1, 699)):
        blk, off = _place(c, r, np.array([tok]))
        c.cache[blk, 0, :, off] = 0x40                  # 2 against 1
    got = _run(c)
    ref, _ = _reference(c)
    # p is 1 and its product with V exact but for per-token scales (2^-10)
    assert np.all(np.abs(got - ref) <= (2.0 ** -8 + (2.0 ** -10 if per_token else 0)) * np.abs(ref))


@pytest.mark.parametrize("D,per_token", VARIANTS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1e4, 3e6, 2e7, 6e7])
def test_large_logits_that_differ_little(D, per_token, sign, size):
    """Logits around +-`size` whose differences are a few of float32's steps there and
    grow along the sequence, V the same everywhere: the rows' weights sum to 1."""
    c = Chunk(52, [(70, 1500), (1, 3000)], 2, 3, D, 16, per_token)
    r = synth.rng(53)
    q = np.ones_like(decode_bf16(c.q_bits))
    q[..., 0] = 2.0 ** -15 * 2.0 ** r.integers(0, 8, q.shape[:2])
    c.q_bits = synth.round_to_bf16_bits(q)
    c.scale = float(sign * size / 0.01 / D)
    c.ks[:] = 0.01
    c.vs[:] = 0.5
    c.cache[:, 0], c.cache[:, 1] = 0x38, 0x3C           # 1 and 1.5
    for req, L in enumerate(c.lens):
        pos = np.arange(L)
        blk, off = _place(c, req, pos)
        c.cache[blk, 0, :, off, 0] = np.clip(pos * 100 // L + r.integers(0, 20, L), 0, 119)[:, None]   # 0 to 240
    got = _run(c)
    # (p in f16 against a sum of p in float32, the V scale exact)
    assert np.all(np.abs(got - 0.75) <= 0.75 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18))


# ------------------------------------------------------------------ batches
@pytest.mark.parametrize("D,per_token", VARIANTS)
def test_single_tokens_beside_a_chunk(D, per_token):
    """One new token each of 60 requests over caches of 1 to 1500, two chunks among
    them: more items than CTAs, cut between the heads and in the chunks."""
    r = synth.rng(56)
    reqs = [(1, int(n)) for n in r.integers(1, 1500, 60)]
    reqs[17], reqs[40] = (200, 1400), (90, 90)
    _check(Chunk(57, reqs, 3, 4, D, 32, per_token, pad=5))


# ------------------------------------------------------------------ lengths
def test_longest_request():
    """2^31 - 16 tokens, all of one page but the last 16: the weights are equal and
    their sums exact, and a NaN in the last token's V makes its dim NaN."""
    bs, L = 16, (1 << 31) - 16
    table = torch.zeros(1, L // bs, dtype=torch.int32, device=dev())
    table[0, -1] = 1
    cache = torch.zeros(2, 2, 1, bs, 64, dtype=torch.uint8, device=dev())
    cache[:, 1] = 0x38                                  # 1
    cache[1, 1, 0, 15, 5] = 0x7F
    scale = torch.tensor([0.5], device=dev())
    out = qpa.pa_chunk_fp8(torch.ones(1, 1, 64, dtype=torch.bfloat16, device=dev()), cache, table, _i32([0, 1]), _i32([L]),
                           scale, scale, 1)
    _clean()
    want = torch.full((64,), 0.5)
    want[5] = float("nan")
    assert torch.equal(out.float().cpu().flatten().nan_to_num(9.0), want.nan_to_num(9.0))


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("per_token", [False, True])
def test_append_every_significand_of_a_scale(per_token):
    """All 128 significands that a bf16 scale can have, per tensor and as the
    largest element's, against all significands of 18 binades, both signs."""
    sig = np.arange(128, 256) / 128
    x = np.stack([np.concatenate([s * 2.0 ** -k for k in range(18)]) for s in (sig, -sig)]).reshape(1, -1)
    for top in sig:
        if per_token:        # 127 elements beside the largest
            n = -(-x.size // 127)
            y = np.zeros(n * 127)
            y[:x.size] = x[0]
            y[np.abs(y) > top] = 0
            v = np.concatenate([np.full((n, 1), top), y.reshape(n, 127)], axis=1)
            s = np.zeros((-(-n // 16), 1, 16), np.float32)
        else:
            v = x.reshape(-1, 128) * 2.0 ** 8
            s = np.array([top], np.float32)
        n = len(v)
        bits = synth.round_to_bf16_bits(v).reshape(n, 1, 128)
        cache = np.zeros((-(-n // 16), 2, 1, 16, 128), np.uint8)
        _check_append(bits, bits[::-1].copy(), cache, np.arange(n, dtype=np.int64), s, s)


# ------------------------------------------------------------------ host
def test_slot_maps_of_different_sizes_from_two_threads():
    """Calls with more than 5119 requests take more shared memory than a launch may
    without a limit of its own; sizes at once do not disturb each other. (The C
    entry in tight loops: the binding's host time would keep the calls apart.)"""
    lib, bad = qpa.load_library(), []

    def work(R, stream, t):
        d = qpa.SlotDesc(R, 16, 1, R, R, 0, 0)
        args = [ctypes.c_void_p(x.data_ptr()) for x in t] + [ctypes.byref(d), ctypes.c_void_p(stream.cuda_stream)]
        bad.extend(st for st in (lib.paged_slot_map(*args) for _ in range(20000)) if st)

    threads, outs = [], []
    for R in (16384, 6000, 11000):
        new, old, free = _i32(np.ones(R)), _i32(np.zeros(R)), _i32(np.arange(R))
        table, start, lens, pos, taken = (torch.zeros(n, dtype=torch.int32, device=dev()) for n in (R, R + 1, R, R, 1))
        slots = torch.zeros(R, dtype=torch.int64, device=dev())
        outs.append(slots)
        threads.append(threading.Thread(target=work, args=(R, torch.cuda.Stream(), (
            new, old, table, free, start, lens, slots, pos, taken))))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _clean()
    assert not bad, f"{len(bad)} calls failed with {set(bad)}"
    for x in outs:
        assert torch.equal(x.cpu(), 16 * torch.arange(x.numel()))


def test_two_errors_are_both_reported():
    """paged_slot_map out of blocks, then a chunk call with a bad block id: one
    query reports the one, the next the other."""
    qpa.paged_slot_map(_i32([5]), _i32([0]), _i32([[0]]), _i32([]), 16, 5)
    c = Chunk(51, [(4, 40)], 1, 2, 128, 16)
    c.table[0, 1] = 9999
    qpa.pa_chunk_fp8(**c.tensors())
    torch.cuda.synchronize()
    assert [qpa.kernel_error() for _ in range(3)] == [6, 3, 0]
