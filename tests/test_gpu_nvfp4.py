"""The 4-bit cache on the GPU against the float64 oracle: the append's bytes, the
values read back (of the fp8 cache too), the decode, and a server's steps with all
of them.

Tolerances. Bytes and values read back are equal. A decode's error is the rounding
of the result, 2^-8 of it (bf16, half a step), and for errors of the probabilities
sum p |v| times: half a step of f16, 2^-11 (of a weight and, the other way, of their
sum); e^x - 1 for a logit's error x, twice (a weight and the sum); 2^-18 for
exponentials and sums of float32. A weight enters in f16 relative to a reference that
lies 2^8 or more below the largest weight, so one in f16's subnormals (steps of 2^-24)
is off by at most 2^-25 there, 2^-33 of the largest weight, and the sum of weights is
at least the largest: 2^-33 sum |v| for the weights, and 2^-33 of the result per token
for their sum."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev

pytestmark = pytest.mark.gpu


def t32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def f32(x):
    return torch.tensor([x], dtype=torch.float32, device=dev())


def done():
    torch.cuda.synchronize()
    assert qpa.kernel_error() == 0


def bf16_of(x):
    """float64 -> bf16 bits, rounded once (ties to even), by the neighbours' distances."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        top = x.astype(np.float32).view(np.uint32) >> 16
        best = None
        for d in (-1, 0, 1):
            bits = (top.astype(np.int64) + d).clip(0, 0xFFFF).astype(np.uint16)
            dist = np.abs(oracle.decode_bf16(bits) - x)
            if best is None:
                best, near = bits, dist
            else:
                take = (dist < near) | ((dist == near) & (bits % 2 == 0)) | np.isnan(near)
                best, near = np.where(take, bits, best), np.where(take, dist, near)
    return best.astype(np.uint16)


def same_bf16(got, want):
    """bf16 tensor == float64 values rounded once; NaN where the value is NaN."""
    g = got.view(torch.int16).cpu().numpy().view(np.uint16)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(oracle.decode_bf16(g)), nan)
    ok = (g == bf16_of(np.where(nan, 0.0, want))) | nan | ((want == 0) & (g & 0x7FFF == 0))
    assert ok.all(), (int((~ok).sum()), want[~ok][:4], oracle.decode_bf16(g)[~ok][:4])


def rand_cache(r, NB, Hk, bs, D, planes=2, smax=100):
    """Random codes and scales: every code, scales of all sizes below smax."""
    codes = r.integers(0, 256, (NB, planes, Hk, bs * D // 2), dtype=np.uint8)
    scales = r.integers(0, smax, (NB, planes, Hk, bs * D // 16), dtype=np.uint8)
    return np.concatenate([codes, scales], axis=-1).reshape(NB, planes, Hk, bs, D // 16 * 9)


def rand_table(r, lens, bs, spare=2, cols=1):
    """(table, number of blocks): each sequence its own blocks, in any order; -1 behind them."""
    need = [-(-int(x) // bs) for x in lens]
    NB = sum(need) + spare
    ids = r.permutation(NB)
    table = np.full((len(lens), max(need + [0]) + cols), -1, dtype=np.int32)
    o = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[o:o + n]
        o += n
    return table, NB


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("T,Hk,D,bs,planes,fused", [
    (1, 1, 64, 16, 2, False), (1, 1, 128, 256, 1, False), (7, 3, 128, 16, 2, True), (130, 8, 128, 64, 2, True),
    (33, 5, 64, 32, 2, False), (300, 1, 128, 128, 1, False), (9, 40, 128, 16, 2, False), (2000, 2, 64, 128, 2, True)])
@pytest.mark.parametrize("g", [0.031, 1.0])
def test_append(T, Hk, D, bs, planes, fused, g):
    r = synth.rng(T * 7 + Hk + D)
    NB = -(-T // bs) + 3
    x = r.standard_normal((T, 4 * Hk, D)) * np.exp(2 * r.standard_normal((T, 4 * Hk, 1)))
    x[:, :, ::D // 4] *= 20
    bits = synth.round_to_bf16_bits(x)
    slots = r.permutation(NB * bs)[:T].astype(np.int64)
    slots[r.random(T) < 0.1] = -1
    before = r.integers(0, 256, (NB, planes, Hk, bs, D // 16 * 9), dtype=np.uint8)
    kb, vb = bits[:, 2 * Hk:3 * Hk], bits[:, 3 * Hk:]
    if fused:
        q = bf16_tensor(bits, dev())
        k, v = q[:, 2 * Hk:3 * Hk], q[:, 3 * Hk:]
    else:
        k, v = bf16_tensor(kb, dev()), bf16_tensor(vb, dev())
    cache = torch.from_numpy(before).to(dev())
    two = planes == 2
    got = qpa.kv_append_nvfp4(k, v if two else None, cache, torch.from_numpy(slots).to(dev()), f32(g),
                              f32(g / 3) if two else None)
    done()
    want = oracle.kv_append_nvfp4(kb, vb if two else None, before, slots, g, g / 3)
    assert got is cache and np.array_equal(cache.cpu().numpy(), want)


def _append_rows(x, g):
    """Codes and scales that the kernel gives for x [T, 1, 64] (float64 values that bf16 holds)."""
    T = x.shape[0]
    NB = -(-T // 16)
    bits = synth.round_to_bf16_bits(x)
    with np.errstate(invalid="ignore"):
        assert np.array_equal(oracle.decode_bf16(bits), x, equal_nan=True)
    cache = torch.zeros(NB, 1, 1, 16, 36, dtype=torch.uint8, device=dev())
    qpa.kv_append_nvfp4(bf16_tensor(bits, dev()), None, cache, torch.arange(T, device=dev()), f32(g), None)
    want = oracle.kv_append_nvfp4(bits, None, np.zeros(cache.shape, dtype=np.uint8), np.arange(T), g, None)
    return cache.cpu().numpy(), want


def test_append_at_the_borders():
    """For many scales, values at and next to each midpoint between codes, and group
    maxima at and next to each midpoint between scales."""
    r = synth.rng(11)
    gs = [np.float32(x) for x in (1.0, 0.5, 3.0, 1 / 3, 0.1, 7.0 / 64, 1.7014118e38, 2.0 ** -126)]
    gs += [np.float32(x) for x in np.exp(r.uniform(-60, 60, 60))]
    gs += [np.float32((1 + i / 64) * 2.0 ** -5) for i in range(64)]        # few bits: many exact midpoints
    e4, mids = oracle.decode_e4m3fn(np.arange(127, dtype=np.uint8)), np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5])
    top = oracle.decode_bf16(np.uint16(0x7F7F))
    for g in gs:
        rows = []
        for s in r.integers(1, 126, 24):
            near = oracle.decode_bf16(bf16_of(mids * e4[s] * float(g)))
            grp = np.zeros(64)
            grp[0] = oracle.decode_bf16(bf16_of(6 * e4[s] * float(g)))     # the group's largest
            grp[1:8], grp[16], grp[17:24] = near, grp[0], -near * (1 + 2.0 ** -7)
            grp[32] = oracle.decode_bf16(bf16_of(6 * (e4[s] + e4[s + 1]) / 2 * float(g)))
            grp[48] = grp[32] * (1 - 2.0 ** -7)
            rows.append(oracle.decode_bf16(bf16_of(np.clip(grp, -top, top))))
        got, want = _append_rows(np.array(rows)[:, None, :], float(g))
        assert np.array_equal(got, want), g
    done()


@pytest.mark.parametrize("g", [1.0, 1e-30, 1e-38, 1e-42, 1e30, 3e38, 0.0, -1.0, np.inf, np.nan])
def test_append_special_values(g):
    x = np.zeros((12, 1, 64))
    r = synth.rng(5)
    x[1:] = oracle.decode_bf16(synth.round_to_bf16_bits(r.standard_normal((11, 1, 64))))
    x[2, 0, 5], x[3, 0, 20], x[4, 0, 63], x[5, 0, :16] = np.nan, np.inf, -np.inf, np.inf
    x[6] *= 2.0 ** -100
    x[7] *= 2.0 ** 100
    x[8] = 2.0 ** -133                                                     # subnormal
    x[9, 0, ::2] = oracle.decode_bf16(np.uint16(0x7F7F))
    x[10, 0, 3] = -0.0
    got, want = _append_rows(x, g)
    assert np.array_equal(got, want)
    done()


def test_append_skips_and_reports_slots_past_the_pool():
    bits = synth.round_to_bf16_bits(synth.rng(6).standard_normal((4, 1, 64)))
    cache = torch.full((2, 1, 1, 16, 36), 9, dtype=torch.uint8, device=dev())
    slots = torch.tensor([3, 32, 2 ** 40, -5], device=dev())
    qpa.kv_append_nvfp4(bf16_tensor(bits, dev()), None, cache, slots, f32(1.0), None)
    assert qpa.kernel_error() == 3
    want = oracle.kv_append_nvfp4(bits, None, np.full((2, 1, 1, 16, 36), 9, dtype=np.uint8), [3, -1, -1, -1], 1.0, None)
    assert np.array_equal(cache.cpu().numpy(), want)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("lens,Hk,D,bs,planes", [
    ([1], 1, 64, 16, 2), ([100], 2, 64, 32, 2), ([0, 17, 0, 300, 16, 1], 3, 128, 16, 2), ([500, 3], 8, 128, 256, 2),
    ([65, 64, 63], 1, 128, 64, 1), ([33] * 40, 20, 64, 128, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gather_nvfp4(lens, Hk, D, bs, planes, dtype):
    r = synth.rng(sum(lens) + Hk)
    table, NB = rand_table(r, lens, bs)
    cache = rand_cache(r, NB, Hk, bs, D, planes, smax=128)                 # 127: NaN
    # windows: whole requests, their last tokens, none, and more rows than tokens
    n = [int(r.choice([x, (x + 1) // 2, 0, x + 3])) for x in lens]
    start = np.concatenate([[2], 2 + np.cumsum(n)])
    T = int(start[-1]) + 3
    outs = [torch.full((T, Hk, D), 7.0, dtype=dtype, device=dev()) for _ in range(planes)]
    wide = torch.full((len(lens), table.shape[1] + 5), -1, dtype=torch.int32, device=dev())
    wide[:, :table.shape[1]] = t32(table)
    gs = [0.037, 1.9]
    k, v = qpa.kv_gather_nvfp4(torch.from_numpy(cache).to(dev()), wide[:, :table.shape[1]], t32(start), t32(lens),
                               f32(gs[0]), f32(gs[1]) if planes == 2 else None, T, outs[0], outs[-1] if planes == 2 else None,
                               dtype)
    done()
    rows, blk, off, zero = oracle.gather_rows(table, start, lens, bs)
    for plane, got in enumerate([k, v][:planes]):
        want = np.full((T, Hk, D), 7.0)
        want[zero] = 0.0
        want[rows] = oracle.values_nvfp4(cache, plane, gs[plane], blk, off)
        if dtype == torch.bfloat16:
            same_bf16(got, want)
        else:
            assert np.array_equal(got.cpu().numpy(), want.astype(np.float32), equal_nan=True)
    assert (v is None) == (planes == 1)


@pytest.mark.parametrize("lens,Hk,D,bs,per_token", [
    ([1], 1, 64, 16, False), ([0, 37, 129], 4, 128, 16, True), ([400, 1, 90], 5, 64, 64, True), ([513], 8, 128, 256, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gather_fp8(lens, Hk, D, bs, per_token, dtype):
    r = synth.rng(sum(lens) + Hk + 1)
    table, NB = rand_table(r, lens, bs)
    cache = r.integers(0, 256, (NB, 2, Hk, bs, D), dtype=np.uint8)
    sc = [np.exp(r.standard_normal((NB, Hk, bs) if per_token else 1)).astype(np.float32) for _ in range(2)]
    start = np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1])
    got = qpa.kv_gather_fp8(torch.from_numpy(cache).to(dev()), t32(table), t32(start), t32(lens),
                            *[torch.from_numpy(x).to(dev()) for x in sc], T, out_dtype=dtype)
    done()
    rows, blk, off, _ = oracle.gather_rows(table, start, lens, bs)
    for plane in range(2):
        s = sc[plane].astype(np.float64)
        want = oracle.decode_e4m3fn(cache[blk, plane, :, off]) * (s[blk, :, off][..., None] if per_token else s[0])
        if dtype == torch.bfloat16:
            same_bf16(got[plane], want)
        else:
            assert np.array_equal(got[plane].cpu().numpy(), want.astype(np.float32), equal_nan=True)


def test_gather_bad_blocks_and_clamped_lengths():
    r = synth.rng(8)
    cache = rand_cache(r, 4, 1, 16, 64)
    table = np.array([[1, 99, 3], [-1, 2, 0]], dtype=np.int32)
    lens, start = [48, 1000], [0, 48, 96]                                   # the second is clamped to 48
    k, v = qpa.kv_gather_nvfp4(torch.from_numpy(cache).to(dev()), t32(table), t32(start), t32(lens), f32(1.0), f32(1.0), 96)
    assert qpa.kernel_error() == 3
    fixed = np.array([[1, 0, 3], [0, 2, 0]])
    rows, blk, off, _ = oracle.gather_rows(fixed, start, [48, 48], 16)
    for plane, got in enumerate((k, v)):
        same_bf16(got, oracle.values_nvfp4(cache, plane, 1.0, blk, off))


# ------------------------------------------------------------------ decode
class Case:
    def __init__(self, lens, Hk, G, D, bs, seed=0, qamp=1.0, gs=(0.05, 0.3), outliers=True):
        r = synth.rng(1000 + seed + sum(lens) + Hk * G)
        self.table, NB = rand_table(r, lens, bs)
        self.lens, self.G, self.gs = np.asarray(lens), G, gs
        x = r.standard_normal((2, NB * bs, Hk, D))
        if outliers:
            x[0, :, :, ::D // 4] *= 8
        kb, vb = synth.round_to_bf16_bits(x)
        self.cache = oracle.kv_append_nvfp4(kb, vb, np.zeros((NB, 2, Hk, bs, D // 16 * 9), dtype=np.uint8),
                                            np.arange(NB * bs), *gs)
        self.q = synth.round_to_bf16_bits(qamp * r.standard_normal((len(lens), Hk * G, D)))

    def run(self, q=None, table=None, cache=None, **kw):
        q = bf16_tensor(self.q, dev()) if q is None else q
        cache = torch.from_numpy(self.cache).to(dev()) if cache is None else cache
        return qpa.pa_decode_nvfp4(q, cache, t32(self.table) if table is None else table, t32(self.lens),
                                   f32(self.gs[0]), f32(self.gs[1]), self.G, **kw)

    def check(self, out, softmax_scale=None, seqs=None):
        assert out.dtype == torch.bfloat16
        got = out.float().cpu().numpy().astype(np.float64)
        want, bound, total, slack = oracle.pa_decode_nvfp4(self.q, self.cache, self.table, self.lens, *self.gs, self.G, softmax_scale)
        tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(slack)[..., None] + 2.0 ** -18)
        tol += 2.0 ** -33 * (total + self.lens[:, None, None] * np.abs(want))
        bad = ~(np.abs(got - want) <= tol)
        if seqs is not None:
            bad = bad[seqs]
        assert not bad.any(), (int(bad.sum()), np.abs(got - want).max(), (np.abs(got - want) / tol).max())
        assert not got[self.lens == 0].any()


@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [127, 128, 129], [15, 16, 17, 255, 256, 257, 0], [1000] * 3, [4097]])
@pytest.mark.parametrize("Hk,G,D,bs", [(1, 1, 128, 16), (2, 8, 128, 32), (3, 5, 64, 16), (1, 16, 128, 256), (2, 12, 64, 128),
                                       (1, 64, 128, 64), (2, 33, 64, 16)])
def test_decode(lens, Hk, G, D, bs):
    c = Case(lens, Hk, G, D, bs)
    out = c.run()
    done()
    c.check(out)


@pytest.mark.parametrize("lens,Hk,G,D,bs", [([70001], 1, 16, 128, 128), ([30000, 1, 9000], 2, 4, 64, 16),
                                            (list(range(0, 2000, 31)), 4, 3, 128, 16), ([300] * 200, 2, 8, 128, 64),
                                            ([700, 2], 80, 2, 128, 16), ([150] * 3, 170, 1, 64, 32)])
def test_decode_splits(lens, Hk, G, D, bs):
    """Ranges that cut a sequence many times, span many sequences, and more heads than SMs."""
    c = Case(lens, Hk, G, D, bs, outliers=False)
    out = c.run()
    done()
    c.check(out)


@pytest.mark.parametrize("qamp,scale", [(1e-3, None), (30.0, None), (400.0, 0.25), (1.0, 1e-4), (2.0, -0.1), (0.0, None)])
def test_decode_logit_ranges(qamp, scale):
    for D, G in ((128, 8), (64, 16)):
        c = Case([400, 90], 2, G, D, 16, qamp=qamp)
        out = c.run(softmax_scale=scale)
        done()
        c.check(out, scale)


def test_decode_large_and_small_queries():
    """Rows and scale groups of a row that differ by many powers of two; a row of zeros."""
    c = Case([333], 2, 8, 128, 16)
    q = oracle.decode_bf16(c.q)
    q[0, 1] *= 2.0 ** -60
    q[0, 2, 16:32] *= 2.0 ** -30
    q[0, 3, 5] = 200.0
    q[0, 4] = 0.0
    q[0, 5, :64] = 0.0
    q[0, 6] *= 2.0 ** -126
    c.q = synth.round_to_bf16_bits(q)
    out = c.run()
    done()
    c.check(out)


def test_decode_queries_that_are_not_finite_stay_in_their_rows():
    c = Case([200, 77], 2, 4, 128, 16)
    q = oracle.decode_bf16(c.q)
    clean = c.run()
    q[0, 1, 7], q[1, 6, 100], q[0, 5, 0] = np.nan, np.inf, -np.inf
    bits = np.where(np.isfinite(q), c.q, np.where(np.isnan(q), 0x7FC0, np.where(q > 0, 0x7F80, 0xFF80))).astype(np.uint16)
    out = c.run(q=bf16_tensor(bits, dev()))
    done()
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 1] = bad[1, 6] = bad[0, 5] = True
    bad = bad.to(dev())
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("D,bs,L", [(128, 16, 201), (64, 64, 130), (128, 256, 383)])
def test_decode_tokens_past_the_end_have_no_influence(D, bs, L):
    """Blocks filled with NaN scales behind the last token, and in every other block."""
    c = Case([L, 5], 2, 8, D, bs)
    clean = c.run()
    cache = c.cache.reshape(c.cache.shape[0], 2, 2, -1).copy()
    sc = cache[..., bs * D // 2:].reshape(cache.shape[0], 2, 2, bs, D // 16)
    code = cache[..., :bs * D // 2].reshape(cache.shape[0], 2, 2, bs, D // 2)
    live = np.zeros((cache.shape[0], bs), dtype=bool)
    for s in range(2):
        for t in range(c.lens[s]):
            live[c.table[s, t // bs], t % bs] = True
    for b, o in zip(*np.nonzero(~live)):
        sc[b, :, :, o], code[b, :, :, o] = 0x7F, 0xFF
    cache = np.concatenate([code.reshape(*cache.shape[:3], -1), sc.reshape(*cache.shape[:3], -1)], -1)
    out = c.run(cache=torch.from_numpy(cache.reshape(c.cache.shape)).to(dev()))
    done()
    assert torch.equal(out, clean)


def test_decode_nan_scales_that_are_seen():
    c = Case([150, 60], 2, 4, 128, 16)
    clean = c.run()
    codes, scales = oracle.nvfp4._split(c.cache)
    scales[c.table[0, 70 // 16], 1, 1, 70 % 16, 3] = 0x7F                   # V of token 70, head 1, dims 48 .. 63
    scales[c.table[1, 10 // 16], 0, 0, 10 % 16, 2] = 0x7F                   # K of token 10, head 0 of the second
    out = c.run(cache=torch.from_numpy(oracle.nvfp4._join(codes, scales)).to(dev()))
    done()
    want = torch.zeros(2, 8, 128, dtype=torch.bool, device=dev())
    want[0, 4:, 48:64] = True
    want[1, :4] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], clean[~want])


def test_decode_strided_and_bad_blocks():
    c = Case([90, 300, 40], 2, 4, 128, 16)
    wide = torch.zeros(3, 20, 128, dtype=torch.bfloat16, device=dev())
    wide[:, 5:13] = bf16_tensor(c.q, dev())
    table = torch.full((3, c.table.shape[1] + 7), 99999, dtype=torch.int32, device=dev())
    table[:, :c.table.shape[1]] = t32(c.table)
    plain = c.run()
    out = c.run(q=wide[:, 5:13], table=table[:, :c.table.shape[1]])
    done()
    assert torch.equal(out, plain)
    c.check(out)
    bad = c.table.copy()
    bad[1, 3], bad[1, 5] = -7, 1 << 30
    out = c.run(table=t32(bad))
    assert qpa.kernel_error() == 3
    c.table = bad.copy()
    c.table[1, 3] = c.table[1, 5] = 0
    c.check(out)


def test_decode_workspace_needs_no_initialisation_and_calls_repeat():
    c = Case([3000, 1, 500], 2, 8, 128, 16)
    d = qpa.nvfp4_desc(bf16_tensor(c.q, dev()), torch.from_numpy(c.cache).to(dev()), t32(c.table), 8)
    n = qpa.pa_decode_nvfp4_workspace_size(d)
    outs = [c.run(workspace=torch.full((n,), fill, dtype=torch.uint8, device=dev())) for fill in (0, 0xFF, 0x7F)]
    done()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    c.check(outs[0])


def test_decode_pages_past_4_gib():
    """Blocks at the end of a pool of 4.8 GB: offsets past 32 bits."""
    r = synth.rng(21)
    Hk, bs, D = 8, 128, 128
    NB = (1 << 32) // (2 * Hk * bs * 72) + 40
    pool = torch.zeros(NB, 2, Hk, bs, 72, dtype=torch.uint8, device=dev())
    lens, G = [500, 129], 4
    kb, vb = (synth.round_to_bf16_bits(r.standard_normal((629, Hk, D))) for _ in range(2))
    table = np.array([[NB - 1, NB - 5, 3, NB - 2], [NB - 9, NB - 3, 0, 0]], dtype=np.int32)
    tok = np.concatenate([np.arange(x) for x in lens])
    req = np.repeat([0, 1], lens)
    slots = table[req, tok // bs].astype(np.int64) * bs + tok % bs
    qpa.kv_append_nvfp4(bf16_tensor(kb, dev()), bf16_tensor(vb, dev()), pool, torch.from_numpy(slots).to(dev()), f32(.1), f32(.1))
    q = synth.round_to_bf16_bits(r.standard_normal((2, Hk * G, D)))
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), pool, t32(table), t32(lens), f32(.1), f32(.1), G)
    k, v = qpa.kv_gather_nvfp4(pool, t32(table), t32([0, 500, 629]), t32(lens), f32(.1), f32(.1), 629)
    done()
    used = np.unique(table)
    small = pool[torch.from_numpy(used).to(dev()).long()].cpu().numpy()
    c = Case.__new__(Case)
    c.q, c.cache, c.table, c.lens, c.gs, c.G = q, small, np.searchsorted(used, table), np.array(lens), (.1, .1), G
    c.check(out)
    rows, blk, off, _ = oracle.gather_rows(c.table, [0, 500, 629], lens, bs)
    same_bf16(k, oracle.values_nvfp4(small, 0, .1, blk, off))
    same_bf16(v, oracle.values_nvfp4(small, 1, .1, blk, off))


# ------------------------------------------------------------------ together
def test_scorer_pages_are_written_and_scored():
    """Keys appended to one-plane pages, scored by nvfp4_index_score."""
    r = synth.rng(31)
    k = synth.round_to_bf16_bits(r.standard_normal((300, 1, 128)))
    slots = np.concatenate([2 * 128 + np.arange(128), 0 * 128 + np.arange(128), 3 * 128 + np.arange(44)])
    pages = torch.zeros(4, 9216, dtype=torch.uint8, device=dev())
    qpa.kv_append_nvfp4(bf16_tensor(k, dev()), None, pages.view(4, 1, 1, 128, 72), torch.from_numpy(slots).to(dev()),
                        f32(1.0), None)
    q = synth.round_to_e4m3_bytes(r.standard_normal((2, 2, 128)))
    table = np.array([[2, 0, 3]], dtype=np.int32)
    got = qpa.nvfp4_index_score(torch.from_numpy(q).to(dev()), pages, t32(table), t32([300]), 2, 4)
    done()
    want = oracle.nvfp4_index_score(q, pages.cpu().numpy(), table, np.array([300]), 2, 4)
    g = got.cpu().double().numpy()
    assert np.array_equal(np.isneginf(g), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.all(np.abs(g[fin] - want[fin]) <= 1e-4 * np.maximum(np.abs(want[fin]), 1))


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_server(captured):
    """Three steps: slots, append, decode, the step's tokens read back; eagerly on a
    side stream, or as two captured graphs with a workspace each that run at the
    same time."""
    r = synth.rng(41)
    Hk, G, D, bs, R = 2, 4, 128, 16, 3
    steps = [[33, 0, 7], [1, 20, 1], [1, 1, 1]]
    cap = max(sum(s) for s in steps)
    copies = 2 if captured else 1
    side = torch.cuda.Stream()
    states = []
    for _ in range(copies):
        st = dict(table=torch.full((R, 8), -1, dtype=torch.int32, device=dev()), old=t32([0] * R), new=t32([0] * R),
                  free=t32(r.permutation(24)), k=torch.zeros(cap, Hk, D, dtype=torch.bfloat16, device=dev()),
                  cache=torch.zeros(*qpa.nvfp4_cache_shape(24, Hk, bs, D), dtype=torch.uint8, device=dev()),
                  q=torch.zeros(R, Hk * G, D, dtype=torch.bfloat16, device=dev()), ks=f32(.07), vs=f32(.2))
        st["v"] = torch.zeros_like(st["k"])
        states.append(st)

    def step(st, stream=None):
        start, lens, slots, _, taken = qpa.paged_slot_map(st["new"], st["old"], st["table"], st["free"], bs, cap, stream=stream)
        qpa.kv_append_nvfp4(st["k"], st["v"], st["cache"], slots, st["ks"], st["vs"], stream=stream)
        out = qpa.pa_decode_nvfp4(st["q"], st["cache"], st["table"], lens, st["ks"], st["vs"], G, stream=stream)
        k, v = qpa.kv_gather_nvfp4(st["cache"], st["table"], start, lens, st["ks"], st["vs"], cap, stream=stream)
        return dict(start=start, lens=lens, slots=slots, taken=taken, out=out, k=k, v=v)

    graphs = []
    if captured:
        step(states[0])                                                    # (writes blocks that the steps write again)
        torch.cuda.synchronize()
        for st in states:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                res = step(st)
            graphs.append((g, res))
    held = [np.zeros(R, dtype=int)] * copies
    table = [np.full((R, 8), -1) for _ in range(copies)]
    cache = [s["cache"].cpu().numpy() for s in states]
    for i, new in enumerate(steps):
        n = sum(new)
        data = [synth.round_to_bf16_bits(r.standard_normal((2, cap, Hk, D))) for _ in range(copies)]
        qs = [synth.round_to_bf16_bits(r.standard_normal((R, Hk * G, D))) for _ in range(copies)]
        for st, x, q in zip(states, data, qs):
            st["k"].copy_(bf16_tensor(x[0], dev()))
            st["v"].copy_(bf16_tensor(x[1], dev()))
            st["q"].copy_(bf16_tensor(q, dev()))
            st["new"].copy_(t32(new))
        torch.cuda.synchronize()
        if captured:
            for j, (g, _) in enumerate(graphs):
                with torch.cuda.stream([side, torch.cuda.Stream()][j]):
                    g.replay()
            res = [x for _, x in graphs]
        else:
            res = [step(states[0], side)]
        torch.cuda.synchronize()
        assert qpa.kernel_error() == 0
        for j, (st, out) in enumerate(zip(states, res)):
            start, lens, tab, slots, _, taken, short = oracle.paged_slot_map(new, held[j], table[j], st["free"].cpu().numpy(),
                                                                             bs, cap)
            assert not short and np.array_equal(st["table"].cpu().numpy(), tab)
            cache[j] = oracle.kv_append_nvfp4(data[j][0], data[j][1], cache[j], slots, .07, .2)
            assert np.array_equal(st["cache"].cpu().numpy(), cache[j])
            c = Case.__new__(Case)
            c.q, c.cache, c.table, c.lens, c.gs, c.G = qs[j], cache[j], tab, lens, (.07, .2), G
            c.check(out["out"])
            rows, blk, off, _ = oracle.gather_rows(tab, start, lens, bs)
            assert len(rows) == n
            same_bf16(out["k"][:n], oracle.values_nvfp4(cache[j], 0, .07, blk, off))
            same_bf16(out["v"][:n], oracle.values_nvfp4(cache[j], 1, .2, blk, off))
            held[j], table[j] = lens, tab
            st["old"].copy_(t32(lens))
            st["free"].copy_(torch.roll(st["free"], -int(taken)))


def test_fp8_pages_are_written_and_read_back():
    r = synth.rng(51)
    k, v = (synth.round_to_bf16_bits(r.standard_normal((70, 2, 64))) for _ in range(2))
    cache = torch.zeros(8, 2, 2, 16, 64, dtype=torch.uint8, device=dev())
    ks, vs = (torch.zeros(8, 2, 16, device=dev()) for _ in range(2))
    table = t32(r.permutation(8)[None, :5])
    _, lens, slots, _, _ = qpa.paged_slot_map(t32([70]), t32([0]), torch.full((1, 5), -1, dtype=torch.int32, device=dev()),
                                              table[0].contiguous(), 16, 70)
    qpa.kv_append_fp8(bf16_tensor(k, dev()), bf16_tensor(v, dev()), cache, slots, ks, vs)
    gk, gv = qpa.kv_gather_fp8(cache, table, t32([0, 70]), lens, ks, vs, 70, out_dtype=torch.float32)
    done()
    for got, bits in ((gk, k), (gv, v)):
        x = oracle.decode_bf16(bits)
        # half a step of e4m3 (2^-4), or of its subnormals (2^-10 of the scale: a / 448), and of the scale's own rounding
        tol = 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * np.abs(x).max(-1, keepdims=True) / 448 + 2.0 ** -22 * np.abs(x)
        assert np.all(np.abs(got.cpu().numpy() - x) <= tol)
