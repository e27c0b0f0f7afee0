"""GPU parity of the serving-step entry points (paged_slot_map, kv_append_fp8,
pa_chunk_fp8) against the float64 oracle, alone and together.

Slots, tables, lengths and e4m3 codes have to be equal. The tolerance of the
attention, per element, with A = sum_t p_t |v_t| from the oracle:
    2^-8 |ref|                      the output's rounding to bf16
  + 2^-11 A                         the probabilities' rounding to f16
  + 2^-10 A                         per-token scales: the V scale's rounding to f16 and
                                    that of the scaled V, 2^-11 each
  + 2 (dq + da) A                   a logit error e changes p by e^(+-e): dq from the
                                    query's residue (2^-18 of the row's largest |q| per
                                    dim), da from float32 sums of D products, the scale
                                    product and the exponential (2^-24 each step)
  + L 2^-24 max|v|                  probabilities below f16's normals round to multiples of
                                    2^-24 (half a step each, doubled by the V scale's
                                    power of two), against a largest one of at least 1
  + 2^-18 A                         float32 sums of p and p v, the merge of split rows
"""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from oracle.formats import decode_bf16, decode_e4m3fn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _clean():
    torch.cuda.synchronize()
    assert qpa.kernel_error() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


# ------------------------------------------------------------------ slots
def _slot_case(seed, new, ctx, bs, spare=4, extra_cols=2):
    r = synth.rng(seed)
    held = [-(-c // bs) for c in ctx]
    need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    maxb = max([1] + need) + extra_cols
    ids = r.permutation(sum(need) + spare + 3).astype(np.int64)
    table = np.full((len(new), maxb), -7)
    o = 0
    for i, n in enumerate(held):
        table[i, :n] = ids[o:o + n]
        o += n
    return table, ids[o:o + sum(need) - sum(held) + spare]


def _check_slots(new, ctx, table, free, bs, max_tokens, table_t=None, err=None):
    table_t = _i32(table) if table_t is None else table_t
    start, lens, tab, slots, pos, taken, short = oracle.paged_slot_map(new, ctx, table, free, bs, max_tokens)
    new_t, ctx_t, free_t = _i32(new), _i32(ctx), _i32(free)
    for _ in range(2):                                  # the same inputs again give the same result
        got = qpa.paged_slot_map(new_t, ctx_t, table_t, free_t, bs, max_tokens)
        torch.cuda.synchronize()
        want_err = (6 if short else 0) if err is None else err
        assert qpa.kernel_error() == want_err
        for g, w, name in zip(got, (start, lens, slots, pos, [taken]),
                              ("query_start", "seq_lens", "slots", "positions", "num_taken")):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w)), name
        assert np.array_equal(table_t.cpu().numpy(), tab)
    assert np.array_equal(new_t.cpu().numpy(), new) and np.array_equal(ctx_t.cpu().numpy(), ctx)


@pytest.mark.parametrize("batch,new_hi,ctx_hi,bs,pad", [(1, 1, 1, 16, 0), (1, 2000, 0, 16, 7), (3, 0, 50, 32, 5),
                                                        (37, 1, 900, 16, 0), (100, 70, 3000, 64, 33),
                                                        (511, 9, 300, 128, 1), (513, 5, 300, 256, 0),
                                                        (2049, 3, 100, 16, 100)])
def test_slots_tables_and_lengths(batch, new_hi, ctx_hi, bs, pad):
    r = synth.rng(batch)
    new, ctx = r.integers(0, new_hi + 1, batch), r.integers(0, ctx_hi + 1, batch)
    ctx[r.random(batch) < 0.2] = (ctx_hi // bs) * bs    # ends exactly on a block
    table, free = _slot_case(batch, new.tolist(), ctx.tolist(), bs)
    _check_slots(new, ctx, table, free, bs, int(new.sum()) + pad)


def test_slots_of_the_most_requests():
    new, ctx = np.ones(qpa.SLOT_MAP_MAX_REQS, dtype=np.int64), np.arange(qpa.SLOT_MAP_MAX_REQS) % 31
    table, free = _slot_case(1, new.tolist(), ctx.tolist(), 16)
    _check_slots(new, ctx, table, free, 16, len(new))


def test_slots_empty_calls():
    _check_slots(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 3), int), np.zeros(0, int), 16, 5)
    _check_slots(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 3), int), np.zeros(0, int), 16, 0)
    _check_slots(np.zeros(2, int), np.array([3, 0]), np.array([[5], [9]]), np.zeros(0, int), 16, 0)


def test_slots_with_too_few_rows_blocks_or_columns():
    new, ctx = np.array([40, 3, 25, 0]), np.array([5, 16, 0, 70])
    table, free = _slot_case(2, new.tolist(), ctx.tolist(), 16, spare=0)
    _check_slots(new, ctx, table, free, 16, 50)                  # the last tokens get no row
    _check_slots(new, ctx, table, free[:2], 16, 80)              # out of blocks
    _check_slots(new, ctx, table, free[:0], 16, 80)
    _check_slots(new, ctx, table[:, :2], free, 16, 80)           # out of columns
    _check_slots(np.array([-3, 4]), np.array([-1, 2]), np.array([[1], [2]]), [], 16, 6)   # negatives are 0


def test_slots_with_a_negative_block():
    table = np.array([[-1, -1], [3, -1]])
    _check_slots(np.array([2, 1]), np.array([4, 4]), table, [8], 16, 4, err=3)
    _check_slots(np.array([2, 1]), np.array([16, 4]), np.array([[6, -1], [3, -1]]), [-5], 16, 4, err=3)


def test_slots_strided_table_and_given_outputs():
    new, ctx = np.array([40, 3, 25]), np.array([5, 16, 0])
    table, free = _slot_case(3, new.tolist(), ctx.tolist(), 16)
    wide = torch.full((3, table.shape[1] + 9), 123456, dtype=torch.int32, device=dev())
    wide[:, :table.shape[1]] = _i32(table)
    _check_slots(new, ctx, table, free, 16, 70, table_t=wide[:, :table.shape[1]])
    assert bool((wide[:, table.shape[1]:] == 123456).all())
    slots = torch.empty(70, dtype=torch.int64, device=dev())
    got = qpa.paged_slot_map(_i32(new), _i32(ctx), _i32(table), _i32(free), 16, 70, slots=slots)
    assert got[2] is slots
    _clean()


# ------------------------------------------------------------------ append
def _append(k_bits, v_bits, cache, slots, ks, vs, fused=False):
    if fused:       # k and v as slices of a wider projection
        wide = torch.zeros(k_bits.shape[0], 3 * k_bits.shape[1], k_bits.shape[2], dtype=torch.bfloat16, device=dev())
        Hk = k_bits.shape[1]
        wide[:, Hk:2 * Hk], wide[:, 2 * Hk:] = bf16_tensor(k_bits, dev()), bf16_tensor(v_bits, dev())
        k, v = wide[:, Hk:2 * Hk], wide[:, 2 * Hk:]
    else:
        k, v = bf16_tensor(k_bits, dev()), bf16_tensor(v_bits, dev())
    c = torch.from_numpy(cache).to(dev())
    ks, vs = torch.from_numpy(np.array(ks)).to(dev()), torch.from_numpy(np.array(vs)).to(dev())
    out = qpa.kv_append_fp8(k, v, c, torch.from_numpy(slots).to(dev()), ks, vs)
    assert out is c
    torch.cuda.synchronize()
    return c.cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy()


def _check_append(k_bits, v_bits, cache, slots, ks, vs, fused=False, err=0):
    got = _append(k_bits, v_bits, cache, slots, ks, vs, fused)
    assert qpa.kernel_error() == err
    want = oracle.kv_append_fp8(k_bits, v_bits, cache, slots, ks, vs)
    for g, w, name in zip(got, want, ("cache", "k_scale", "v_scale")):
        assert np.array_equal(g.view(np.uint8), np.asarray(w).view(np.uint8)), name


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("T,Hk,D,bs,fused", [(1, 1, 64, 16, False), (1, 1, 128, 16, True), (7, 3, 128, 32, True),
                                             (33, 8, 64, 64, False), (130, 5, 128, 128, False), (301, 2, 64, 256, True),
                                             (9, 20, 128, 16, False), (5, 70, 64, 16, True)])
def test_append_codes_and_scales(T, Hk, D, bs, fused, per_token):
    r = synth.rng(T * 7 + Hk + D)
    k, v = (synth.round_to_bf16_bits(r.standard_normal((T, Hk, D)) * np.exp(r.uniform(-4, 4, (T, Hk, 1))))
            for _ in range(2))
    NB = -(-T // bs) + 2
    cache = r.integers(0, 256, (NB, 2, Hk, bs, D)).astype(np.uint8)
    slots = r.permutation(NB * bs)[:T].astype(np.int64)
    slots[r.random(T) < 0.15] = -1
    if per_token:
        ks, vs = (r.random((NB, Hk, bs)).astype(np.float32) for _ in range(2))
    else:
        ks, vs = np.array([0.37], np.float32), np.array([0.004], np.float32)
    _check_append(k, v, cache, slots, ks, vs, fused)


@pytest.mark.parametrize("scale", [1.0, 0.125, 3.0, 0.75, 1 / 448, 0.1, 1e-3, 7e4, 1e-35, 1e35, 2.0 ** -126, -0.5])
def test_append_every_bf16_value(scale):
    """Every bf16 bit pattern, NaN and infinities among them: ties, borders,
    subnormal codes and saturation."""
    bits = np.arange(65536, dtype=np.uint16).reshape(256, 2, 128)
    cache = np.zeros((16, 2, 2, 16, 128), np.uint8)
    s = np.array([scale], np.float32)
    _check_append(bits, bits[::-1].copy(), cache, np.arange(256, dtype=np.int64), s, s)


@pytest.mark.parametrize("scale", [np.nextafter(np.float32(1), np.float32(2)), np.nextafter(np.float32(1), np.float32(0)),
                                   np.nextafter(np.float32(0.75), np.float32(1)), 130 / 448, 250 / 448,
                                   -np.nextafter(np.float32(131 / 21), np.float32(9)), 2.0 ** 99, 2.0 ** -99])
def test_append_scales_beside_ties(scale):
    """Scales a unit away from those that make ties, where x / scale falls within
    2^-24 of a midpoint between two codes."""
    test_append_every_bf16_value(scale)


@pytest.mark.parametrize("scale", [0.0, -0.0, np.inf, -np.inf, np.nan])
def test_append_scales_that_are_no_scales(scale):
    """Division as IEEE has it: by 0 saturated infinities (NaN for 0 / 0), by
    infinity zeros, by NaN NaN."""
    bits = np.array([0, 0x8000, 0x3F80, 0xC000, 0x7F80, 0xFF80, 0x7FC0, 1] * 8, np.uint16).reshape(1, 1, 64)
    with np.errstate(all="ignore"):
        want = oracle.e4m3_nearest(decode_bf16(bits[0, 0]) / np.float64(scale), 1.0)
    s = np.array([scale], np.float32)
    got, _, _ = _append(bits, bits, np.zeros((1, 2, 1, 16, 64), np.uint8), np.zeros(1, np.int64), s, s)
    assert np.array_equal(got[0, 0, 0, 0], want) and np.array_equal(got[0, 1, 0, 0], want)
    _clean()


@pytest.mark.parametrize("lead", [2.0 ** -126, 2.0 ** -81, 2.0 ** -79, 1.0, 2.0 ** 127])
def test_append_per_token_every_largest_significand(lead):
    """Vectors of every significand of the largest element, their elements all
    significands of the 11 binades below it, both signs."""
    sig = np.arange(128, 256) / 128
    top = sig * lead
    x = np.stack([np.concatenate([[t], s * lead * 2.0 ** -k]) for t in top for k in range(12) for s in (sig[:127], -sig[1:])])
    x[np.abs(x) > np.abs(x[:, :1])] = 0
    bits = synth.round_to_bf16_bits(x).reshape(-1, 8, 128)
    T = len(bits)
    cache = np.zeros((T // 16, 2, 8, 16, 128), np.uint8)
    z = np.zeros((T // 16, 8, 16), np.float32)
    _check_append(bits, bits[::-1].copy(), cache, np.arange(T, dtype=np.int64), z, z)


def test_append_per_token_extremes():
    """Zero vectors, subnormal ones, infinities and NaN beside finite values."""
    x = np.zeros((6, 1, 64), np.float32)
    x[1, 0, 3] = 1e-40
    x[2, 0, :5] = [1e-38, -2e-38, 3e-39, 0, 1e-41]
    x[3, 0, :3] = [np.inf, -1.0, 1e38]
    x[4, 0, :3] = [np.nan, 5.0, -0.001]
    x[5, 0, :] = 3e38
    b = synth.round_to_bf16_bits(x)
    cache = np.full((1, 2, 1, 16, 64), 0x55, np.uint8)
    z = np.zeros((1, 1, 16), np.float32)
    _check_append(b, b[::-1].copy(), cache, np.arange(6, dtype=np.int64), z, z)


def test_append_skips_padding_and_refuses_far_slots():
    r = synth.rng(9)
    k = synth.round_to_bf16_bits(r.standard_normal((5, 2, 128)))
    cache = np.full((2, 2, 2, 16, 128), 0x3C, np.uint8)
    one = np.ones(1, np.float32)
    _check_append(k, k, cache, np.full(5, -1, np.int64), one, one)
    _check_append(k, k, cache, np.array([32, 0, 1 << 40, -9, 31], np.int64), one, one, err=3)
    _check_append(k[:0], k[:0], cache, np.zeros(0, np.int64), one, one)


# ------------------------------------------------------------------ chunk attention
class Chunk:
    """A ragged batch: requests of (new, total) tokens, stale slots and unused
    table entries poisoned, queries padded by rows of no request."""

    def __init__(self, seed, reqs, Hk, G, D=128, bs=16, per_token=False, pad=0, q_scale=1.5, softmax_scale=None):
        r = synth.rng(seed)
        self.G, self.scale, self.per_token, self.bs = G, softmax_scale, per_token, bs
        new, tot = [a for a, _ in reqs], [b for _, b in reqs]
        need = [-(-t // bs) for t in tot]
        NB = sum(need) + 2
        self.table = np.full((len(reqs), max([1] + need) + 1), 1 << 30)
        perm, o = r.permutation(NB), 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[o:o + n]
            o += n
        x = r.standard_normal((NB, 2, Hk, bs, D))
        if per_token:
            self.ks, self.vs = (np.exp(r.uniform(np.log(0.002), np.log(0.05), (NB, Hk, bs))).astype(np.float32)
                                for _ in range(2))
            x[:, 0] /= self.ks[..., None]
            x[:, 1] /= self.vs[..., None]
        else:
            self.ks, self.vs = np.array([0.011], np.float32), np.array([0.0173], np.float32)
            x[:, 0] /= self.ks
            x[:, 1] /= self.vs
        self.cache = synth.round_to_e4m3_bytes(x)
        for i, t in enumerate(tot):          # stale slots: NaN codes (and NaN scales)
            if t % bs:
                b = self.table[i, t // bs]
                self.cache[b, :, :, t % bs:] = 0x7F
                if per_token:
                    self.ks[b, :, t % bs:] = self.vs[b, :, t % bs:] = np.nan
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.lens = np.array(tot)
        T = int(self.start[-1]) + pad
        self.q_bits = synth.round_to_bf16_bits(q_scale * r.standard_normal((T, Hk * G, D)))

    def tensors(self):
        return dict(q=bf16_tensor(self.q_bits, dev()), kv_cache=torch.from_numpy(self.cache).to(dev()),
                    block_table=_i32(self.table), query_start=_i32(self.start), seq_lens=_i32(self.lens),
                    k_scale=torch.from_numpy(self.ks).to(dev()), v_scale=torch.from_numpy(self.vs).to(dev()),
                    query_group=self.G, softmax_scale=self.scale)

    def reference(self):
        return oracle.pa_chunk_fp8(self.q_bits, self.cache, self.table, self.start, self.lens, self.ks, self.vs, self.G,
                                   self.scale)

    def tolerance(self, ref, bound):
        D = self.q_bits.shape[2]
        scale = abs(self.scale) if self.scale is not None else D ** -0.5
        kv = decode_e4m3fn(self.cache)
        if self.per_token:
            kv[:, 0] *= self.ks[..., None].astype(np.float64)
            kv[:, 1] *= self.vs[..., None].astype(np.float64)
        else:
            kv[:, 0] *= float(self.ks[0])
            kv[:, 1] *= float(self.vs[0])
        kv = np.nan_to_num(kv)
        k1, vmax = np.abs(kv[:, 0]).sum(axis=-1).max(), np.abs(kv[:, 1]).max()
        qmax = np.abs(decode_bf16(self.q_bits)).max(axis=-1, keepdims=True)
        dq = scale * 2.0 ** -18 * qmax * k1
        da = scale * qmax * k1 * (D + 4) * 2.0 ** -24 + 2.0 ** -22
        pv = 2.0 ** -11 + (2.0 ** -10 if self.per_token else 0.0) + 2.0 ** -18
        return (2.0 ** -8 * np.abs(ref) + pv * bound + 2 * (dq + da) * bound
                + int(self.lens.max(initial=0)) * 2.0 ** -24 * vmax)


def _check_chunk(c, **kw):
    t = {**c.tensors(), **kw}
    out = torch.full(tuple(t["q"].shape), 77.0, dtype=torch.bfloat16, device=dev())
    got = qpa.pa_chunk_fp8(out=out, **t)
    _clean()
    _compare(c, got)
    return t, out


def _compare(c, got, ref=None):
    got = got.double().cpu().numpy()
    ref, bound = c.reference() if ref is None else ref
    nobody = np.isnan(bound).all(axis=(1, 2))
    assert np.all(got[nobody] == 77.0), "rows of no request were written"
    live = ~nobody
    tol = c.tolerance(ref, bound)
    nan = np.isnan(ref[live])
    assert np.array_equal(np.isnan(got[live]), nan), "NaN pattern differs"
    err, lim = np.abs(got[live] - ref[live])[~nan], tol[live][~nan]
    assert np.all(err <= lim), f"worst {np.max(err / lim):.3g} of the tolerance"


CASES = [
    # requests (new, total), Hk, G, D, bs, per_token, pad
    ([(1, 1)], 1, 1, 128, 16, False, 0),
    ([(1, 127), (1, 128), (1, 129), (1, 1000)], 2, 8, 128, 16, False, 3),
    ([(5, 5), (0, 40), (3, 200), (17, 17)], 2, 4, 128, 16, False, 1),
    ([(130, 130)], 1, 2, 128, 32, False, 0),
    ([(128, 128), (129, 257)], 1, 1, 128, 64, False, 5),
    ([(300, 700)], 2, 1, 64, 128, False, 0),
    ([(64, 1024), (31, 513)], 2, 8, 128, 128, False, 0),
    ([(90, 400), (1, 2500), (2, 3)], 3, 3, 128, 256, False, 2),
    ([(33, 100), (7, 300)], 2, 5, 64, 16, False, 0),
    ([(6, 600)], 1, 64, 128, 16, False, 0),
    ([(9, 9), (40, 333)], 1, 7, 64, 32, False, 1),
    ([(1, 1), (12, 300)], 2, 8, 128, 16, True, 0),
    ([(260, 261)], 1, 1, 64, 64, True, 2),
    ([(70, 900), (1, 2000), (0, 0)], 2, 4, 128, 256, True, 0),
    ([(50, 50), (3, 1100)], 3, 5, 64, 16, True, 4),
    ([(30, 200), (15, 15)], 1, 33, 64, 128, False, 0),
    ([(1, 20000)], 1, 4, 128, 64, False, 0),               # one item over many CTAs
    ([(1, 9000), (40, 12000)], 1, 4, 64, 16, True, 0),
]


@pytest.mark.parametrize("reqs,Hk,G,D,bs,per_token,pad", CASES)
def test_chunk_parity(reqs, Hk, G, D, bs, per_token, pad):
    _check_chunk(Chunk(len(reqs) + 10 * G + D, reqs, Hk, G, D, bs, per_token, pad))


def test_chunk_many_short_requests():
    r = synth.rng(77)
    reqs = [(int(n), int(n + c)) for n, c in zip(r.integers(0, 4, 700), r.integers(0, 40, 700))]
    _check_chunk(Chunk(78, reqs, 1, 2, 64, 16))


def test_chunk_longer_prompt():
    _check_chunk(Chunk(79, [(1100, 1500)], 1, 2, 128, 16))


def test_chunk_rows_without_a_token_give_zero():
    """More query rows than cached tokens: the first rows see none."""
    for per_token in (False, True):
        c = Chunk(5, [(40, 40), (300, 20), (7, 0), (4, 9)], 2, 3, 64, 16, per_token)
        t, out = _check_chunk(c)
        assert bool((out[40:40 + 280] == 0).all()) and bool((out[340:347] == 0).all())


@pytest.mark.parametrize("scale", [-0.3, 1e-30, 3.0, 0.02])
def test_chunk_softmax_scales(scale):
    """Negative, vanishing and steep scales."""
    _check_chunk(Chunk(6, [(20, 150), (3, 300)], 1, 4, 128, 16, softmax_scale=scale))


def test_chunk_zero_and_negative_k_scale():
    for s in (0.0, -0.011):
        c = Chunk(8, [(20, 150)], 1, 4, 128, 16)
        c.ks[:] = s
        _check_chunk(c)
    c = Chunk(9, [(20, 150)], 1, 4, 128, 16, per_token=True)
    r = synth.rng(10)
    c.ks *= np.where(r.random(c.ks.shape) < 0.5, -1, 1).astype(np.float32)
    c.vs *= np.where(r.random(c.vs.shape) < 0.5, -1, 1).astype(np.float32)
    live = ~np.isnan(c.vs)
    c.vs[live & (r.random(c.vs.shape) < 0.2)] = 0
    _check_chunk(c)


def test_chunk_growing_logits():
    """Keys that grow along the sequence: the running maximum moves in every
    tile, by little and by much."""
    for step in (0.002, 0.2):
        c = Chunk(11, [(30, 900)], 1, 4, 128, 16)
        pos = np.arange(900)
        blk, off = c.table[0, pos // 16], pos % 16
        base = decode_bf16(c.q_bits)[0, 0]
        x = base[None] * (step * pos)[:, None] / np.abs(base).max()
        c.cache[blk, 0, 0, off] = synth.round_to_e4m3_bytes(x)
        _check_chunk(c)


def test_chunk_v_scales_growing_and_falling():
    c = Chunk(12, [(30, 900), (30, 900)], 1, 4, 128, 16, per_token=True)
    pos = np.arange(900)
    for r, f in ((0, 1.02), (1, 1 / 1.02)):
        blk, off = c.table[r, pos // 16], pos % 16
        c.vs[blk, 0, off] = (1e-3 * f ** pos).astype(np.float32)
    _check_chunk(c)


def test_chunk_extreme_queries():
    """Row magnitudes near both ends of bf16, a zero row, an element far below
    its row's largest; a row with an infinity or NaN is NaN and no other is."""
    c = Chunk(13, [(8, 200)], 1, 4, 128, 16)
    q = decode_bf16(c.q_bits)
    q[0] *= 2.0 ** -120
    q[1] = 0
    q[2, :, 0] = 300.0
    q[2, :, 1:] *= 1e-4
    q[5, 1, 7], q[6, 2, 9], q[6, 3, 100] = np.nan, np.inf, -np.inf
    c.q_bits = synth.round_to_bf16_bits(q)
    ref, bound = c.reference()
    for row, head in ((5, 1), (6, 2), (6, 3)):
        ref[row, head] = bound[row, head] = np.nan
    out = torch.full(tuple(c.q_bits.shape), 77.0, dtype=torch.bfloat16, device=dev())
    qpa.pa_chunk_fp8(out=out, **c.tensors())
    _clean()
    with np.errstate(invalid="ignore"):
        # (the tolerance of the other rows must not pick up the NaN)
        _compare(c, out, (ref, bound))


def test_chunk_nan_in_tokens_that_a_row_does_not_see():
    """A NaN code in K or V of a new token reaches the rows that see the token
    (for V only that dim), and no earlier row."""
    for per_token in (False, True):
        c = Chunk(14, [(60, 300), (40, 40)], 2, 4, 128, 16, per_token)
        for req, tok, kv, h, d in ((0, 270, 1, 0, 5), (0, 290, 0, 1, 6), (1, 17, 1, 1, 127), (1, 30, 0, 0, 0),
                                   (0, 100, 1, 1, 64)):
            c.cache[c.table[req, tok // 16], kv, h, tok % 16, d] = 0x7F if d % 2 else 0xFF
        _check_chunk(c)


def test_chunk_strided_inputs():
    c = Chunk(15, [(20, 90), (33, 33)], 2, 3, 64, 16, pad=2)
    t = c.tensors()
    T = t["q"].shape[0]
    wide = torch.zeros(T, 11, 64, dtype=torch.bfloat16, device=dev())
    wide[:, 2:8] = t["q"]
    tab = torch.full((2, t["block_table"].shape[1] + 5), -1, dtype=torch.int32, device=dev())
    tab[:, :-5] = t["block_table"]
    _check_chunk(c, q=wide[:, 2:8], block_table=tab[:, :-5])


def test_chunk_invalid_block_reads_block_0():
    c = Chunk(16, [(4, 40)], 1, 2, 128, 16)
    want = c.table.copy()
    c.table[0, 1] = 9999
    t = c.tensors()
    out = torch.full(tuple(t["q"].shape), 77.0, dtype=torch.bfloat16, device=dev())
    qpa.pa_chunk_fp8(out=out, **t)
    torch.cuda.synchronize()
    assert qpa.kernel_error() == 3
    want[0, 1] = 0
    c.table = want
    _compare(c, out)


def test_chunk_single_tokens_agree_with_the_decode():
    c = Chunk(17, [(1, 500), (1, 33), (1, 1)], 2, 8, 128, 16)
    t = c.tensors()
    a = qpa.pa_chunk_fp8(**t).double()
    b = qpa.pa_decode_fp8(t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["k_scale"], t["v_scale"], 4, 8)
    _clean()
    ref, bound = c.reference()
    assert np.all(np.abs((a - b.double()).cpu().numpy()) <= 2 * c.tolerance(ref, bound))


def test_chunk_two_streams_at_once_and_graph_replay():
    """Overlapping calls with a workspace each, then a captured call replayed
    on new queries, against the eager results (equal: the split is fixed)."""
    c1, c2 = Chunk(18, [(200, 900)], 2, 4, 128, 16), Chunk(19, [(150, 700), (1, 50)], 2, 4, 64, 32, True)
    t1, t2 = c1.tensors(), c2.tensors()
    e1, e2 = qpa.pa_chunk_fp8(**t1), qpa.pa_chunk_fp8(**t2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.empty_like(e1), torch.empty_like(e2)
    w1 = qpa.alloc_workspace(qpa.pa_chunk_fp8_workspace_size(qpa.chunk_desc(t1["q"], t1["kv_cache"], t1["block_table"], 4, False)), dev())
    w2 = qpa.alloc_workspace(qpa.pa_chunk_fp8_workspace_size(qpa.chunk_desc(t2["q"], t2["kv_cache"], t2["block_table"], 4, True)), dev())
    torch.cuda.synchronize()
    for _ in range(5):
        qpa.pa_chunk_fp8(out=o1, workspace=w1, stream=s1, **t1)
        qpa.pa_chunk_fp8(out=o2, workspace=w2, stream=s2, **t2)
    torch.cuda.synchronize()
    assert torch.equal(o1, e1) and torch.equal(o2, e2)

    g = torch.cuda.CUDAGraph()
    o3 = torch.empty_like(e1)
    with torch.cuda.graph(g):
        qpa.pa_chunk_fp8(out=o3, workspace=w1, **t1)
    t1["q"].mul_(0.5)
    g.replay()
    want = qpa.pa_chunk_fp8(**t1)
    _clean()
    assert torch.equal(o3, want)


def test_memory_of_a_call_on_another_stream():
    """Outputs and workspace that the binding allocates belong to the stream of
    the call: a block that the current stream has freed, with a write to it still
    queued there, is not handed out."""
    c = Chunk(9, [(200, 900), (1, 5000)], 2, 8)
    t = c.tensors()
    want = qpa.pa_chunk_fp8(**t).clone()
    new, free, table = _i32([3, 2]), _i32(range(8)), _i32(np.zeros((2, 4)))
    side = torch.cuda.Stream()
    n = qpa.pa_chunk_fp8_workspace_size(qpa.chunk_desc(t["q"], t["kv_cache"], t["block_table"], c.G, False))
    freed = [torch.empty(k, dtype=torch.uint8, device=dev()) for k in (n, want.nbytes, 12, 8, 40, 20, 4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                      # some tens of ms before the writes
    for x in freed:
        x.fill_(255)
    del freed, x
    got = qpa.pa_chunk_fp8(**t, stream=side)
    got2 = qpa.paged_slot_map(new, new, table, free, 16, 5, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert got2[0].tolist() == [0, 3, 5] and got2[1].tolist() == [6, 4] and got2[3].tolist() == [3, 4, 5, 2, 3]
    _clean()


def test_pages_past_4_gib():
    """Blocks at the end of a cache of more than 2^32 bytes: append there, then
    attend over them, beside blocks at its start."""
    Hk, bs, D = 8, 16, 128
    NB = (1 << 32) // (2 * Hk * bs * D) + 5000
    r = synth.rng(31)
    blocks = np.array([NB - 1, 3, NB - 77, NB // 2 + 9, 0, NB - 4999])
    T = 90
    k, v, q = (synth.round_to_bf16_bits(r.standard_normal((T, h, D))) for h in (Hk, Hk, Hk))
    pos = np.arange(T)
    slots = (blocks[pos // bs] * bs + pos % bs).astype(np.int64)
    for per_token in (False, True):
        cache = torch.empty(NB, 2, Hk, bs, D, dtype=torch.uint8, device=dev())
        n = (NB, Hk, bs) if per_token else (1,)
        ks, vs = torch.full(n, 0.01, device=dev()), torch.full(n, 0.02, device=dev())
        qpa.kv_append_fp8(bf16_tensor(k, dev()), bf16_tensor(v, dev()), cache, torch.from_numpy(slots).to(dev()), ks, vs)
        out = qpa.pa_chunk_fp8(bf16_tensor(q, dev()), cache, _i32(blocks[None]), _i32([0, T]), _i32([T]), ks, vs, 1)
        _clean()
        # the oracle on the six blocks, numbered 0..5
        small = np.zeros((6, 2, Hk, bs, D), np.uint8)
        sk, sv = (np.full((6, Hk, bs) if per_token else (1,), x, np.float32) for x in (0.01, 0.02))
        small, sk, sv = oracle.kv_append_fp8(k, v, small, pos, sk, sv)
        idx = torch.from_numpy(blocks).to(dev())
        live = np.ones((6, 2, Hk, bs, D), bool)
        live[5, :, :, T - 80:] = False                  # slots that nothing wrote
        assert np.array_equal(cache[idx].cpu().numpy()[live], small[live])
        c = Chunk.__new__(Chunk)
        c.G, c.scale, c.per_token, c.bs = 1, None, per_token, bs
        c.q_bits, c.cache, c.table, c.start, c.lens, c.ks, c.vs = q, small, np.arange(6)[None], [0, T], np.array([T]), sk, sv
        _compare(c, out)
        del cache


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,per_token", [(128, False), (64, True)])
def test_steps_of_a_server(D, per_token):
    """Three steps of a small server in one captured graph per shape: slots from
    lengths, append, chunk attention (prompts, then single tokens beside a
    chunk), and the multi-token decode on the same pages; each checked against
    the oracle run on the oracle's own pages."""
    Hk, G, bs, NB, maxb = 2, 4, 16, 64, 12
    r = synth.rng(20)
    steps = [np.array([37, 5, 0]), np.array([1, 90, 16]), np.array([1, 1, 1])]
    free = r.permutation(NB)
    table, lens = np.full((3, maxb), -1), np.zeros(3, int)
    cache = np.zeros((NB, 2, Hk, bs, D), np.uint8)
    ks, vs = ((np.zeros((NB, Hk, bs), np.float32),) * 2 if per_token else
              (np.array([0.01], np.float32), np.array([0.02], np.float32)))
    t_table, t_lens = _i32(table), _i32(lens)
    t_cache = torch.from_numpy(cache).to(dev())
    t_ks, t_vs = torch.from_numpy(ks.copy()).to(dev()), torch.from_numpy(vs.copy()).to(dev())
    for new in steps:
        T = int(new.sum()) + 3
        q, k, v = (synth.round_to_bf16_bits(r.standard_normal((T, h, D))) for h in (Hk * G, Hk, Hk))
        # the library, through a captured graph
        t_new, t_free = _i32(new), _i32(free)
        tq, tk, tv = (bf16_tensor(x, dev()) for x in (q, k, v))
        out = torch.full((T, Hk * G, D), 77.0, dtype=torch.bfloat16, device=dev())
        ws = qpa.alloc_workspace(qpa.pa_chunk_fp8_workspace_size(qpa.chunk_desc(tq, t_cache, t_table, G, per_token)), dev())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            start, tot, slots, pos, taken = qpa.paged_slot_map(t_new, t_lens, t_table, t_free, bs, T)
            qpa.kv_append_fp8(tk, tv, t_cache, slots, t_ks, t_vs)
            qpa.pa_chunk_fp8(tq, t_cache, t_table, start, tot, t_ks, t_vs, G, out=out, workspace=ws)
        g.replay()
        _clean()
        # the oracle
        o_start, o_lens, table, o_slots, _, o_taken, short = oracle.paged_slot_map(new, lens, table, free, bs, T)
        assert not short and int(taken) == o_taken
        cache, ks, vs = oracle.kv_append_fp8(k, v, cache, o_slots, ks, vs)
        assert np.array_equal(t_cache.cpu().numpy(), cache) and np.array_equal(t_ks.cpu().numpy(), ks)
        c = Chunk.__new__(Chunk)
        c.G, c.scale, c.per_token, c.bs = G, None, per_token, bs
        c.q_bits, c.cache, c.table, c.start, c.lens, c.ks, c.vs = q, cache, table, o_start, o_lens, ks, vs
        _compare(c, out)
        free, lens = free[o_taken:], o_lens
        t_lens = tot.clone()
    # the last step brought one token to each: the decode reads the same pages
    dec = qpa.pa_decode_fp8_ext(tq[:3].view(3, 1, Hk * G, D), t_cache, t_table, t_lens, t_ks, t_vs, 4, G)
    _clean()
    ref, bound = c.reference()
    err = np.abs(dec.double().cpu().numpy().reshape(3, Hk * G, D) - ref[:3])
    assert np.all(err <= c.tolerance(ref, bound)[:3] + 2.0 ** -8 * bound[:3])
