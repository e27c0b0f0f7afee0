"""The 4-bit cache's calls at their limits: sequences up to the last 32-bit length,
thousands of sequences, calls of different shapes from several host threads, and as
a thread's first CUDA call."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import Case, done, f32, rand_cache, rand_table, same_bf16, t32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(128, 4), (64, 12)])
def test_one_sequence_of_2_to_the_31_tokens(D, G):
    """The longest length a table can hold; its entries name three blocks, so the
    attention is that over their tokens, each weighed by how often it comes.

    Tolerance: 2^-8 of the result, and for weights as in the other tests. A float32 sum
    of n terms in order is off by at most n 2^-23 of the sum of their magnitudes (each
    addition rounds or cuts off one unit); a warp adds 2 sums of 16 tokens per tile, every
    third (every second, with more than 8 rows) of its range's 2^24 / 152 tiles."""
    r = synth.rng(D)
    bs, NB = 256, 3
    maxb = (2 ** 31 - 1) // bs
    table = r.integers(0, NB, (1, maxb), dtype=np.int32)
    L = maxb * bs - 5
    cache = rand_cache(r, NB, 1, bs, D, smax=48)
    q = synth.round_to_bf16_bits(0.3 * r.standard_normal((1, G, D)))
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), torch.from_numpy(table).to(dev()),
                              t32([L]), f32(.2), f32(.2), G)
    done()
    count = np.zeros((NB, bs))
    count += np.bincount(table[0], minlength=NB)[:, None]
    count[table[0, -1], -5:] -= 1
    blk, off = np.repeat(np.arange(NB), bs), np.tile(np.arange(bs), NB)
    K, V = (oracle.values_nvfp4(cache, i, .2, blk, off)[:, 0] for i in range(2))
    x = oracle.decode_bf16(q)[0] @ K.T / np.sqrt(D)
    w = np.exp(x - x.max(axis=1, keepdims=True)) * count.reshape(-1)
    w /= w.sum(axis=1, keepdims=True)
    want, bound = w @ V, w @ np.abs(V)
    adds = 2 * 2 ** 24 / 152 / (3 if G <= 8 else 2)
    qq = np.abs(oracle.decode_bf16(q)[0])
    slack = (qq.max(axis=1) * 2.0 ** -16 * np.abs(K).sum(axis=1).max()) / np.sqrt(D) + 2.0 ** -21 * np.abs(x).max(axis=1)
    tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(slack)[:, None] + 2 * adds * 2.0 ** -23)
    err = np.abs(out[0].float().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()


def test_last_tokens_of_a_long_sequence_read_back():
    r = synth.rng(3)
    bs = 256
    maxb = (2 ** 31 - 1) // bs
    table = torch.full((1, maxb), -1, dtype=torch.int32, device=dev())
    table[0, -2:] = t32([2, 0])
    L = maxb * bs - 7
    cache = rand_cache(r, 3, 2, bs, 64)
    k, v = qpa.kv_gather_nvfp4(torch.from_numpy(cache).to(dev()), table, t32([0, 300]), t32([L]), f32(1.0), f32(1.0), 300)
    done()
    off = np.arange(L - 300, L)
    blk = np.where(off // bs == maxb - 1, 0, 2)
    same_bf16(k, oracle.values_nvfp4(cache, 0, 1.0, blk, off % bs))
    same_bf16(v, oracle.values_nvfp4(cache, 1, 1.0, blk, off % bs))


def test_thousands_of_sequences():
    r = synth.rng(4)
    lens = r.integers(0, 40, 3001)
    c = Case.__new__(Case)
    c.table, NB = rand_table(r, lens, 16)
    c.cache, c.lens, c.G, c.gs = rand_cache(r, NB, 1, 16, 64, smax=60), lens, 2, (.1, .1)
    c.q = synth.round_to_bf16_bits(r.standard_normal((3001, 2, 64)))
    out = c.run()
    start = np.concatenate([[0], np.cumsum(lens)])
    k, v = qpa.kv_gather_nvfp4(torch.from_numpy(c.cache).to(dev()), t32(c.table), t32(start), t32(lens), f32(.1), f32(.1),
                               int(start[-1]))
    done()
    rows, blk, off, _ = oracle.gather_rows(c.table, start, lens, 16)
    same_bf16(k, oracle.values_nvfp4(c.cache, 0, .1, blk, off))
    same_bf16(v, oracle.values_nvfp4(c.cache, 1, .1, blk, off))
    c.check(out)


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _call(c):
    """(a function of a stream handle that decodes case c through the C ABI, its output, what it has to be)"""
    q, cache, table, lens = bf16_tensor(c.q, dev()), torch.from_numpy(c.cache).to(dev()), t32(c.table), t32(c.lens)
    ks, vs = f32(c.gs[0]), f32(c.gs[1])
    want = c.run()
    out = torch.zeros_like(want)
    d = qpa.nvfp4_desc(q, cache, table, c.G)
    ws = qpa.alloc_workspace(qpa.pa_decode_nvfp4_workspace_size(d), dev())
    keep = (q, cache, table, lens, ks, vs, d, ws)
    return lambda s, k=keep: qpa.load_library().pa_decode_nvfp4(*[_p(t) for t in k[:6]], _p(out), ctypes.byref(k[6]), _p(k[7]),
                                                                k[7].nbytes, s), out, want


def _together(calls, times):
    bad = []

    def work(call, stream):
        bad.extend(st for st in (call(ctypes.c_void_p(stream.cuda_stream)) for _ in range(times)) if st)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done()
    return bad


def test_first_cuda_call_of_a_thread():
    call, out, want = _call(Case([300, 7], 2, 4, 128, 16))
    assert not _together([call], 1)
    assert torch.equal(out, want)


def test_decodes_of_different_shapes_from_several_threads():
    """The kernel's four forms, a stream and a workspace each."""
    calls = [_call(Case([700, 40], 2, G, D, 16)) for D, G in ((128, 4), (128, 16), (64, 4), (64, 40))]
    assert not _together([c for c, _, _ in calls], 300)
    assert all(torch.equal(o, w) for _, o, w in calls)


def test_graph_replays_see_new_inputs_and_lengths():
    """One captured decode: other queries, lengths and blocks each time, a length of 0 among them."""
    c = Case([500, 1, 260], 2, 8, 128, 16)
    q, table, lens = bf16_tensor(c.q, dev()), t32(c.table), t32(c.lens)
    cache, ks, vs = torch.from_numpy(c.cache).to(dev()), f32(c.gs[0]), f32(c.gs[1])
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = qpa.pa_decode_nvfp4(q, cache, table, lens, ks, vs, 8)
    r = synth.rng(9)
    for new in ([500, 1, 260], [0, 1, 129], [13, 0, 0], [400, 1, 260]):
        c.lens = np.array(new)
        c.q = synth.round_to_bf16_bits(r.standard_normal(c.q.shape))
        q.copy_(bf16_tensor(c.q, dev()))
        lens.copy_(t32(new))
        g.replay()
        done()
        c.check(out)


def test_outputs_and_rows_of_no_request_stay():
    """Rows of the outputs behind the last request, and an out tensor of the caller's."""
    c = Case([40, 3], 1, 4, 64, 16)
    big = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device=dev())
    got = c.run(out=big[1:3])
    done()
    c.check(got)
    assert got.data_ptr() == big[1:3].data_ptr() and bool((big[0] == 3).all()) and bool((big[3:] == 3).all())


def test_last_tile_below_2_to_the_31():
    """Tokens up to 2^31 - 17 in blocks of 16: the last tile's end lies past 32 bits. All but the last 130 tokens
    have keys of 0 and values of NaN-free block 1; behind the last token are NaN scales."""
    r = synth.rng(77)
    bs, D = 16, 64
    maxb = (2 ** 31 - 1) // bs
    L = maxb * bs - 1
    table = torch.ones(1, maxb, dtype=torch.int32, device=dev())
    table[0, -9:] = t32(np.arange(2, 11))
    cache = rand_cache(r, 11, 1, bs, D, smax=48)
    codes, scales = oracle.nvfp4._split(cache)
    scales[0], scales[10, :, :, -1] = 0x7F, 0x7F
    codes[1, 0] = 0
    codes[2:11, 0] &= 0x77                                                  # positive keys, scales up to 0.9375
    cache = oracle.nvfp4._join(codes, scales)
    # logits (base e) of the last tokens about 100 above the others': 2^31 e^-50 is nothing
    q = synth.round_to_bf16_bits(np.full((1, 1, D), 16.0))
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), table, t32([L]), f32(1.0), f32(1.0), 1)
    done()
    blk, off = np.repeat(np.arange(2, 11), bs)[:-1], np.tile(np.arange(bs), 9)[:-1]
    K, V = (oracle.values_nvfp4(cache, i, 1.0, blk, off)[:, 0] for i in range(2))
    x = 16.0 * K.sum(axis=1) / 8
    assert x.max() > 60
    w = np.exp(x - x.max())
    w /= w.sum()
    want, bound = w @ V, w @ np.abs(V)
    # 2^-8 of the result; weights as in the other tests (the query is exact); the 2^31 others: below 2^31 e^-60
    tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(2.0 ** -21 * x.max()) + 2.0 ** -18)
    tol = tol + 2.0 ** 31 * np.exp(-60.0) * (np.abs(V).max() + 6 * 0.9375) + 2.0 ** -33 * (np.abs(V).sum(axis=0) + 144 * np.abs(want))
    err = np.abs(out[0, 0].float().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("amp", [-1e20, -1e33, -1e36])
def test_logits_far_below_zero(amp):
    """Equal keys, logits of down to -10^36: the result is the mean of the values (2^-8 of it, and the weights are
    exact: 2^-18 sum |v| for the sums)."""
    r = synth.rng(78)
    lens = [300, 1000]
    table, NB = rand_table(r, lens, 16)
    cache = rand_cache(r, NB, 1, 16, 64, smax=60)
    codes, scales = oracle.nvfp4._split(cache)
    codes[:, 0], scales[:, 0] = 0x22, 0x38                                  # 1 x 1
    cache = oracle.nvfp4._join(codes, scales)
    q = synth.round_to_bf16_bits(np.full((2, 3, 64), amp))
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), t32(table), t32(lens), f32(1.0), f32(.3), 3)
    done()
    for s, L in enumerate(lens):
        V = oracle.values_nvfp4(cache, 1, .3, table[s, np.arange(L) // 16], np.arange(L) % 16)[:, 0]
        want = V.mean(axis=0)
        err = np.abs(out[s].float().cpu().numpy() - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(V).mean(axis=0))


@pytest.mark.parametrize("fp4", [True, False])
def test_every_value_read_back_with_many_scales(fp4):
    """All codes with all group scales (fp8: all codes), scales of few bits (many midpoints) and of many: rounded once."""
    r = synth.rng(79)
    gs = [(1 + i / 128) * 2.0 ** r.integers(-60, 60) for i in range(128)] + list(np.exp(r.uniform(-60, 60, 60)))
    gs += [np.nextafter(np.float32(m / x), np.float32(d)) for x in (3, 5, 7, 9, 11, 13, 15, 21, 27, 33, 39, 45)
           for m in (257, 259, 301, 511) for d in (0, 1e9)] + [-0.3, 0.0]
    gs = np.array(gs, dtype=np.float32)
    D, bs = 64, 256
    if fp4:
        code = np.tile((np.arange(16) + 16 * ((np.arange(16) + 1) % 16)).astype(np.uint8)[::2], (bs, 4))
        sc = (np.arange(bs * 4) % 128).astype(np.uint8)
        cache = np.concatenate([code.reshape(-1), sc])[None, None, None].reshape(1, 1, 1, bs, 36)
    else:
        cache = np.resize(np.arange(256, dtype=np.uint8), (1, 2, 1, bs, D))
    dc = torch.from_numpy(cache).to(dev())
    for g in gs:
        if fp4:
            k, _ = qpa.kv_gather_nvfp4(dc, t32([[0]]), t32([0, bs]), t32([bs]), f32(float(g)), None, bs)
            want = oracle.values_nvfp4(cache, 0, g, np.zeros(bs, dtype=int), np.arange(bs))
        else:
            k, _ = qpa.kv_gather_fp8(dc, t32([[0]]), t32([0, bs]), t32([bs]), f32(float(g)), f32(1.0), bs)
            want = oracle.decode_e4m3fn(cache[0, 0, 0])[:, None] * float(g)
        with np.errstate(invalid="ignore"):
            same_bf16(k, want)
    done()


@pytest.mark.parametrize("D,G,bs,cols", [(128, 8, 16, 32), (64, 24, 256, 2), (128, 16, 64, 8)])
def test_tables_of_512_tokens_leave_the_workspace_alone(D, G, bs, cols):
    c = Case([bs * cols, 1, 130, 0], 2, G, D, bs)
    table = t32(c.table[:, :cols])
    d = qpa.nvfp4_desc(bf16_tensor(c.q, dev()), torch.from_numpy(c.cache).to(dev()), table, G)
    ws = torch.full((qpa.pa_decode_nvfp4_workspace_size(d),), 0x5A, dtype=torch.uint8, device=dev())
    outs = [c.run(table=table, workspace=ws), c.run(table=table), c.run(table=table)]
    done()
    assert bool((ws == 0x5A).all()) and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    c.check(outs[0])
