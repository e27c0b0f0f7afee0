"""GPU tests of the entry points called from host threads: as a thread's first CUDA
call, and from several threads at once, a stream, a workspace and sizes of its own
in each.

The C entries are called, and in tight loops: the binding's own CUDA calls would
come first, and its host time keep the calls apart."""
import ctypes
import threading

import pytest
import torch

import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import UqDev, dev
from test_gpu_step import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _together(calls, times):
    """Each call (a function of a stream handle) `times` times in a thread of its own;
    the statuses other than 0."""
    bad = []

    def work(call, stream):
        bad.extend(st for st in (call(ctypes.c_void_p(stream.cuda_stream)) for _ in range(times)) if st)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert qpa.kernel_error() == 0
    return bad


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _uq_call(c, out, d, ws):
    return lambda s: qpa.load_library().uq_decode_hd256(_p(c.q), _p(c.kv), _p(c.cent), _p(c.bt), _p(c.sl), 1, _p(out),
                                                        ctypes.byref(d), _p(ws), ws.nbytes, s)


def test_first_cuda_call_of_a_thread():
    """A call that encodes a tensor map needs a context that is current in its thread;
    torch has made none there yet."""
    c = UqDev(synth.make_uq_case(4, [40]))
    want, ws, d = c.run(1)
    out = torch.zeros_like(want)
    assert not _together([_uq_call(c, out, d, ws)], 1)
    assert torch.equal(out, want)

    t = Chunk(5, [(20, 90)], 2, 4).tensors()
    want = qpa.pa_chunk_fp8(**t)
    out = torch.zeros_like(want)
    cd = qpa.chunk_desc(t["q"], t["kv_cache"], t["block_table"], 4, False)
    ws = qpa.alloc_workspace(qpa.pa_chunk_fp8_workspace_size(cd), dev())
    names = ("q", "kv_cache", "block_table", "query_start", "seq_lens", "k_scale", "v_scale")
    assert not _together([lambda s: qpa.load_library().pa_chunk_fp8(*[_p(t[n]) for n in names], _p(out), ctypes.byref(cd),
                                                                    _p(ws), ws.nbytes, s)], 1)
    assert torch.equal(out, want)


@pytest.mark.parametrize("fp8", [True, False])
def test_combines_of_different_partition_counts(fp8):
    """Empty slots of 6000 to 20000 partitions, or of an eighth of that with 8 slots
    each (48 to 160 KB of weights in shared memory), give 0."""
    lib, calls, outs = qpa.load_library(), [], []
    for P in (20000, 6000, 11000) if fp8 else (2500, 750, 1400):
        D = 128 if fp8 else 256
        q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=dev())
        table = torch.zeros(1, 1, dtype=torch.int32, device=dev())
        if fp8:
            d = qpa.fp8_desc(q, torch.zeros(1, 2, 1, 16, D, dtype=torch.uint8, device=dev()), table, 1, None, torch.float32)
            ws = torch.zeros(qpa.pa_decode_fp8_workspace_size(d, P), dtype=torch.uint8, device=dev())
            fn = lib.pa_decode_fp8_combine
        else:
            d = UqDev(synth.make_uq_case(3, [5], num_kv_heads=1, query_group=1)).desc()
            ws = torch.zeros(qpa.uq_decode_hd256_workspace_size(d, P), dtype=torch.uint8, device=dev())
            fn = lib.uq_decode_hd256_combine
        out = torch.full((1, 1, D), 9.0, device=dev())
        outs.append(out)
        calls.append(lambda s, fn=fn, P=P, out=out, d=d, ws=ws: fn(P, _p(out), ctypes.byref(d), _p(ws), ws.nbytes, s))
    bad = _together(calls, 5000)
    assert not bad, f"{len(bad)} calls failed with {set(bad)}"
    assert all(bool((o == 0).all()) for o in outs)


def test_hd256_decodes_of_different_head_counts():
    """1, 2 and 4 KV heads take rings of different sizes."""
    calls, outs = [], []
    for Hk in (1, 2, 4):
        c = UqDev(synth.make_uq_case(4, [40], num_kv_heads=Hk, query_group=8))
        want, ws, d = c.run(1)
        out = torch.zeros_like(want)
        outs.append((out, want, c))
        calls.append(_uq_call(c, out, d, ws))
    bad = _together(calls, 5000)
    assert not bad, f"{len(bad)} calls failed with {set(bad)}"
    assert all(torch.equal(o, w) for o, w, _ in outs)
