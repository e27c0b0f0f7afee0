"""Refusals of the 4-bit cache's entry points and of reading back, without a GPU: by
the C ABI and by the binding."""
import ctypes

import pytest
import torch

import quantized_paged_attention_gb300 as qpa_pkg

NULL = ctypes.c_void_p(0)


def at(i, off=0):
    """Distinct addresses 16 MiB apart, never dereferenced: every call below is
    refused (or has nothing to do)."""
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


@pytest.fixture(scope="module")
def qpa():
    import __graft_entry__
    __graft_entry__.build()
    qpa_pkg.load_library()
    return qpa_pkg


def _set(d, kw, **base):
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def _call(fn, n, ptrs, desc, *rest):
    p = {i: at(i) for i in range(n)}
    p.update(ptrs or {})
    return fn(*[p[i] for i in range(n)], ctypes.byref(desc) if desc is not None else None, *rest)


# ------------------------------------------------------------------ append
def _append(qpa, ptrs=None, **kw):
    d = _set(qpa.Append4Desc(), kw, num_tokens=3, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=4, planes=2)
    return _call(qpa.load_library().kv_append_nvfp4, 6, ptrs, d, None)


def test_append_refusals(qpa):
    for kw in (dict(num_tokens=-1), dict(num_kv_heads=0), dict(num_kv_heads=65537), dict(head_dim=96),
               dict(head_dim=256), dict(block_size=48), dict(num_blocks=0), dict(planes=0), dict(planes=3)):
        assert _append(qpa, **kw) == -2, kw
    for i in range(6):
        assert _append(qpa, {i: NULL}) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 4), (4, 2), (5, 2)):
        assert _append(qpa, {i: at(i, off)}) == -3, i
    for s in ("k_stride_tok", "k_stride_head", "v_stride_tok", "v_stride_head"):
        assert _append(qpa, **{s: 100}) == -3 and _append(qpa, **{s: -8}) == -3
    assert _append(qpa, {i: NULL for i in range(6)}, num_tokens=0) == 0
    assert qpa.load_library().kv_append_nvfp4(*[at(i) for i in range(6)], None, None) == -1


def test_append_overlaps(qpa):
    row, cache = 2 * 128 * 2, 4 * 2 * 2 * 16 * 72
    assert _append(qpa, {0: at(2, cache - 16)}) == -7
    assert _append(qpa, {1: at(2, -3 * row + 16)}) == -7
    assert _append(qpa, {3: at(2, 64)}) == -7
    assert _append(qpa, {4: at(2, cache - 4)}) == -7 and _append(qpa, {5: at(2)}) == -7
    assert _append(qpa, {0: at(2, cache // 2 - 16)}, planes=1) == -7     # one plane: half the bytes


# ------------------------------------------------------------------ reading back
def _gather(qpa, name="kv_gather_nvfp4", ptrs=None, **kw):
    d = _set(qpa.GatherDesc(), kw, num_reqs=2, num_tokens=5, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=4,
             max_blocks_per_seq=4, planes=2)
    return _call(getattr(qpa.load_library(), name), 8, ptrs, d, None)


@pytest.mark.parametrize("name", ["kv_gather_nvfp4", "kv_gather_fp8"])
def test_gather_refusals(qpa, name):
    for kw in (dict(num_reqs=-1), dict(num_tokens=-1), dict(num_kv_heads=0), dict(num_kv_heads=65537), dict(head_dim=32),
               dict(block_size=8), dict(num_blocks=0), dict(max_blocks_per_seq=0), dict(planes=3), dict(out_dtype=2),
               dict(kv_scale_per_token=2), dict(table_stride=3), dict(max_blocks_per_seq=1 << 28)):
        assert _gather(qpa, name, **kw) == -2, kw
    for i in range(8):
        assert _gather(qpa, name, {i: NULL}) == -1, i
    for i, off in ((0, 8), (1, 2), (2, 2), (3, 2), (4, 2), (5, 2), (6, 8), (7, 8)):
        assert _gather(qpa, name, {i: at(i, off)}) == -3, i
    nothing = {i: NULL for i in range(8)}
    assert _gather(qpa, name, nothing, num_tokens=0) == 0 and _gather(qpa, name, nothing, num_reqs=0) == 0
    out = 5 * 2 * 128 * 2                                              # bytes of an output (num_tokens x heads x D, float32: twice)
    assert _gather(qpa, name, {7: at(6, 2 * out - 16)}) == -7
    assert _gather(qpa, name, {7: at(6, 2 * out)}, out_dtype=0, num_reqs=0) == 0
    assert _gather(qpa, name, {6: at(0, 16)}) == -7 and _gather(qpa, name, {7: at(3, -16)}) == -7
    assert _gather(qpa, name, {6: at(1, 4 * 8 - 16)}) == -7 and _gather(qpa, name, {6: at(2)}) == -7


def test_gather_nvfp4_has_no_scales_per_token(qpa):
    assert _gather(qpa, kv_scale_per_token=1) == -2


# ------------------------------------------------------------------ decode
def _desc(qpa, **kw):
    return _set(qpa.Nvfp4Desc(), kw, num_seqs=2, num_kv_heads=2, query_group=4, head_dim=128, block_size=16, num_blocks=4,
                max_blocks_per_seq=4)


def _decode(qpa, ptrs=None, ws_bytes=None, **kw):
    p = {i: at(i) for i in range(8)}
    p.update(ptrs or {})
    n = qpa.pa_decode_nvfp4_workspace_size(_desc(qpa)) if ws_bytes is None else ws_bytes
    return qpa.load_library().pa_decode_nvfp4(*[p[i] for i in range(7)], ctypes.byref(_desc(qpa, **kw)), p[7], n, None)


def test_decode_refusals(qpa):
    for kw in (dict(num_seqs=-1), dict(num_kv_heads=0), dict(num_kv_heads=65537), dict(query_group=0), dict(query_group=65),
               dict(head_dim=256), dict(block_size=24), dict(num_blocks=0), dict(max_blocks_per_seq=0),
               dict(table_stride=3), dict(max_blocks_per_seq=1 << 28), dict(num_seqs=1 << 28)):
        assert _decode(qpa, **kw) == -2, kw
        assert qpa.pa_decode_nvfp4_workspace_size(_desc(qpa, **kw)) == 0
    for i in range(8):
        assert _decode(qpa, {i: NULL}) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 2), (5, 2), (6, 8), (7, 128)):
        assert _decode(qpa, {i: at(i, off)}) == -3, i
    assert _decode(qpa, q_stride_seq=1028) == -3 and _decode(qpa, q_stride_head=-8) == -3
    n = qpa.pa_decode_nvfp4_workspace_size(_desc(qpa))
    assert n > 0 and _decode(qpa, ws_bytes=n - 1) == -4
    assert _decode(qpa, {i: NULL for i in range(8)}, num_seqs=0) == 0
    row = 8 * 128 * 2
    assert _decode(qpa, {6: at(0, 2 * row - 16)}) == -7                  # out in q
    assert _decode(qpa, {7: at(6, -256)}) == -7 or n <= 256              # the workspace's end in out
    assert _decode(qpa, {6: at(1, 4 * 2 * 2 * 16 * 72 - 16)}) == -7      # out in the cache


# ------------------------------------------------------------------ binding
def _t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


U8, I32, I64, F = torch.uint8, torch.int32, torch.int64, torch.float32


def test_binding_append():
    ok = dict(k=_t(3, 2, 128), v=_t(3, 2, 128), kv_cache=_t(4, 2, 2, 16, 72, dtype=U8), slots=_t(3, dtype=I64),
              k_scale=_t(1, dtype=F), v_scale=_t(1, dtype=F))
    for kw in (dict(k=_t(3, 2, 64)), dict(k=_t(3, 2, 128, dtype=torch.float16)), dict(v=None), dict(v_scale=None),
               dict(v=None, v_scale=None), dict(kv_cache=_t(4, 1, 2, 16, 72, dtype=U8)), dict(slots=_t(3, dtype=I32)),
               dict(kv_cache=_t(4, 2, 2, 16, 70, dtype=U8)), dict(kv_cache=_t(4, 3, 2, 16, 72, dtype=U8)),
               dict(kv_cache=_t(4, 2, 2, 16, 144, dtype=U8)[..., ::2]), dict(k_scale=_t(2, dtype=F)),
               dict(v_scale=_t(1)), dict(k=_t(3, 2, 256)[..., ::2]), dict(slots=_t(6, dtype=I64)[::2])):
        with pytest.raises(ValueError):
            qpa_pkg.kv_append_nvfp4(**{**ok, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        qpa_pkg.kv_append_nvfp4(**ok)


def test_binding_gather():
    ok = dict(kv_cache=_t(4, 2, 2, 16, 72, dtype=U8), block_table=_t(2, 4, dtype=I32), query_start=_t(3, dtype=I32),
              seq_lens=_t(2, dtype=I32), k_scale=_t(1, dtype=F), v_scale=_t(1, dtype=F), num_tokens=5)
    bad = (dict(block_table=_t(2, 4, dtype=I64)), dict(query_start=_t(2, dtype=I32)), dict(seq_lens=_t(3, dtype=I32)),
           dict(num_tokens=-1), dict(num_tokens=(1 << 32) + 5), dict(out_dtype=torch.float16), dict(out_k=_t(5, 2, 64)),
           dict(out_v=_t(5, 2, 128, dtype=F)), dict(out_k=_t(10, 2, 128)[::2]), dict(query_start=_t(6, dtype=I32)[::2]),
           dict(block_table=_t(2, 8, dtype=I32)[:, ::2]))
    for kw in bad + (dict(v_scale=None), dict(k_scale=_t(4, 2, 16, dtype=F))):
        with pytest.raises(ValueError):
            qpa_pkg.kv_gather_nvfp4(**{**ok, **kw})
    one = dict(ok, kv_cache=_t(4, 1, 2, 16, 72, dtype=U8))
    for kw in (dict(), dict(v_scale=None, out_v=_t(5, 2, 128))):
        with pytest.raises(ValueError, match="one plane"):
            qpa_pkg.kv_gather_nvfp4(**{**one, **kw})
    fp8 = dict(ok, kv_cache=_t(4, 2, 2, 16, 128, dtype=U8))
    for kw in bad + (dict(k_scale=_t(4, 2, 8, dtype=F)), dict(kv_cache=_t(4, 1, 2, 16, 128, dtype=U8))):
        with pytest.raises(ValueError):
            qpa_pkg.kv_gather_fp8(**{**fp8, **kw})
    for call, args in ((qpa_pkg.kv_gather_nvfp4, ok), (qpa_pkg.kv_gather_fp8, fp8)):
        with pytest.raises(ValueError, match="CUDA"):
            call(**args)


def test_binding_decode(qpa):
    ok = dict(q=_t(2, 8, 128), kv_cache=_t(4, 2, 2, 16, 72, dtype=U8), block_table=_t(2, 4, dtype=I32),
              seq_lens=_t(2, dtype=I32), k_scale=_t(1, dtype=F), v_scale=_t(1, dtype=F), query_group=4)
    bad = (dict(q=_t(2, 8, 64)), dict(q=_t(2, 8, 128, dtype=F)), dict(query_group=2), dict(q=_t(2, 8, 256)[..., ::2]),
           dict(kv_cache=_t(4, 1, 2, 16, 72, dtype=U8)), dict(block_table=_t(3, 4, dtype=I32)), dict(seq_lens=_t(3, dtype=I32)),
           dict(seq_lens=_t(2, dtype=I64)), dict(out=_t(2, 8, 128, dtype=F)), dict(out=_t(2, 4, 128)),
           dict(k_scale=_t(4, 2, 16, dtype=F)), dict(workspace=_t(1 << 20, dtype=U8)[::2]),
           dict(q=_t(1, 8, 128).expand(2, 8, 128)), dict(block_table=_t(2, 1 << 31, dtype=I32)))
    for kw in bad:
        with pytest.raises(ValueError):
            qpa_pkg.pa_decode_nvfp4(**{**ok, **kw})
    other = qpa_pkg.nvfp4_desc(ok["q"], ok["kv_cache"], ok["block_table"], 4, 0.5)
    other.num_kv_heads = 1
    with pytest.raises(ValueError, match="describe"):
        qpa_pkg.pa_decode_nvfp4(**ok, desc=other)
    with pytest.raises(ValueError, match="CUDA"):
        qpa_pkg.pa_decode_nvfp4(**ok)
