"""Refusals of the serving-step entry points, without a GPU: bad arguments are
turned away on the host before any launch, by the C ABI and by the binding."""
import ctypes

import pytest
import torch

NULL = ctypes.c_void_p(0)


def at(i, off=0):
    """Distinct addresses 16 MiB apart, never dereferenced: every call below is
    refused (or has nothing to do)."""
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


@pytest.fixture(scope="module")
def qpa():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_paged_attention_gb300 as qpa
    qpa.load_library()
    return qpa


def _set(d, kw, **base):
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def _slot(qpa, ptrs=None, **kw):
    d = _set(qpa.SlotDesc(), kw, num_reqs=4, block_size=16, max_blocks_per_seq=8, num_free=32, max_tokens=64)
    p = {i: at(i) for i in range(9)}
    p.update(ptrs or {})
    return qpa.load_library().paged_slot_map(*[p[i] for i in range(9)], ctypes.byref(d), None)


@pytest.mark.parametrize("kw", [dict(num_reqs=-1), dict(num_reqs=16385), dict(block_size=24), dict(block_size=0),
                                dict(max_blocks_per_seq=0), dict(num_free=-1), dict(max_tokens=-1), dict(reserved=1),
                                dict(table_stride=7), dict(max_blocks_per_seq=1 << 28, table_stride=1 << 28)])
def test_slot_map_shapes(qpa, kw):
    assert _slot(qpa, **kw) == -2


def test_slot_map_pointers(qpa):
    for i in range(9):
        assert _slot(qpa, {i: NULL}) == -1, i
        assert _slot(qpa, {i: at(i, 2)}) == -3, i
    assert _slot(qpa, {6: at(6, 4)}) == -3                       # slots are 8-byte
    assert qpa.load_library().paged_slot_map(*[at(i) for i in range(9)], None, None) == -1


def test_slot_map_overlaps(qpa):
    assert _slot(qpa, {5: at(1)}) == -7                           # seq_lens in place of cached_lens
    assert _slot(qpa, {4: at(5, 12)}) == -7                       # query_start's 20 bytes into seq_lens
    assert _slot(qpa, {2: at(3, 16)}) == -7                       # the table inside the free list
    assert _slot(qpa, {7: at(6, 508)}) == -7                      # positions over the last slot
    assert _slot(qpa, {8: at(2, 4 * 31)}) == -7                   # num_taken in the table's last entry


def _append(qpa, ptrs=None, **kw):
    d = _set(qpa.AppendDesc(), kw, num_tokens=3, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=4)
    p = {i: at(i) for i in range(6)}
    p.update(ptrs or {})
    return qpa.load_library().kv_append_fp8(*[p[i] for i in range(6)], ctypes.byref(d), None)


def test_append_refusals(qpa):
    for kw in (dict(num_tokens=-1), dict(num_kv_heads=0), dict(head_dim=96), dict(block_size=48), dict(num_blocks=0),
               dict(kv_scale_per_token=2)):
        assert _append(qpa, **kw) == -2, kw
    for i in range(6):
        assert _append(qpa, {i: NULL}) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 4), (4, 2), (5, 2)):
        assert _append(qpa, {i: at(i, off)}) == -3, i
    for s in ("k_stride_tok", "k_stride_head", "v_stride_tok", "v_stride_head"):
        assert _append(qpa, **{s: 100}) == -3 and _append(qpa, **{s: -8}) == -3
    assert _append(qpa, {i: NULL for i in range(6)}, num_tokens=0) == 0


def test_append_overlaps(qpa):
    row, cache = 2 * 128 * 2, 4 * 2 * 2 * 16 * 128                # bytes of a token's heads, of the cache
    assert _append(qpa, {0: at(2, cache - 16)}) == -7             # k begins in the cache's end
    assert _append(qpa, {1: at(2, -3 * row + 16)}) == -7          # v ends in its beginning
    assert _append(qpa, {1: at(2, -5 * row + 16)}, v_stride_tok=2 * row // 2) == -7   # strided: 2 x 2 rows + 1
    assert _append(qpa, {3: at(2, 64)}) == -7
    assert _append(qpa, {4: at(2, cache - 4)}) == -7
    assert _append(qpa, {5: at(4, 4 * 2 * 16 * 4 - 4)}, kv_scale_per_token=1) == -7   # written scales over each other


def _chunk_desc(qpa, **kw):
    return _set(qpa.ChunkDesc(), kw, num_reqs=2, num_tokens=5, num_kv_heads=2, query_group=4, head_dim=128,
                block_size=16, num_blocks=4, max_blocks_per_seq=4)


def _chunk(qpa, ptrs=None, ws_bytes=None, **kw):
    d = _chunk_desc(qpa, **kw)
    p = {i: at(i) for i in range(9)}
    p.update(ptrs or {})
    n = qpa.pa_chunk_fp8_workspace_size(_chunk_desc(qpa)) if ws_bytes is None else ws_bytes
    return qpa.load_library().pa_chunk_fp8(*[p[i] for i in range(8)], ctypes.byref(d), p[8], n, None)


def test_chunk_refusals(qpa):
    bad = (dict(num_reqs=-1), dict(num_tokens=-1), dict(num_kv_heads=0), dict(query_group=0), dict(query_group=65),
           dict(head_dim=256), dict(block_size=8), dict(num_blocks=0), dict(max_blocks_per_seq=0),
           dict(kv_scale_per_token=-1), dict(table_stride=3), dict(max_blocks_per_seq=1 << 28))
    for kw in bad:
        assert _chunk(qpa, **kw) == -2, kw
        assert qpa.pa_chunk_fp8_workspace_size(_chunk_desc(qpa, **kw)) == 0
    for i in range(9):
        assert _chunk(qpa, {i: NULL}) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 2), (5, 2), (6, 2), (7, 8), (8, 128)):
        assert _chunk(qpa, {i: at(i, off)}) == -3, i
    assert _chunk(qpa, {5: at(5, 4)}, kv_scale_per_token=1) == -3
    assert _chunk(qpa, q_stride_tok=1028) == -3 and _chunk(qpa, q_stride_head=-8) == -3
    n = qpa.pa_chunk_fp8_workspace_size(_chunk_desc(qpa))
    assert n > 0 and _chunk(qpa, ws_bytes=n - 1) == -4
    assert _chunk(qpa, num_reqs=0) == 0 and _chunk(qpa, {i: NULL for i in range(9)}, num_tokens=0) == 0


def test_chunk_overlaps(qpa):
    out = 5 * 8 * 128 * 2
    ws = qpa.pa_chunk_fp8_workspace_size(_chunk_desc(qpa))
    assert _chunk(qpa, {7: at(0)}) == -7                          # in place
    assert _chunk(qpa, {7: at(0, -out + 16)}) == -7
    assert _chunk(qpa, {8: at(0, -ws + 256)}, ws_bytes=ws) == -7 and _chunk(qpa, {7: at(8, 256)}) == -7
    assert _chunk(qpa, {7: at(1, 4 * 2 * 2 * 16 * 128 - 16)}) == -7
    assert _chunk(qpa, {3: at(7, 8)}) == -7 and _chunk(qpa, {4: at(8, 4)}) == -7 and _chunk(qpa, {6: at(7, 4)}) == -7


def test_descriptor_layouts(qpa):
    assert ctypes.sizeof(qpa.SlotDesc) == 32 and qpa.SlotDesc.table_stride.offset == 24
    assert ctypes.sizeof(qpa.AppendDesc) == 56 and qpa.AppendDesc.k_stride_tok.offset == 24
    assert ctypes.sizeof(qpa.ChunkDesc) == 64 and qpa.ChunkDesc.q_stride_tok.offset == 40


def test_status_string_of_overlap(qpa):
    assert b"overlap" in qpa.load_library().qpa_status_string(-7)


# ------------------------------------------------------------------ the binding
def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_refuses_cpu_tensors(qpa):
    with pytest.raises(ValueError, match="CUDA"):
        qpa.paged_slot_map(_i32(2), _i32(2), _i32(2, 4), _i32(3), 16, 8)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(1, 2, 1, 16, 64, dtype=torch.uint8)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        qpa.kv_append_fp8(k, k, cache, torch.zeros(2, dtype=torch.int64), one, one)
    with pytest.raises(ValueError, match="CUDA"):
        qpa.pa_chunk_fp8(k, cache, _i32(1, 1), _i32(2), _i32(1), one, one, 1)


def test_binding_refuses_wrong_types_and_shapes(qpa):
    i, one = _i32, torch.ones(1)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(1, 2, 1, 16, 64, dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int64)
    bad = [
        lambda: qpa.paged_slot_map(i(2).long(), i(2), i(2, 4), i(3), 16, 8),
        lambda: qpa.paged_slot_map(i(2), i(3), i(2, 4), i(3), 16, 8),
        lambda: qpa.paged_slot_map(i(2), i(2), i(4, 2).t(), i(3), 16, 8),
        lambda: qpa.paged_slot_map(i(2), i(2), i(2, 4), i(3), 16, 8, slots=i(8)),
        lambda: qpa.paged_slot_map(i(2), i(2), i(2, 4), i(3), 16, 8, positions=i(7)),
        lambda: qpa.kv_append_fp8(k.float(), k, cache, slots, one, one),
        lambda: qpa.kv_append_fp8(k, k[:1], cache, slots, one, one),
        lambda: qpa.kv_append_fp8(k, k, cache[:, :1], slots, one, one),
        lambda: qpa.kv_append_fp8(k, k, cache, slots.int(), one, one),
        lambda: qpa.kv_append_fp8(k, k, cache, slots, torch.ones(2), one),
        lambda: qpa.kv_append_fp8(k, k, cache, slots, torch.ones(1, 1, 16), one),
        lambda: qpa.kv_append_fp8(k.expand(2, 1, 64)[:, :1].transpose(0, 2), k, cache, slots, one, one),
        lambda: qpa.pa_chunk_fp8(k, cache, i(1, 1), i(3), i(1), one, one, 1),
        lambda: qpa.pa_chunk_fp8(k, cache, i(1, 1), i(2), i(1), one, one, 2),
        lambda: qpa.pa_chunk_fp8(k, cache, i(1, 1), i(2), i(1), one, one, 1, out=k.float()),
        lambda: qpa.pa_chunk_fp8(k[:1].expand(2, 1, 64), cache, i(1, 1), i(2), i(1), one, one, 1),
        lambda: qpa.pa_chunk_fp8(k, cache, i(1, 1), i(2), i(1), one, one, 1,
                                 desc=qpa.chunk_desc(k[:1], cache, i(1, 1), 1, False)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", n)
