"""Quantised paged-attention decode for GB300 (sm_103a).

A thin ctypes binding over the C ABI of ``libqpa.so`` (declared in
``include/qpa.h``). It only marshals arguments: every step of the decode runs
in the library's CUDA kernels. PyTorch supplies device memory and streams.
There is no CPU fallback: if the library is missing or a tensor is not on a
CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqpa.so")

QPA_OK = 0
QPA_OUT_F32 = 0
QPA_OUT_BF16 = 1
QPA_UQ_UE8M0_SCALES = 1
QPA_UQ_Q_HAIRCUT = 2
QPA_UQ_ROT_PERM = 4
QPA_IDX_PER_TOKEN = 1
QPA_IDX_SHARED_PAGES = 2
QPA_TEST_WITHHOLD_ARRIVAL = 1
SLOT_MAP_MAX_REQS = 16384
_lib = None


class QpaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = _lib.qpa_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn} failed: {msg} ({status})")


class Fp8Desc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("query_group", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("q_stride_seq", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("softmax_scale", ctypes.c_float), ("test_flags", ctypes.c_int32)]


class Fp8ExtDesc(ctypes.Structure):
    _fields_ = [("base", Fp8Desc), ("query_len", ctypes.c_int32), ("kv_scale_per_token", ctypes.c_int32),
                ("q_stride_tok", ctypes.c_int64)]


class UqDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("query_group", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("padded_slot", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("q_stride_seq", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("softmax_scale", ctypes.c_float)]


class IdxDesc(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int32), ("query_len", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_cols", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("q_stride_tok", ctypes.c_int64),
                ("q_stride_head", ctypes.c_int64), ("s_stride_head", ctypes.c_int64),
                ("s_stride_row", ctypes.c_int64)]


class SlotDesc(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("num_free", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32), ("table_stride", ctypes.c_int64)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("kv_scale_per_token", ctypes.c_int32), ("k_stride_tok", ctypes.c_int64),
                ("k_stride_head", ctypes.c_int64), ("v_stride_tok", ctypes.c_int64),
                ("v_stride_head", ctypes.c_int64)]


class ChunkDesc(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("query_group", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("kv_scale_per_token", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("q_stride_tok", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("table_stride", ctypes.c_int64)]


_P = ctypes.c_void_p
_SIGS = {
    "qpa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qpa_version": (ctypes.c_int, []),
    "qpa_kernel_error": (ctypes.c_int, [_P]),
    "pa_decode_fp8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Fp8Desc), ctypes.c_int]),
    "pa_decode_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                     ctypes.POINTER(Fp8Desc), _P, ctypes.c_size_t, _P]),
    "pa_decode_fp8_partition": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int,
                                               ctypes.POINTER(Fp8Desc), _P, ctypes.c_size_t, _P]),
    "pa_decode_fp8_combine": (ctypes.c_int, [ctypes.c_int, _P, ctypes.POINTER(Fp8Desc), _P,
                                             ctypes.c_size_t, _P]),
    "pa_decode_fp8_static": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                            ctypes.POINTER(Fp8Desc), _P]),
    "pa_decode_fp8_ext_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Fp8ExtDesc), ctypes.c_int]),
    "pa_decode_fp8_ext": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                         ctypes.POINTER(Fp8ExtDesc), _P, ctypes.c_size_t, _P]),
    "uq_decode_hd256_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(UqDesc), ctypes.c_int]),
    "uq_decode_hd256": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.POINTER(UqDesc), _P,
                                       ctypes.c_size_t, _P]),
    "uq_decode_hd256_partition": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, ctypes.POINTER(UqDesc),
                                                 _P, ctypes.c_size_t, _P]),
    "uq_decode_hd256_combine": (ctypes.c_int, [ctypes.c_int, _P, ctypes.POINTER(UqDesc), _P,
                                               ctypes.c_size_t, _P]),
    "nvfp4_index_score": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.POINTER(IdxDesc), _P]),
    "paged_slot_map": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(SlotDesc), _P]),
    "kv_append_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(AppendDesc), _P]),
    "pa_chunk_fp8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(ChunkDesc)]),
    "pa_chunk_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(ChunkDesc), _P,
                                    ctypes.c_size_t, _P]),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libqpa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libqpa.so not found at {path}; build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def declared_symbols():
    return list(_SIGS)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("qpa runs on CUDA tensors only (no CPU path)")


def _check(fn, st):
    if st != QPA_OK:
        raise QpaError(fn, st)


def kernel_error(stream=None) -> int:
    """Synchronise the stream and return/clear the device error word."""
    return load_library().qpa_kernel_error(_stream(stream))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns blocks aligned to at least 512 bytes
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------- fp8
def fp8_desc(q, kv_cache, block_table, query_group, softmax_scale=None, out_dtype=torch.float32):
    B, Hq, D = q.shape
    NB, two, Hk, bs, D2 = kv_cache.shape
    assert two == 2 and D2 == D and Hq == Hk * query_group
    d = Fp8Desc()
    d.num_seqs, d.num_kv_heads, d.query_group, d.head_dim = B, Hk, query_group, D
    d.block_size, d.num_blocks, d.max_blocks_per_seq = bs, NB, block_table.shape[1]
    d.out_dtype = QPA_OUT_BF16 if out_dtype == torch.bfloat16 else QPA_OUT_F32
    if q.stride(2) != 1:
        raise ValueError("q must be contiguous along head_dim")
    d.q_stride_seq, d.q_stride_head = q.stride(0), q.stride(1)
    d.softmax_scale = 0.0 if softmax_scale is None else float(softmax_scale)
    return d


def pa_decode_fp8_workspace_size(desc: Fp8Desc, num_partitions: int) -> int:
    return int(load_library().pa_decode_fp8_workspace_size(ctypes.byref(desc), num_partitions))


def pa_decode_fp8(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions: int,
                  query_group: int, out=None, workspace=None, softmax_scale=None,
                  out_dtype=torch.float32, stream=None, desc=None):
    """fp8 paged-attention decode. q bf16 [B, Hq, 128]; kv_cache uint8
    [NB, 2, Hk, bs, 128]; block_table int32 [B, maxb]; seq_lens int32 [B];
    k_scale / v_scale float32 [1] on the device. Returns out [B, Hq, 128]."""
    lib = load_library()
    _need_cuda(q, kv_cache, block_table, seq_lens, k_scale, v_scale)
    if desc is None:
        desc = fp8_desc(q, kv_cache, block_table, query_group, softmax_scale, out_dtype)
    if out is None:
        odt = torch.bfloat16 if desc.out_dtype == QPA_OUT_BF16 else torch.float32
        out = torch.empty((q.shape[0], q.shape[1], q.shape[2]), dtype=odt, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(pa_decode_fp8_workspace_size(desc, num_partitions), q.device)
    st = lib.pa_decode_fp8(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), _ptr(k_scale),
                           _ptr(v_scale), num_partitions, _ptr(out), ctypes.byref(desc),
                           _ptr(workspace), workspace.numel(), _stream(stream))
    _check("pa_decode_fp8", st)
    return out


def pa_decode_fp8_partition(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions,
                            desc, workspace, stream=None):
    st = load_library().pa_decode_fp8_partition(
        _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), _ptr(k_scale), _ptr(v_scale),
        num_partitions, ctypes.byref(desc), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("pa_decode_fp8_partition", st)


def pa_decode_fp8_combine(num_partitions, out, desc, workspace, stream=None):
    st = load_library().pa_decode_fp8_combine(num_partitions, _ptr(out), ctypes.byref(desc),
                                              _ptr(workspace), workspace.numel(), _stream(stream))
    _check("pa_decode_fp8_combine", st)


def fp8_ext_desc(q, kv_cache, block_table, query_group, per_token, softmax_scale=None,
                 out_dtype=torch.float32):
    """Descriptor of pa_decode_fp8_ext for q bf16 [B, QL, Hq, 128]."""
    B, QL, Hq, D = q.shape
    NB, two, Hk, bs, D2 = kv_cache.shape
    assert two == 2 and D2 == D and Hq == Hk * query_group
    if q.stride(3) != 1:
        raise ValueError("q must be contiguous along head_dim")
    d = Fp8ExtDesc()
    b = d.base
    b.num_seqs, b.num_kv_heads, b.query_group, b.head_dim = B, Hk, query_group, D
    b.block_size, b.num_blocks, b.max_blocks_per_seq = bs, NB, block_table.shape[1]
    b.out_dtype = QPA_OUT_BF16 if out_dtype == torch.bfloat16 else QPA_OUT_F32
    b.q_stride_seq, b.q_stride_head = q.stride(0), q.stride(2)
    b.softmax_scale = 0.0 if softmax_scale is None else float(softmax_scale)
    d.query_len = QL
    d.kv_scale_per_token = 1 if per_token else 0
    d.q_stride_tok = q.stride(1)
    return d


def pa_decode_fp8_ext_workspace_size(desc: Fp8ExtDesc, num_partitions: int) -> int:
    return int(load_library().pa_decode_fp8_ext_workspace_size(ctypes.byref(desc), num_partitions))


def pa_decode_fp8_ext(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions: int,
                      query_group: int, out=None, workspace=None, softmax_scale=None,
                      out_dtype=torch.float32, stream=None, desc=None):
    """fp8 decode of QL query tokens per sequence. q bf16 [B, QL, Hq, 128];
    k_scale / v_scale float32 [1] (per-tensor) or [NB, Hk, bs] (per-token) on
    the device. Returns out [B, QL, Hq, 128]."""
    lib = load_library()
    _need_cuda(q, kv_cache, block_table, seq_lens, k_scale, v_scale)
    per_token = k_scale.numel() > 1 or k_scale.dim() == 3
    if desc is None:
        desc = fp8_ext_desc(q, kv_cache, block_table, query_group, per_token, softmax_scale, out_dtype)
    if out is None:
        odt = torch.bfloat16 if desc.base.out_dtype == QPA_OUT_BF16 else torch.float32
        out = torch.empty(tuple(q.shape), dtype=odt, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(pa_decode_fp8_ext_workspace_size(desc, num_partitions), q.device)
    st = lib.pa_decode_fp8_ext(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), _ptr(k_scale),
                               _ptr(v_scale), num_partitions, _ptr(out), ctypes.byref(desc),
                               _ptr(workspace), workspace.numel(), _stream(stream))
    _check("pa_decode_fp8_ext", st)
    return out


def fp8_workspace_views(workspace, desc: Fp8Desc, num_partitions: int):
    """(O, m, l) float32 views of the partition partials in a workspace."""
    rows = desc.num_seqs * desc.num_kv_heads * num_partitions * desc.query_group
    up = lambda x: (x + 255) // 256 * 256
    m_off = up(rows * desc.head_dim * 4)
    l_off = up(m_off + rows * 4)
    f = workspace.view(torch.uint8)
    shp = (desc.num_seqs, desc.num_kv_heads, num_partitions, desc.query_group)
    O = f[:rows * desc.head_dim * 4].view(torch.float32).view(*shp, desc.head_dim)
    m = f[m_off:m_off + rows * 4].view(torch.float32).view(*shp)
    l = f[l_off:l_off + rows * 4].view(torch.float32).view(*shp)
    return O, m, l


def pa_decode_fp8_static(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions: int,
                         query_group: int, out=None, softmax_scale=None, out_dtype=torch.float32,
                         stream=None, desc=None):
    """pa_decode_fp8 without a workspace: for callers that cannot allocate
    device memory. The partials go to the library's static device array
    (8 MiB per GPU); calls that overlap on the GPU race on it."""
    lib = load_library()
    _need_cuda(q, kv_cache, block_table, seq_lens, k_scale, v_scale, out)
    if desc is None:
        desc = fp8_desc(q, kv_cache, block_table, query_group, softmax_scale, out_dtype)
    if out is None:
        raise ValueError("pa_decode_fp8_static writes into a caller-provided `out` tensor")
    st = lib.pa_decode_fp8_static(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
                                  _ptr(k_scale), _ptr(v_scale), num_partitions, _ptr(out),
                                  ctypes.byref(desc), _stream(stream))
    _check("pa_decode_fp8_static", st)
    return out


# --------------------------------------------------------------------- uq hd256
def uq_desc(q, kv_cache, block_table, query_group, softmax_scale=None, out_dtype=torch.float32,
            scale_format="e4m3", q_haircut=False, rot_perm=False):
    """scale_format: "e4m3" or "ue8m0" group scale bytes; q_haircut: round
    softmax_scale * q_r to e4m3 before the QK product; rot_perm: the cache is
    in the domain of the column-permuted rotation."""
    if scale_format not in ("e4m3", "ue8m0"):
        raise ValueError(f"scale_format {scale_format!r}")
    B, Hq, D = q.shape
    NB, bs, Hk, slot = kv_cache.shape
    assert D == 256 and Hq == Hk * query_group
    if q.stride(2) != 1:
        raise ValueError("q must be contiguous along head_dim")
    d = UqDesc()
    d.num_seqs, d.num_kv_heads, d.query_group, d.head_dim = B, Hk, query_group, D
    d.block_size, d.num_blocks, d.max_blocks_per_seq, d.padded_slot = bs, NB, block_table.shape[1], slot
    d.out_dtype = QPA_OUT_BF16 if out_dtype == torch.bfloat16 else QPA_OUT_F32
    d.q_stride_seq, d.q_stride_head = q.stride(0), q.stride(1)
    d.softmax_scale = 0.0 if softmax_scale is None else float(softmax_scale)
    d.flags = ((QPA_UQ_UE8M0_SCALES if scale_format == "ue8m0" else 0) | (QPA_UQ_Q_HAIRCUT if q_haircut else 0)
               | (QPA_UQ_ROT_PERM if rot_perm else 0))
    return d


def uq_decode_hd256_workspace_size(desc: UqDesc, num_partitions: int) -> int:
    return int(load_library().uq_decode_hd256_workspace_size(ctypes.byref(desc), num_partitions))


def uq_decode_hd256(q, kv_cache, centroids, block_table, seq_lens, num_partitions: int, query_group: int,
                    out=None, workspace=None, softmax_scale=None, out_dtype=torch.float32, stream=None,
                    desc=None, scale_format="e4m3", q_haircut=False, rot_perm=False):
    """4-bit head_dim=256 decode. q bf16 [B, Hq, 256] (not rotated); kv_cache
    uint8 [NB, bs, Hk, padded_slot]; centroids float32 [16]; returns the
    un-rotated out [B, Hq, 256]. scale_format / q_haircut / rot_perm as in uq_desc."""
    lib = load_library()
    _need_cuda(q, kv_cache, centroids, block_table, seq_lens)
    if desc is None:
        desc = uq_desc(q, kv_cache, block_table, query_group, softmax_scale, out_dtype, scale_format, q_haircut,
                       rot_perm)
    if out is None:
        odt = torch.bfloat16 if desc.out_dtype == QPA_OUT_BF16 else torch.float32
        out = torch.empty((q.shape[0], q.shape[1], 256), dtype=odt, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(uq_decode_hd256_workspace_size(desc, num_partitions), q.device)
    st = lib.uq_decode_hd256(_ptr(q), _ptr(kv_cache), _ptr(centroids), _ptr(block_table), _ptr(seq_lens),
                             num_partitions, _ptr(out), ctypes.byref(desc), _ptr(workspace), workspace.numel(),
                             _stream(stream))
    _check("uq_decode_hd256", st)
    return out


def uq_decode_hd256_partition(q, kv_cache, centroids, block_table, seq_lens, num_partitions, desc, workspace,
                              stream=None):
    st = load_library().uq_decode_hd256_partition(
        _ptr(q), _ptr(kv_cache), _ptr(centroids), _ptr(block_table), _ptr(seq_lens), num_partitions,
        ctypes.byref(desc), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("uq_decode_hd256_partition", st)


def uq_decode_hd256_combine(num_partitions, out, desc, workspace, stream=None):
    st = load_library().uq_decode_hd256_combine(num_partitions, _ptr(out), ctypes.byref(desc), _ptr(workspace),
                                                workspace.numel(), _stream(stream))
    _check("uq_decode_hd256_combine", st)


# --------------------------------------------------------------------- nvfp4 index scorer
def idx_desc(q_codes, pages, block_table, query_len, num_cols, scores=None, per_token=False, shared_pages=False):
    """num_cols counts blocks, or tokens with per_token (one column per token);
    shared_pages: score page by page over groups of 8 requests, loading a page
    that several requests map once (for requests that share pages)."""
    RQ, H, D = q_codes.shape
    assert D == 128 and RQ % query_len == 0
    d = IdxDesc()
    d.num_reqs, d.query_len, d.num_heads, d.head_dim = RQ // query_len, query_len, H, D
    d.num_blocks, d.max_blocks_per_seq, d.num_cols = pages.shape[0], block_table.shape[1], num_cols
    d.page_stride = pages.stride(0) * pages.element_size()
    d.q_stride_tok, d.q_stride_head = q_codes.stride(0), q_codes.stride(1)
    if scores is not None:
        d.s_stride_head, d.s_stride_row = scores.stride(0), scores.stride(1)
    d.flags = (QPA_IDX_PER_TOKEN if per_token else 0) | (QPA_IDX_SHARED_PAGES if shared_pages else 0)
    return d


def nvfp4_index_score(q_codes, pages, block_table, seq_lens, query_len: int, num_cols: int, scores=None,
                      stream=None, desc=None, per_token=False, shared_pages=False):
    """Paged NVFP4 index scores. q_codes uint8 (e4m3) [R*QL, H, 128]; pages
    uint8 [NB, 9216]; returns float32 scores [H, R*QL, num_cols] (columns are
    blocks, or tokens with per_token)."""
    lib = load_library()
    _need_cuda(q_codes, pages, block_table, seq_lens, scores)
    if scores is None:
        scores = torch.empty((q_codes.shape[1], q_codes.shape[0], num_cols), dtype=torch.float32,
                             device=q_codes.device)
    if desc is None:
        desc = idx_desc(q_codes, pages, block_table, query_len, num_cols, scores, per_token, shared_pages)
    st = lib.nvfp4_index_score(_ptr(q_codes), _ptr(pages), _ptr(block_table), _ptr(seq_lens), _ptr(scores),
                               ctypes.byref(desc), _stream(stream))
    _check("nvfp4_index_score", st)
    return scores


# --------------------------------------------------------------------- serving step
# These calls take a few microseconds on the GPU, so their checks are written
# out straight: a helper per property costs more than the kernel.
def _fail(msg):
    raise ValueError(msg)


def _rows(block_table):
    """(max_blocks, row stride or 0) of an int32 block table with contiguous rows."""
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        _fail("block_table must be int32 [num_reqs, max_blocks]")
    R, maxb = block_table.shape
    if maxb >= 1 << 31:
        _fail("block_table must have less than 2^31 columns")
    if R > 0 and maxb > 1 and block_table.stride(1) != 1:
        _fail("block_table must have contiguous rows")
    if R <= 1:
        return maxb, 0
    stride = block_table.stride(0)
    if stride < maxb:
        _fail("block_table rows must not overlap")
    return maxb, stride


def _dim_stride(t, i):
    """Stride of dimension i for a descriptor, where 0 means contiguous: a
    dimension of one element has no stride; an expanded one is refused."""
    if t.shape[i] <= 1:
        return 0
    s = t.stride(i)
    if s <= 0:
        _fail("expanded tensors are not supported")
    return s


def _launch(fn, index, stream, *args):
    """Call an entry point on `stream` (default: the device's current stream)
    with device `index`, that of all the call's tensors, current."""
    lib = _lib if _lib is not None else load_library()
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device_index != index:
            _fail("the stream must belong to the tensors' device")
        raw = stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = getattr(lib, fn)(*args, raw)
    else:
        with torch.cuda.device(index):
            st = getattr(lib, fn)(*args, raw)
    if st != QPA_OK:
        raise QpaError(fn, st)


def _empty(shape, dtype, device, stream):
    """Memory for a launch on `stream`, from that stream's own pool: another
    stream's may still be in use there by work queued before."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _device_of(*ts):
    """Index of the CUDA device that holds every tensor."""
    index = ts[0].get_device()
    for t in ts:
        if t.get_device() != index or index < 0:
            _fail("qpa runs on CUDA tensors only (no CPU path), all of them on one device")
    return index


def paged_slot_map(new_lens, cached_lens, block_table, free_blocks, block_size: int, max_tokens: int,
                   query_start=None, seq_lens=None, slots=None, positions=None, num_taken=None, stream=None):
    """Block table, slots and lengths of a step from the requests' lengths.

    new_lens, cached_lens int32 [R] (R <= 16384); block_table int32
    [R, max_blocks], rows contiguous, extended in place; free_blocks int32 [F]:
    ids are taken from its front. Returns (query_start int32 [R+1], seq_lens
    int32 [R], slots int64 [max_tokens], positions int32 [max_tokens],
    num_taken int32 [1]), written into the tensors passed for them if any
    (a captured graph keeps its own)."""
    i32 = torch.int32
    R = new_lens.numel()
    for t in (new_lens, cached_lens, free_blocks):
        if t.dtype != i32 or not t.is_contiguous():
            _fail("new_lens, cached_lens and free_blocks must be contiguous int32")
    maxb, stride = _rows(block_table)
    # (ctypes cuts a number to its field's 32 bits without a word)
    if not (0 <= max_tokens < 1 << 31 and 0 <= block_size < 1 << 31 and free_blocks.numel() < 1 << 31):
        _fail("max_tokens, block_size and the free list's length must be below 2^31 and not negative")
    if cached_lens.numel() != R or block_table.shape[0] != R:
        _fail("new_lens, cached_lens and block_table must have one entry per request")
    for t, n, dt in ((query_start, R + 1, i32), (seq_lens, R, i32), (slots, max_tokens, torch.int64),
                     (positions, max_tokens, i32), (num_taken, 1, i32)):
        if t is not None and (t.dtype != dt or t.numel() != n or not t.is_contiguous()):
            _fail(f"an output has to be contiguous, {dt}, of {n} elements")
    dev = new_lens.device
    if query_start is None:
        query_start = _empty(R + 1, i32, dev, stream)
    if seq_lens is None:
        seq_lens = _empty(R, i32, dev, stream)
    if slots is None:
        slots = _empty(max_tokens, torch.int64, dev, stream)
    if positions is None:
        positions = _empty(max_tokens, i32, dev, stream)
    if num_taken is None:
        num_taken = _empty(1, i32, dev, stream)
    index = _device_of(new_lens, cached_lens, block_table, free_blocks, query_start, seq_lens, slots, positions,
                       num_taken)
    d = SlotDesc(R, block_size, maxb, free_blocks.numel(), max_tokens, 0, stride)
    _launch("paged_slot_map", index, stream, new_lens.data_ptr(), cached_lens.data_ptr(), block_table.data_ptr(),
            free_blocks.data_ptr(), query_start.data_ptr(), seq_lens.data_ptr(), slots.data_ptr(),
            positions.data_ptr(), num_taken.data_ptr(), ctypes.byref(d))
    return query_start, seq_lens, slots, positions, num_taken


def _cache_shape(kv_cache):
    if kv_cache.dtype != torch.uint8 or kv_cache.dim() != 5 or kv_cache.shape[1] != 2 or not kv_cache.is_contiguous():
        _fail("kv_cache must be contiguous uint8 [num_blocks, 2, num_kv_heads, block_size, head_dim]")
    NB, _, Hk, bs, D = kv_cache.shape
    return NB, Hk, bs, D


def _per_token_scales(NB, Hk, bs, k_scale, v_scale):
    """True for [num_blocks, Hk, bs] scale tensors, False for one value each."""
    f32 = torch.float32
    if k_scale.dtype != f32 or v_scale.dtype != f32 or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        _fail("k_scale and v_scale must be contiguous float32")
    if k_scale.dim() == 3:
        if tuple(k_scale.shape) != (NB, Hk, bs) or tuple(v_scale.shape) != (NB, Hk, bs):
            _fail("per-token scales must be [num_blocks, num_kv_heads, block_size]")
        return True
    if k_scale.numel() != 1 or v_scale.numel() != 1:
        _fail("per-tensor scales must have one element")
    return False


def kv_append_fp8(k, v, kv_cache, slots, k_scale, v_scale, stream=None):
    """Quantise new keys and values into the paged fp8 cache, in place.

    k, v bf16 [T, Hk, D] (slices of a fused projection allowed); kv_cache uint8
    [NB, 2, Hk, bs, D]; slots int64 [T], negative = skip the row; k_scale /
    v_scale float32 with one element (read) or [NB, Hk, bs] (computed per token
    and written). Returns kv_cache."""
    NB, Hk, bs, D = _cache_shape(kv_cache)
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or slots.dtype != torch.int64:
        _fail("k and v must be bfloat16, slots int64")
    T = slots.numel()
    if tuple(k.shape) != (T, Hk, D) or tuple(v.shape) != (T, Hk, D) or not slots.is_contiguous():
        _fail("k and v must be [num_tokens, num_kv_heads, head_dim] with a row per (contiguous) slot")
    if T and (k.stride(2) != 1 or v.stride(2) != 1):
        _fail("k and v must be contiguous along head_dim")
    per_token = _per_token_scales(NB, Hk, bs, k_scale, v_scale)
    index = _device_of(k, v, kv_cache, slots, k_scale, v_scale)
    d = AppendDesc(T, Hk, D, bs, NB, 1 if per_token else 0, _dim_stride(k, 0), _dim_stride(k, 1), _dim_stride(v, 0),
                   _dim_stride(v, 1))
    _launch("kv_append_fp8", index, stream, k.data_ptr(), v.data_ptr(), kv_cache.data_ptr(), slots.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), ctypes.byref(d))
    return kv_cache


def chunk_desc(q, kv_cache, block_table, query_group, per_token, softmax_scale=None):
    """Descriptor of pa_chunk_fp8 for q bf16 [T, Hq, D]."""
    NB, Hk, bs, D = _cache_shape(kv_cache)
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[1] != Hk * query_group or q.shape[2] != D:
        _fail("q must be bfloat16 [num_tokens, num_kv_heads*query_group, head_dim]")
    T = q.shape[0]
    if T and q.stride(2) != 1:
        _fail("q must be contiguous along head_dim")
    maxb, stride = _rows(block_table)
    return ChunkDesc(block_table.shape[0], T, Hk, query_group, D, bs, NB, maxb, 1 if per_token else 0,
                     0.0 if softmax_scale is None else float(softmax_scale), _dim_stride(q, 0), _dim_stride(q, 1),
                     stride)


def pa_chunk_fp8_workspace_size(desc: ChunkDesc) -> int:
    return int(load_library().pa_chunk_fp8_workspace_size(ctypes.byref(desc)))


def pa_chunk_fp8(q, kv_cache, block_table, query_start, seq_lens, k_scale, v_scale, query_group: int, out=None,
                 workspace=None, softmax_scale=None, stream=None, desc=None):
    """Attention of a chunk of new tokens per request over the paged fp8 cache.

    q bf16 [T, Hq, D]; kv_cache uint8 [NB, 2, Hk, bs, D] (the new tokens are in
    it, see kv_append_fp8); block_table int32 [R, max_blocks]; query_start int32
    [R+1]; seq_lens int32 [R] counting the new tokens; k_scale / v_scale float32
    with one element or [NB, Hk, bs]. Returns out bf16 [T, Hq, D]; rows outside
    every request's range are not written. `workspace` may be kept between calls;
    a `desc` (from chunk_desc) is compared with the tensors' own and saves no time."""
    NB, Hk, bs, _ = _cache_shape(kv_cache)
    per_token = _per_token_scales(NB, Hk, bs, k_scale, v_scale)
    if softmax_scale is None and desc is not None:
        softmax_scale = desc.softmax_scale
    want = chunk_desc(q, kv_cache, block_table, query_group, per_token, softmax_scale)
    if desc is not None and bytes(desc) != bytes(want):
        _fail("desc does not describe these tensors")
    R = want.num_reqs
    if query_start.dtype != torch.int32 or seq_lens.dtype != torch.int32 or not query_start.is_contiguous() or \
            not seq_lens.is_contiguous() or query_start.numel() != R + 1 or seq_lens.numel() != R:
        _fail("query_start must be contiguous int32 with one entry more than requests, seq_lens with one per request")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, q.device, stream)
    elif out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        _fail("out must be contiguous bfloat16 of the shape of q")
    if workspace is None:
        workspace = _empty(max(pa_chunk_fp8_workspace_size(want), 256), torch.uint8, q.device, stream)
    elif not workspace.is_contiguous():
        _fail("workspace must be contiguous")
    index = _device_of(q, kv_cache, block_table, query_start, seq_lens, k_scale, v_scale, out, workspace)
    _launch("pa_chunk_fp8", index, stream, q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(),
            query_start.data_ptr(), seq_lens.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), out.data_ptr(),
            ctypes.byref(want), workspace.data_ptr(), workspace.nbytes)
    return out
