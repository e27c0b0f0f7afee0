"""The 4-bit (NVFP4) paged cache, restated in float64 numpy: the quantising
append, reading tokens back, and the attention of one new token per sequence.

A (block, plane, head) chunk holds block_size * D/2 bytes of e2m1 codes (dim 2i in
the low nibble of byte i) and block_size * D/16 e4m3 scales; a value is code *
scale * the tensor's scale.

Pins (tests/test_oracle_nvfp4.py): values that the formats hold come back
unchanged, every code is the nearest by exact rational arithmetic, the pages agree
with the scorer's reading of them.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import decode_bf16, decode_e2m1, decode_e4m3fn, unpack_nibbles
from .step import BF16_MAX

_E4M3 = decode_e4m3fn(np.arange(127, dtype=np.uint8))     # the non-negative finite values, increasing
_E2M1 = decode_e2m1(np.arange(8, dtype=np.uint8))


def _nearest(a, unit, values):
    """Index of the value v with v * unit nearest to a (>= 0), ties to the even
    index: decided by comparing a with midpoint * unit, products of at most 35 bits."""
    a, unit = np.broadcast_arrays(np.asarray(a, dtype=np.float64), np.asarray(unit, dtype=np.float64))
    code = np.zeros(a.shape, dtype=np.int64)
    for lo in range(len(values) - 1):
        mid = (values[lo] + values[lo + 1]) / 2 * unit
        code += (a > mid) | ((a == mid) & (lo % 2 == 1))
    return code


def quantise_nvfp4(x, g):
    """x [..., D] -> (codes uint8 [..., D/2], scales uint8 [..., D/16])."""
    x = np.asarray(x, dtype=np.float64)
    grp = x.reshape(*x.shape[:-1], -1, 16)
    g = float(g)
    bad = np.isnan(grp).any(axis=-1) | (not (g > 0 and math.isfinite(g)))
    grp = np.where(bad[..., None], 0.0, grp)
    unit = g if not bad.all() else 1.0
    a = np.minimum(np.abs(grp), BF16_MAX).max(axis=-1)
    s = np.maximum(_nearest(a, 6.0 * unit, _E4M3), 1)
    code = _nearest(np.minimum(np.abs(grp), BF16_MAX), (_E4M3[s] * unit)[..., None], _E2M1)
    code = np.where(bad[..., None], 0, code | np.signbit(grp) * 8).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0x7F, s).astype(np.uint8)


def _split(kv_cache):
    """(codes [NB, planes, Hk, bs, D/2], scales [NB, planes, Hk, bs, D/16]) of a cache, as copies."""
    NB, planes, Hk, bs, row = kv_cache.shape
    D = row // 9 * 16
    flat = np.asarray(kv_cache).reshape(NB, planes, Hk, bs * row)
    return (flat[..., :bs * D // 2].reshape(NB, planes, Hk, bs, D // 2).copy(),
            flat[..., bs * D // 2:].reshape(NB, planes, Hk, bs, D // 16).copy())


def _join(codes, scales):
    NB, planes, Hk, bs, half = codes.shape
    return np.concatenate([codes.reshape(NB, planes, Hk, -1), scales.reshape(NB, planes, Hk, -1)],
                          axis=-1).reshape(NB, planes, Hk, bs, half // 8 * 9)


def kv_append_nvfp4(k_bits, v_bits, kv_cache, slots, k_scale, v_scale):
    """The cache after the append; k_bits, v_bits [T, Hk, D] bf16 bits (v_bits None: one plane)."""
    codes, scales = _split(kv_cache)
    NB, _, _, bs, _ = codes.shape
    live = [(t, int(s)) for t, s in enumerate(np.asarray(slots)) if 0 <= s < NB * bs]
    rows, at = np.array([t for t, _ in live], dtype=int), np.array([s for _, s in live], dtype=int)
    for plane, (bits, g) in enumerate([(k_bits, k_scale)] + ([] if v_bits is None else [(v_bits, v_scale)])):
        c, s = quantise_nvfp4(decode_bf16(np.asarray(bits)[rows]), np.float32(g))
        codes[at // bs, plane, :, at % bs] = c
        scales[at // bs, plane, :, at % bs] = s
    return _join(codes, scales)


def values_nvfp4(kv_cache, plane, g, blk, off):
    """Values [len(blk), Hk, D] of the tokens (blk, off)."""
    codes, scales = _split(kv_cache)
    c, s = decode_e2m1(unpack_nibbles(codes[blk, plane, :, off])), decode_e4m3fn(scales[blk, plane, :, off])
    return c * np.repeat(s, 16, axis=-1) * float(np.float32(g))


def gather_rows(block_table, query_start, seq_lens, block_size):
    """(row, block, offset) arrays of the rows that hold a token, and the rows that are 0."""
    rows, blk, off, zero = [], [], [], []
    for r, L in enumerate(np.asarray(seq_lens)):
        a, b = int(query_start[r]), int(query_start[r + 1])
        for i in range(b - a):
            t = int(L) - (b - a) + i
            if t < 0:
                zero.append(a + i)
            else:
                rows.append(a + i)
                blk.append(int(block_table[r, t // block_size]))
                off.append(t % block_size)
    return (np.array(x, dtype=np.int64) for x in (rows, blk, off, zero))


def pa_decode_nvfp4(q_bits, kv_cache, block_table, seq_lens, k_scale, v_scale, query_group, softmax_scale=None):
    """(out, bound, total, slack) float64 [B, Hq, D] (slack [B, Hq]): the attention;
    sum_t p_t |v_t|, by which relative errors of the probabilities scale; sum_t |v_t|,
    by which absolute ones do; and the largest error of a logit for queries within 2^-17 of their group's largest and 2^-31 of
    their row's, and sums of float32."""
    q = decode_bf16(q_bits)
    B, Hq, D = q.shape
    Hk, bs = kv_cache.shape[2], kv_cache.shape[3]
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    out, bound, total, slack = *(np.zeros((B, Hq, D)) for _ in range(3)), np.zeros((B, Hq))
    for s, L in enumerate(np.asarray(seq_lens)):
        L = int(L)
        if L == 0:
            continue
        tok = np.arange(L)
        blk, off = np.asarray(block_table)[s, tok // bs].astype(np.int64), tok % bs
        with np.errstate(invalid="ignore", over="ignore"):
            K, V = values_nvfp4(kv_cache, 0, k_scale, blk, off), values_nvfp4(kv_cache, 1, v_scale, blk, off)
            for h in range(Hk):
                hs = slice(h * query_group, (h + 1) * query_group)
                x = scale * (q[s, hs] @ K[:, h].T)
                w = np.exp(x - x.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[s, hs], bound[s, hs], total[s, hs] = w @ V[:, h], w @ np.abs(V[:, h]), np.abs(V[:, h]).sum(axis=0)
                near = np.repeat(np.abs(q[s, hs]).reshape(query_group, -1, 16).max(axis=-1), 16, axis=-1)
                # 6 terms of 3 bits: half of the last step, 2^-2 8^-5 of the power of two at or above the group's
                # largest; groups far below the row's largest: 2^-31 of that
                err = (near * 2.0 ** -17 + np.abs(q[s, hs]) * 2.0 ** -20
                       + np.abs(q[s, hs]).max(axis=-1, keepdims=True) * 2.0 ** -31) @ np.abs(K[:, h]).T
                slack[s, hs] = abs(scale) * err.max(axis=1) + 2.0 ** -21 * np.abs(x).max(axis=1)
    return out, bound, total, slack
