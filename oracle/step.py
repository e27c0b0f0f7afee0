"""The serving step around the fp8 paged cache, restated in float64 numpy:
slots and block tables from request lengths, the quantising append, and the
attention of a chunk of new tokens per request. Plain loops, one definition
after the other; shares only the format decoders with the decode oracle."""
from __future__ import annotations

import math

import numpy as np

from .formats import decode_bf16, decode_e4m3fn

INT32_MAX = 2 ** 31 - 1


def paged_slot_map(new_lens, cached_lens, block_table, free_blocks, block_size: int, max_tokens: int):
    """(query_start, seq_lens, block_table, slots, positions, num_taken,
    short): short is true when a block or a table column was missing."""
    bs = block_size
    table = np.array(block_table, dtype=np.int64)
    maxb = table.shape[1]
    start, lens, slots, pos, k, short = [0], [], [], [], 0, False
    for r, (n, c) in enumerate(zip(new_lens, cached_lens)):
        n, c = max(0, int(n)), max(0, int(c))
        held, need = -(-c // bs), -(-(c + n) // bs)
        blk = {}
        for e in range(held, need):
            if k < len(free_blocks) and e < maxb:
                blk[e] = table[r, e] = int(free_blocks[k])
            else:
                short = True
            k += 1
        for p in range(c, c + n):
            e = p // bs
            b = blk.get(e, -1) if e >= held else (int(table[r, e]) if e < maxb else -1)
            slots.append(b * bs + p % bs if b >= 0 else -1)
            pos.append(p)
            short = short or e >= maxb
        start.append(min(start[-1] + n, INT32_MAX))
        lens.append(min(c + n, INT32_MAX))
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    pos = (pos + [0] * max_tokens)[:max_tokens]
    return (np.array(start), np.array(lens, dtype=np.int64), table, np.array(slots, dtype=np.int64),
            np.array(pos, dtype=np.int64), k, short)


_CODE_VALUES = decode_e4m3fn(np.arange(127, dtype=np.uint8))     # the non-negative finite codes, increasing


def e4m3_nearest(x: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Code of the e4m3 value nearest to x / s (ties to the even code,
    saturating), decided by comparing |x| with midpoint * |s|: exact for x of
    8 and s of 24 significant bits, since the product has at most 29."""
    x, s = np.broadcast_arrays(np.asarray(x, dtype=np.float64), np.asarray(s, dtype=np.float64))
    ax, as_ = np.abs(x), np.abs(s)
    code = np.zeros(x.shape, dtype=np.int64)
    with np.errstate(invalid="ignore"):
        for lo in range(126):
            mid = (_CODE_VALUES[lo] + _CODE_VALUES[lo + 1]) / 2 * as_
            code += (ax > mid) | ((ax == mid) & (lo % 2 == 1))
    code = code | (np.signbit(x) ^ np.signbit(s)) * 0x80
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


BF16_MAX = float(np.float32(3.3895314e38))


def token_scale(x: np.ndarray) -> np.ndarray:
    """Per-token scale of vectors x [..., D]: largest |x| / 448 in float32, at
    least 2^-126 (NaN ignored, infinities as the largest bf16)."""
    a = np.nan_to_num(np.abs(np.asarray(x, dtype=np.float64)), nan=0.0, posinf=BF16_MAX).max(axis=-1)
    return np.maximum((a / 448.0).astype(np.float32), np.float32(2.0 ** -126))


def kv_append_fp8(k_bits, v_bits, kv_cache, slots, k_scale, v_scale):
    """(cache, k_scale, v_scale) after the append; k_bits, v_bits [T, Hk, D]
    bf16 bits; k_scale / v_scale floats, or [NB, Hk, bs] arrays (written)."""
    cache = np.array(kv_cache)
    NB, _, Hk, bs, D = cache.shape
    scales = [np.array(k_scale, dtype=np.float32), np.array(v_scale, dtype=np.float32)]
    x = [decode_bf16(k_bits), decode_bf16(v_bits)]
    for t, slot in enumerate(np.asarray(slots)):
        if slot < 0 or slot >= NB * bs:
            continue
        b, o = int(slot) // bs, int(slot) % bs
        for kv in range(2):
            s = scales[kv]
            if s.ndim == 3:
                s[b, :, o] = token_scale(x[kv][t])
                row = s[b, :, o][:, None]
            else:
                row = np.float64(s.reshape(-1)[0])
            cache[b, kv, :, o] = e4m3_nearest(x[kv][t], row)
    return cache, scales[0], scales[1]


def pa_chunk_fp8(q_bits, kv_cache, block_table, query_start, seq_lens, k_scale, v_scale, query_group: int,
                 softmax_scale: float | None = None):
    """(out, bound) float64 [T, Hq, D]: the attention and sum_t p_t |v_t|, by
    which errors of the probabilities scale. Rows of no request are NaN."""
    q = decode_bf16(q_bits)
    T, Hq, D = q.shape
    NB, _, Hk, bs, _ = kv_cache.shape
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    per_token = np.ndim(k_scale) == 3
    out, bound = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    for r, L in enumerate(np.asarray(seq_lens)):
        L = int(L)
        a, b = int(query_start[r]), int(query_start[r + 1])
        tok = np.arange(L)
        blk, off = np.asarray(block_table)[r, tok // bs].astype(np.int64), tok % bs
        for h in range(Hk):
            k = decode_e4m3fn(kv_cache[blk, 0, h, off])
            v = decode_e4m3fn(kv_cache[blk, 1, h, off])
            if per_token:
                k = k * np.asarray(k_scale, dtype=np.float64)[blk, h, off][:, None]
                v = v * np.asarray(v_scale, dtype=np.float64)[blk, h, off][:, None]
            else:
                k, v = k * float(np.asarray(k_scale).reshape(-1)[0]), v * float(np.asarray(v_scale).reshape(-1)[0])
            heads = slice(h * query_group, (h + 1) * query_group)
            for i in range(b - a):
                n = max(0, L - (b - a) + i + 1)
                if n == 0:
                    out[a + i, heads] = bound[a + i, heads] = 0.0
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (q[a + i, heads] @ k[:n].T)
                    w = np.exp(s - s.max(axis=1, keepdims=True))
                    w /= w.sum(axis=1, keepdims=True)
                    out[a + i, heads] = w @ v[:n]
                    bound[a + i, heads] = w @ np.abs(v[:n])
    return out, bound
