"""The operators around the 4-bit (NVFP4) paged cache, as measured.

A server that keeps its keys and values in 4 bits quantises the new tokens into
the pages (kv_append_nvfp4), reads a request's tokens back for a dense prompt
attention or to hand them on (kv_gather_nvfp4, and kv_gather_fp8 for the fp8
pages), and decodes one token per request over the pages (pa_decode_nvfp4).
`own` selects the library's kernels or the plain form in elementary torch
operations. The pages' codes hold no value by themselves, so an append is
followed by reading the new tokens back, in both forms.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 128 running requests
        dict(name="append_decode_128", op="append", batch=128, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=300, heads=8,
             head_dim=128, block_size=16, fused_qkv=True, lens_seed=1),
        # the new tokens of two long prompts, read out of the fused projection's output
        dict(name="append_prompts_16k", op="append", batch=2, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, heads=8,
             head_dim=128, block_size=16, fused_qkv=True, lens_seed=2),
        # chunks of odd lengths behind cached tokens, head_dim 64, an odd head count
        dict(name="append_chunks_d64", op="append", batch=23, new_lo=1, new_hi=401, ctx_lo=0, ctx_hi=700, heads=5,
             head_dim=64, block_size=128, fused_qkv=False, lens_seed=3),
        # a short request read back: latency
        dict(name="read_short", op="read4", batch=1, len_lo=100, len_hi=100, heads=2, head_dim=64, block_size=32,
             lens_seed=4),
        # the contexts of six requests, for a dense prompt attention
        dict(name="read_contexts", op="read4", batch=6, len_lo=1500, len_hi=9000, heads=8, head_dim=128, block_size=16,
             lens_seed=5),
        # the same of fp8 pages with scales per tensor
        dict(name="read_fp8_contexts", op="read8", batch=6, len_lo=1500, len_hi=9000, heads=8, head_dim=128,
             block_size=64, per_token=False, lens_seed=6),
        # fp8 pages with scales per token, short ragged requests, head_dim 64
        dict(name="read_fp8_scales_d64", op="read8", batch=37, len_lo=1, len_hi=600, heads=4, head_dim=64,
             block_size=16, per_token=True, lens_seed=7),
        # the smallest decode: four short requests
        dict(name="decode_short", op="decode", batch=4, len_lo=1, len_hi=200, heads=2, group=4, head_dim=128,
             block_size=16, lens_seed=8),
        # sixteen long requests of one length: the bandwidth-bound end
        dict(name="decode_16x16k", op="decode", batch=16, len_lo=16384, len_hi=16384, heads=8, group=8, head_dim=128,
             block_size=16, lens_seed=9),
        # a ragged batch, odd group
        dict(name="decode_ragged_64", op="decode", batch=64, len_lo=1, len_hi=16384, heads=8, group=5, head_dim=128,
             block_size=64, lens_seed=10),
        # one long document, wide group: split over the length
        dict(name="decode_long_128k", op="decode", batch=1, len_lo=131071, len_hi=131071, heads=4, group=16,
             head_dim=128, block_size=128, lens_seed=11),
        # head_dim 64
        dict(name="decode_d64", op="decode", batch=32, len_lo=1000, len_hi=12000, heads=8, group=8, head_dim=64,
             block_size=32, lens_seed=12),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read4", "read8", "decode", "decode"])
    case = dict(op=op, heads=rng.choice([1, 2, 3, 4, 5, 8]), head_dim=rng.choice([64, 128, 128]),
                block_size=rng.choice([16, 32, 64, 128, 256]), lens_seed=rng.randrange(1 << 30))
    if op == "append":
        while True:
            case.update(batch=_logint(rng, 1, 256), new_lo=1, new_hi=_logint(rng, 1, 16384), ctx_lo=0,
                        ctx_hi=_logint(rng, 1, 4096))
            if case["batch"] * case["new_hi"] <= 16384 and case["batch"] * case["ctx_hi"] <= 200000:
                return dict(case, fused_qkv=rng.random() < 0.5)
    while True:
        case.update(batch=_logint(rng, 1, 64), len_lo=1, len_hi=_logint(rng, 1, 131072))
        if op == "decode":
            case.update(group=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 24]))
        if op == "read8":
            case.update(per_token=rng.random() < 0.5)
        # (the plain form pads every request to the longest one)
        if case["batch"] * case["len_hi"] <= (1 << 20 if op == "decode" else 1 << 16) and \
                work(case)["bytes"] <= (6e8 if op == "decode" else 3e8):
            return case


def _lens(case):
    r = random.Random(case["lens_seed"])
    if case["op"] == "append":
        return [(r.randint(case["new_lo"], case["new_hi"]), r.randint(case["ctx_lo"], case["ctx_hi"]))
                for _ in range(case["batch"])]
    return [(0, r.randint(case["len_lo"], case["len_hi"])) for _ in range(case["batch"])]


def work(case):
    lens = _lens(case)
    h, d = case["heads"], case["head_dim"]
    new, tot = sum(n for n, _ in lens), sum(n + c for n, c in lens)
    page = 2 * h * (d // 2 + d // 16)                 # 4-bit bytes of a token
    if case["op"] == "append":
        # bf16 in, pages out, and the pages' values in bf16 again
        return {"bytes": new * (2 * 2 * h * d + 2 * page + 2 * 2 * h * d + 8), "flops": 4 * new * h * d}
    if case["op"] == "read4":
        return {"bytes": tot * (page + 2 * 2 * h * d), "flops": 4 * tot * h * d}
    if case["op"] == "read8":
        return {"bytes": tot * h * (2 * d + (8 if case["per_token"] else 0) + 2 * 2 * d), "flops": 2 * tot * h * d}
    return {"bytes": tot * page + 2 * 2 * case["batch"] * h * case["group"] * d, "flops": 4 * d * h * case["group"] * tot}


# ------------------------------------------------------------------ inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _blocks(n, bs):
    return (n + bs - 1) // bs


def _keys(shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    # a few channels an order larger, as trained models have them
    x[..., :: shape[-1] // 4] *= 8
    return x


def _pages4(x, scale):
    """x [blocks, heads, block_size, D] as 4-bit chunks [blocks, heads, block_size, 9 D / 16]."""
    nb, h, bs, d = x.shape
    x = (x / scale).view(nb, h, bs, d // 16, 16)
    s = (x.abs().amax(-1) / 6).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    a = x.abs() / s.float()[..., None]
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a > m
    code = (code | (x < 0).to(torch.uint8) << 3).view(nb, h, bs, d)
    code = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat([code.reshape(nb, h, -1), s.view(torch.uint8).reshape(nb, h, -1)], -1).view(nb, h, bs, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    lens = _lens(case)
    # another seed gives the same requests in another order
    order = torch.randperm(case["batch"], generator=g, device="cuda").tolist()
    new, tot = [lens[i][0] for i in order], [sum(lens[i]) for i in order]
    h, d, bs, op = case["heads"], case["head_dim"], case["block_size"], case["op"]
    used = [_blocks(x, bs) for x in tot]
    nb, maxb = sum(used) + 3, max(used)
    table = torch.zeros(case["batch"], maxb, dtype=torch.int32, device="cuda")
    held = torch.arange(maxb, device="cuda")[None, :] < _i32(used)[:, None]
    table[held] = torch.randperm(nb, generator=g, device="cuda").int()[:sum(used)]
    st.update(block_table=table, seq_lens=_i32(tot))
    # rows of the step: the new tokens, or every token of a request
    rows = new if op == "append" else tot
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    st.update(query_start=_i32(start), rows=start[-1])
    st.update(k_scale=torch.tensor([0.031], device="cuda"), v_scale=torch.tensor([0.0043], device="cuda"))
    if op == "append":
        if case["fused_qkv"]:
            # keys and values as slices of [rows][query heads + 2 heads][D], two query heads per KV head
            qkv = _keys((start[-1], 4 * h, d), g).bfloat16()
            k, v = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
        else:
            k, v = _keys((start[-1], h, d), g).bfloat16(), _keys((start[-1], h, d), g).bfloat16()
        req = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), torch.tensor(new, device="cuda"))
        pos = (st["seq_lens"] - st["query_start"][1:])[req].long() + torch.arange(start[-1], device="cuda")
        st.update(k=k, v=v, slots=table[req, pos // bs].long() * bs + pos % bs,
                  kv_cache=torch.zeros(nb, 2, h, bs, d // 2 + d // 16, dtype=torch.uint8, device="cuda"))
        return st
    fp8 = op == "read8"
    cache = torch.empty(nb, 2, h, bs, d if fp8 else d // 2 + d // 16, dtype=torch.uint8, device="cuda")
    if fp8 and case["per_token"]:
        st.update(k_scale=torch.empty(nb, h, bs, device="cuda"), v_scale=torch.empty(nb, h, bs, device="cuda"))
    step = max(1, (1 << 26) // (h * bs * d))
    for b0 in range(0, nb, step):
        b1 = min(nb, b0 + step)
        for kv, sc in ((0, st["k_scale"]), (1, st["v_scale"])):
            x = _keys((b1 - b0, h, bs, d), g)
            if not fp8:
                cache[b0:b1, kv] = _pages4(x, sc)
                continue
            if case["per_token"]:
                sc[b0:b1] = x.abs().amax(-1) / 448
                x = x / sc[b0:b1, :, :, None]
            else:
                x = x / sc
            cache[b0:b1, kv] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    st.update(kv_cache=cache)
    if op == "decode":
        # queries that give the softmax clear peaks without one token taking all
        st.update(q=(0.4 * torch.randn(case["batch"], h * case["group"], d, generator=g, device="cuda")).bfloat16())
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "read4": _plain_read, "read8": _plain_read, "decode": _plain_decode}[state["op"]](state)


def _run_own(s):
    import quantized_paged_attention_gb300 as qpa
    if s["op"] == "decode":
        return qpa.pa_decode_nvfp4(s["q"], s["kv_cache"], s["block_table"], s["seq_lens"], s["k_scale"], s["v_scale"],
                                   s["group"])
    if s["op"] == "append":
        qpa.kv_append_nvfp4(s["k"], s["v"], s["kv_cache"], s["slots"], s["k_scale"], s["v_scale"])
    read = qpa.kv_gather_fp8 if s["op"] == "read8" else qpa.kv_gather_nvfp4
    k, v = read(s["kv_cache"], s["block_table"], s["query_start"], s["seq_lens"], s["k_scale"], s["v_scale"], s["rows"])
    return dict(k=k, v=v)


def _values4(chunk, head_dim):
    """[..., block_size, 9 D / 16] bytes as float32 values [..., block_size, D], without the tensor's scale."""
    bs = chunk.shape[-2]
    flat = chunk.flatten(-2)
    code, scale = flat[..., :bs * head_dim // 2], flat[..., bs * head_dim // 2:]
    code = torch.stack([code & 15, code >> 4], -1).long()
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=chunk.device)
    val = lut[code].view(*flat.shape[:-1], bs, head_dim // 16, 16)
    scale = scale.contiguous().view(torch.float8_e4m3fn).float().view(*flat.shape[:-1], bs, head_dim // 16, 1)
    return (val * scale).flatten(-2)


def _plain_read(s):
    bs, start, n = s["block_size"], s["query_start"].long(), s["rows"]
    row = torch.arange(n, device=start.device)
    req = torch.searchsorted(start[1:], row, right=True)
    pos = s["seq_lens"].long()[req] - start[1:][req] + row
    blk, off = s["block_table"][req, pos // bs].long(), pos % bs
    if s["op"] == "read8":
        val = s["kv_cache"].view(torch.float8_e4m3fn)[blk, :, :, off].float()             # [rows, 2, heads, D]
        if s["per_token"]:
            ks, vs = s["k_scale"][blk, :, off][..., None], s["v_scale"][blk, :, off][..., None]
        else:
            ks, vs = s["k_scale"], s["v_scale"]
    else:
        half, grp = s["head_dim"] // 2, s["head_dim"] // 16
        page = s["kv_cache"].flatten(3)                                                  # [blocks, 2, heads, chunk]
        at = off[:, None] * half + torch.arange(half, device=off.device)
        sat = bs * half + off[:, None] * grp + torch.arange(grp, device=off.device)
        both = page[blk[:, None], :, :, torch.cat([at, sat], 1)]                          # [rows, bytes, 2, heads]
        val = _values4(both.permute(0, 2, 3, 1)[..., None, :], s["head_dim"])[..., 0, :]
        ks, vs = s["k_scale"], s["v_scale"]
    return dict(k=(val[:, 0] * ks).bfloat16(), v=(val[:, 1] * vs).bfloat16())


def _round_e4m3(x):
    """float64, positive -> the nearest e4m3 value (ties to even, saturating), exact."""
    a = x.clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.exp2(((e - 1).clamp(min=-6) - 3).double())
    return (torch.round(a / step) * step).clamp(max=448.0)


def _round_e2m1(a):
    """Magnitudes, float64 -> codes 0 to 7 of the nearest e2m1 values; a tie goes to the even code."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())


def _quantise(x, scale):
    """[rows, heads, D] -> (code bytes [rows, heads, D / 2], e4m3 scales [rows, heads, D / 16])."""
    t, h, d = x.shape
    # in 64 bits: codes and scales turn on values next to a border
    x = x.double().reshape(t, h, d // 16, 16)
    s = _round_e4m3(x.abs().amax(-1) / (6 * scale.double())).clamp(min=2.0 ** -9)
    code = _round_e2m1(x.abs() / (s * scale.double())[..., None]) | (x < 0).byte() << 3
    code = code.view(t, h, d)
    return code[..., 0::2] | code[..., 1::2] << 4, s.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    bs, half, grp = s["block_size"], s["head_dim"] // 2, s["head_dim"] // 16
    page = s["kv_cache"].flatten(3)
    blk, off = s["slots"] // bs, s["slots"] % bs
    at = off[:, None] * half + torch.arange(half, device=off.device)
    sat = bs * half + off[:, None] * grp + torch.arange(grp, device=off.device)
    kc, ks = _quantise(s["k"], s["k_scale"])
    vc, vs = _quantise(s["v"], s["v_scale"])
    page[blk[:, None], :, :, at] = torch.stack([kc, vc], 1).permute(0, 3, 1, 2)
    page[blk[:, None], :, :, sat] = torch.stack([ks, vs], 1).permute(0, 3, 1, 2)
    return _plain_read(s)


def _plain_decode(s):
    h, grp, d, lens = s["heads"], s["group"], s["head_dim"], s["seq_lens"].long()
    page = s["kv_cache"][s["block_table"].long()]                       # [B, blocks, 2, heads, block_size, bytes]
    kv = _values4(page, d).permute(2, 0, 3, 1, 4, 5).flatten(3, 4)      # [2, B, heads, tokens, D]
    q = s["q"].float().view(-1, h, grp, d)
    sc = torch.matmul(q, kv[0].transpose(2, 3)) * (s["k_scale"] / math.sqrt(d))
    sc = sc.masked_fill(torch.arange(sc.shape[-1], device=q.device) >= lens[:, None, None, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.matmul(p, kv[1]) / p.sum(-1, keepdim=True) * s["v_scale"]
    return o.flatten(1, 2).bfloat16()


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _decode_e2m1(code):
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
    return torch.where(code >= 8, -mag, mag)


def _decode_e4m3(code):
    c = code.long()
    e, m = (c >> 3 & 15).double(), (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _token_values(s, kv, head, blk, off):
    """Values of one head's tokens (block, offset) in 64 bits."""
    d, bs = s["head_dim"], s["block_size"]
    sc = s["k_scale"] if kv == 0 else s["v_scale"]
    if s["op"] == "read8":
        x = _decode_e4m3(s["kv_cache"][blk, kv, head, off])
        return x * (sc[blk, head, off].double()[:, None] if s["per_token"] else sc.double())
    flat = s["kv_cache"].view(s["kv_cache"].shape[0], 2, s["heads"], -1)
    dim = torch.arange(d, device=blk.device)
    byte = flat[blk[:, None], kv, head, off[:, None] * (d // 2) + dim // 2].long()
    code = torch.where(dim % 2 == 0, byte & 15, byte >> 4)
    scale = flat[blk[:, None], kv, head, bs * (d // 2) + off[:, None] * (d // 16) + dim // 16]
    return _decode_e2m1(code) * _decode_e4m3(scale) * sc.double()


def exact(case, seed):
    s = prepare(case, seed)
    bs, h, d = case["block_size"], case["heads"], case["head_dim"]
    tot, start = s["seq_lens"].tolist(), s["query_start"].tolist()
    if case["op"] == "append":
        # every candidate's distance from the exact quotient; the nearest wins, of two the even code
        e4 = _decode_e4m3(torch.arange(1, 127, device="cuda"))
        e2 = _decode_e2m1(torch.arange(8, device="cuda"))
        out = {}
        for name, x, sc in (("k", s["k"], s["k_scale"].double()), ("v", s["v"], s["v_scale"].double())):
            x = x.double().reshape(-1, 16)
            want = x.abs().max(1).values / (6 * sc)
            up = torch.searchsorted(e4, want).clamp(1, 125)
            lo, hi = e4[up - 1], e4[up]
            even = torch.where(up % 2 == 0, lo, hi)                     # (e4 holds the codes from 1 on)
            near = torch.where(want - lo == hi - want, even, torch.where(want - lo < hi - want, lo, hi))
            real = near * sc
            ratio = x.abs() / real[:, None]
            up = torch.searchsorted(e2, ratio).clamp(1, 7)
            lo, hi = e2[up - 1], e2[up]
            pick = torch.where(ratio - lo == hi - ratio, torch.where(up % 2 == 1, lo, hi),
                               torch.where(ratio - lo < hi - ratio, lo, hi))
            out[name] = (torch.copysign(pick, x) * real[:, None]).view(-1, h, d)
        return out
    if case["op"] in ("read4", "read8"):
        out = torch.zeros(2, s["rows"], h, d, dtype=torch.float64, device="cuda")
        for r, n in enumerate(tot):
            t = torch.arange(n, device="cuda")
            blk, off = s["block_table"][r].long()[t // bs], t % bs
            for kv in range(2):
                for i in range(h):
                    out[kv, start[r]:start[r + 1], i] = _token_values(s, kv, i, blk, off)
        return dict(k=out[0], v=out[1])
    grp = case["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(tot):
        t = torch.arange(n, device="cuda")
        blk, off = s["block_table"][r].long()[t // bs], t % bs
        for i in range(h):
            k, v = _token_values(s, 0, i, blk, off), _token_values(s, 1, i, blk, off)
            w = torch.softmax(s["q"][r, i * grp:(i + 1) * grp].double() @ k.T / d ** 0.5, -1)
            out[r, i * grp:(i + 1) * grp] = w @ v
    return out
