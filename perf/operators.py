"""The operators of a serving step around the fp8 paged cache, as measured.

A server that decodes with pa_decode_fp8 takes a batch through three steps
before and beside it: the block table, slots and lengths of the step are made
from the requests' lengths (paged_slot_map), the new tokens' keys and values
are quantised into the pages (kv_append_fp8), and a chunk of new tokens per
request attends to the pages (pa_chunk_fp8). Each case is one call of one of
them; `own` selects the library's kernels or the plain form in elementary
torch operations.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of 256 running requests: the plan of a decode step
        dict(name="plan_decode_256", op="plan", batch=256, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=16384,
             block_size=16, max_len=16400, pad=0, lens_seed=1),
        # decode rows beside prompt chunks of odd sizes, requests without a new token, padded to a graph's size
        dict(name="plan_mixed_600", op="plan", batch=600, new_lo=0, new_hi=57, ctx_lo=0, ctx_hi=32768,
             block_size=64, max_len=33000, pad=515, lens_seed=2),
        # eight long prompts admitted at once
        dict(name="plan_prompts", op="plan", batch=8, new_lo=9000, new_hi=16384, ctx_lo=0, ctx_hi=0,
             block_size=16, max_len=16384, pad=0, lens_seed=3),
        # a decode step's new keys and values, per-tensor scales
        dict(name="append_decode_128", op="append", tokens=128, heads=8, head_dim=128, block_size=16,
             per_token=False, fused_qkv=True, pad=0, lens_seed=4),
        # the new tokens of a long prompt, read out of the fused projection's output
        dict(name="append_prompt_16k", op="append", tokens=16384, heads=8, head_dim=128, block_size=16,
             per_token=False, fused_qkv=True, pad=0, lens_seed=5),
        # per-token scales, head_dim 64, an odd token count and padded rows
        dict(name="append_scales_d64", op="append", tokens=5003, heads=8, head_dim=64, block_size=128,
             per_token=True, fused_qkv=False, pad=117, lens_seed=6),
        # the smallest call: a few tokens of one request on one KV head
        dict(name="chunk_short", op="chunk", batch=1, new_lo=37, new_hi=37, ctx_lo=163, ctx_hi=163, heads=1, group=8,
             head_dim=128, block_size=16, per_token=False, lens_seed=7),
        # a whole prompt without context: the compute-bound end
        dict(name="chunk_prompt_8k", op="chunk", batch=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, heads=8,
             group=8, head_dim=128, block_size=16, per_token=False, lens_seed=8),
        # one chunk of a long document whose earlier chunks are cached
        dict(name="chunk_long_context", op="chunk", batch=1, new_lo=1024, new_hi=1024, ctx_lo=65536, ctx_hi=65536,
             heads=8, group=4, head_dim=128, block_size=64, per_token=False, lens_seed=9),
        # chunked prefill batched with requests that bring a few tokens: ragged, odd group
        dict(name="chunk_ragged_24", op="chunk", batch=24, new_lo=1, new_hi=700, ctx_lo=0, ctx_hi=9000, heads=4,
             group=5, head_dim=128, block_size=16, per_token=False, lens_seed=10),
        # head_dim 64 with per-token scales
        dict(name="chunk_scales_d64", op="chunk", batch=6, new_lo=200, new_hi=1500, ctx_lo=0, ctx_hi=4000, heads=8,
             group=8, head_dim=64, block_size=32, per_token=True, lens_seed=11),
        # one new token for each of 64 requests over long caches: the form for single tokens, bound by bytes
        dict(name="chunk_single_64", op="chunk", batch=64, new_lo=1, new_hi=1, ctx_lo=1023, ctx_hi=16383, heads=8,
             group=8, head_dim=128, block_size=16, per_token=False, lens_seed=12),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "chunk", "chunk"])
    seed = rng.randrange(1 << 30)
    bs = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        while True:
            batch = _logint(rng, 1, 2048)
            new_hi = _logint(rng, 1, 16384)
            if batch * new_hi <= 1 << 18:
                break
        ctx_hi = _logint(rng, 1, 32768)
        return dict(op=op, batch=batch, new_lo=rng.choice([0, 1]), new_hi=new_hi, ctx_lo=0, ctx_hi=ctx_hi,
                    block_size=bs, max_len=ctx_hi + new_hi, pad=rng.choice([0, _logint(rng, 1, 2000)]), lens_seed=seed)
    per_token = rng.random() < 0.5
    head_dim = rng.choice([64, 128, 128])
    if op == "append":
        return dict(op=op, tokens=_logint(rng, 1, 16384), heads=rng.choice([1, 2, 4, 5, 8]), head_dim=head_dim,
                    block_size=bs, per_token=per_token, fused_qkv=rng.random() < 0.5,
                    pad=rng.choice([0, _logint(rng, 1, 500)]), lens_seed=seed)
    while True:
        case = dict(op=op, batch=_logint(rng, 1, 64), new_lo=1, new_hi=_logint(rng, 1, 4096), ctx_lo=0,
                    ctx_hi=_logint(rng, 1, 65536), heads=rng.choice([1, 2, 3, 4, 8]),
                    group=rng.choice([1, 2, 3, 4, 5, 8, 16]), head_dim=head_dim, block_size=bs, per_token=per_token,
                    lens_seed=seed)
        w = work(case)
        # (also bounds the plain form's launches and the cache's size)
        if w["flops"] <= 5e11 and w["bytes"] <= 1.5e9 and case["batch"] * case["new_hi"] <= 40000:
            return case


def _lens(case):
    """(new tokens, cached tokens) of every request."""
    r = random.Random(case["lens_seed"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    return new, ctx


def _blocks(n, bs):
    return (n + bs - 1) // bs


def work(case):
    op = case["op"]
    if op == "plan":
        new, ctx = _lens(case)
        bs = case["block_size"]
        taken = sum(_blocks(c + n, bs) - _blocks(c, bs) for n, c in zip(new, ctx))
        # lengths in; lengths, starts, slots and positions out; the taken ids read and put into the table
        return {"bytes": 16 * case["batch"] + 12 * (sum(new) + case["pad"]) + 8 * taken, "flops": 0}
    if op == "append":
        n = case["tokens"] * case["heads"]
        b = 2 * n * case["head_dim"] * 3 + 8 * (case["tokens"] + case["pad"])
        return {"bytes": b + (8 * n if case["per_token"] else 0), "flops": 2 * n * case["head_dim"]}
    new, ctx = _lens(case)
    d, hk, g = case["head_dim"], case["heads"], case["group"]
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    kv = sum(n + c for n, c in zip(new, ctx)) * hk * (2 * d + (8 if case["per_token"] else 0))
    return {"bytes": kv + 2 * 2 * sum(new) * hk * g * d, "flops": 4 * d * hk * g * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op == "plan":
        new, ctx = _lens(case)
        # another seed gives the same requests other block ids and another order
        order = torch.randperm(case["batch"], generator=g, device="cuda").tolist()
        new, ctx = [new[i] for i in order], [ctx[i] for i in order]
        bs = case["block_size"]
        maxb = _blocks(case["max_len"], bs)
        held = sum(_blocks(c, bs) for c in ctx)
        taken = sum(_blocks(c + n, bs) for c, n in zip(ctx, new)) - held
        ids = torch.randperm(held + taken + 64, generator=g, device="cuda").int()
        col = torch.arange(maxb, device="cuda")
        nb = _i32([_blocks(c, bs) for c in ctx]).long()
        table = torch.full((case["batch"], maxb), -1, dtype=torch.int32, device="cuda")
        table[col[None, :] < nb[:, None]] = ids[:held]
        st.update(new_lens=_i32(new), cached_lens=_i32(ctx), block_table=table, free_blocks=ids[held:].contiguous(),
                  max_tokens=sum(new) + case["pad"])
    elif op == "append":
        t, hk, d, bs = case["tokens"], case["heads"], case["head_dim"], case["block_size"]
        rows = t + case["pad"]
        if case["fused_qkv"]:
            # keys and values as slices of [rows][query heads + 2 Hk][D], two query heads per KV head
            qkv = torch.randn(rows, 4 * hk, d, generator=g, device="cuda").bfloat16()
            k, v = qkv[:, 2 * hk:3 * hk], qkv[:, 3 * hk:]
        else:
            k = torch.randn(rows, hk, d, generator=g, device="cuda").bfloat16()
            v = torch.randn(rows, hk, d, generator=g, device="cuda").bfloat16()
        # a few channels carry keys an order larger, as they do in trained models
        k[:, :, :: max(1, d // 4)] *= 12
        nb = _blocks(t, bs) + 2
        # the pool is as large as the step fills, the blocks in any order
        perm = torch.randperm(nb, generator=g, device="cuda")
        pos = torch.arange(t, device="cuda")
        slot = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        slot[:t] = perm[pos // bs] * bs + pos % bs
        cache = torch.zeros(nb, 2, hk, bs, d, dtype=torch.uint8, device="cuda")
        if case["per_token"]:
            ks = torch.zeros(nb, hk, bs, device="cuda")
            vs = torch.zeros(nb, hk, bs, device="cuda")
        else:
            ks, vs = torch.tensor([0.113], device="cuda"), torch.tensor([0.0101], device="cuda")
        st.update(k=k, v=v, kv_cache=cache, slots=slot, k_scale=ks, v_scale=vs)
    else:
        new, ctx = _lens(case)
        order = torch.randperm(case["batch"], generator=g, device="cuda").tolist()
        new, ctx = [new[i] for i in order], [ctx[i] for i in order]
        hk, grp, d, bs = case["heads"], case["group"], case["head_dim"], case["block_size"]
        tot = [n + c for n, c in zip(new, ctx)]
        used = sum(_blocks(x, bs) for x in tot)
        nb = used + 3
        maxb = max(_blocks(x, bs) for x in tot)
        perm = torch.randperm(nb, generator=g, device="cuda").int()
        table = torch.zeros(case["batch"], maxb, dtype=torch.int32, device="cuda")
        o = 0
        for i, x in enumerate(tot):
            n = _blocks(x, bs)
            table[i, :n] = perm[o:o + n]
            o += n
        cache = torch.empty(nb, 2, hk, bs, d, dtype=torch.uint8, device="cuda")
        if case["per_token"]:
            ks = torch.empty(nb, hk, bs, device="cuda")
            vs = torch.empty(nb, hk, bs, device="cuda")
        else:
            ks, vs = torch.tensor([4.5 / E4M3_MAX], device="cuda"), torch.tensor([5.0 / E4M3_MAX], device="cuda")
        step = max(1, (1 << 27) // (hk * bs * d))
        for b0 in range(0, nb, step):
            b1 = min(nb, b0 + step)
            for kv, sc in ((0, ks), (1, vs)):
                x = torch.randn(b1 - b0, hk, bs, d, generator=g, device="cuda")
                if case["per_token"]:
                    s = x.abs().amax(dim=-1) / E4M3_MAX
                    sc[b0:b1] = s
                    x = x / s[..., None]
                else:
                    x = x / sc
                cache[b0:b1, kv] = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        # queries large enough that the softmax has clear peaks
        q = (1.5 * torch.randn(sum(new), hk * grp, d, generator=g, device="cuda")).bfloat16()
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        st.update(q=q, kv_cache=cache, block_table=table, query_start=_i32(start), seq_lens=_i32(tot), k_scale=ks,
                  v_scale=vs, new=new, tot=tot)
        if own:
            import quantized_paged_attention_gb300 as qpa
            st["desc"] = qpa.chunk_desc(q, cache, table, grp, case["per_token"])
            st["workspace"] = qpa.alloc_workspace(qpa.pa_chunk_fp8_workspace_size(st["desc"]), q.device)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "append": _plain_append, "chunk": _plain_chunk}[state["op"]](state)


def _run_own(s):
    import quantized_paged_attention_gb300 as qpa
    if s["op"] == "plan":
        start, lens, slots, pos, taken = qpa.paged_slot_map(s["new_lens"], s["cached_lens"], s["block_table"],
                                                            s["free_blocks"], s["block_size"], s["max_tokens"])
        return dict(query_start=start, seq_lens=lens, slots=slots, positions=pos, taken=taken,
                    block_table=s["block_table"])
    if s["op"] == "append":
        qpa.kv_append_fp8(s["k"], s["v"], s["kv_cache"], s["slots"], s["k_scale"], s["v_scale"])
        return _append_out(s)
    return qpa.pa_chunk_fp8(s["q"], s["kv_cache"], s["block_table"], s["query_start"], s["seq_lens"], s["k_scale"],
                            s["v_scale"], s["group"], workspace=s["workspace"], desc=s["desc"])


def _append_out(s):
    out = dict(kv_cache=s["kv_cache"].view(torch.float8_e4m3fn))
    if s["per_token"]:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _plain_plan(s):
    new, old, table, free = s["new_lens"].long(), s["cached_lens"].long(), s["block_table"], s["free_blocks"]
    bs, n = s["block_size"], s["max_tokens"]
    zero = torch.zeros(1, dtype=torch.int64, device=new.device)
    start = torch.cat([zero, torch.cumsum(new, 0)])
    nb_old, nb_new = (old + bs - 1) // bs, (old + new + bs - 1) // bs
    base = torch.cat([zero, torch.cumsum(nb_new - nb_old, 0)])
    col = torch.arange(table.shape[1], device=new.device)[None, :]
    src = (base[:-1, None] + col - nb_old[:, None]).clamp(0, free.numel() - 1)
    fresh = (col >= nb_old[:, None]) & (col < nb_new[:, None])
    table.copy_(torch.where(fresh, free[src], table))
    i = torch.arange(n, device=new.device)
    req = torch.searchsorted(start[1:], i, right=True)
    live = req < new.numel()
    req = req.clamp(max=new.numel() - 1)
    pos = old[req] + i - start[req]
    blk = table[req, (pos // bs).clamp(0, table.shape[1] - 1)].long()
    return dict(query_start=start.int(), seq_lens=(old + new).int(),
                slots=torch.where(live, blk * bs + pos % bs, -1),
                positions=torch.where(live, pos, 0).int(), taken=base[-1:].int(), block_table=table)


def _round_e4m3(x):
    """float64 -> the nearest e4m3 value (ties to even, saturating), exact."""
    a = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(a)
    step = torch.exp2(((e - 1).clamp(min=-6) - 3).double())
    r = (torch.round(a / step) * step).clamp(max=E4M3_MAX)
    return torch.copysign(torch.where(x.isnan(), x, r), x).float().to(torch.float8_e4m3fn)


def _plain_append(s):
    cache, slots, bs = s["kv_cache"], s["slots"], s["block_size"]
    rows = torch.nonzero(slots >= 0).flatten()
    blk, off = slots[rows] // bs, slots[rows] % bs
    for kv, (x, sc) in enumerate(((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))):
        x = x[rows]
        if s["per_token"]:
            amax = torch.nan_to_num(x.float().abs(), nan=0.0, posinf=float(torch.finfo(torch.bfloat16).max)).amax(-1)
            # divided in 64 bits: the codes below turn on the stored scale's last bit
            scale = (amax.double() / E4M3_MAX).float().clamp(min=2.0 ** -126)
            sc[blk, :, off] = scale
        else:
            scale = sc[None, :].expand(x.shape[0], x.shape[1])
        cache[blk, kv, :, off] = _round_e4m3(x.double() / scale.double()[..., None]).view(torch.uint8)
    return _append_out(s)


def _plain_chunk(s):
    q, cache, grp, bs = s["q"], s["kv_cache"], s["group"], s["block_size"]
    hk, d = s["heads"], s["head_dim"]
    out = torch.empty_like(q)
    t0 = 0
    for r, (n, tot) in enumerate(zip(s["new"], s["tot"])):
        if n == 0:
            continue
        blk = s["block_table"][r, :_blocks(tot, bs)].long()
        page = cache[blk].view(torch.float8_e4m3fn).float()                  # [blocks, 2, Hk, bs, D]
        if s["per_token"]:
            page[:, 0] *= s["k_scale"][blk][..., None]
            page[:, 1] *= s["v_scale"][blk][..., None]
        else:
            page[:, 0] *= s["k_scale"]
            page[:, 1] *= s["v_scale"]
        kv = page.permute(1, 2, 0, 3, 4).reshape(2, hk, -1, d)[:, :, :tot]
        rows = max(1, (1 << 29) // (hk * grp * tot))
        for a in range(0, n, rows):
            b = min(n, a + rows)
            qr = q[t0 + a:t0 + b].float().view(b - a, hk, grp, d).permute(1, 2, 0, 3)
            see = tot - n + b                                                  # the block's last row sees so many
            sc = torch.matmul(qr.reshape(hk, -1, d), kv[0, :, :see].transpose(1, 2)) * (1.0 / math.sqrt(d))
            sc = sc.view(hk, grp, b - a, see)
            lim = torch.arange(tot - n + a, tot - n + b, device=q.device)
            mask = torch.arange(see, device=q.device)[None, :] > lim[:, None]
            sc.masked_fill_(mask, float("-inf"))
            p = torch.exp(sc - sc.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(hk, -1, see), kv[1, :, :see]).view(hk, grp, b - a, d)
            out[t0 + a:t0 + b] = o.permute(2, 0, 1, 3).reshape(b - a, hk * grp, d).to(out.dtype)
        t0 += n
    return out


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    bs = case["block_size"]
    if case["op"] == "plan":
        new, old = s["new_lens"].tolist(), s["cached_lens"].tolist()
        table, free = s["block_table"].tolist(), s["free_blocks"].tolist()
        start, slots, pos, k = [0], [], [], 0
        for r, (n, c) in enumerate(zip(new, old)):
            for e in range(_blocks(c, bs), _blocks(c + n, bs)):
                table[r][e] = free[k]
                k += 1
            for p in range(c, c + n):
                slots.append(table[r][p // bs] * bs + p % bs)
                pos.append(p)
            start.append(start[-1] + n)
        pad = s["max_tokens"] - len(slots)
        return dict(query_start=_i32(start), seq_lens=_i32([a + b for a, b in zip(new, old)]),
                    slots=torch.tensor(slots + [-1] * pad, dtype=torch.int64, device="cuda"),
                    positions=_i32(pos + [0] * pad), taken=_i32([k]), block_table=_i32(table))
    if case["op"] == "append":
        # the nearest of the 127 non-negative e4m3 values, found among their borders
        code = torch.arange(127, device="cuda")
        e, m = code // 8, (code % 8).double()
        val = torch.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
        mid = (val[1:] + val[:-1]) / 2
        t = s["slots"]
        out = s["kv_cache"].view(torch.float8_e4m3fn).double()
        scales = [s["k_scale"].double(), s["v_scale"].double()]
        live = [i for i, x in enumerate(t.tolist()) if x >= 0]
        blk, off = t[live] // bs, t[live] % bs
        for kv, x in enumerate((s["k"], s["v"])):
            x = x[live].double()
            sc = scales[kv]
            if case["per_token"]:
                row = x.abs().max(dim=-1).values / 448
                sc[blk, :, off] = row
                # the codes are relative to the scale as it is stored, in 32 bits
                x = x / row.float().double()[:, :, None]
            else:
                x = x / sc
            a = x.abs()
            lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
            idx = torch.where((lo != hi) & (lo % 2 == 0), lo, hi)              # a tie goes to the even code
            out[blk, kv, :, off] = torch.copysign(val[idx], x)
        res = dict(kv_cache=out)
        if case["per_token"]:
            res.update(k_scale=scales[0], v_scale=scales[1])
        return res
    if work(case)["flops"] > 2.5e12:
        return None
    # one (request, KV head, block of rows) after another
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pool = s["kv_cache"].view(torch.float8_e4m3fn)
    first = 0
    grp, d = case["group"], case["head_dim"]
    for r in range(case["batch"]):
        n, tot = s["new"][r], s["tot"][r]
        ids = torch.arange(tot, device="cuda")
        blk, off = s["block_table"][r].long()[ids // bs], ids % bs
        for h in range(case["heads"]):
            k, v = pool[blk, 0, h, off].double(), pool[blk, 1, h, off].double()
            if case["per_token"]:
                k = k * s["k_scale"][blk, h, off].double()[:, None]
                v = v * s["v_scale"][blk, h, off].double()[:, None]
            else:
                k, v = k * s["k_scale"].double(), v * s["v_scale"].double()
            step = max(1, (1 << 28) // (tot * grp))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                last = tot - n + i1
                qq = s["q"][first + i0:first + i1, h * grp:(h + 1) * grp].double()
                logit = torch.einsum("igd,td->igt", qq, k[:last]) / d ** 0.5
                seen = ids[:last][None, :] <= torch.arange(tot - n + i0, last, device="cuda")[:, None]
                logit = logit.masked_fill(~seen[:, None, :], -math.inf)
                w = torch.softmax(logit, dim=-1)
                out[first + i0:first + i1, h * grp:(h + 1) * grp] = torch.einsum("igt,td->igd", w, v[:last])
        first += n
    return out
