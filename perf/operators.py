"""Measured cases of the attention token mixer: the page plan of a serving step, the cache append,
attention of new tokens over a paged cache, and attention over whole packed prompts.

Each operator has a plain form (elementary torch operations in FP32), the framework's call (where
`own` is set) and a definition in 64 bits (`exact`). Head layouts: 32 query heads on 8 key/value heads
of 128 is a common grouped layout; 24 on 4 of 256 is the 6144-wide token mixer with 64 KiB of FP16 keys
and values per position over 16 attention layers; 16 on 2 of 64 a small one.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _plan(name, requests, ctx, new, page, lens):
    return {"name": name, "op": "plan", "requests": requests, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "chunk": 0, "page": page, "lens": lens}


def _append(name, tokens, kv_heads, dim, page, dtype):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype}


def _paged(name, requests, ctx, new, chunk, heads, kv_heads, dim, page, dtype, lens):
    return {"name": name, "op": "paged", "requests": requests, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "chunk": chunk, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype, "lens": lens}


def _prompt(name, requests, new, chunk, heads, kv_heads, dim, dtype, lens):
    return {"name": name, "op": "prompt", "requests": requests, "ctx_lo": 0, "ctx_hi": 0, "new_lo": new[0],
            "new_hi": new[1], "chunk": chunk, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "lens": lens}


def listed():
    return [
        # four requests verify eight speculated tokens each: the smallest step, where latency counts
        _plan("plan_verify", 4, (1000, 30000), (8, 8), 64, 1),
        # a large server step: hundreds of decodes and short prompts admitted together
        _plan("plan_wave", 700, (0, 12000), (1, 181), 16, 2),
        # the keys and values of one verify step of eight requests
        _append("append_verify", 64, 4, 256, 64, "f16"),
        # a wave of prompts: 16K tokens of 8 x 128
        _append("append_wave", 16411, 8, 128, 16, "bf16"),
        # one user, one token, a short context: latency
        _paged("decode_one", 1, (4097, 4097), (1, 1), 0, 24, 4, 256, 64, "f16", 3),
        # 64 users decoding, ragged contexts up to 16K
        _paged("decode_batch", 64, (700, 16384), (1, 1), 0, 32, 8, 128, 16, "bf16", 4),
        # 16 users verify eight speculated tokens each
        _paged("verify_batch", 16, (2000, 32768), (8, 8), 0, 24, 4, 256, 64, "f16", 5),
        # a 64-row prefill chunk behind 96K tokens of context
        _paged("chunk64_96k", 1, (98304, 98304), (64, 64), 0, 24, 4, 256, 128, "f16", 6),
        # one prompt's chunk scheduled together with decoding users
        _paged("chunk_mixed", 16, (300, 6000), (1, 1), 1024, 32, 8, 128, 32, "f16", 7),
        # short chat turns packed together, small heads
        _prompt("prompt_packed", 24, (1, 700), 0, 16, 2, 64, "bf16", 8),
        # one whole long prompt
        _prompt("prompt_long", 1, (8192, 8192), 0, 32, 8, 128, "bf16", 9),
        # a few ragged prompts with wide heads
        _prompt("prompt_wide", 3, (900, 2500), 5003, 24, 4, 256, "f16", 10),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["plan", "append", "paged", "paged", "prompt"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8]) if dim < 256 else rng.choice([1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    lens = rng.randrange(1 << 20)
    if op == "plan":
        lo = rng.choice([0, 1, 500])
        new = _spread(rng, 1, 150)
        c = _plan("", _spread(rng, 1, 800), (lo, lo + _spread(rng, 1, 12000)), (rng.choice([1, new]), new), page, lens)
    elif op == "append":
        c = _append("", _spread(rng, 1, 16384), kv_heads, dim, page, dtype)
    elif op == "paged":
        kind = rng.choice(["decode", "verify", "chunk"])
        if kind == "chunk":
            requests, ctx, new, chunk = _spread(rng, 1, 6), (1, _spread(rng, 1, 6000)), (1, 1), _spread(rng, 33, 1024)
        else:
            requests = _spread(rng, 1, 48)
            ctx = (1, _spread(rng, 1, 12000))
            new, chunk = ((1, 1) if kind == "decode" else (2, rng.choice([4, 8, 16]))), 0
        c = _paged("", requests, ctx, new, chunk, kv_heads * group, kv_heads, dim, page, dtype, lens)
    else:
        most = _spread(rng, 1, 2048)
        requests = max(1, min(_spread(rng, 1, 24), 8192 // most))
        c = _prompt("", requests, (1, most), 0, kv_heads * group, kv_heads, dim, dtype, lens)
    c.pop("name")
    return c


def _lengths(case):
    """(cached, new) tokens of each request, from the case alone."""
    rng = random.Random(case["lens"])
    lo, hi = case["ctx_lo"], case["ctx_hi"]
    cached = [lo if lo == hi else max(lo, _spread(rng, max(lo, 1), hi) - (1 if lo == 0 else 0))
              for _ in range(case["requests"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    if case["chunk"]:
        new[0] = case["chunk"]
    return cached, new


def _ceil(a, b):
    return -(-a // b)


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * gain).to(TYPES[case["dtype"]])

    if case["op"] == "append":
        T, page = case["tokens"], case["page"]
        n_pages = _ceil(T, page) + 7
        shape = (n_pages, page, case["kv_heads"], case["dim"])
        # the tokens of a step fill whole pages here and there in the cache, the last one partly
        pages = torch.randperm(n_pages, generator=g, device=DEV)[:_ceil(T, page)]
        at = torch.arange(T, device=DEV)
        return {"case": case, "k": normal(T, case["kv_heads"], case["dim"]), "v": normal(T, case["kv_heads"], case["dim"]),
                "slots": pages[at // page] * page + at % page, "k_pages": normal(*shape), "v_pages": normal(*shape)}

    cached, new = _lengths(case)
    total = sum(new)
    if case["op"] == "prompt":
        return {"case": case, "q": normal(total, case["heads"], case["dim"], gain=1.5),
                "k": normal(total, case["kv_heads"], case["dim"]), "v": normal(total, case["kv_heads"], case["dim"]),
                "q_start": _ints(_starts(new)), "max_new": max(new), "max_kv": max(new)}

    page = case["page"]
    held = [_ceil(c, page) for c in cached]
    need = [_ceil(c + n, page) for c, n in zip(cached, new)]
    have = held if case["op"] == "plan" else need
    n_pages = sum(need) + 9
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    width = max(need) + 1
    # entries of a table row behind its pages hold nothing of use
    col = torch.arange(width, device=DEV)[None]
    first = _ints(_starts(have)[:-1], torch.int64)[:, None]
    inside = col < _ints(have, torch.int64)[:, None]
    table = torch.where(inside, order[(first + col).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    if case["op"] == "plan":
        # the free pages sit in a ring, from its fifth entry before the end on
        free, head = n_pages - sum(held), n_pages - 5
        ring = order.roll(head - sum(held))
        state = _ints([head, free])
        return {"case": case, "cached": _ints(cached), "new": _ints(new), "table": table, "ring": ring,
                "ring_state": state, "max_tokens": total + 13, "page": page}
    shape = (n_pages, page, case["kv_heads"], case["dim"])
    return {"case": case, "q": normal(total, case["heads"], case["dim"], gain=1.5), "k_pages": normal(*shape),
            "v_pages": normal(*shape), "table": table, "q_start": _ints(_starts(new)),
            "kv_len": _ints([c + n for c, n in zip(cached, new)]), "max_new": max(new),
            "max_kv": max(c + n for c, n in zip(cached, new))}


def _plan_plain(s):
    """Pages for the new tokens from the ring of free pages, in request order; where every token goes."""
    cached, new, page, width = s["cached"].long(), s["new"].long(), s["page"], s["table"].shape[1]
    table, ring = s["table"], s["ring"].long()
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)])
    held, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    take = (need - held).cumsum(0)
    col = torch.arange(width, device=DEV)[None]
    k = (take - (need - held))[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    table.copy_(torch.where(fresh, ring[(s["ring_state"][0] + k) % ring.shape[0]].to(torch.int32), table))
    t = torch.arange(s["max_tokens"], device=DEV)
    r = torch.searchsorted(q_start[1:], t, right=True)
    live = r < new.shape[0]
    r = r.clamp(max=new.shape[0] - 1)
    pos = torch.where(live, cached[r] + t - q_start[r], 0)
    slot = table[r, pos // page].long() * page + pos % page
    state = torch.stack([(s["ring_state"][0] + take[-1]) % ring.shape[0], s["ring_state"][1] - take[-1]])
    return {"table": table, "q_start": q_start.to(torch.int32), "kv_len": (cached + new).to(torch.int32),
            "slots": torch.where(live, slot, -1), "positions": torch.where(live, pos, -1).to(torch.int32),
            "ring_state": state.to(torch.int32)}


def _append_plain(s):
    for pages, rows in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
        pages.view(-1, *pages.shape[2:])[s["slots"]] = rows
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attend(q, k, v, q_start, kv_len, max_new):
    """Causal attention of packed query rows q [T][H][D], the last of each request's keys k, v
    [R][L][Hkv][D] (FP32): row i of request r sees its keys 0 .. kv_len - new + i."""
    T, H, D = q.shape
    R, L, Hkv, _ = k.shape
    new = q_start[1:] - q_start[:-1]
    i = torch.arange(max_new, device=DEV)
    rows = (q_start[:-1, None] + i).clamp(max=T - 1)
    qp = q.float()[rows].view(R, max_new, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)  # [R][Hkv][G][F][D]
    s = torch.matmul(qp, k.permute(0, 2, 3, 1)[:, :, None]).mul_(1.0 / math.sqrt(D))  # [R][Hkv][G][F][L]
    last = (kv_len - new)[:, None] + i
    seen = torch.arange(L, device=DEV) <= last.clamp(max=L)[..., None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]) / total
    lse = (m + total.log())[..., 0]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    at = t - q_start[r]
    return {"out": o[r, :, :, at].reshape(T, H, D).to(q.dtype), "lse": lse[r, :, :, at].reshape(T, H)}


def _paged_plain(s):
    page = s["k_pages"].shape[1]
    table = s["table"][:, : _ceil(s["max_kv"], page)].long().clamp(min=0)
    k, v = (x[table].float().flatten(1, 2) for x in (s["k_pages"], s["v_pages"]))
    return _attend(s["q"], k, v, s["q_start"].long(), s["kv_len"].long(), s["max_new"])


def _prompt_plain(s):
    start = s["q_start"].long()
    rows = (start[:-1, None] + torch.arange(s["max_kv"], device=DEV)).clamp(max=s["k"].shape[0] - 1)
    return _attend(s["q"], s["k"].float()[rows], s["v"].float()[rows], start, start[1:] - start[:-1], s["max_new"])


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "paged": _paged_plain, "prompt": _prompt_plain}[op](s)
    from bit_vector_lut_gb300 import vq3
    if op == "plan":
        p = vq3.paged_plan(s["cached"], s["new"], s["table"], s["ring"], s["ring_state"], s["page"], s["max_tokens"])
        return {"table": s["table"], "q_start": p.q_start, "kv_len": p.kv_len, "slots": p.slots,
                "positions": p.positions, "ring_state": p.ring_state}
    if op == "append":
        vq3.kv_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    if op == "paged":
        out = vq3.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"], s["kv_len"],
                                  max_new=s["max_new"], lse=lse)
    else:
        out = vq3.prompt_attention(s["q"], s["k"], s["v"], s["q_start"], max_new=s["max_new"], lse=lse)
    return {"out": out, "lse": lse}


def work(case):
    if case["op"] == "append":
        row = case["kv_heads"] * case["dim"] * 2
        return {"bytes": case["tokens"] * (4 * row + 8), "flops": 0}
    cached, new = _lengths(case)
    total, R = sum(new), case["requests"]
    if case["op"] == "plan":
        fresh = sum(_ceil(c + n, case["page"]) - _ceil(c, case["page"]) for c, n in zip(cached, new))
        return {"bytes": 4 * (4 * R + 1 + 2 * fresh + 4) + 12 * (total + 13), "flops": 0}
    rows = 2 * case["dim"]
    kv = sum(c + n for c, n in zip(cached, new))
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    read = kv * case["kv_heads"] * 2 * rows + 4 * (2 * R + 1)
    if case["op"] == "paged":
        read += 4 * sum(_ceil(c + n, case["page"]) for c, n in zip(cached, new))
    return {"bytes": read + total * case["heads"] * (2 * rows + 4), "flops": 4 * case["dim"] * case["heads"] * seen}


def exact(case, seed):
    """Attention from its definition, one request and head at a time, in FP64; what only moves or counts has none."""
    if case["op"] in ("plan", "append"):
        return None
    s = prepare(case, seed)
    cached, new = _lengths(case)
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    out = torch.empty(sum(new), H, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(sum(new), H, dtype=torch.float64, device=DEV)
    t0 = 0
    for r in range(case["requests"]):
        n, length = new[r], cached[r] + new[r]
        if case["op"] == "paged":
            pages = s["table"][r, : _ceil(length, case["page"])].long()
            keys, values = (s[x][pages].flatten(0, 1)[:length] for x in ("k_pages", "v_pages"))
        else:
            keys, values = s["k"][t0 : t0 + n], s["v"][t0 : t0 + n]
        last = torch.arange(length - n, length, device=DEV)
        hidden = torch.arange(length, device=DEV)[None] > last[:, None]
        for h in range(H):
            kv = h // (H // Hkv)
            x = s["q"][t0 : t0 + n, h].double() @ keys[:, kv].double().T / D**0.5
            x[hidden] = -math.inf
            top = torch.logsumexp(x, 1)
            lse[t0 : t0 + n, h] = top
            out[t0 : t0 + n, h] = (x - top[:, None]).exp() @ values[:, kv].double()
        t0 += n
    return {"out": out, "lse": lse}
