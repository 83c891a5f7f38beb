"""Measured cases of the hybrid decoder's serving path beside attention: the gated delta rule over packed
requests with their states in slots, the short convolution in front of it, and the append of rotated keys and
values to the paged cache.

Each operator has a plain form (elementary torch operations in FP32, the rotation's angles in FP64), the
framework's call (where `own` is set) and a definition in 64 bits (`exact`). Head layouts: 48 value heads on 16
query/key heads of 128 x 128 is the 6144-wide delta-rule mixer (10240 channels of convolution), 24 query heads
on 4 key/value heads of 256 its attention counterpart; 32 on 8 of 128 a common grouped layout; the others are
small generic ones.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 64  # tokens a step of the plain delta rule


def _delta(name, requests, new, qk_heads, v_heads, d_k, d_v, dtype, lens, chunk=0):
    return {"name": name, "op": "delta", "requests": requests, "new_lo": new[0], "new_hi": new[1], "chunk": chunk,
            "qk_heads": qk_heads, "v_heads": v_heads, "d_k": d_k, "d_v": d_v, "dtype": dtype, "lens": lens}


def _conv(name, requests, new, channels, width, unit_heads, head_dim, bias, dtype, lens):
    return {"name": name, "op": "conv", "requests": requests, "new_lo": new[0], "new_hi": new[1], "chunk": 0,
            "channels": channels, "width": width, "unit_heads": unit_heads, "head_dim": head_dim, "bias": bias,
            "dtype": dtype, "lens": lens}


def _rotary(name, requests, new, ctx, pad, heads, kv_heads, dim, rotated, interleaved, page, dtype, lens):
    return {"name": name, "op": "rotary", "requests": requests, "new_lo": new[0], "new_hi": new[1], "chunk": 0,
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "pad": pad, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotated": rotated, "interleaved": interleaved, "page": page, "dtype": dtype, "lens": lens}


def listed():
    return [
        # one user, one token, a small mixer: latency
        _delta("delta_one", 1, (1, 1), 4, 8, 64, 64, "f16", 1),
        # 64 users decoding
        _delta("delta_decode", 64, (1, 1), 16, 48, 128, 128, "bf16", 2),
        # 16 users verify eight speculated tokens each
        _delta("delta_verify", 16, (8, 8), 16, 48, 128, 128, "f16", 3),
        # one prompt's chunk scheduled together with decoding users
        _delta("delta_mixed", 24, (1, 1), 16, 48, 128, 128, "bf16", 4, chunk=1003),
        # a wave of ragged prompts
        _delta("delta_wave", 16, (1, 1100), 16, 48, 128, 128, "f16", 5),
        # one whole long prompt
        _delta("delta_long", 1, (8192, 8192), 16, 48, 128, 128, "bf16", 6),
        # the convolution of 64 decoding users
        _conv("conv_decode", 64, (1, 1), 10240, 4, 32, 128, False, "bf16", 7),
        # and of a wave of ragged prompts
        _conv("conv_wave", 16, (1, 1100), 10240, 4, 32, 128, False, "f16", 8),
        # a verify step of four users, a quarter of each head rotated, far positions
        _rotary("rotary_verify", 4, (8, 8), (90000, 190000), 5, 24, 4, 256, 64, False, 64, "f16", 9),
        # a wave of prompts, whole heads rotated
        _rotary("rotary_wave", 11, (300, 2500), (0, 0), 13, 32, 8, 128, 128, False, 16, "bf16", 10),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "conv", "rotary"])
    dtype = rng.choice(["f16", "bf16"])
    lens = rng.randrange(1 << 20)
    if op == "delta":
        d_k, d_v = rng.choice([64, 128, 128, 256]), rng.choice([48, 64, 128, 128, 256])
        qk = rng.choice([1, 2, 5, 8, 16])
        v = qk * rng.choice([1, 2, 3])
        kind = rng.choice(["decode", "verify", "prompts", "mixed"])
        room = (48 << 14) / (v * d_k * d_v)  # the largest listed mixer against this one
        total = int(7000 * min(1, room))
        chunk = 0
        if kind == "decode":
            requests, new = _spread(rng, 1, max(1, min(int(60 * room), 400))), (1, 1)
        elif kind == "verify":
            requests, new = _spread(rng, 1, max(1, min(int(40 * room), 200))), (2, rng.choice([3, 4, 8, 16]))
        elif kind == "prompts":
            longest = _spread(rng, 20, min(6000, total))
            requests, new = max(1, min(_spread(rng, 1, 24), total // longest)), (1, longest)
        else:
            requests, new, chunk = _spread(rng, 2, max(2, min(int(24 * room), 40))), (1, 1), _spread(rng, 20, min(2048, total))
        c = _delta("", requests, new, qk, v, d_k, d_v, dtype, lens, chunk)
    elif op == "conv":
        head_dim = rng.choice([64, 128])
        units = rng.choice([0, 2, 10, 32])
        channels = units * head_dim + 8 * _spread(rng, 8, 1024)
        kind = rng.choice(["decode", "prompts"])
        longest = 1 if kind == "decode" else _spread(rng, 4, 6000)
        requests = _spread(rng, 1, 300) if kind == "decode" else max(1, min(_spread(rng, 1, 40), 7000 // longest))
        c = _conv("", requests, (1, longest), channels, rng.choice([2, 3, 4, 4]), units, head_dim, rng.random() < 0.5,
                  dtype, lens)
    else:
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8]) if dim < 256 else rng.choice([1, 2, 4])
        kind = rng.choice(["decode", "prompts"])
        longest = rng.choice([1, 1, 4, 8]) if kind == "decode" else _spread(rng, 16, 4000)
        requests = _spread(rng, 1, 200) if kind == "decode" else max(1, min(_spread(rng, 1, 24), 8000 // longest))
        rotated = rng.choice([x for x in (32, 48, 64, 96, 128, 256) if x <= dim])
        c = _rotary("", requests, (1, longest), (0, _spread(rng, 1, 200000)) if kind == "decode" else (0, 0),
                    rng.choice([0, 3]), kv_heads * rng.choice([1, 2, 4, 6, 8]), kv_heads, dim, rotated,
                    rng.random() < 0.4, rng.choice([16, 32, 64, 128, 256]), dtype, lens)
    c.pop("name")
    return c


def _lengths(case):
    """New tokens of each request, from the case alone."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    if case["chunk"]:
        new[len(new) // 2] = case["chunk"]
    return new


def _cached(case):
    """Tokens that each request has in the cache already."""
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["requests"])]


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, new, R = TYPES[case["dtype"]], _lengths(case), case["requests"]
    T = sum(new)

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * gain).to(dtype)

    s = {"case": case, "q_start": _ints(_starts(new)), "max_new": max(new)}
    if case["op"] != "rotary":
        # every request goes on from its slot of a pool that has a few more
        slots = torch.randperm(R + 2, generator=g, device=DEV)[:R].to(torch.int32)
        s |= {"slots": slots, "tokens": T}
    if case["op"] == "delta":
        H, G, dk, dv = case["v_heads"], case["qk_heads"], case["d_k"], case["d_v"]
        # one buffer of rows, as the convolution leaves it: queries and keys of unit length, then values
        rows = torch.randn(T, 2 * G * dk + H * dv, generator=g, device=DEV)
        heads = rows[:, : 2 * G * dk].view(T, 2 * G, dk)
        heads /= heads.norm(dim=-1, keepdim=True)
        rows = rows.to(dtype)
        q, k, v = rows.split([G * dk, G * dk, H * dv], 1)
        # per head a decay that lasts for some 2 to 1000 tokens, gates around one half
        span = torch.exp(torch.rand(H, generator=g, device=DEV) * math.log(500.0)) * 2
        alpha = torch.exp(-2 * torch.rand(T, H, generator=g, device=DEV) / span)
        s |= {"q": q.view(T, G, dk), "k": k.view(T, G, dk), "v": v.view(T, H, dv), "alpha": alpha,
              "beta": torch.sigmoid(torch.randn(T, H, generator=g, device=DEV)),
              "states": torch.randn(R + 2, H, dk, dv, generator=g, device=DEV) * 0.1}
    elif case["op"] == "conv":
        C, W = case["channels"], case["width"]
        s |= {"x": normal(T, C), "weight": normal(C, W, gain=0.5), "bias": normal(C) if case["bias"] else None,
              "states": normal(R + 2, W - 1, C)}
    else:
        page, P, cached = case["page"], T + case["pad"], _cached(case)
        need = [-(-(c + n) // page) for c, n in zip(cached, new)]
        first = [c // page for c in cached]
        # the pages that the step writes, anywhere in the cache; rows behind the last request have no slot
        pages = sum(n - f for n, f in zip(need, first))
        order = torch.randperm(pages + 5, generator=g, device=DEV)
        slots = torch.full((P,), -1, dtype=torch.int64, device=DEV)
        positions = torch.full((P,), -1, dtype=torch.int32, device=DEV)
        at, t = 0, 0
        for c, n, f, e in zip(cached, new, first, need):
            x = torch.arange(c, c + n, device=DEV)
            positions[t : t + n] = x
            slots[t : t + n] = order[at + x // page - f] * page + x % page
            at, t = at + e - f, t + n
        shape = (pages + 5, page, case["kv_heads"], case["dim"])
        half = case["rotated"] // 2
        s |= {"q": normal(P, case["heads"], case["dim"]), "k": normal(P, case["kv_heads"], case["dim"]),
              "v": normal(P, case["kv_heads"], case["dim"]), "slots": slots, "positions": positions,
              "freq": (1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float(),
              "k_pages": normal(*shape), "v_pages": normal(*shape),
              "q_out": torch.zeros(P, case["heads"], case["dim"], dtype=dtype, device=DEV)}
    return s


def _delta_plain(s):
    """Chunks of 64 tokens, every request's in step: with g_i the product of the gates up to token i,
    U = (I + N)^-1 (V - g K S), N[i][j] = g_i / g_j b_j k_i . k_j below the diagonal, solved row by row for all
    chunks at once; then chunk by chunk O = g Q S + M U and S <- g_C S + K^T (b g_C / g_j U)."""
    case, starts, T = s["case"], s["q_start"].long(), s["tokens"]
    H, G, R = case["v_heads"], case["qk_heads"], case["requests"]
    C = min(CHUNK, s["max_new"])
    n_chunks = -(-s["max_new"] // C)
    L = n_chunks * C
    at = starts[:-1, None] + torch.arange(L, device=DEV)
    live = at < starts[1:, None]
    rows = at.clamp(max=T - 1)

    def padded(x, fill):  # [R][H][chunks][C][..]
        x = torch.where(live.view(R, L, *[1] * (x.dim() - 1)), x[rows].float(), fill)
        x = x.repeat_interleave(H // x.shape[2], 2)
        return x.transpose(1, 2).reshape(R, H, n_chunks, C, *x.shape[3:])

    q, k, v = padded(s["q"], 0.0), padded(s["k"], 0.0), padded(s["v"], 0.0)
    beta, log = padded(s["beta"], 0.0), padded(s["alpha"], 1.0).double().log().cumsum(-1)
    ratio = (log[..., :, None] - log[..., None, :]).exp().float().tril()  # g_i / g_j
    gate, left = log.exp().float()[..., None], (log[..., -1:] - log).exp().float()[..., None]
    N = (ratio * beta[..., None, :] * (k @ k.mT)).tril(-1)
    M = ratio * beta[..., None, :] * (q @ k.mT) * case["d_k"] ** -0.5
    inverse = torch.eye(C, device=DEV).expand_as(N).clone()
    for i in range(1, C):
        inverse[..., i, :] -= (N[..., i, None, :i] @ inverse[..., :i, :])[..., 0, :]
    S = s["states"][s["slots"].long()]
    outs = []
    for c in range(n_chunks):
        u = inverse[:, :, c] @ (v[:, :, c] - gate[:, :, c] * (k[:, :, c] @ S))
        outs.append(gate[:, :, c] * (q[:, :, c] @ S) * case["d_k"] ** -0.5 + M[:, :, c] @ u)
        S = gate[:, :, c, -1:] * S + (k[:, :, c] * (left * beta[..., None])[:, :, c]).mT @ u
    s["states"][s["slots"].long()] = S
    o = torch.stack(outs, 2).reshape(R, H, L, -1).transpose(1, 2)
    return {"out": o[live].to(s["v"].dtype), "states": s["states"]}


def _conv_plain(s):
    """y_t = silu(bias + sum_j w_j x_(t - W + 1 + j)), the inputs before a request's first from its slot."""
    case, starts, W, T = s["case"], s["q_start"].long(), s["case"]["width"], s["tokens"]
    x, at = s["x"].float(), torch.arange(T, device=DEV)
    old = s["states"][s["slots"].long()]
    r = torch.searchsorted(starts[1:].contiguous(), at, right=True)
    back = W - 1 - torch.arange(W, device=DEV)
    src = at[:, None] - back
    before = src < starts[r][:, None]
    y = torch.zeros_like(x) if s["bias"] is None else s["bias"].float().expand_as(x).clone()
    for j in range(W):
        row = (W - 1 + src[:, j] - starts[r]).clamp(min=0, max=W - 2)
        taps = torch.where(before[:, j, None], old[r, row].float(), x[src[:, j].clamp(min=0)])
        y += s["weight"][:, j].float() * taps
    y = y / (1 + torch.exp(-y))
    d = case["unit_heads"] * case["head_dim"]
    if d:
        heads = y[:, :d].view(T, case["unit_heads"], case["head_dim"])
        heads *= (heads.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
    src = starts[1:, None] - (W - 1) + torch.arange(W - 1, device=DEV)
    row = (src - starts[:-1, None] + W - 1).clamp(min=0, max=W - 2)
    kept = torch.where((src < starts[:-1, None])[..., None], old.gather(1, row[..., None].expand_as(old)),
                       s["x"][src.clamp(min=0)])
    s["states"][s["slots"].long()] = kept
    return {"out": y.to(s["x"].dtype), "states": s["states"]}


def _rotate_plain(x, cos, sin, interleaved):
    half = cos.shape[-1]
    y = x.float().clone()
    a, b = (y[..., : 2 * half : 2], y[..., 1 : 2 * half : 2]) if interleaved else (y[..., :half], y[..., half : 2 * half])
    c, s = cos[:, None], sin[:, None]
    first, second = a * c - b * s, b * c + a * s
    a.copy_(first)
    b.copy_(second)
    return y.to(x.dtype)


def _rotary_plain(s):
    live = s["positions"] >= 0
    angle = s["positions"][live].double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"][live] = _rotate_plain(s["q"][live], cos, sin, s["case"]["interleaved"])
    slots = s["slots"][live]
    for pages, rows in ((s["k_pages"], _rotate_plain(s["k"][live], cos, sin, s["case"]["interleaved"])),
                        (s["v_pages"], s["v"][live])):
        pages.view(-1, *pages.shape[2:])[slots] = rows
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(s):
    case = s["case"]
    if not own:
        return {"delta": _delta_plain, "conv": _conv_plain, "rotary": _rotary_plain}[case["op"]](s)
    from bit_vector_lut_gb300 import vq3
    if case["op"] == "delta":
        out = vq3.delta_rule_batch(s["q"], s["k"], s["v"], s["beta"], s["alpha"], s["states"], s["q_start"], s["slots"],
                                   s["slots"], max_new=s["max_new"], scale=case["d_k"] ** -0.5)
        return {"out": out, "states": s["states"]}
    if case["op"] == "conv":
        out = vq3.short_conv(s["x"], s["weight"], s["states"], s["q_start"], s["slots"], s["slots"], bias=s["bias"],
                             unit_heads=case["unit_heads"], head_dim=case["head_dim"])
        return {"out": out, "states": s["states"]}
    vq3.kv_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["k_pages"], s["v_pages"],
                         interleaved=case["interleaved"], q_out=s["q_out"])
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def work(case):
    T, R = sum(_lengths(case)), case["requests"]
    if case["op"] == "delta":
        H, dk, dv = case["v_heads"], case["d_k"], case["d_v"]
        rows = 2 * T * (2 * case["qk_heads"] * dk + 2 * H * dv) + 8 * T * H
        return {"bytes": rows + 8 * R * H * dk * dv + 4 * (3 * R + 1), "flops": 6 * T * H * dk * dv}
    if case["op"] == "conv":
        C, W = case["channels"], case["width"]
        return {"bytes": 4 * T * C + 2 * C * (W + case["bias"]) + 4 * R * (W - 1) * C + 4 * (3 * R + 1),
                "flops": 2 * T * C * W}
    row = 2 * case["dim"]
    return {"bytes": T * (2 * row * (case["heads"] + 2 * case["kv_heads"]) + 12) + 12 * case["pad"] + 2 * case["rotated"],
            "flops": 3 * T * (case["heads"] + case["kv_heads"]) * case["rotated"]}


def _delta_exact(s, new):
    case = s["case"]
    H, R = case["v_heads"], case["requests"]
    group = H // case["qk_heads"]
    pool = s["states"].double()
    S = pool[s["slots"].long()]  # [R][H][dk][dv]
    out = torch.empty(s["tokens"], H, case["d_v"], dtype=torch.float64, device=DEV)
    first = _starts(new)
    order = sorted(range(R), key=lambda r: -new[r])  # the requests that are still going come first
    S = S[torch.tensor(order, device=DEV)]
    for i in range(max(new)):
        going = [r for r in order if new[r] > i]
        m, t = len(going), torch.tensor([first[r] + i for r in going], device=DEV)
        q, k = (s[x][t].double().repeat_interleave(group, 1) for x in ("q", "k"))
        a, b, now = s["alpha"][t].double(), s["beta"][t].double(), S[:m]
        now *= a[..., None, None]
        u = b[..., None] * (s["v"][t].double() - torch.einsum("rhkv,rhk->rhv", now, k))
        now += k[..., None] * u[..., None, :]
        out[t] = torch.einsum("rhkv,rhk->rhv", now, q) * case["d_k"] ** -0.5
    pool[s["slots"].long()[torch.tensor(order, device=DEV)]] = S
    return {"out": out, "states": pool}


def _conv_exact(s, new):
    case = s["case"]
    W, pool, outs, t = case["width"], s["states"].double(), [], 0
    w, kept = s["weight"].double(), s["states"].double()
    for r, n in enumerate(new):
        slot = int(s["slots"][r])
        line = torch.cat([pool[slot], s["x"][t : t + n].double()])  # [W - 1 + n][C]
        y = sum(w[:, j] * line[j : j + n] for j in range(W))
        outs.append(y if s["bias"] is None else y + s["bias"].double())
        kept[slot] = line[n:]
        t += n
    y = torch.cat(outs)
    y = y * torch.sigmoid(y)
    d, heads = case["head_dim"], case["unit_heads"]
    for h in range(heads):
        part = y[:, h * d : (h + 1) * d]
        part /= ((part * part).sum(1, keepdim=True) + 1e-6) ** 0.5
    return {"out": y, "states": kept}


def _rotary_exact(s):
    case, half = s["case"], s["case"]["rotated"] // 2
    rows = torch.nonzero(s["positions"] >= 0)[:, 0]
    turn = torch.polar(torch.ones(len(rows), 1, half, dtype=torch.float64, device=DEV),
                       s["positions"][rows].double()[:, None, None] * s["freq"].double())

    def turned(x):
        x = x[rows].double()
        pair = x[..., : 2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
        pair = pair if case["interleaved"] else pair.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., 2 * half :]], -1)

    q = s["q_out"].double()
    q[rows] = turned(s["q"])
    pages = s["k_pages"].double()
    pages.view(-1, *pages.shape[2:])[s["slots"][rows]] = turned(s["k"])
    return {"q": q, "k_pages": pages, "v_pages": None}


def exact(case, seed):
    """The recurrence token by token, the convolution tap by tap and request by request, the rotation as a product of
    complex numbers, in FP64."""
    s, new = prepare(case, seed), _lengths(case)
    if case["op"] == "delta":
        return _delta_exact(s, new)
    return _conv_exact(s, new) if case["op"] == "conv" else _rotary_exact(s)
