"""Measured cases of the operators between a layer's projections: rotary embedding and the write into a paged
key-value cache, attention of one new token per sequence over that cache, and causal attention over packed prompts.

``run`` computes a case either with the library's calls (``own`` true) or in elementary torch
operations (``own`` false); ``exact`` computes it from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
ROW_BYTES = {"bf16": 2.0, "mxfp8": 1.0 + 1.0 / 32.0}  # a value of the cache


# ------------------------------------------------------------------ cases

def _append(name, T, heads, kv, D, page, fmt, rot, pairs, k_out):
    return {"name": name, "op": "append", "T": T, "heads": heads, "kv": kv, "D": D, "page": page, "fmt": fmt,
            "rot": rot, "pairs": pairs, "k_out": k_out}


def _decode(name, B, lo, hi, heads, kv, D, page, fmt):
    return {"name": name, "op": "decode", "B": B, "lo": lo, "hi": hi, "heads": heads, "kv": kv, "D": D, "page": page,
            "fmt": fmt}


def _prompt(name, n, lo, hi, heads, kv, D):
    return {"name": name, "op": "prompt", "n": n, "lo": lo, "hi": hi, "heads": heads, "kv": kv, "D": D}


def listed():
    return [
        # one decoded token of one sequence: its query and key rotated, its key and value into the cache
        _append("append_T1", 1, 56, 8, 128, 64, "bf16", 128, False, False),
        # a decode batch on an 8-bit cache, half of each head rotated, in neighbouring pairs
        _append("append_T176_mxfp8", 176, 64, 8, 128, 64, "mxfp8", 64, True, False),
        # a prompt: the rotated keys also as rows, for the prompt's own attention
        _append("append_T8192", 8192, 64, 8, 128, 64, "bf16", 128, False, True),
        # one sequence with a short context: latency
        _decode("decode_B1_L1000", 1, 1000, 1000, 56, 8, 128, 64, "bf16"),
        # one sequence with a long context
        _decode("decode_B1_L131072", 1, 131072, 131072, 64, 8, 128, 64, "bf16"),
        # a small batch without shared heads, narrow heads, small pages
        _decode("decode_B15_D64_page16", 15, 1, 4096, 32, 32, 64, 16, "bf16"),
        # a batch of sequences at all stages, some slots of the batch without one
        _decode("decode_B88", 88, 0, 8192, 56, 8, 128, 64, "bf16"),
        # a large batch on an 8-bit cache
        _decode("decode_B176_mxfp8", 176, 1, 8192, 64, 8, 128, 64, "mxfp8"),
        # a short prompt alone
        _prompt("prompt_512", 1, 512, 512, 64, 8, 128),
        # a long prompt
        _prompt("prompt_8192", 1, 8192, 8192, 64, 8, 128),
        # prompts of very different lengths in one call, seven query heads to a key head
        _prompt("prompt_packed_1_3001", 15, 1, 3001, 56, 8, 128),
        # narrow heads, none shared
        _prompt("prompt_packed_D64", 3, 700, 2047, 32, 32, 64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    D = rng.choice((64, 128))
    group = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16))
    kv = rng.choice([n for n in (1, 2, 4, 5, 8, 16, 32) if n * group <= 64])
    return kv * group, kv, D


def draw(rng):
    op = rng.choice(("append", "decode", "prompt"))
    heads, kv, D = _heads(rng)
    page, fmt = rng.choice((16, 32, 64, 128, 256)), rng.choice(("bf16", "bf16", "mxfp8"))
    if op == "append":
        rot = rng.choice((D, D, D // 2, 0))
        most = min(8192, 8192 * 80 * 128 // ((heads + 2 * kv) * D))
        c = _append("", _log_int(rng, 1, most), heads, kv, D, page, fmt, rot, rng.random() < 0.4, rng.random() < 0.5)
    elif op == "decode":
        B = _log_int(rng, 1, 256)
        # (a batch's rows, padded to its longest, take no more than 1.4 GB of a BF16 cache)
        most = max(16, min(131072, int(1.4e9) // (4 * kv * D * B)))
        hi = _log_int(rng, 1, most)
        c = _decode("", B, rng.choice((0, 1, hi)), hi, heads, kv, D, page, fmt)
    else:
        n = _log_int(rng, 1, 64)
        most = int(min(8192, 16384 // n + 1, 8192 * math.sqrt(64 * 128 / (n * heads * D))))
        hi = _log_int(rng, 1, max(1, most))
        c = _prompt("", n, rng.choice((0, 1, hi)), hi, heads, kv, D)
    del c["name"]
    return c


def _lengths(n, lo, hi):
    """n lengths between lo and hi, evenly over the range in a mixed order, the longest among them."""
    if n == 1:
        return [hi]
    golden = (math.sqrt(5) - 1) / 2
    spread = [(i * golden) % 1.0 for i in range(n)]
    top = max(spread)
    return [lo + int(round((hi - lo) * s / top)) for s in spread]


def work(case):
    heads, kv, D = case["heads"], case["kv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        per = (heads + 2 * kv) * D * 2 + heads * D * 2 + 2 * kv * D * ROW_BYTES[case["fmt"]] + 4
        per += kv * D * 2 * case["k_out"] + (4 * case["rot"] + 4 if case["rot"] else 0)
        return {"bytes": T * per, "flops": 3.0 * T * (heads + kv) * case["rot"]}
    if case["op"] == "decode":
        total = sum(_lengths(case["B"], case["lo"], case["hi"]))
        pages = sum(-(-L // case["page"]) for L in _lengths(case["B"], case["lo"], case["hi"]))
        return {"bytes": total * 2 * kv * D * ROW_BYTES[case["fmt"]] + 4 * pages + case["B"] * (4 * heads * D + 4),
                "flops": 4.0 * total * heads * D}
    lengths = _lengths(case["n"], case["lo"], case["hi"])
    return {"bytes": sum(lengths) * (2 * heads + 2 * kv) * D * 2 + 4 * case["n"],
            "flops": sum(2.0 * L * (L + 1) for L in lengths) * heads * D}


# ------------------------------------------------------------------ inputs

def _mxfp8_of(x):
    """E4M3 values and E8M0 bytes of the last dimension's blocks of 32: the smallest power of two that brings a
    block's largest value to 448 or below."""
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, -127, e - 9 + (m > 0.875).int()).clamp(-127, 127)
    q = (b * torch.exp2(-e.to(x.dtype)).unsqueeze(-1)).float().to(torch.float8_e4m3fn).view(x.shape)
    return q, (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    heads, kv, D = case["heads"], case["kv"], case["D"]
    s = {"case": case}

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(torch.bfloat16)

    if case["op"] == "prompt":
        lengths = _lengths(case["n"], case["lo"], case["hi"])
        T = sum(lengths)
        # the rows that the input projection and the rotation leave: queries, keys and values side by side
        qkv = normal(T, heads + 2 * kv, D)
        qkv[:, :heads] *= 1.5
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        s["longest"] = max(lengths)
        s["offsets"] = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(DEV)
        s["out"] = torch.zeros((T, heads, D), dtype=torch.bfloat16, device=DEV)
        return s

    page = case["page"]
    if case["op"] == "append":
        T, rot = case["T"], case["rot"]
        n_pages = -(-T // page) + 3
        s["qkv"] = normal(T, (heads + 2 * kv) * D)
        slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T]  # (batches: a token per sequence)
        if T > 1024:  # a prompt: whole pages, in any order
            slots = torch.randperm(n_pages, generator=g, device=DEV).mul(page).unsqueeze(1)
            slots = (slots + torch.arange(page, device=DEV)).flatten()[:T]
        s["slots"] = slots.to(torch.int32)
        s["rope"] = s["positions"] = None
        if rot:
            n_pos = max(T, 4096)
            s["positions"] = torch.arange(T, device=DEV, dtype=torch.int32) if T > 1024 else \
                torch.randint(0, n_pos, (T,), generator=g, device=DEV, dtype=torch.int32)
            freq = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
            angle = torch.arange(n_pos, device=DEV, dtype=torch.float64).unsqueeze(1) * freq
            s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["q_out"] = torch.zeros((T, heads, D), dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.zeros((T, kv, D), dtype=torch.bfloat16, device=DEV) if case["k_out"] else None
        cache = [normal(n_pages, kv, page, D) for _ in range(2)]
    else:
        B = case["B"]
        lengths = _lengths(B, case["lo"], case["hi"])
        held = [-(-L // page) for L in lengths]
        width = max(1, max(held))
        n_pages = sum(held) + 2
        free = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)  # (past a sequence's end: no page)
        used = torch.arange(width, device=DEV) < torch.tensor(held, device=DEV).unsqueeze(1)
        table[used] = free[:sum(held)]
        s["table"], s["lens"] = table, torch.tensor(lengths, dtype=torch.int32).to(DEV)
        s["q"] = normal(B, heads, D, scale=1.5)
        s["out"] = torch.zeros((B, heads, D), dtype=torch.bfloat16, device=DEV)
        cache = [normal(n_pages, kv, page, D) for _ in range(2)]
    if case["fmt"] == "mxfp8":
        (k, ks), (v, vs) = (_mxfp8_of(c.float()) for c in cache)
    else:
        (k, ks), (v, vs) = ((c, None) for c in cache)
    s["cache"] = (k, v, ks, vs)
    if own:  # the cache that a program holds
        from mxfp4_routed_expert_router_gb300.attention import KvCache
        s["held"] = KvCache(k, v, ks, vs)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[op](state)


def _run_own(op, s):
    from mxfp4_routed_expert_router_gb300 import attention as A
    c = s["case"]
    if op == "append":
        s["held"].append(s["qkv"], c["heads"], s["slots"], s["positions"], s["rope"], c["pairs"], s["q_out"],
                         s["k_out"])
        return _append_outputs(s["q_out"], s["k_out"], s["cache"])
    if op == "decode":
        return {"out": s["held"].decode(s["q"], s["table"], s["lens"], out=s["out"])}
    return {"out": A.prompt(s["q"], s["k"], s["v"], s["offsets"], out=s["out"])}


def _append_outputs(q, k, cache):
    out = {"q": q, "cache_k": cache[0], "cache_v": cache[1]}
    if k is not None:
        out["k"] = k
    if cache[2] is not None:  # E4M3 values and their E8M0 powers of two
        out["cache_k_scales"] = cache[2].view(torch.float8_e8m0fnu)
        out["cache_v_scales"] = cache[3].view(torch.float8_e8m0fnu)
    return out


def _plain_append(s):
    c = s["case"]
    heads, kv, D, rot, page = c["heads"], c["kv"], c["D"], c["rot"], c["page"]
    x = s["qkv"].view(c["T"], heads + 2 * kv, D)
    qk, v = x[:, :heads + kv], x[:, heads + kv:]
    if rot:
        # 64 bits: a rotated value next to a border of the cache's type rounds to its own side
        t = s["rope"][s["positions"].long()].double().unsqueeze(1)
        cos, sin = t[..., :rot // 2], t[..., rot // 2:]
        r = qk[..., :rot].double()
        if c["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        qk = torch.cat((r, qk[..., rot:].double()), -1)
    q, k = qk[:, :heads].to(torch.bfloat16), qk[:, heads:]
    kc, vc, ks, vs = s["cache"]
    at = s["slots"].long()
    pg, row = at // page, at % page
    if ks is None:
        kc[pg, :, row], vc[pg, :, row] = k.to(torch.bfloat16), v
    else:
        (k8, e), (v8, f) = _mxfp8_of(k.double()), _mxfp8_of(v.double())
        kc.view(torch.uint8)[pg, :, row], vc.view(torch.uint8)[pg, :, row] = k8.view(torch.uint8), v8.view(torch.uint8)
        ks[pg, :, row], vs[pg, :, row] = e, f
    return _append_outputs(q, k.to(torch.bfloat16) if c["k_out"] else None, s["cache"])


def _values(codes, scales, at):
    """Pages `at` of a cache as float values."""
    x = codes[at] if scales is None else codes.view(torch.uint8)[at].view(torch.float8_e4m3fn)
    x = x.float()
    if scales is not None:
        x = x * torch.exp2(scales[at].float() - 127).repeat_interleave(32, -1)
    return x


def _plain_decode(s):
    c = s["case"]
    B, heads, kv, D = c["B"], c["heads"], c["kv"], c["D"]
    kc, vc, ks, vs = s["cache"]
    at = s["table"].long().clamp_min(0)
    rows = at.shape[1] * c["page"]
    # [B, pages, kv, page, D] -> [B, kv, rows, D]
    k = _values(kc, ks, at).transpose(1, 2).reshape(B, kv, rows, D)
    q = s["q"].float().view(B, kv, heads // kv, D)
    here = (torch.arange(rows, device=DEV) < s["lens"].unsqueeze(1)).view(B, 1, 1, rows)
    a = (q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(~here, -math.inf)
    del k
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = _values(vc, vs, at).transpose(1, 2).reshape(B, kv, rows, D)
    out = p @ v / torch.where(total > 0, total, 1.0)  # (a sequence of no tokens: zeros)
    return {"out": out.view(B, heads, D).to(torch.bfloat16)}


def _plain_prompt(s):
    c = s["case"]
    n, heads, kv, D = c["n"], c["heads"], c["kv"], c["D"]
    T, L = s["q"].shape[0], s["longest"]
    first, end = s["offsets"][:-1].long().unsqueeze(1), s["offsets"][1:].long().unsqueeze(1)
    at = first + torch.arange(L, device=DEV)  # [n, L] rows, padded to the longest sequence
    here = at < end
    at = at.clamp_max(T - 1)
    q = s["q"][at].float().view(n, L, kv, heads // kv, D).permute(0, 2, 3, 1, 4).reshape(n, kv, -1, D)
    k = s["k"][at].float().permute(0, 2, 3, 1)
    v = s["v"][at].float().transpose(1, 2)
    p = (q @ k).mul_(1 / math.sqrt(D)).view(n, kv, heads // kv, L, L)
    p.masked_fill_(torch.ones((L, L), dtype=torch.bool, device=DEV).triu_(1), -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, kv, -1, L) @ v).view(n, kv, heads // kv, L, D) / total
    out = o.to(torch.bfloat16).permute(0, 3, 1, 2, 4).reshape(n, L, heads, D)
    return {"out": out[here]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](s, case)


def _held(codes, scales):
    x = codes.to(torch.float64)
    return x if scales is None else x.unflatten(-1, (-1, 32)).mul(
        torch.pow(2.0, scales.to(torch.float64) - 127).unsqueeze(-1)).flatten(-2)


def _exact_append(s, case):
    heads, kv, D, rot, page = case["heads"], case["kv"], case["D"], case["rot"], case["page"]
    x = s["qkv"].to(torch.float64).reshape(case["T"], -1, D)
    if rot:  # a turn of the plane of two values, as the product of complex numbers
        t = s["rope"].to(torch.float64)[s["positions"].long()]
        turn = torch.complex(t[:, :rot // 2], t[:, rot // 2:]).unsqueeze(1)
        one = slice(0, rot, 2) if case["pairs"] else slice(0, rot // 2)
        two = slice(1, rot, 2) if case["pairs"] else slice(rot // 2, rot)
        z = torch.complex(x[:, :heads + kv, one].contiguous(), x[:, :heads + kv, two].contiguous()) * turn
        x = x.clone()
        x[:, :heads + kv, one], x[:, :heads + kv, two] = z.real, z.imag
    out = {"q": x[:, :heads]}
    page_of, row = torch.div(s["slots"], page, rounding_mode="floor").long(), torch.remainder(s["slots"], page).long()
    for name, new, codes, scales in (("k", x[:, heads:heads + kv], s["cache"][0], s["cache"][2]),
                                     ("v", x[:, heads + kv:], s["cache"][1], s["cache"][3])):
        held = codes.to(torch.float64)
        if scales is None:
            held[page_of, :, row] = new
        else:
            b = new.reshape(*new.shape[:-1], -1, 32)
            p = torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 448.0)).clamp(-127, 127)
            y = b / torch.pow(2.0, p)
            step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            held[page_of, :, row] = ((y / step).round() * step).reshape(new.shape)
            power = torch.pow(2.0, scales.to(torch.float64) - 127)
            power[page_of, :, row] = torch.pow(2.0, p).squeeze(-1)
            out[f"cache_{name}_scales"] = power
        out[f"cache_{name}"] = held
    if case["k_out"]:
        out["k"] = x[:, heads:heads + kv]
    return out


def _exact_decode(s, case):
    heads, kv, D, page = case["heads"], case["kv"], case["D"], case["page"]
    kc, vc, ks, vs = s["cache"]
    out = torch.zeros((case["B"], heads, D), dtype=torch.float64, device=DEV)
    for b, L in enumerate(_lengths(case["B"], case["lo"], case["hi"])):
        if L == 0:
            continue
        pages = s["table"][b, :-(-L // page)].long()

        def rows(codes, scales):  # [kv, L, D]
            x = codes.view(torch.uint8)[pages].view(codes.dtype)
            return _held(x, None if scales is None else scales[pages]).transpose(0, 1).reshape(kv, -1, D)[:, :L]

        q = s["q"][b].to(torch.float64).reshape(kv, -1, D)
        w = torch.softmax(torch.einsum("hgd,hld->hgl", q, rows(kc, ks)) * D ** -0.5, dim=2)
        out[b] = torch.einsum("hgl,hld->hgd", w, rows(vc, vs)).reshape(heads, D)
    return {"out": out}


def _exact_prompt(s, case):
    heads, kv, D = case["heads"], case["kv"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    a = 0
    for L in _lengths(case["n"], case["lo"], case["hi"]):
        q, k, v = (s[x][a:a + L].to(torch.float64) for x in "qkv")
        for h in range(heads):
            j = h // (heads // kv)
            for r in range(0, L, 2048):  # a block of rows and the keys up to its last row
                e = min(L, r + 2048)
                w = q[r:e, h] @ k[:e, j].T * D ** -0.5
                w += torch.full_like(w, -math.inf).triu(r + 1)
                out[a + r:a + e, h] = torch.softmax(w, dim=1) @ v[:e, j]
        a += L
    return {"out": out}
