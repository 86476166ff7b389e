"""Measured cases of the operators around the MoE layer: the residual addition with an RMS norm
(BF16 and MXFP8 outputs), group-limited routing, and the linear layer with 4-bit (or BF16) weights.

``run`` computes a case either with the library's calls (``own`` true) or in elementary torch
operations (``own`` false); ``exact`` computes it from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ROW_BYTES = {"bf16": 2.0, "f32": 4.0, "mxfp8": 1.0 + 1.0 / 32.0}
WEIGHT_BITS = {"mxfp4": 4.25, "int4g32": 4.75, "bf16": 16.0}


# ------------------------------------------------------------------ cases

def _norm(name, T, H, residual, delta, y, q, pad=0):
    return {"name": name, "op": "norm", "T": T, "H": H, "residual": residual, "delta": delta, "y": y, "q": q,
            "pad": pad}


def _route(name, T, E, k, groups, kept, score, group_score, bias, renorm, masked, logits="normal"):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "groups": groups, "kept": kept, "score": score,
            "group_score": group_score, "bias": bias, "renorm": renorm, "masked": masked, "logits": logits}


def _linear(name, T, N, K, fmt, x, out):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "fmt": fmt, "x": x, "out": out}


def listed():
    return [
        # the norm before the experts: one decoded token, both outputs
        _norm("norm_T1", 1, 7168, "bf16", "bf16", True, True),
        # a ragged batch of narrow rows cut out of wider buffers
        _norm("norm_T333_H2080", 333, 2080, "bf16", "bf16", True, False, pad=64),
        # a decode batch on an FP32 residual stream (the layer's own output type)
        _norm("norm_T176", 176, 7168, "f32", "f32", True, True),
        # a prompt
        _norm("norm_T8192", 8192, 7168, "f32", "f32", True, True),
        # the routing of one decoded token over the 256-expert layer
        _route("route_T1", 1, 256, 8, 8, 4, "sigmoid", "top2", True, True, 0),
        # softmax scores, uneven expert count, some experts switched off
        _route("route_T176_E250", 176, 250, 6, 5, 3, "softmax", "max", False, False, 7),
        # a prompt with skewed expert popularity
        _route("route_T8192", 8192, 256, 8, 8, 4, "sigmoid", "top2", True, True, 0, "zipf"),
        # the router's own product for one token
        _linear("linear_bf16_T1_router", 1, 256, 7168, "bf16", "bf16", "f32"),
        # an attention output projection for one token
        _linear("linear_mxfp4_T1", 1, 7168, 7168, "mxfp4", "bf16", "f32"),
        # a wide input projection on the norm's 8-bit output
        _linear("linear_mxfp4_T1_wide", 1, 36864, 7168, "mxfp4", "mxfp8", "bf16"),
        # a projection of a small decode batch from the dense width
        _linear("linear_int4_T15", 15, 7168, 18432, "int4g32", "bf16", "bf16"),
        # a short prompt
        _linear("linear_mxfp4_T512", 512, 7168, 7168, "mxfp4", "bf16", "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _off_3072(size, step):
    return size + step if size == 3072 else size


def draw(rng):
    op = rng.choice(("norm", "route", "linear"))
    if op == "norm":
        H = _off_3072(32 * _log_int(rng, 2, 512), 32)
        T = _off_3072(_log_int(rng, 1, max(1, min(8192, 8192 * 7168 // H))), 1)
        y, q = rng.choice(((True, True), (True, False), (False, True)))
        c = _norm("", T, H, rng.choice(("bf16", "f32")), rng.choice(("none", "bf16", "f32")), y, q,
                  rng.choice((0, 0, 8, 264)))
    elif op == "route":
        groups = rng.choice((1, 1, 2, 3, 4, 8, 16, 24))
        E = groups * _log_int(rng, 4, 1024 // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(16, kept * (E // groups)))
        T = _off_3072(_log_int(rng, 1, max(1, 8192 * 256 // max(E, 256))), 1)
        c = _route("", T, E, k, groups, kept, rng.choice(("sigmoid", "softmax")), rng.choice(("top2", "max")),
                   rng.random() < 0.6, rng.random() < 0.7, rng.choice((0, 0, E // 8)), rng.choice(("normal", "zipf")))
    else:
        K = _off_3072(32 * _log_int(rng, 4, 576), 32)
        N = _off_3072(_log_int(rng, 16, min(36864, 36864 * 7168 // K)), 1)
        T = _log_int(rng, 1, max(1, min(512, 512 * 7168 * 7168 // (N * K))))
        c = _linear("", T, N, K, rng.choice(("mxfp4", "mxfp4", "int4g32", "bf16")), rng.choice(("bf16", "mxfp8")),
                    rng.choice(("f32", "bf16")))
    del c["name"]
    return c


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        per = ROW_BYTES[case["residual"]] * 2  # read, and the sum written
        per += ROW_BYTES[case["delta"]] if case["delta"] != "none" else 0.0
        per += 2.0 * case["y"] + ROW_BYTES["mxfp8"] * case["q"]
        return {"bytes": T * H * per + 4.0 * H, "flops": 6.0 * T * H}
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": 4.0 * T * E + 4.0 * E * case["bias"] + 8.0 * T * k, "flops": 8.0 * T * E}
    N, K = case["N"], case["K"]
    return {"bytes": N * K * WEIGHT_BITS[case["fmt"]] / 8 + T * K * ROW_BYTES[case["x"]] + T * N * ROW_BYTES[case["out"]],
            "flops": 2.0 * T * N * K}


# ------------------------------------------------------------------ inputs

def _rows(T, H, pad, dtype, gen=None, scale=1.0):
    """[T, H] rows inside a buffer whose rows are `pad` elements wider."""
    buf = torch.zeros((T, H + pad), dtype=dtype, device=DEV) if gen is None else \
        torch.randn((T, H + pad), generator=gen, device=DEV).mul_(scale).to(dtype)
    return buf[:, :H]


def _mxfp8_of(x):
    """Codes (E4M3) and scales (E8M0 bytes) of float rows, as a program stores them."""
    b = x.float().view(x.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1) / 448.0)
    s = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    q = (b * torch.exp2(-s.float()).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(x.shape), (s + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    T, s = case["T"], {"case": case}
    if case["op"] == "norm":
        H, pad = case["H"], case["pad"]
        types = {"bf16": torch.bfloat16, "f32": torch.float32}
        s["residual"] = _rows(T, H, pad, types[case["residual"]], g, 3.0)
        s["delta"] = None if case["delta"] == "none" else _rows(T, H, pad, types[case["delta"]], g, 1.0)
        s["gain"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
        s["sum"] = _rows(T, H, pad, types[case["residual"]])
        s["y"] = _rows(T, H, pad, torch.bfloat16) if case["y"] else None
        s["q"] = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device=DEV) if case["q"] else None
        s["q_scales"] = torch.zeros((T, H // 32), dtype=torch.uint8, device=DEV) if case["q"] else None
    elif case["op"] == "route":
        E, k = case["E"], case["k"]
        lg = torch.randn((T, E), generator=g, device=DEV)
        if case["logits"] == "zipf":  # log-popularity of a shuffled power law, Gumbel noise per token
            r = torch.arange(1, E + 1, device=DEV, dtype=torch.float64) ** -1.1
            u = torch.rand((T, E), generator=g, device=DEV).clamp_min(1e-9)
            lg = ((r / r.sum()).log()[torch.randperm(E, generator=g, device=DEV)].float() - (-u.log()).log())
        if case["masked"]:  # experts that take no tokens (being moved, or lost)
            lg[:, torch.randperm(E, generator=g, device=DEV)[:case["masked"]]] = -math.inf
        s["logits"] = lg.contiguous()
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        s["scale"] = 2.5
        s["ids"] = torch.zeros((T, k), dtype=torch.int32, device=DEV)
        s["w"] = torch.zeros((T, k), dtype=torch.float32, device=DEV)
    else:
        N, K, fmt = case["N"], case["K"], case["fmt"]
        if fmt == "bf16":
            s["codes"], s["scales"], s["zeros"] = \
                (0.02 * torch.randn((N, K), generator=g, device=DEV)).to(torch.bfloat16), None, None
        else:
            s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
            if fmt == "mxfp4":
                s["scales"] = torch.randint(117, 122, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
                s["zeros"] = None
            else:
                s["scales"] = torch.exp2(torch.rand((N, K // 32), generator=g, device=DEV) * 4 - 11).half()
                s["zeros"] = torch.randint(6, 11, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        x = torch.randn((T, K), generator=g, device=DEV)
        s["x"], s["x_scales"] = (x.to(torch.bfloat16), None) if case["x"] == "bf16" else _mxfp8_of(x)
        s["out"] = torch.zeros((T, N), dtype={"f32": torch.float32, "bf16": torch.bfloat16}[case["out"]], device=DEV)
        if own:  # the handle that a program loads once for its weights
            from mxfp4_routed_expert_router_gb300.linear import QuantLinear
            s["linear"] = QuantLinear(fmt, s["codes"], s["scales"], s["zeros"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    return {"norm": _plain_norm, "route": _plain_route, "linear": _plain_linear}[op](state)


def _run_own(op, s):
    from mxfp4_routed_expert_router_gb300 import binding as B
    c = s["case"]
    if op == "norm":
        B.moe_add_rmsnorm(s["residual"], s["delta"], s["gain"], EPS, s["sum"], s["y"], s["q"], s["q_scales"])
        return _norm_outputs(s["sum"], s["y"], s["q"], s["q_scales"])
    if op == "route":
        B.moe_route_grouped(s["logits"], s["bias"], c["T"], c["E"], c["k"], c["groups"], c["kept"],
                            B.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else B.MOE_SCORE_SOFTMAX,
                            B.MOE_GROUP_TOP2 if c["group_score"] == "top2" else B.MOE_GROUP_MAX,
                            c["renorm"], s["scale"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    return {"out": s["linear"].forward(s["x"], s["x_scales"], out=s["out"])}


def _norm_outputs(total, y, q, q_scales):
    out = {"sum": total}
    if y is not None:
        out["y"] = y
    if q is not None:  # E4M3 values and their E8M0 powers of two
        out["q"] = q
        out["q_scales"] = q_scales.view(torch.float8_e8m0fnu)
    return out


def _plain_norm(s):
    r = s["residual"].float()
    if s["delta"] is not None:
        r = r + s["delta"].float()
    total = r.to(s["residual"].dtype)
    r = total.float()
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["gain"]
    q = sc = None
    if s["q"] is not None:
        b = n.view(n.shape[0], -1, 32)
        # the smallest power of two that brings the block's largest value to 448 or below
        m, e = torch.frexp(b.abs().amax(-1))
        e = torch.where(m == 0, -127, e - 9 + (m > 0.875).int()).clamp(-127, 127)
        q = (b * torch.exp2(-e.float()).unsqueeze(-1)).to(torch.float8_e4m3fn).view(n.shape)
        sc = (e + 127).to(torch.uint8)
    return _norm_outputs(total, n.to(torch.bfloat16) if s["y"] is not None else None, q, sc)


def _plain_route(s):
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    lg = s["logits"].double()  # 64 bits: selections turn on values next to a border
    open_ = lg > -math.inf
    if c["score"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-lg))
    else:
        ex = torch.exp(lg - lg.amax(-1, keepdim=True))
        sc = ex / ex.sum(-1, keepdim=True)
    key = sc if s["bias"] is None else sc + s["bias"].double()
    key = key.masked_fill(~open_, -math.inf)
    top = torch.sort(key.view(T, G, E // G), dim=-1, descending=True, stable=True).values
    gs = top[..., 0]
    if c["group_score"] == "top2" and E > G:
        gs = gs + torch.where(top[..., 1] > -math.inf, top[..., 1], 0.0)
    gi = torch.sort(gs, dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
    in_kept = torch.zeros((T, G), dtype=torch.bool, device=lg.device).scatter_(1, gi, True)
    key = key.view(T, G, E // G).masked_fill(~in_kept.unsqueeze(-1), -math.inf).view(T, E)
    top = torch.sort(key, dim=-1, descending=True, stable=True)
    ids = top.indices[:, :k]
    full = top.values[:, :k] > -math.inf
    w = torch.where(full, sc.gather(1, ids), 0.0)
    if c["renorm"]:
        tot = w.sum(-1, keepdim=True)
        w = torch.where(tot > 0, w / tot, 0.0)
    return {"ids": torch.where(full, ids, -1).int(), "w": (w * s["scale"]).float()}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_linear(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = (x.view(-1, K // 32, 32) * torch.exp2(s["x_scales"].float() - 127).unsqueeze(-1)).view(-1, K)
    if c["fmt"] == "bf16":
        w = s["codes"].float()
    else:
        nib = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(N, K // 32, 32)
        if c["fmt"] == "mxfp4":
            table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=x.device)
            w = table[nib.int()] * torch.exp2(s["scales"].float() - 127).unsqueeze(-1)
        else:
            w = (nib.float() - s["zeros"].float().unsqueeze(-1)) * s["scales"].float().unsqueeze(-1)
        w = w.view(N, K)
    return {"out": (x @ w.t()).to(s["out"].dtype)}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "route": _exact_route, "linear": _exact_linear}[case["op"]](s, case)


def _exact_norm(s, case):
    r = s["residual"].to(torch.float64)
    if s["delta"] is not None:
        r = r.add(s["delta"].to(torch.float64))
    # the stream holds the sum in its own type, and the norm is that of what it holds
    total = r.to(s["residual"].dtype).to(torch.float64)
    rms = (torch.linalg.vector_norm(total, dim=1, keepdim=True).square() / case["H"] + EPS).sqrt()
    n = total / rms * s["gain"].to(torch.float64)
    out = {"sum": total}
    if case["y"]:
        out["y"] = n
    if case["q"]:
        b = n.reshape(-1, 32)
        p = torch.ceil(torch.log2(b.abs().max(dim=1, keepdim=True).values / 448.0)).clamp(-127, 127)
        v = b / torch.pow(2.0, p)
        step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        out["q"] = ((v / step).round() * step).reshape(n.shape)
        out["q_scales"] = torch.pow(2.0, p).reshape(n.shape[0], -1)
    return out


def _exact_route(s, case):
    """The ids are whole numbers that any two sides agree on; the weights follow from the definition by repeated maxima."""
    lg = s["logits"].to(torch.float64)
    T, E = lg.shape
    G = case["groups"]
    if case["score"] == "sigmoid":
        score = torch.sigmoid(lg)
    else:
        score = torch.softmax(lg, dim=1)
    key = score.clone()
    if s["bias"] is not None:
        key += s["bias"].to(torch.float64)
    key[torch.isinf(lg)] = -math.inf
    left, total = key.reshape(T, G, -1).clone(), 0.0
    for i in range(2 if case["group_score"] == "top2" and E > G else 1):
        best = left.max(dim=2, keepdim=True)
        total = total + (best.values if i == 0 else best.values.nan_to_num(neginf=0.0)).squeeze(2)
        left.scatter_(2, best.indices, -math.inf)
    left = torch.full((T, G, E // G), -math.inf, dtype=torch.float64, device=lg.device)
    for _ in range(case["kept"]):
        g = total.argmax(dim=1)
        left[torch.arange(T), g] = key.reshape(T, G, -1)[torch.arange(T), g]
        total[torch.arange(T), g] = -math.inf
    left, got = left.reshape(T, E), []
    for _ in range(case["k"]):
        best = left.max(dim=1, keepdim=True)
        got.append(score.gather(1, best.indices).masked_fill(torch.isinf(best.values), 0.0))
        left.scatter_(1, best.indices, -math.inf)
    w = torch.cat(got, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "w": w.nan_to_num(0.0) * s["scale"]}


def _exact_linear(s, case):
    N, K = case["N"], case["K"]
    x = s["x"].to(torch.float64)
    if s["x_scales"] is not None:
        x = x * torch.pow(2.0, s["x_scales"].to(torch.float64) - 127).repeat_interleave(32, dim=1)
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
    for r in range(0, N, 8192):
        codes = s["codes"][r:r + 8192]
        if case["fmt"] == "bf16":
            w = codes.to(torch.float64)
        else:
            w = torch.empty((codes.shape[0], K), dtype=torch.float64, device=x.device)
            for half in (0, 1):
                c = (codes >> (4 * half)).bitwise_and(15)
                if case["fmt"] == "mxfp4":  # sign, two exponent bits, one mantissa bit
                    e, m = (c >> 1).bitwise_and(3).double(), c.bitwise_and(1).double()
                    v = torch.where(e == 0, m / 2, torch.pow(2.0, e - 1) * (1 + m / 2))
                    w[:, half::2] = torch.where(c >= 8, -v, v)
                else:
                    w[:, half::2] = c.double()
            if case["fmt"] == "int4g32":
                w -= s["zeros"][r:r + 8192].double().repeat_interleave(32, dim=1)
                w *= s["scales"][r:r + 8192].double().repeat_interleave(32, dim=1)
            else:
                w *= torch.pow(2.0, s["scales"][r:r + 8192].double() - 127).repeat_interleave(32, dim=1)
        out[:, r:r + 8192] = x @ w.T
    return {"out": out}
