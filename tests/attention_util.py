"""Plain forms of the attention operators in 64 bits, and caches for their tests."""
import numpy as np
import torch


def e4m3_blocks(x):
    """E4M3 values, and E8M0 bytes, of float64 values in blocks of 32: the smallest power of two with amax <= 448 * 2^p,
    each value rounded once, to nearest even; values that are not finite become NaN (beside an infinity the byte is
    247).  Returns (values * 2^p, bytes)."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.nanmax(np.abs(np.where(np.isnan(b), 0, b)), axis=-1, keepdims=True)
    with np.errstate(all="ignore"):
        m, e = np.frexp(amax)
        p = np.where(amax == 0, -127, e - 9 + (m > 0.875))
        p = np.where(np.isinf(amax), 120, np.clip(p, -127, 127)).astype(np.int64)
        y = b * 2.0 ** -p
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
        q = np.round(y / step) * step * 2.0 ** p
    q[~np.isfinite(b)] = np.nan
    return q.reshape(x.shape), (p + 127).astype(np.uint8)[..., 0]


def cache_values(c):
    """k, v of a KvCache as float64 [n_pages, n_kv_heads, page_size, head_dim]."""
    out = []
    for t, s in ((c.k, c.k_scales), (c.v, c.v_scales)):
        x = t.float().double()
        if s is not None:
            e = s.double()
            e = torch.where(e == 255, float("nan"), torch.exp2(e - 127))
            x = x * e.repeat_interleave(32, -1)
        out.append(x)
    return out


def random_cache(n_pages, kv, page, D, fmt, seed, spread=1):
    """A cache of normal values; with MXFP8, scale bytes in 127 - spread .. 127 + spread."""
    from mxfp4_routed_expert_router_gb300.attention import KvCache
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (n_pages, kv, page, D)
    x = [torch.randn(shape, generator=g, device="cuda") for _ in range(2)]
    if fmt == "bf16":
        return KvCache(*[t.bfloat16() for t in x])
    s = [torch.randint(127 - spread, 128 + spread, shape[:3] + (D // 32,), generator=g, device="cuda",
                       dtype=torch.uint8) for _ in range(2)]
    return KvCache(*[t.to(torch.float8_e4m3fn) for t in x], *s)


def paged(lens, page, n_pages, width, seed):
    """A table [B, width] of distinct pages for sequences of these lengths; -1 where a sequence has none."""
    rng = np.random.default_rng(seed)
    free = list(rng.permutation(n_pages))
    table = np.full((len(lens), width), -1, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = free.pop()
    return torch.from_numpy(table).cuda()


def attend(q, k, v, scale, visible=None):
    """softmax(scale q k^T) v in 64 bits for q [h, n, D], k, v [h, L, D] and a mask [n, L] (True: seen).  Returns the
    output, sum p |v| and the largest sum |q||k| * scale, for tolerances.  What is not seen does not count, be it finite
    or not."""
    s = q @ k.transpose(-1, -2) * scale
    mag = (q.abs() @ k.abs().transpose(-1, -2) * scale)
    if visible is not None:
        s = s.masked_fill(~visible, -torch.inf)
        mag = mag.masked_fill(~visible, 0)
    p = torch.softmax(s, -1)
    if visible is not None:  # (0 * inf)
        o = torch.stack([torch.stack([p[h, i, visible[i]] @ v[h, visible[i]] for i in range(q.shape[1])])
                         for h in range(q.shape[0])]) if not torch.isfinite(v).all() else p @ v
    else:
        o = p @ v
    return o, p @ torch.nan_to_num(v.abs(), posinf=0.0), mag.amax(-1, keepdim=True)


def tolerance(o, pv, mag, D, vmax=0.0):
    """Bound of the kernels' error against ``attend``:
    * the output rounds to BF16: 2^-8 of it;
    * each probability rounds to BF16 for the product with v (FP16 with MXFP8, which is finer): 2^-8 of sum p |v|;
    * a score is D exact products added in FP32 (truncating at worst 2^-22 of the sum of magnitudes at each of the D / 16
      steps) and one multiplication by scale * log2 e; the exponential is good to 2^-21: the probabilities' relative
      error, twice for the quotient;
    * the FP32 sums of p v: 2^-16 of sum p |v| covers 2^18 truncated terms of random sign and thousands of one;
    * vmax, with MXFP8: a P below FP16's normal range is off by 2^-25 of the scale of its pass, which is at most 2^8
      above the token's own: 2^-17 of |v| for each of the 16 tokens of a step, whose largest p is 1 there."""
    ds = 2 * ((D / 16 + 2) * 2.0 ** -22 * mag * 1.45 + 2.0 ** -21)
    return 2.0 ** -8 * o.abs() + (2.0 ** -8 + ds + 2.0 ** -16) * pv * 1.01 + 2.0 ** -13 * vmax + 1e-30
