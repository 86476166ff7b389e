"""moe_attention_decode on the GPU against its definition in 64 bits; the tolerance is derived in attention_util."""
import numpy as np
import pytest
import torch

from attention_util import attend, cache_values, paged, random_cache, tolerance

pytestmark = pytest.mark.gpu


def expected(c, q, table, lens, scale):
    """(output, tolerance) [B, heads, D]"""
    k, v = cache_values(c)
    B, heads, D = q.shape
    out, tol = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = table[b, :-(-n // c.page_size)].long()
        kb, vb = (x[at].transpose(0, 1).reshape(c.n_kv_heads, -1, D)[:, :n] for x in (k, v))
        o, pv, mag = attend(q[b].double().view(c.n_kv_heads, -1, D), kb, vb, scale)
        vmax = vb.abs().amax((1, 2), keepdim=True) if c.k_scales is not None else 0.0
        t = tolerance(o, pv, mag, D, vmax)
        out[b], tol[b] = o.reshape(heads, D), t.reshape(heads, D)
    return out, tol


def check(got, want):
    out, tol = want
    err = (got.double() - out).abs()
    assert torch.all(err <= tol), (err / tol.clamp_min(1e-30)).max()


def make(lens, heads, kv, D, page, fmt, seed, scale=None, spread=1, spare=3, width=None, q_scale=1.5):
    held = sum(-(-n // page) for n in lens)
    c = random_cache(held + spare, kv, page, D, fmt, seed, spread)
    width = max(1, max(-(-n // page) for n in lens)) if width is None else width
    table = paged(lens, page, held + spare, width, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    q = (torch.randn((len(lens), heads, D), generator=g, device="cuda") * q_scale).bfloat16()
    return c, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


CASES = [
    ([1], 1, 1, 64, 16), ([1], 8, 8, 128, 64), ([63], 8, 1, 128, 64), ([64], 7, 1, 64, 64), ([65], 9, 1, 128, 32),
    ([1000], 56, 8, 128, 64), ([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0], 12, 4, 64, 16),
    ([0, 0, 300, 0], 6, 2, 128, 128), ([5000], 16, 1, 128, 256), ([3, 4097, 1, 900], 32, 32, 64, 16),
    ([700] * 40, 40, 8, 128, 64), ([20000, 3], 64, 4, 128, 64), ([333, 100], 48, 2, 64, 32),
    ([37 * i % 500 for i in range(200)], 8, 2, 64, 32), ([1] * 300, 4, 4, 128, 16), ([257], 40, 1, 64, 256),
    ([256, 0, 1, 255] * 60, 4, 2, 64, 64), ([512, 400], 12, 2, 128, 32), ([513, 400], 12, 2, 128, 16),
    ([1024, 7, 0, 700] * 5, 20, 5, 64, 128), ([256] * 160, 8, 1, 128, 64), ([3] * 1500, 2, 1, 64, 16),
]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens,heads,kv,D,page", CASES)
def test_decode_matches_its_definition(lens, heads, kv, D, page, fmt):
    c, q, table, n = make(lens, heads, kv, D, page, fmt, len(lens) + heads)
    got = c.decode(q, table, n)
    want = expected(c, q, table, lens, D ** -0.5)
    torch.cuda.synchronize()
    check(got, want)
    assert torch.equal(c.decode(q, table, n), got)  # the same, call by call


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [6, 40])
def test_mxfp8_scales_far_apart(D, spread):
    """Blocks whose powers of two differ by up to 2^80 among the tokens of a step, large ones with small probabilities."""
    lens = [100, 1, 16, 700]
    c, q, table, n = make(lens, 8, 2, D, 32, "mxfp8", 77, spread=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    c.v_scales.copy_(torch.randint(127 - spread, 128 + spread, c.v_scales.shape, generator=g, device="cuda"))
    check(c.decode(q, table, n), expected(c, q, table, lens, D ** -0.5))
    # a token that cannot be chosen has the largest values: the others' sum must not lose its bits
    c.v_scales.fill_(127)
    first = table[0, 0].item()
    c.k[first, :, 3] = q[0].view(2, 4, D).float().mean(1).mul(-30).to(torch.float8_e4m3fn)
    c.v_scales[first, :, 3] = 160
    out, _ = expected(c, q, table, lens, D ** -0.5)
    c2 = c.v_scales.clone()
    got = c.decode(q, table, n)
    k, v = cache_values(c)
    _, tol = expected(c, q, table, lens, D ** -0.5)
    err = (got.double() - out).abs()
    # (the tolerance's vmax counts the token's own 2^33: what it may add is its probability's share, sum p |v|, alone)
    at = table[0, :4].long()
    kb, vb = (x[at].transpose(0, 1).reshape(2, -1, D)[:, :100] for x in (k, v))
    o, pv, mag = attend(q[0].double().view(2, -1, D), kb, vb, D ** -0.5)
    tight = tolerance(o, pv, mag, D, 448.0 * 2).reshape(8, D)
    assert torch.all(err[0] <= tight), (err[0] / tight).max()
    assert torch.all(err <= tol) and torch.equal(c2, c.v_scales)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_what_a_sequence_does_not_hold_may_be_anything(fmt):
    lens = [5, 70, 0, 129, 200]
    c, q, table, n = make(lens, 16, 2, 128, 64, fmt, 31, width=6)
    want = expected(c, q, table, lens, 0.2)
    got = c.decode(q, table, n, scale=0.2)
    check(got, want)
    used = torch.zeros((c.k.shape[0], 64), dtype=torch.bool, device="cuda")
    for b, L in enumerate(lens):
        for i in range(L):
            used[table[b, i // 64].item(), i % 64] = True
    for t in (c.k, c.v):
        if fmt == "bf16":
            t.copy_(t.masked_fill(~used[:, None, :, None], float("nan")))
        else:
            raw = t.view(torch.uint8)
            raw.copy_(raw.masked_fill(~used[:, None, :, None], 0x7F))
    if fmt == "mxfp8":
        for s in (c.k_scales, c.v_scales):
            s.copy_(s.masked_fill(~used[:, None, :, None], 255))
    assert torch.equal(c.decode(q, table, n, scale=0.2), got)
    if fmt == "bf16":
        for t in (c.k, c.v):
            t.copy_(t.masked_fill(~used[:, None, :, None], float("-inf")))
        assert torch.equal(c.decode(q, table, n, scale=0.2), got)
    # and what it does hold reaches its heads, and no other sequence
    page = table[3, 1].item()
    c.v[page, 1, 7] = float("nan")
    again = c.decode(q, table, n, scale=0.2)
    assert torch.isnan(again[3, 8:]).all() and torch.equal(again[3, :8], got[3, :8])
    assert torch.equal(again[:3], got[:3]) and torch.equal(again[4:], got[4:])


def test_large_scores_and_one_hot_rows():
    """Scores of hundreds: the maximum carries the softmax; and of -thousands everywhere."""
    for fmt in ("bf16", "mxfp8"):
        c, q, table, n = make([300, 77], 8, 2, 64, 32, fmt, 41, q_scale=60.0)
        check(c.decode(q, table, n), expected(c, q, table, [300, 77], 0.125))
        c.k.copy_(c.k.float().abs().to(c.k.dtype))
        q2 = -q.abs()
        check(c.decode(q2, table, n), expected(c, q2, table, [300, 77], 0.125))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_bad_lengths_and_pages(fmt):
    from mxfp4_routed_expert_router_gb300 import attention as A, binding as B
    A.sync()
    lens = [100, 50, 300, 80]
    c, q, table, n = make(lens, 8, 2, 64, 32, fmt, 51)
    good = c.decode(q, table, n)
    A.sync()
    cases = []
    for bad in (-1, table.shape[1] * 32 + 1, 2 ** 31 - 1, -2 ** 31):
        m = n.clone()
        m[1] = bad
        cases.append((table, m))
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = bad
        cases.append((t, n))
    for t, m in cases:
        got = c.decode(q, t, m)
        with pytest.raises(B.MoeError) as e:
            A.sync()
        assert e.value.status == B.MOE_EDEVICE
        A.sync()
        assert torch.isnan(got[1]).all()
        for b in (0, 2, 3):
            check(got[b:b + 1], [x[b:b + 1] for x in expected(c, q, table, lens, 0.125)])
    t = table.clone()
    t[1, 2:] = 10 ** 6  # (past the sequence's end: not read)
    assert torch.equal(c.decode(q, t, n), good)
    A.sync()


def test_strided_rows_streams_and_graphs():
    lens = [900, 0, 64, 2000]
    c, q, table, n = make(lens, 8, 2, 128, 64, "bf16", 61)
    want = c.decode(q, table, n)
    wide = torch.zeros((4, 12 * 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :1024] = q.view(4, -1)
    out = torch.full((4, 1040), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :1024].view(4, 8, 128)
    c.decode(wide.view(4, 12, 128)[:, :8], table, n, out=view)
    assert torch.equal(view, want) and torch.all(out[:, 1024:] == 7.0)
    sides = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):  # several streams at a time, each with its workspace
        for s in sides:
            with torch.cuda.stream(s):
                got.append(c.decode(q, table, n))
        got.append(c.decode(q, table, n, stream=sides[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    g = torch.cuda.CUDAGraph()
    buf = torch.zeros_like(q)
    with torch.cuda.graph(g):
        c.decode(q, table, n, out=buf)
    m = n.clone()
    n.copy_(torch.tensor([1, 128, 0, 777], dtype=torch.int32))
    t2 = paged([1, 128, 0, 777], 64, c.k.shape[0], table.shape[1], 5)
    table.copy_(t2)
    g.replay()
    torch.cuda.synchronize()
    check(buf, expected(c, q, table, [1, 128, 0, 777], 128 ** -0.5))
    assert m.tolist() == lens


def test_no_sequences_and_tables_wider_than_needed():
    c, q, table, n = make([10, 200], 8, 2, 64, 16, "bf16", 71, width=4000)
    check(c.decode(q, table, n), expected(c, q, table, [10, 200], 0.125))
    assert c.decode(q[:0], table[:0], n[:0]).shape == (0, 8, 64)


@pytest.mark.parametrize("fmt,n_pages", [("bf16", 40000), ("mxfp8", 80000)])
def test_a_cache_whose_offsets_pass_32_bits(fmt, n_pages):
    """5 GB of keys and as much of values: tokens written to and read from its last pages, and its first ones."""
    from mxfp4_routed_expert_router_gb300 import attention as A
    kv, heads, page, D = 8, 16, 64, 128
    c = A.KvCache.empty(n_pages, kv, page, D, fmt)
    assert c.k.numel() * c.k.element_size() > 2 ** 32
    lens = [130, 70]
    pages = [[n_pages - 1, 0, n_pages - 3], [n_pages - 2, 1, 2]]
    table = torch.tensor(pages, dtype=torch.int32, device="cuda")
    slots = [pages[s][i // page] * page + i % page for s, n in enumerate(lens) for i in range(n)]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((200, (heads + 2 * kv) * D), generator=g, device="cuda").bfloat16()
    q = c.append(x, heads, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    used = torch.unique(table).long()
    small = A.KvCache(*[t.view(torch.uint8)[used].view(t.dtype).contiguous() if t is not None else None
                        for t in (c.k, c.v, c.k_scales, c.v_scales)])
    local = torch.searchsorted(used, table.long()).int()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = c.decode(q[[129, 199]].contiguous(), table, n)
    check(got, expected(small, q[[129, 199]], local, lens, D ** -0.5))
    assert torch.equal(small.decode(q[[129, 199]].contiguous(), local, n), got)
    if fmt == "bf16":
        at = torch.tensor(slots, device="cuda")
        v = x.view(200, -1, D)[:, heads + kv:]
        assert torch.equal(c.v[at // page, :, at % page], v)
