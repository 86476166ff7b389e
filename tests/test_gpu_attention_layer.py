"""The attention operators together, as a decoder layer runs them: prompts into the cache, then token by token.

Tolerances are those of attention_util: the rows that prompt and decode attention see are the same BF16 rows, and the
cache holds them exactly (BF16) or as the MXFP8 values that the reference reads back.
"""
import numpy as np
import pytest
import torch

from attention_util import attend, cache_values, tolerance
from test_gpu_linear import Weight

from mxfp4_routed_expert_router_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

HEADS, KV, D, PAGE = 8, 2, 64, 16
ROW = (HEADS + 2 * KV) * D


def _attention(fmt, n_pages=40, **kw):
    from mxfp4_routed_expert_router_gb300 import attention as A
    return A.Attention(HEADS, A.KvCache.empty(n_pages, KV, PAGE, D, fmt), A.rope_table(512, D), **kw)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pages:
    """Pages of a few sequences, in any order, as a serving program keeps them."""

    def __init__(self, n_seqs, width, seed):
        self.table = np.random.default_rng(seed).permutation(n_seqs * width).reshape(n_seqs, width).astype(np.int32)

    def slot(self, s, pos):
        return int(self.table[s, pos // PAGE]) * PAGE + pos % PAGE


def _rows_of(att, pages, s, n):
    """k, v of a sequence's first n tokens as the cache holds them, [KV, n, D] float64."""
    at = [pages.slot(s, i) for i in range(n)]
    return [x.transpose(1, 2).reshape(-1, KV, D)[at].transpose(0, 1) for x in cache_values(att.cache)]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("pairs", [False, True])
def test_prompts_and_then_token_by_token(fmt, pairs):
    att = _attention(fmt, pairs=pairs)
    lens, steps = [37, 1, 100, 16], 20
    pages = Pages(4, 10, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    T = sum(lens)
    qkv = torch.randn((T + 3, ROW), generator=g, device="cuda").bfloat16()  # (three rows of padding)
    pos = [i for n in lens for i in range(n)] + [0, 0, 0]
    slots = [pages.slot(s, i) for s, n in enumerate(lens) for i in range(n)] + [-1] * 3
    offsets = _i32(np.cumsum([0] + lens))
    rows = qkv.clone()
    out = att.prompt(rows, _i32(slots), _i32(pos), offsets)
    att_q = rows.view(T + 3, -1, D)[:, :HEADS]
    assert not out[T:].any()
    for s, n in enumerate(lens):  # the prompt's own rows: BF16 keys, whatever the cache holds
        a = sum(lens[:s])
        k, v = (rows.view(T + 3, -1, D)[a:a + n, HEADS + i * KV:HEADS + (i + 1) * KV].double().transpose(0, 1)
                .repeat_interleave(HEADS // KV, 0) for i in (0, 1))
        o, pv, mag = attend(att_q[a:a + n].double().transpose(0, 1), k, v, D ** -0.5,
                            torch.ones((n, n), dtype=torch.bool, device="cuda").tril())
        err = (out[a:a + n].view(n, HEADS, D).double().transpose(0, 1) - o).abs()
        assert torch.all(err <= tolerance(o, pv, mag, D))
        if fmt == "bf16":
            kc, vc = _rows_of(att, pages, s, n)
            assert torch.equal(kc.repeat_interleave(HEADS // KV, 0), k)
            assert torch.equal(vc.repeat_interleave(HEADS // KV, 0), v)
    # decode: sequence 1 ends after 5 steps, and a slot of the batch is never used
    held = list(lens) + [0]
    table = _i32(np.vstack([pages.table, np.full((1, 10), -1)]))
    for step in range(steps):
        new = torch.randn((5, ROW), generator=g, device="cuda").bfloat16()
        live = [s < 4 and not (s == 1 and step >= 5) for s in range(5)]
        slots = [pages.slot(s, held[s]) if live[s] else -1 for s in range(5)]
        positions = [held[s] if live[s] else 0 for s in range(5)]
        for s in range(5):
            held[s] += live[s]
        n = [held[s] if live[s] else 0 for s in range(5)]
        got = att.decode(new, _i32(slots), _i32(positions), table, _i32(n)).view(5, HEADS, D)
        q = new.view(5, -1, D)[:, :HEADS]
        for s in range(5):
            if not live[s]:
                assert not got[s].any()
                continue
            k, v = _rows_of(att, pages, s, n[s])
            o, pv, mag = attend(q[s].double().view(KV, -1, D), k, v, D ** -0.5)
            vmax = v.abs().amax((1, 2), keepdim=True) if fmt == "mxfp8" else 0.0
            err = (got[s].double().view(KV, -1, D) - o).abs()
            assert torch.all(err <= tolerance(o, pv, mag, D, vmax)), (step, s)
    from mxfp4_routed_expert_router_gb300 import attention as A
    A.sync()


def _block(seed, fmt="bf16", **kw):
    from mxfp4_routed_expert_router_gb300 import layer
    from mxfp4_routed_expert_router_gb300.block import MoeBlock, Routing
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    H, E = 256, 16
    ws = [Weight("mxfp4", H, HEADS * D, seed + 1, 115, 119), Weight("bf16", E, H, seed + 2),
          Weight("int4g32", ROW, H, seed + 3)]
    gain = torch.ones(H, device="cuda")
    args = dict(gain=gain, out_proj=QuantLinear("mxfp4", *ws[0].args), in_proj=QuantLinear("int4g32", *ws[2].args),
                in_gain=gain, attention=_attention(fmt))
    return MoeBlock(layer.MoeLayer(wl.custom("layer", 1, H, 128, E, 1, 4, seed)), QuantLinear("bf16", *ws[1].args),
                    Routing(4, 4, 2), **{**args, **kw})


def test_block_runs_the_whole_layer():
    """decode and prompt of a block are its parts one after the other, also captured and on another stream."""
    b = _block(5)
    pages, H = Pages(3, 8, 4), 256
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    lens = [40, 7, 60]
    T = sum(lens)
    res = torch.randn((T, H), generator=g, device="cuda")
    slots = _i32([pages.slot(s, i) for s, n in enumerate(lens) for i in range(n)])
    pos, off = _i32([i for n in lens for i in range(n)]), _i32(np.cumsum([0] + lens))
    want = res.clone()
    qkv = b.project_in(want)
    b.forward(b.attention.prompt(qkv, slots, pos, off), want)
    got = res.clone()
    assert b.prompt(got, slots, pos, off).data_ptr() == got.data_ptr()
    assert torch.equal(got, want)
    one = torch.randn((3, H), generator=g, device="cuda")
    s1, p1 = _i32([pages.slot(s, n) for s, n in enumerate(lens)]), _i32(lens)
    table, n1 = torch.from_numpy(pages.table).cuda(), _i32([n + 1 for n in lens])
    want = one.clone()
    b.forward(b.attention.decode(b.project_in(want), s1, p1, table, n1), want)
    got = one.clone()
    b.decode(got, s1, p1, table, n1)
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = one.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b.decode(got, s1, p1, table, n1)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    buf, pbuf = one.clone(), res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.prompt(pbuf, slots, pos, off)
        b.decode(buf, s1, p1, table, n1)
    for _ in range(2):
        buf.copy_(one), pbuf.copy_(res)
        b.attention.cache.k.zero_(), b.attention.cache.v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want)
    b.layer.sync()


def test_steps_enqueued_at_once():
    """Kernels of one step start while those of the step before still end: forty steps enqueued at once give what they
    give one at a time."""
    b = _block(7, "mxfp8")
    b.attention = _attention("mxfp8")
    pages, H, steps = Pages(4, 8, 8), 256, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    res = [torch.randn((4, H), generator=g, device="cuda") for _ in range(steps)]
    table = torch.from_numpy(pages.table).cuda()
    args = [(_i32([pages.slot(s, i) for s in range(4)]), _i32([i] * 4), table, _i32([i + 1] * 4)) for i in range(steps)]
    want = []
    for r, a in zip(res, args):
        x = r.clone()
        torch.cuda.synchronize()
        want.append(b.decode(x, *a))
        torch.cuda.synchronize()
    for _ in range(3):
        got = [r.clone() for r in res]
        b.attention.cache.k.view(torch.uint8).zero_()
        for x, a in zip(got, args):
            b.decode(x, *a)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_parts_that_do_not_fit_are_refused():
    from mxfp4_routed_expert_router_gb300 import attention as A, binding as B
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    b = _block(11)
    wrong_in = QuantLinear("bf16", torch.zeros((ROW - 64, 256), dtype=torch.bfloat16, device="cuda"))
    wrong_out = QuantLinear("bf16", torch.zeros((256, 256), dtype=torch.bfloat16, device="cuda"))
    cache = b.attention.cache
    res = torch.zeros((2, 256), device="cuda")
    table, i2 = _i32([[0], [1]]), _i32([0, 1])
    for call in (lambda: _block(11, in_proj=None), lambda: _block(11, in_proj=wrong_in), lambda: _block(11, out_proj=None),
                 lambda: _block(11, out_proj=wrong_out), lambda: A.Attention(7, cache), lambda: A.Attention(0, cache),
                 lambda: A.Attention(8, cache, torch.zeros(8, 64)),
                 lambda: A.Attention(8, cache, torch.zeros(8, 64, device="cuda").half()),
                 lambda: _block(11, attention=None).decode(res, i2, i2, table, i2),
                 lambda: b.decode(res[:, :128], i2, i2, table, i2), lambda: b.prompt(res.half(), i2, i2, i2),
                 lambda: b.attention.decode(torch.zeros((2, ROW - 64), dtype=torch.bfloat16, device="cuda"), i2, i2,
                                            table, i2),
                 lambda: b.decode(res, i2, None, table, i2)):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.status == B.MOE_EINVAL
    assert not res.any()
