"""A call of Attention or MoeBlock that is refused has written nothing: neither the rows, nor the cache, nor the residual
stream."""
import pytest
import torch

from test_gpu_attention_layer import ROW, _attention, _block, _i32

pytestmark = pytest.mark.gpu

TABLES = [
    ("page_table", lambda a: a.update(table=a["table"][:1])), ("page_table", lambda a: a.update(table=a["table"].long())),
    ("page_table", lambda a: a.update(table=a["table"].t())), ("page_table", lambda a: a.update(table=a["table"].cpu())),
    ("page_table", lambda a: a.update(table=a["table"][:, :0])), ("lens", lambda a: a.update(lens=a["lens"][:1])),
    ("lens", lambda a: a.update(lens=a["lens"].long())), ("lens", lambda a: a.update(lens=a["lens"].cpu())),
    ("page_table", lambda a: a.update(table=a["table"][0])), ("slots", lambda a: a.update(slots=a["slots"].long())),
    ("positions", lambda a: a.update(pos=None)),
]
OFFSETS = [
    ("offsets", lambda a: a.update(off=a["off"].long())), ("offsets", lambda a: a.update(off=a["off"].cpu())),
    ("offsets", lambda a: a.update(off=a["off"][:0])), ("offsets", lambda a: a.update(off=a["off"].view(2, 1))),
    ("offsets", lambda a: a.update(off=_i32([0, 1, 2, 2])[::2])), ("offsets", lambda a: a.update(off=_i32([0] * 65538))),
    ("slots", lambda a: a.update(slots=a["slots"][:1])), ("positions", lambda a: a.update(pos=None)),
]


def _arguments():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    return dict(qkv=torch.randn((2, ROW), generator=g, device="cuda").bfloat16(), slots=_i32([3, 20]), pos=_i32([3, 4]),
                table=_i32([[0, 2, 4], [1, 3, 5]]), lens=_i32([4, 5]), off=_i32([0, 2]))


def _refused(call, touched):
    from mxfp4_routed_expert_router_gb300 import binding as B
    was = [t.clone() for t in touched]
    with pytest.raises(B.MoeError) as e:
        call()
    torch.cuda.synchronize()
    assert e.value.status == B.MOE_EINVAL
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(touched, was))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_refused_steps_leave_rows_and_cache(fmt):
    att = _attention(fmt)
    cache = [t for t in (att.cache.k, att.cache.v, att.cache.k_scales, att.cache.v_scales) if t is not None]
    for t in cache:
        t.view(torch.uint8).fill_(0x21)
    for _, change in TABLES:
        a = _arguments()
        change(a)
        _refused(lambda: att.decode(a["qkv"], a["slots"], a["pos"], a["table"], a["lens"]), cache + [a["qkv"]])
    for _, change in OFFSETS:
        a = _arguments()
        change(a)
        _refused(lambda: att.prompt(a["qkv"], a["slots"], a["pos"], a["off"]), cache + [a["qkv"]])
    rows = torch.zeros((65537, ROW), dtype=torch.bfloat16, device="cuda")
    n = torch.full((65537,), -1, dtype=torch.int32, device="cuda")
    n[0] = 5
    _refused(lambda: att.decode(rows, n, n, n.view(-1, 1), n), cache + [rows])
    a = _arguments()  # and the calls as they should be
    att.decode(a["qkv"], a["slots"], a["pos"], a["table"], a["lens"])
    assert not torch.all(cache[0].view(torch.uint8) == 0x21)


def test_prompts_of_more_heads_than_a_key_head_serves():
    from mxfp4_routed_expert_router_gb300 import attention as A
    att = A.Attention(65, A.KvCache.empty(2, 1, 16, 64))
    qkv = torch.ones((2, 67 * 64), dtype=torch.bfloat16, device="cuda")
    _refused(lambda: att.prompt(qkv, _i32([0, 1]), None, _i32([0, 2])), [att.cache.k, att.cache.v, qkv])
    got = att.decode(qkv, _i32([0, 16]), None, _i32([[0], [1]]), _i32([1, 1]))
    assert torch.all(got == 1)


def test_heads_and_scales_that_no_call_takes_are_refused_at_once():
    from mxfp4_routed_expert_router_gb300 import attention as A, binding as B
    cache = A.KvCache.empty(2, 2, 16, 64)
    for heads, scale in ((2, 0.0), (2, -1.0), (2, float("nan")), (2, float("inf")), (2, 3e38), (1026, 0.1), (3, 0.1)):
        with pytest.raises(B.MoeError) as e:
            A.Attention(heads, cache, scale=scale)
        assert e.value.status == B.MOE_EINVAL


def test_refused_steps_of_a_block_leave_the_residual_stream():
    b = _block(13)
    cache = [b.attention.cache.k, b.attention.cache.v]
    res = torch.ones((2, 256), device="cuda")
    for _, change in TABLES:
        a = _arguments()
        change(a)
        _refused(lambda: b.decode(res, a["slots"], a["pos"], a["table"], a["lens"]), cache + [res])
    for _, change in OFFSETS:
        a = _arguments()
        change(a)
        _refused(lambda: b.prompt(res, a["slots"], a["pos"], a["off"]), cache + [res])
