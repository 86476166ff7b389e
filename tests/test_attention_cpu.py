"""Refusals of the attention operators that need no GPU: every argument is checked on the host before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_gb300 import build
    build.build()
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


CACHE = dict(k=256, v=256, ks=None, vs=None, type=0, n_pages=4, page=64, kv=2, dim=64)


def _cache(b, **kw):
    v = {**CACHE, **kw}
    return b.MoeKvCache(*[v[k] for k in CACHE])


BAD_CACHES = [
    (dict(type=1), "MOE_EINVAL"), (dict(type=3), "MOE_EINVAL"), (dict(dim=32), "MOE_EDIMS"), (dict(dim=96), "MOE_EDIMS"),
    (dict(dim=256), "MOE_EDIMS"), (dict(page=8), "MOE_EDIMS"), (dict(page=48), "MOE_EDIMS"),
    (dict(page=512), "MOE_EDIMS"), (dict(page=0), "MOE_EDIMS"), (dict(kv=0), "MOE_EINVAL"), (dict(kv=1025), "MOE_EINVAL"),
    (dict(n_pages=0), "MOE_EINVAL"), (dict(n_pages=1 << 26), "MOE_EINVAL"), (dict(k=None), "MOE_EINVAL"),
    (dict(v=None), "MOE_EINVAL"), (dict(k=264), "MOE_EINVAL"), (dict(v=258), "MOE_EINVAL"), (dict(type=2), "MOE_EINVAL"),
    (dict(type=2, ks=256), "MOE_EINVAL"), (dict(type=2, ks=264, vs=256), "MOE_EINVAL"),
]

APPEND = dict(qkv=256, ld=512, T=2, heads=4, slots=256, pos=256, rope=256, n_pos=8, rot=64, style=0, q=256, qld=256,
              ko=256, kld=128)


def _append(b, cache=None, **kw):
    v = {**APPEND, **kw}
    c = _cache(b) if cache is None else cache
    return b.lib.moe_kv_append(ctypes.byref(c), *[v[k] for k in APPEND], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "MOE_EINVAL"), (dict(T=(1 << 24) + 1), "MOE_EINVAL"), (dict(heads=0), "MOE_EINVAL"),
    (dict(heads=1025), "MOE_EINVAL"), (dict(style=2), "MOE_EINVAL"), (dict(rot=8), "MOE_EDIMS"),
    (dict(rot=0), "MOE_EDIMS"), (dict(rot=40), "MOE_EDIMS"), (dict(rot=128), "MOE_EDIMS"), (dict(n_pos=0), "MOE_EDIMS"),
    (dict(qkv=None), "MOE_EINVAL"), (dict(slots=None), "MOE_EINVAL"), (dict(pos=None), "MOE_EINVAL"),
    (dict(ld=511), "MOE_EINVAL"), (dict(ld=504), "MOE_EINVAL"), (dict(qld=248), "MOE_EINVAL"),
    (dict(kld=120), "MOE_EINVAL"), (dict(ld=516), "MOE_EINVAL"), (dict(qkv=264), "MOE_EINVAL"),
    (dict(q=258), "MOE_EINVAL"), (dict(qld=260), "MOE_EINVAL"), (dict(ko=264), "MOE_EINVAL"), (dict(rope=264), "MOE_EINVAL"),
    (dict(slots=258), "MOE_EINVAL"), (dict(pos=257), "MOE_EINVAL"), (dict(T=0), "MOE_OK"),
    (dict(T=0, qkv=None, slots=None), "MOE_OK"),
])
def test_append_refusals(b, kw, status):
    assert _append(b, **kw) == getattr(b, status)


DECODE = dict(q=256, qld=256, B=2, heads=4, table=256, max_pages=4, lens=256, scale=0.1, out=256, old=256, ws=256,
              n=1 << 30)


def _decode(b, cache=None, **kw):
    v = {**DECODE, **kw}
    c = _cache(b) if cache is None else cache
    return b.lib.moe_attention_decode(ctypes.byref(c), *[v[k] for k in DECODE], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "MOE_EINVAL"), (dict(B=65537), "MOE_EINVAL"), (dict(heads=0), "MOE_EINVAL"), (dict(heads=3), "MOE_EINVAL"),
    (dict(heads=1026), "MOE_EINVAL"), (dict(max_pages=0), "MOE_EINVAL"), (dict(max_pages=1 << 25), "MOE_EINVAL"),
    (dict(scale=float("nan")), "MOE_EINVAL"), (dict(scale=float("inf")), "MOE_EINVAL"), (dict(scale=0.0), "MOE_EINVAL"),
    (dict(scale=-1.0), "MOE_EINVAL"), (dict(scale=3e38), "MOE_EINVAL"), (dict(q=None), "MOE_EINVAL"),
    (dict(table=None), "MOE_EINVAL"), (dict(lens=None), "MOE_EINVAL"), (dict(out=None), "MOE_EINVAL"),
    (dict(qld=248), "MOE_EINVAL"), (dict(old=0), "MOE_EINVAL"), (dict(q=264), "MOE_EINVAL"), (dict(qld=260), "MOE_EINVAL"),
    (dict(out=258), "MOE_EINVAL"), (dict(table=258), "MOE_EINVAL"), (dict(lens=257), "MOE_EINVAL"),
    (dict(ws=None), "MOE_EWORKSPACE"), (dict(ws=128), "MOE_EWORKSPACE"), (dict(n=16), "MOE_EWORKSPACE"),
    (dict(B=0), "MOE_OK"), (dict(B=0, q=None, ws=None), "MOE_OK"),
])
def test_decode_refusals(b, kw, status):
    assert _decode(b, **kw) == getattr(b, status)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(b, kw, status):
    c = _cache(b, **kw)
    assert _append(b, c, heads=2, rope=None) == getattr(b, status)
    assert _decode(b, c, heads=c.n_kv_heads) == getattr(b, status)
    assert b.lib.moe_attention_decode(None, 256, 256, 2, 4, 256, 4, 256, 0.1, 256, 256, 256, 1 << 30, None) == b.MOE_EINVAL


def test_decode_workspace(b):
    n = b.moe_attention_decode_workspace_bytes
    assert n(0, 4, 2, 64) == 0 and n(1, 3, 2, 64) == 0 and n(1, 4, 2, 96) == 0 and n(65537, 4, 2, 64) == 0
    assert n(1, 4, 2, 64) > 0 and n(1, 32, 2, 64) > n(1, 16, 2, 64)  # (above 8 heads a key head: parts of 16)


PROMPT = dict(q=256, qld=256, k=256, kld=128, v=256, vld=128, T=8, offsets=256, n=2, heads=4, kv=2, dim=64, scale=0.1,
              out=256, old=256)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "MOE_EINVAL"), (dict(T=(1 << 24) + 1), "MOE_EINVAL"), (dict(n=-1), "MOE_EINVAL"),
    (dict(n=65537), "MOE_EINVAL"), (dict(dim=32), "MOE_EDIMS"), (dict(dim=192), "MOE_EDIMS"), (dict(heads=0), "MOE_EINVAL"),
    (dict(kv=0), "MOE_EINVAL"), (dict(heads=5), "MOE_EINVAL"), (dict(heads=65, kv=1), "MOE_EINVAL"),
    (dict(heads=1026), "MOE_EINVAL"), (dict(scale=0.0), "MOE_EINVAL"), (dict(scale=float("nan")), "MOE_EINVAL"),
    (dict(scale=-0.1), "MOE_EINVAL"), (dict(scale=3e38), "MOE_EINVAL"), (dict(q=None), "MOE_EINVAL"),
    (dict(k=None), "MOE_EINVAL"), (dict(v=None), "MOE_EINVAL"), (dict(offsets=None), "MOE_EINVAL"),
    (dict(out=None), "MOE_EINVAL"), (dict(qld=248), "MOE_EINVAL"), (dict(kld=120), "MOE_EINVAL"),
    (dict(vld=64), "MOE_EINVAL"), (dict(old=128), "MOE_EINVAL"), (dict(q=264), "MOE_EINVAL"), (dict(kld=132), "MOE_EINVAL"),
    (dict(v=258), "MOE_EINVAL"), (dict(out=264), "MOE_EINVAL"), (dict(offsets=258), "MOE_EINVAL"), (dict(T=0), "MOE_OK"),
    (dict(n=0), "MOE_OK"), (dict(T=0, q=None), "MOE_OK"),
])
def test_prompt_refusals(b, kw, status):
    v = {**PROMPT, **kw}
    assert b.lib.moe_attention_prompt(*[v[k] for k in PROMPT], None) == getattr(b, status)


def test_wrappers_check_shapes_types_and_devices(b):
    import torch
    from mxfp4_routed_expert_router_gb300 import attention as A
    bf, i32 = torch.bfloat16, torch.int32
    c = _cache(b)
    qkv = torch.zeros((3, 512), dtype=bf)
    ok = dict(qkv=qkv, heads=4, slots=torch.zeros(3, dtype=i32), pos=torch.zeros(3, dtype=i32), rope=torch.zeros(8, 64),
              style=0, q=torch.zeros((3, 4, 64), dtype=bf), ko=torch.zeros((3, 2, 64), dtype=bf))

    def append(**kw):
        v = {**ok, **kw}
        b.moe_kv_append(c, *[v[k] for k in ok])

    def decode(q=torch.zeros((3, 4, 64), dtype=bf), table=torch.zeros((3, 2), dtype=i32),
               lens=torch.zeros(3, dtype=i32), out=torch.zeros((3, 4, 64), dtype=bf)):
        b.moe_attention_decode(c, q, table, lens, 0.1, out, None, 0)

    def prompt(q=torch.zeros((3, 4, 64), dtype=bf), k=torch.zeros((3, 2, 64), dtype=bf),
               v=torch.zeros((3, 2, 64), dtype=bf), off=torch.zeros(2, dtype=i32), out=torch.zeros((3, 4, 64), dtype=bf)):
        b.moe_attention_prompt(q, k, v, off, 0.1, out)

    calls = [lambda kw=kw: append(**kw) for kw in (
        dict(qkv=qkv.float()), dict(qkv=qkv[:, :500]), dict(qkv=qkv.t()), dict(qkv=qkv[0]), dict(heads=5),
        dict(slots=torch.zeros(2, dtype=i32)), dict(slots=torch.zeros(3)), dict(slots=torch.zeros(6, dtype=i32)[::2]),
        dict(pos=None), dict(pos=torch.zeros(3, dtype=torch.int64)), dict(rope=torch.zeros(8, 64, dtype=bf)),
        dict(rope=torch.zeros(64)), dict(rope=torch.zeros(64, 8).t()), dict(q=ok["q"].float()), dict(q=ok["q"][:2]),
        dict(q=torch.zeros((3, 64, 4), dtype=bf).transpose(1, 2)), dict(q=torch.zeros((4, 3, 64), dtype=bf).transpose(0, 1)),
        dict(ko=ok["q"]), dict())]  # (the last one: right but for its device)
    calls += [lambda kw=kw: decode(**kw) for kw in (
        dict(q=torch.zeros((3, 256), dtype=bf)), dict(q=torch.zeros((3, 4, 64))), dict(q=torch.zeros((3, 4, 32), dtype=bf)),
        dict(table=torch.zeros((2, 2), dtype=i32)), dict(table=torch.zeros((3, 2))),
        dict(table=torch.zeros((2, 3), dtype=i32).t()), dict(lens=torch.zeros(4, dtype=i32)),
        dict(lens=torch.zeros(3, dtype=torch.int64)), dict(out=torch.zeros((3, 4, 64))),
        dict(out=torch.zeros((2, 4, 64), dtype=bf)), dict())]
    calls += [lambda kw=kw: prompt(**kw) for kw in (
        dict(q=torch.zeros((3, 256), dtype=bf)), dict(q=torch.zeros((3, 4, 64))), dict(k=torch.zeros((2, 2, 64), dtype=bf)),
        dict(v=torch.zeros((3, 1, 64), dtype=bf)), dict(off=torch.zeros(2)), dict(off=torch.zeros(0, dtype=i32)),
        dict(off=torch.zeros(4, dtype=i32)[::2]), dict(out=torch.zeros((3, 4, 32), dtype=bf)), dict())]
    z = torch.zeros
    calls += [lambda: A.KvCache(z((2, 2, 64, 64)), z((2, 2, 64, 64))),
              lambda: A.KvCache(z((2, 2, 64, 64), dtype=bf), z((2, 2, 64, 32), dtype=bf)),
              lambda: A.KvCache(z((2, 64, 64), dtype=bf), z((2, 64, 64), dtype=bf)),
              lambda: A.KvCache(z((2, 2, 64, 64), dtype=bf), z((2, 2, 64, 64), dtype=bf), z(1), z(1)),
              lambda: A.KvCache(*[z((2, 2, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)] * 2),
              lambda: A.KvCache(*[z((2, 2, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)] * 2,
                                *[z((2, 2, 64, 4), dtype=torch.uint8)] * 2),
              lambda: A.KvCache(*[z((2, 2, 64, 64), dtype=bf)] * 2),  # (not on a GPU)
              lambda: A.KvCache.empty(2, 2, fmt="fp16")]
    for i, call in enumerate(calls):
        with pytest.raises(b.MoeError) as e:
            call()
        assert e.value.status == b.MOE_EINVAL, i
