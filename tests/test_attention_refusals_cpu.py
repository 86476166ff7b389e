"""Refusals of Attention that need no GPU: what no call takes is refused when it is made, and a call is checked as a whole
before its first write (of which a stand-in for the cache would tell)."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_gb300 import build
    build.build()
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


def _cache(b, kv=2, page=16, device=-1):
    c = b.MoeKvCache(256, 256, None, None, b.MOE_ROWS_BF16, 4, page, kv, 64)
    c.device = device
    wrote = []
    return types.SimpleNamespace(c=c, n_kv_heads=kv, head_dim=64, device=torch.device("cpu"), wrote=wrote,
                                 append=lambda *a: wrote.append("append"), decode=lambda *a: wrote.append("decode"))


@pytest.mark.parametrize("heads,scale", [(2, 0.0), (2, -1.0), (2, float("nan")), (2, float("inf")), (2, 3e38), (2, 1e-60),
                                         (1026, 0.1), (3, 0.1), (0, 0.1)])
def test_heads_and_scales(b, heads, scale):
    from mxfp4_routed_expert_router_gb300 import attention as A
    with pytest.raises(b.MoeError) as e:
        A.Attention(heads, _cache(b), scale=scale)
    assert e.value.status == b.MOE_EINVAL


def test_checks_come_before_writes(b, monkeypatch):
    from mxfp4_routed_expert_router_gb300 import attention as A
    monkeypatch.setattr(b, "_gpu_of", lambda t, cache=None: -1)  # (host tensors as if on the current device)
    cache = _cache(b)
    att = A.Attention(4, cache)
    i32 = torch.int32
    qkv, z = torch.zeros((3, 512), dtype=torch.bfloat16), torch.zeros
    table, lens, off = z((3, 2), dtype=i32), z(3, dtype=i32), z(2, dtype=i32)
    steps = [(qkv, z((2, 2), dtype=i32), lens), (qkv, z((3, 2)), lens), (qkv, z((2, 3), dtype=i32).t(), lens),
             (qkv, z((3, 0), dtype=i32), lens), (qkv, z(3, dtype=i32), lens), (qkv, table, z(2, dtype=i32)),
             (qkv, table, z(3)), (qkv, table, z(6, dtype=i32)[::2]), (qkv[:, :500], table, lens), (qkv[0], table, lens),
             (torch.tensor(0.0), table, lens),
             (qkv[:1].expand(65537, 512), z((65537, 1), dtype=i32), z(65537, dtype=i32))]
    for rows, t, n in steps:
        with pytest.raises(b.MoeError) as e:
            att.decode(rows, None, None, t, n)
        assert e.value.status == b.MOE_EINVAL and not cache.wrote
    for rows, o in ((qkv, z(2)), (qkv, z((2, 1), dtype=i32)), (qkv, z(0, dtype=i32)), (qkv, z(4, dtype=i32)[::2]),
                    (qkv, z(65538, dtype=i32)), (qkv[:, :500], off)):
        with pytest.raises(b.MoeError) as e:
            att.prompt(rows, None, None, o)
        assert e.value.status == b.MOE_EINVAL and not cache.wrote
    many = A.Attention(65, _cache(b, kv=1))
    with pytest.raises(b.MoeError) as e:
        many.prompt(z((3, 67 * 64), dtype=torch.bfloat16), None, None, off)
    assert e.value.status == b.MOE_EINVAL and not many.cache.wrote
    wide = types.SimpleNamespace(**{**vars(_cache(b, page=256)), "wrote": cache.wrote, "append": cache.append})
    with pytest.raises(b.MoeError) as e:
        A.Attention(4, wide).decode(qkv[:1], None, None, torch.empty((1, 1 << 23), dtype=i32), z(1, dtype=i32))
    assert e.value.status == b.MOE_EINVAL and not cache.wrote
