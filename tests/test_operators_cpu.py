"""Refusals of the operators around the layer that need no GPU: every argument
is checked on the host before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_gb300 import build
    build.build()
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


NORM = dict(residual=256, rt=0, rld=64, delta=256, dt=0, dld=64, gain=256, gt=1, eps=1e-6, T=2, H=64, sum=256, sld=64,
            y=256, yld=64, q=256, qld=64, qs=256)


def _norm(b, **kw):
    v = {**NORM, **kw}
    return b.lib.moe_add_rmsnorm(*[v[k] for k in NORM], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "MOE_EINVAL"), (dict(T=(1 << 24) + 1), "MOE_EINVAL"), (dict(H=0), "MOE_EDIMS"),
    (dict(H=48), "MOE_EDIMS"), (dict(H=65568), "MOE_EDIMS"), (dict(rt=2), "MOE_EINVAL"), (dict(dt=2), "MOE_EINVAL"),
    (dict(gt=-1), "MOE_EINVAL"), (dict(eps=-1.0), "MOE_EINVAL"), (dict(eps=float("nan")), "MOE_EINVAL"),
    (dict(eps=float("inf")), "MOE_EINVAL"), (dict(residual=None), "MOE_EINVAL"),
    (dict(sum=None, y=None, q=None), "MOE_EINVAL"), (dict(qs=None), "MOE_EINVAL"), (dict(rld=63), "MOE_EINVAL"),
    (dict(dld=32), "MOE_EINVAL"), (dict(sld=0), "MOE_EINVAL"), (dict(yld=-64), "MOE_EINVAL"), (dict(qld=8), "MOE_EINVAL"),
    (dict(residual=264), "MOE_EINVAL"), (dict(rld=68), "MOE_EINVAL"), (dict(delta=258), "MOE_EINVAL"),
    (dict(y=272 + 2), "MOE_EINVAL"), (dict(q=257), "MOE_EINVAL"), (dict(qld=72), "MOE_EINVAL"),
    (dict(gain=260), "MOE_EINVAL"), (dict(T=0), "MOE_OK"), (dict(T=0, residual=None), "MOE_OK"),
])
def test_norm_refusals(b, kw, status):
    assert _norm(b, **kw) == getattr(b, status)


ROUTE = dict(logits=256, bias=256, T=2, E=64, k=4, G=8, KG=2, score=1, gs=1, renorm=1, scale=1.0, ids=256, w=256)


def _route(b, **kw):
    v = {**ROUTE, **kw}
    return b.lib.moe_route_grouped(*[v[k] for k in ROUTE], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "MOE_EINVAL"), (dict(T=(1 << 24) + 1), "MOE_EINVAL"), (dict(E=0), "MOE_EINVAL"),
    (dict(E=1025), "MOE_EINVAL"), (dict(G=0), "MOE_EINVAL"), (dict(G=7), "MOE_EINVAL"), (dict(G=64), "MOE_EINVAL"),
    (dict(KG=0), "MOE_EINVAL"), (dict(KG=9), "MOE_EINVAL"), (dict(k=0), "MOE_EINVAL"), (dict(k=17), "MOE_EINVAL"),
    (dict(k=33, KG=8), "MOE_EINVAL"), (dict(score=2), "MOE_EINVAL"), (dict(gs=-1), "MOE_EINVAL"),
    (dict(logits=None), "MOE_EINVAL"), (dict(ids=None), "MOE_EINVAL"), (dict(w=None), "MOE_EINVAL"),
    (dict(logits=258), "MOE_EINVAL"), (dict(bias=257), "MOE_EINVAL"), (dict(ids=262), "MOE_EINVAL"),
    (dict(T=0), "MOE_OK"), (dict(T=0, logits=None), "MOE_OK"),
])
def test_route_refusals(b, kw, status):
    assert _route(b, **kw) == getattr(b, status)


def test_linear_refusals(b):
    L = b.lib
    h = ctypes.c_void_p()
    mx = b.MoeMx(256, 256, None)

    def load(N=16, K=64, fmt=b.MOE_W_MXFP4, w=mx, out=h):
        return L.moe_linear_load(N, K, fmt, None if w is None else ctypes.byref(w), None,
                                 None if out is None else ctypes.byref(out))

    assert load(w=None) == b.MOE_EINVAL and load(out=None) == b.MOE_EINVAL
    assert load(fmt=5) == b.MOE_EINVAL
    assert load(N=0) == b.MOE_EINVAL and load(N=(1 << 20) + 1) == b.MOE_EINVAL
    for K in (0, 31, 48, 65568):
        assert load(K=K) == b.MOE_EDIMS
    assert load(w=b.MoeMx(None, 256, None)) == b.MOE_EINVAL
    assert load(w=b.MoeMx(256, None, None)) == b.MOE_EINVAL
    assert load(fmt=b.MOE_W_INT4G32, w=b.MoeMx(256, 257, None)) == b.MOE_EINVAL
    assert b"2-byte aligned" in L.moe_last_error()
    assert h.value is None
    assert L.moe_linear_forward(None, 256, 0, 64, None, 1, 256, 1, 16, 0, None, 0, None) == b.MOE_EINVAL
    assert L.moe_linear_workspace_bytes(None, 4) == 0
    assert L.moe_linear_sync_status(None, None) == b.MOE_EINVAL
    L.moe_linear_free(None)  # no-op


def test_wrappers_check_shapes_and_types(b):
    import torch
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    x = torch.zeros((3, 64))
    for call in (lambda: b.moe_add_rmsnorm(x, x[:2], None, 1e-6, x),
                 lambda: b.moe_add_rmsnorm(x, None, torch.ones(63), 1e-6, x),
                 lambda: b.moe_add_rmsnorm(x, None, None, 1e-6, x.bfloat16()),
                 lambda: b.moe_add_rmsnorm(x, None, None, 1e-6, None, x),
                 lambda: b.moe_add_rmsnorm(x.half(), None, None, 1e-6, x.half()),
                 lambda: b.moe_add_rmsnorm(x.t(), None, None, 1e-6, None),
                 lambda: b.moe_add_rmsnorm(x, None, None, 1e-6, None, None, x.to(torch.float8_e4m3fn),
                                           torch.zeros((3, 3), dtype=torch.uint8)),
                 lambda: QuantLinear("mxfp3", x),
                 lambda: QuantLinear("mxfp4", x, x),
                 lambda: QuantLinear("mxfp4", torch.zeros((4, 32), dtype=torch.uint8)),
                 lambda: QuantLinear("mxfp4", torch.zeros((4, 32), dtype=torch.uint8),
                                     torch.zeros((4, 3), dtype=torch.uint8)),
                 lambda: QuantLinear("int4g32", torch.zeros((4, 32), dtype=torch.uint8),
                                     torch.zeros((4, 2), dtype=torch.uint8)),
                 lambda: QuantLinear("bf16", torch.zeros((4, 64)))):
        with pytest.raises(b.MoeError) as e:
            call()
        assert e.value.status == b.MOE_EINVAL


def _refused(b, calls):
    for i, call in enumerate(calls):
        with pytest.raises(b.MoeError) as e:
            call()
        assert e.value.status == b.MOE_EINVAL, i


def test_route_wrapper_checks_shapes_and_types(b, monkeypatch):
    """Bare addresses reach the library only from tensors of the right type and size."""
    import torch
    T, E, k = 3, 16, 4
    reached = []
    monkeypatch.setattr(b, "_stream", lambda s: None)
    monkeypatch.setattr(b.lib, "moe_route_grouped", lambda *a: reached.append(a) or 0)
    good = dict(logits=torch.zeros(T, E), bias=torch.zeros(E), ids=torch.zeros((T, k), dtype=torch.int32),
                w=torch.zeros(T, k))

    def call(**kw):
        v = {**good, **kw}
        b.moe_route_grouped(v["logits"], v["bias"], T, E, k, 4, 2, b.MOE_SCORE_SIGMOID, b.MOE_GROUP_MAX, True, 1.0,
                            v["ids"], v["w"])

    _refused(b, [lambda kw=kw: call(**kw) for kw in (
        dict(logits=good["logits"].bfloat16()), dict(logits=good["logits"].double()), dict(logits=torch.zeros(T, E - 1)),
        dict(logits=torch.zeros(T - 1, E)), dict(logits=torch.zeros(E, T).t()), dict(logits=torch.zeros(T, 2 * E)[:, :E]),
        dict(logits=torch.zeros(T, 2 * E)),
        dict(logits=torch.zeros(E, T)), dict(bias=torch.zeros(E, dtype=torch.bfloat16)), dict(bias=torch.zeros(E - 1)),
        dict(bias=torch.zeros(2 * E)[::2]), dict(ids=good["ids"].long()), dict(ids=good["ids"].float()),
        dict(ids=torch.zeros((T, k - 1), dtype=torch.int32)), dict(ids=torch.zeros(T * k - 1, dtype=torch.int32)),
        dict(w=good["w"].half()), dict(w=torch.zeros(T, k - 1)), dict(w=torch.zeros(k, T).t()))])
    assert not reached
    call()
    call(bias=None)
    call(logits=torch.zeros(T + 2, E), ids=torch.zeros(T * k, dtype=torch.int32), w=torch.zeros(T + 1, k))
    call(logits=256, bias=512, ids=1024, w=2048)  # plain addresses
    assert len(reached) == 4 and reached[3][0] == 256


def test_linear_wrapper_checks_the_scales_of_x(b, monkeypatch):
    """E8M0 scales are bytes: a wider type of the same shape would be read as other numbers."""
    import torch
    T, K = 3, 64
    reached = []
    monkeypatch.setattr(b, "_stream", lambda s: None)
    monkeypatch.setattr(b.lib, "moe_linear_forward", lambda *a: reached.append(a) or 0)
    x, y = torch.zeros(T, K).to(torch.float8_e4m3fn), torch.zeros(T, 8)
    good = torch.zeros((T, K // 32), dtype=torch.uint8)
    _refused(b, [lambda sc=sc: b.moe_linear_forward(1, x, sc, y) for sc in (
        good.float(), good.to(torch.float16), good.int(), good[:2], good[:, :1], torch.zeros((2, T), dtype=torch.uint8).t(),
        torch.zeros((T, 4), dtype=torch.uint8)[:, ::2], good.view(-1))])
    assert not reached
    for sc in (good, good.view(torch.float8_e8m0fnu), None):
        b.moe_linear_forward(1, x, sc, y)
    assert len(reached) == 3


def test_quant_linear_checks_the_scales_of_x(b, monkeypatch):
    import torch
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    reached = []
    monkeypatch.setattr(b, "_stream", lambda s: None)
    monkeypatch.setattr(b.lib, "moe_linear_forward", lambda *a: reached.append(a) or 0)
    lin = QuantLinear.__new__(QuantLinear)
    lin.handle, lin.N, lin.K, lin._no_ws, lin.device = None, 8, 64, 8, torch.device("cpu")
    x, out = torch.zeros(3, 64).to(torch.float8_e4m3fn), torch.zeros(3, 8)
    _refused(b, [lambda dt=dt: lin.forward(x, torch.zeros((3, 2), dtype=dt), out=out)
                 for dt in (torch.float32, torch.float16, torch.int64)])
    assert not reached
    lin.forward(x, torch.zeros((3, 2), dtype=torch.uint8), out=out)
    assert len(reached) == 1


class _Calls:
    """Stands for the library: records which entry points a block reaches."""

    def __init__(self, b, monkeypatch):
        import torch
        self.names = []
        monkeypatch.setattr(b, "_stream", lambda s: None)
        monkeypatch.setattr(b, "_current_stream", lambda: 11)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        for name in ("moe_add_rmsnorm", "moe_linear_forward", "moe_forward_routed"):
            monkeypatch.setattr(b.lib, name, lambda *a, name=name: self.names.append((name, a)) or 0)
        real = b.lib.moe_route_grouped  # (argument checks only: no tokens reach a kernel)
        monkeypatch.setattr(b.lib, "moe_route_grouped",
                            lambda *a: self.names.append(("moe_route_grouped", a)) or (real(*a) if a[2] == 0 else 0))
        monkeypatch.setattr(b.lib, "moe_workspace_bytes", lambda h, T, k: 4096 * T)


def _linear(N, K):
    import torch
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    lin = QuantLinear.__new__(QuantLinear)
    lin.handle, lin.N, lin.K, lin._no_ws, lin.device = None, N, K, 1 << 20, torch.device("cpu")
    return lin


def _layer(H, E, k):
    import types

    import torch
    from mxfp4_routed_expert_router_gb300.layer import MoeLayer
    layer = MoeLayer.__new__(MoeLayer)
    layer.handle, layer._ws, layer.dense, layer.device = None, None, False, torch.device("cpu")
    layer.cfg, layer.config = types.SimpleNamespace(hidden=H, n_experts=E, k=k), types.SimpleNamespace(k_max=k)
    return layer


def test_block_refuses_rows_that_the_experts_cannot_take(b, monkeypatch):
    """The residual stream goes to the experts as dense FP32 rows: any other is refused before it is touched."""
    import torch
    from mxfp4_routed_expert_router_gb300.block import MoeBlock, Routing
    calls = _Calls(b, monkeypatch)
    T, H, E = 5, 64, 16
    block = MoeBlock(_layer(H, E, 4), _linear(E, H), Routing(4, 4, 2))
    attn = torch.zeros((T, H), dtype=torch.bfloat16)
    calls.names.clear()
    good = torch.zeros(T, H)
    _refused(b, [lambda r=r: block.forward(attn, r) for r in (
        good.bfloat16(), good.double(), torch.zeros(T, 2 * H)[:, :H], torch.zeros(2 * T, H)[::2], torch.zeros(H, T).t(),
        torch.zeros(T, 32), torch.zeros(T, 96), torch.zeros(T * H))])
    assert not calls.names
    block.forward(attn, good)
    assert [n for n, _ in calls.names] == ["moe_add_rmsnorm", "moe_linear_forward", "moe_route_grouped",
                                           "moe_forward_routed"]


def test_block_refuses_parts_that_do_not_fit(b, monkeypatch):
    import torch
    from mxfp4_routed_expert_router_gb300.block import MoeBlock, Routing
    _Calls(b, monkeypatch)
    H, E = 64, 16
    good = dict(layer=_layer(H, E, 4), router=_linear(E, H), routing=Routing(4, 4, 2), bias=torch.zeros(E),
                out_proj=_linear(H, 96), in_proj=_linear(200, H))
    MoeBlock(**good)
    dense = _layer(H, E, 4)
    dense.dense = True
    _refused(b, [lambda kw=kw: MoeBlock(**{**good, **kw}) for kw in (
        dict(bias=torch.zeros(E, dtype=torch.bfloat16)), dict(bias=torch.zeros(E + 1)), dict(bias=torch.zeros(2 * E)[::2]),
        dict(router=_linear(E, 96)), dict(out_proj=_linear(96, H)), dict(in_proj=_linear(200, 96)),
        dict(routing=Routing(5, 4, 2)), dict(routing=Routing(4, 3, 2)), dict(routing=Routing(4, 4, 5)),
        dict(routing=Routing(0, 4, 2)), dict(routing=Routing(4, 4, 2, score=7)), dict(layer=dense))])


def test_block_workspaces_of_streams_and_captures(b, monkeypatch):
    """The experts' workspace is the stream's, or the captured call's own: never one that calls on two streams share,
    nor one that a later call of more tokens frees while a graph still holds its address."""
    import gc

    import torch
    from mxfp4_routed_expert_router_gb300 import linear
    from mxfp4_routed_expert_router_gb300.block import MoeBlock, Routing
    calls = _Calls(b, monkeypatch)
    now = dict(stream=11, capturing=False)
    monkeypatch.setattr(b, "_current_stream", lambda: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(linear, "_workspaces", linear._Workspaces())
    H, E = 64, 16
    block = MoeBlock(_layer(H, E, 4), _linear(E, H), Routing(4, 4, 2))

    kept = []  # captured calls' memory belongs to their graphs: here every tensor made while capturing lives on
    empty = torch.empty
    monkeypatch.setattr(linear.torch, "empty",
                        lambda *a, **kw: (kept.append(empty(*a, **kw)) or kept[-1]) if now["capturing"] else empty(*a, **kw))

    def ran(T, stream, capturing=False):
        now.update(stream=stream, capturing=capturing)
        calls.names.clear()
        block.forward(torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros(T, H))
        at, size = [a for n, a in calls.names if n == "moe_forward_routed"][0][8:10]
        assert at and size >= 4096 * T
        return at, size

    one, other = ran(3, 11), ran(3, 22)
    assert one[0] != other[0], "two streams share the experts' workspace"
    assert ran(2, 11)[0] == one[0], "the stream's calls share it"
    graph = ran(1, 11, capturing=True)
    mine = [t for t in kept if t.data_ptr() == graph[0]]
    assert mine and graph[0] not in (one[0], other[0]), "a captured call has bytes of its graph's own"
    bigger = ran(300, 11)
    gc.collect()
    assert bigger[0] != graph[0] and ran(3, 22) == other
    assert block.layer._ws is None
    calls.names.clear()
