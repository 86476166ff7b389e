"""MoeBlock on the GPU against its definition in 64 bits (NumPy, and the CPU oracle for the experts).

The experts' output is held to the layer's bound, 1e-2 of its rms.  Everything
else is FP32 sums of exact products and one rounding of x: below 1e-4 of the
stream's rms at these sizes; 4-bit projections of the norm's MXFP8 rows also
carry E4M3's 2^-4 of each value, below 2^-4 * sum |n||w| / sqrt(count) * 4.
"""
import numpy as np
import pytest
import torch

import oracle
from parity_util import oracle_weights
from test_gpu_linear import Weight
from test_gpu_route_grouped import expected as expected_routing

from mxfp4_routed_expert_router_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

H, A, E = 256, 192, 16


def _block(seed):
    from mxfp4_routed_expert_router_gb300 import layer
    from mxfp4_routed_expert_router_gb300.block import MoeBlock, Routing
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    cfg = wl.custom("block", 1, H, 128, E, 1, 4, seed)
    rng = np.random.default_rng(seed)
    ws = {"out": Weight("mxfp4", H, A, seed + 1, 115, 119), "router": Weight("bf16", E, H, seed + 2),
          "in": Weight("int4g32", 320, H, seed + 3)}
    gain = torch.from_numpy(1 + 0.1 * rng.standard_normal(H)).float()
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b = MoeBlock(layer.MoeLayer(cfg), QuantLinear("bf16", *ws["router"].args), Routing(4, 4, 2, scale=1.5),
                 gain.cuda(), torch.from_numpy(bias).cuda(), QuantLinear("mxfp4", *ws["out"].args),
                 QuantLinear("int4g32", *ws["in"].args), gain.cuda())
    return cfg, b, ws, gain.numpy().astype(np.float64), bias


def _norm(r, gain):
    return r / np.sqrt((r * r).mean(1, keepdims=True) + 1e-6) * gain


@pytest.mark.parametrize("T", [1, 7, 40, 300])
def test_block_matches_its_definition(T):
    cfg, b, ws, gain, bias = _block(50)
    rng = np.random.default_rng(T)
    res = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    attn = torch.from_numpy(rng.standard_normal((T, A)).astype(np.float32)).to(torch.bfloat16)
    stream = res.cuda()
    got_in = b.project_in(stream).float().cpu().numpy().astype(np.float64)
    n = _norm(res.double().numpy(), gain)
    tol = 2.0 ** -8 * np.abs(n @ ws["in"].w.T) + 2.0 ** -4 * np.sqrt((n ** 2) @ (ws["in"].w.T ** 2)) * 4 + 1e-4
    assert np.all(np.abs(got_in - n @ ws["in"].w.T) <= tol)
    out = b.forward(attn.cuda(), stream)
    b.layer.sync()
    assert out.data_ptr() == stream.data_ptr()
    r = res.double().numpy() + attn.double().numpy() @ ws["out"].w.T
    x = torch.from_numpy(_norm(r, gain)).to(torch.bfloat16)
    logits = x.double().numpy() @ ws["router"].w.T
    ids, w = expected_routing(logits, bias, 4, 4, 2, "sigmoid", "top2", True, 1.5)
    y = oracle.moe_layer_routed(oracle_weights(cfg, range(E)), x.view(torch.int16).numpy().view(np.uint16), ids,
                                w.astype(np.float32))
    err = np.abs(out.cpu().numpy().astype(np.float64) - (r + y))
    assert err.max() <= 1e-2 * np.sqrt(np.mean(y ** 2)) + 1e-4 * np.sqrt(np.mean(r ** 2))


def test_block_in_a_graph_and_on_a_side_stream():
    cfg, b, *_ = _block(60)
    for T in (1, 24):
        attn = torch.randn((T, A), device="cuda").bfloat16()
        res = torch.randn((T, H), device="cuda")
        want = b.forward(attn, res.clone()).clone()
        side = torch.cuda.Stream()
        got = res.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            b.forward(attn, got)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        buf = res.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.forward(attn, buf)
        buf.copy_(res)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want)


@pytest.mark.parametrize("T", [1, 6, 20])
def test_block_steps_without_waiting(T):
    """Kernels of one step start while those of the step before still end: many steps enqueued at once, other work
    between them, give what the same steps give one at a time."""
    cfg, b, *_ = _block(70)
    steps = 40
    attn = [torch.randn((T, A), device="cuda").bfloat16() for _ in range(steps)]
    res0 = torch.randn((T, H), device="cuda")
    one, want = res0.clone(), []
    for a in attn:
        q = b.project_in(one)
        torch.cuda.synchronize()
        b.forward(a, one)
        torch.cuda.synchronize()
        want.append((q.clone(), one.clone()))
        one.mul_(0.5)
        torch.cuda.synchronize()
    for _ in range(5):
        res, got = res0.clone(), []
        for a in attn:
            q = b.project_in(res)
            b.forward(a, res)
            got.append((q, res.clone()))
            res.mul_(0.5)
        torch.cuda.synchronize()
        for (q, r), (wq, wr) in zip(got, want):
            assert torch.equal(q, wq) and torch.equal(r, wr)


def test_operators_in_a_graph_beside_copies():
    """Captured after and between copies and memsets, as a serving step is."""
    cfg, b, *_ = _block(80)
    T = 5
    host_attn = torch.randn((T, A)).bfloat16().pin_memory()
    host_res = torch.randn((T, H)).pin_memory()
    attn, res = torch.zeros((T, A), device="cuda", dtype=torch.bfloat16), torch.zeros((T, H), device="cuda")
    out = torch.empty((T, H), device="cuda")
    b.project_in(res)
    b.forward(attn, res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.copy_(host_attn, non_blocking=True)
        res.copy_(host_res, non_blocking=True)
        q = b.project_in(res)
        b.forward(attn, res)
        out.copy_(res)
        res.zero_()
        q2 = b.project_in(out)
    for i in range(4):
        host_attn.copy_(torch.randn((T, A)).bfloat16())
        host_res.copy_(torch.randn((T, H)))
        g.replay()
        torch.cuda.synchronize()
        r = host_res.cuda()
        assert torch.equal(b.project_in(r), q)
        b.forward(host_attn.cuda(), r)
        assert torch.equal(out, r) and torch.equal(b.project_in(r), q2) and not res.any()


def test_block_graph_outlives_larger_calls():
    """A graph captured with one token is replayed after calls and captures of many, and after other tensors have
    taken whatever memory those gave back."""
    cfg, b, *_ = _block(90)
    attn = {T: torch.randn((T, A), device="cuda").bfloat16() for T in (1, 24, 300)}
    res = {T: torch.randn((T, H), device="cuda") for T in attn}
    want, graphs, bufs = {}, {}, {}
    for T in attn:
        want[T] = b.forward(attn[T], res[T].clone()).clone()
        bufs[T] = res[T].clone()
        graphs[T] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[T]):
            b.forward(attn[T], bufs[T])
    torch.cuda.synchronize()
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 18, 1 << 22, 1 << 24, 1 << 24)]
    for T in attn:
        bufs[T].copy_(res[T])
        graphs[T].replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[T], want[T])
    assert all((o == 7).all() for o in others)


def test_block_on_streams_at_a_time():
    """One block on three streams without an order between them: each gets what it gets alone."""
    cfg, b, *_ = _block(91)
    sizes = (3, 24, 70)
    attn = [torch.randn((T, A), device="cuda").bfloat16() for T in sizes]
    res = [torch.randn((T, H), device="cuda") for T in sizes]
    want = []
    for a, r in zip(attn, res):
        one = r.clone()
        for _ in range(4):
            b.forward(a, one)
        torch.cuda.synchronize()
        want.append(one)
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [r.clone() for r in res]
    torch.cuda.synchronize()
    for i in range(4):
        for s, a, g in zip(streams, attn, got):
            with torch.cuda.stream(s):
                b.forward(a, g)
    torch.cuda.synchronize()
    b.layer.sync()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
