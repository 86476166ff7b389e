"""moe_linear_forward on the GPU against a plain NumPy form in 64 bits.

Tolerances.  4-bit weights decode exactly and x keeps its value, so what is left
is FP32 accumulation: per sum at most K / 16 matrix instructions and 32 further
additions, each off by at most 2^-23 of the terms so far: (K / 16 + 32) * 2^-23 *
sum |x||w| for every value (group-32 INT4 sums q and z apart: |s|(q + z) in place
of |w|).  BF16 results round by 2^-8 of the value more.
"""
import threading

import numpy as np
import pytest
import torch

from mxfp4_routed_expert_router_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def _mods():
    from mxfp4_routed_expert_router_gb300 import binding
    from mxfp4_routed_expert_router_gb300.linear import QuantLinear
    return binding, QuantLinear


def _nibbles(codes):
    return np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)


class Weight:
    """A random weight: what the library takes, its values and the terms that the error bound counts."""

    def __init__(self, fmt, N, K, seed, e_lo=117, e_hi=122, with_zeros=True):
        rng = np.random.default_rng(seed)
        self.fmt, self.N, self.K = fmt, N, K
        if fmt == "bf16":
            v = torch.from_numpy((rng.standard_normal((N, K)) * 0.05).astype(np.float32)).to(torch.bfloat16)
            self.args = (v.cuda(),)
            self.w = v.float().numpy().astype(np.float64)
            self.terms = np.abs(self.w)
            return
        if fmt == "mxfp4":
            codes, scales = wl.mx_matrix(rng, N, K, e_lo, e_hi)
            self.args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
            self.w = E2M1[_nibbles(codes)] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
            self.terms = np.abs(self.w)
            return
        codes, bits, zeros = wl.i4_matrix(rng, N, K, 2.0 ** -9, 2.0 ** -5, 0, 15, signed_scales=True)
        if not with_zeros:
            zeros[:] = 8
        s = np.repeat(bits.view(np.float16).astype(np.float64), 32, 1)
        z = np.repeat(zeros.astype(np.float64), 32, 1)
        self.args = (torch.from_numpy(codes).cuda(), torch.from_numpy(bits.view(np.float16)).cuda(),
                     torch.from_numpy(zeros).cuda() if with_zeros else None)
        self.w = s * (_nibbles(codes) - z)
        self.terms = np.abs(s) * (_nibbles(codes) + z)


def _mx8(rng, T, K):
    """Random MXFP8 rows, their values, and the tensors."""
    codes = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32) * 100).to(torch.float8_e4m3fn)
    sc = rng.integers(115, 123, (T, K // 32), dtype=np.uint8)
    v = codes.float().numpy().astype(np.float64) * np.repeat(2.0 ** (sc.astype(np.float64) - 127), 32, 1)
    return v, codes.cuda(), torch.from_numpy(sc).cuda()


def _x(rng, T, K, xt, pad=0):
    if xt == "mxfp8":
        v, c, sc = _mx8(rng, T, K)
        if pad:
            buf = torch.zeros((T, K + pad), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            buf[:, :K].copy_(c)
            c = buf[:, :K]
        return v, c, sc
    t = torch.from_numpy(rng.standard_normal((T, K + pad)).astype(np.float32)).to(torch.bfloat16)
    return t[:, :K].float().numpy().astype(np.float64), t.cuda()[:, :K], None


def _check(got, x, W, out_bf16=False, base=None):
    ref = x @ W.w.T
    tol = (W.K / 16 + 32) * 2.0 ** -23 * (np.abs(x) @ W.terms.T)
    if base is not None:
        ref = ref + base
        tol = tol + 2.0 ** -23 * np.abs(ref)
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = got.float().cpu().numpy().astype(np.float64)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(got - ref).max())


FMTS = ["mxfp4", "int4g32", "bf16"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(1, 32), (17, 96), (130, 256), (256, 1056), (1000, 288), (61, 4128)])
def test_linear_token_counts(fmt, N, K):
    _, Linear = _mods()
    W = Weight(fmt, N, K, seed=N + K)
    lin = Linear(fmt, *W.args)
    rng = np.random.default_rng(5)
    for T in (1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 70):
        x, xt, _ = _x(rng, T, K, "bf16")
        _check(lin.forward(xt), x, W)
    lin.sync()
    lin.free()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T", [1, 2, 4, 7, 24, 130])
def test_linear_rows_and_outputs(fmt, xt, T):
    """Both row types of x, both types of y, accumulation, strided rows on both sides."""
    _, Linear = _mods()
    N, K = 203, 608
    W = Weight(fmt, N, K, seed=T)
    lin = Linear(fmt, *W.args)
    rng = np.random.default_rng(T)
    for pad in (0, 32):
        x, xd, sc = _x(rng, T, K, xt, pad)
        buf = torch.full((T, N + pad), 3.0, device="cuda")
        _check(lin.forward(xd, sc, out=buf[:, :N]), x, W)
        assert torch.all(buf[:, N:] == 3.0)
        base = torch.randn((T, N), device="cuda")
        acc = base.clone()
        _check(lin.forward(xd, sc, out=acc, accumulate=True), x, W, base=base.cpu().numpy().astype(np.float64))
        half = torch.full((T, N + pad), 3.0, device="cuda", dtype=torch.bfloat16)
        _check(lin.forward(xd, sc, out=half[:, :N]), x, W, out_bf16=True)
        assert torch.all(half[:, N:] == 3.0)
    lin.free()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [(1, 7168, 7168), (15, 2048, 18432), (1, 48, 65536), (16, 32, 65536), (40, 16, 65536),
                                   (200, 520, 2048), (513, 300, 1024)])
def test_linear_large_shapes(fmt, T, N, K):
    _, Linear = _mods()
    W = Weight(fmt, N, K, seed=N)
    lin = Linear(fmt, *W.args)
    x, xd, _ = _x(np.random.default_rng(1), T, K, "bf16")
    _check(lin.forward(xd), x, W)
    lin.sync()
    lin.free()


@pytest.mark.parametrize("T", [1, 2, 3, 8, 30, 150])
def test_linear_wide_exponents(T):
    """MXFP4 block exponents over the format's range, x rows at both ends of BF16's."""
    _, Linear = _mods()
    N, K = 64, 512
    # (products stay inside FP32's normal range)
    for lo, hi, powers in ((0, 3, (60,)), (60, 190, (-60, 0, 40)), (100, 160, (-60, 0, 60))):
        W = Weight("mxfp4", N, K, seed=hi, e_lo=lo, e_hi=hi)
        lin = Linear("mxfp4", *W.args)
        rng = np.random.default_rng(hi)
        t = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
        for p in powers:
            xs = t * 2.0 ** p
            x = xs.float().cpu().numpy().astype(np.float64)
            _check(lin.forward(xs), x, W)
        lin.free()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 3, 8, 20, 140])
def test_linear_rows_of_zeros_and_non_finite_rows(fmt, T):
    _, Linear = _mods()
    N, K = 70, 320
    W = Weight(fmt, N, K, seed=3)
    lin = Linear(fmt, *W.args)
    x, xd, _ = _x(np.random.default_rng(2), T, K, "bf16")
    xd[0] = 0
    x[0] = 0
    assert torch.all(lin.forward(xd)[0] == 0)
    if T > 2:
        xd[1, 7] = float("nan")
        xd[2, 33] = float("inf")
    got = lin.forward(xd)
    if T > 2:
        assert torch.all(torch.isnan(got[1])) and not torch.any(torch.isfinite(got[2]))
    rest = [0] + list(range(3, T))
    _check(got[rest], x[rest], W)
    lin.free()


def test_linear_int4_without_zero_points():
    _, Linear = _mods()
    W = Weight("int4g32", 90, 224, seed=8, with_zeros=False)
    lin = Linear("int4g32", *W.args)
    for T in (1, 6, 40):
        x, xd, _ = _x(np.random.default_rng(T), T, 224, "bf16")
        _check(lin.forward(xd), x, W)
    lin.free()


def test_linear_repeats_bit_for_bit():
    _, Linear = _mods()
    for fmt in FMTS:
        W = Weight(fmt, 500, 7168, seed=4)
        lin = Linear(fmt, *W.args)
        for T in (1, 5, 16, 200):
            _, xd, _ = _x(np.random.default_rng(T), T, 7168, "bf16")
            first = lin.forward(xd)
            for _ in range(3):
                assert torch.equal(lin.forward(xd), first)
        lin.free()


def test_linear_streams_graphs_and_freed_weights():
    _, Linear = _mods()
    W = Weight("mxfp4", 300, 1024, seed=6)
    lin = Linear("mxfp4", *W.args)
    for a in W.args:
        a.zero_()  # the library has its own copy
    rng = np.random.default_rng(6)
    for T in (1, 12, 160):
        x, xd, _ = _x(rng, T, 1024, "bf16")
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(3)]
        outs = [torch.empty((T, 300), device="cuda") for _ in side]
        torch.cuda.synchronize()
        for _ in range(5):
            for s, o in zip(side, outs):  # one handle on several streams at a time
                lin.forward(xd, out=o, stream=s)
        torch.cuda.synchronize()
        for o in outs:
            _check(o, x, W)
        buf = torch.zeros_like(xd)
        out = torch.empty((T, 300), device="cuda")
        lin.forward(buf, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.forward(buf, out=out)
        buf.copy_(xd)
        g.replay()
        torch.cuda.synchronize()
        _check(out, x, W)
    lin.free()


def test_linear_calls_share_a_streams_workspace():
    """Calls of several layers and sizes on one stream, without waiting, and a captured call replayed on another."""
    _, Linear = _mods()
    Ws = [Weight("mxfp4", 260, 512, seed=8), Weight("int4g32", 130, 1024, seed=9)]
    lins = [Linear(W.fmt, *W.args) for W in Ws]
    rng = np.random.default_rng(8)
    calls = []  # sizes that grow, so that the workspace is replaced while calls are in flight
    for T in (9, 40, 17, 300, 11, 700):
        for W, lin in zip(Ws, lins):
            x, xd, _ = _x(rng, T, W.K, "bf16")
            calls.append((lin, W, x, xd, torch.empty((T, W.N), device="cuda")))
    buf = [torch.zeros((50, W.K), dtype=torch.bfloat16, device="cuda") for W in Ws]
    got = [torch.empty((50, W.N), device="cuda") for W in Ws]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for lin, b, o in zip(lins, buf, got):
            lin.forward(b, out=o)
    fresh = [_x(rng, 50, W.K, "bf16") for W in Ws]
    for b, f in zip(buf, fresh):
        b.copy_(f[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(side):
            g.replay()
        for lin, _, _, xd, o in calls:
            lin.forward(xd, out=o)
    torch.cuda.synchronize()
    for lin, W, x, _, o in calls:
        _check(o, x, W)
    for W, f, o in zip(Ws, fresh, got):
        _check(o, f[0], W)
    for lin in lins:
        lin.free()


def test_linear_threads_on_one_stream():
    """Two threads whose calls interleave on the same stream do not share a workspace."""
    _, Linear = _mods()
    W = Weight("mxfp4", 200, 512, seed=10)
    lin = Linear(W.fmt, *W.args)
    rng = np.random.default_rng(10)
    xs = [[_x(rng, T, 512, "bf16") for T in (20, 65, 9)] for _ in range(2)]
    outs = [[torch.empty((x[0].shape[0], 200), device="cuda") for x in row] for row in xs]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(30):
            for x, o in zip(xs[i], outs[i]):
                lin.forward(x[1], out=o)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for row, out in zip(xs, outs):
        for x, o in zip(row, out):
            _check(o, x[0], W)
    lin.free()


def test_linear_refusals():
    B, Linear = _mods()
    W = Weight("mxfp4", 40, 64, seed=1)
    lin = Linear("mxfp4", *W.args)
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 40), 5.0, device="cuda")

    def refused(status, call):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.status == status

    refused(B.MOE_EINVAL, lambda: lin.forward(x[:, :32], out=out))
    refused(B.MOE_EINVAL, lambda: lin.forward(x.float(), out=out))
    refused(B.MOE_EINVAL, lambda: lin.forward(x, out=out[:, :39]))
    refused(B.MOE_EINVAL, lambda: lin.forward(x, out=out.bfloat16(), accumulate=True))
    refused(B.MOE_EINVAL, lambda: lin.forward(x, accumulate=True))
    refused(B.MOE_EINVAL, lambda: lin.forward(x.to(torch.float8_e4m3fn), out=out))
    odd = torch.zeros((3, 65), dtype=torch.bfloat16, device="cuda")
    refused(B.MOE_EINVAL, lambda: lin.forward(odd[:, :64], out=out))
    refused(B.MOE_EINVAL, lambda: lin.forward(odd[:, 1:], out=out))
    bad = W.args[1].clone()
    bad[7, 1] = 255
    refused(B.MOE_ESCALE, lambda: Linear("mxfp4", W.args[0], bad))
    I4 = Weight("int4g32", 40, 64, seed=1)
    z = I4.args[2].clone()
    z[3, 0] = 16
    refused(B.MOE_ESCALE, lambda: Linear("int4g32", I4.args[0], I4.args[1], z))
    s = I4.args[1].clone()
    s[0, 1] = float("inf")
    refused(B.MOE_ESCALE, lambda: Linear("int4g32", I4.args[0], s))
    torch.cuda.synchronize()
    assert torch.all(out == 5.0)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert lin.forward(e).shape == (0, 40)
    lin.free()


@pytest.mark.parametrize("fmt", FMTS + ["mxfp4 wide"])
@pytest.mark.parametrize("T", [9, 33, 65, 97, 128, 129, 300])
def test_linear_gemm_ring_depths(fmt, T):
    """The tcgen05 GEMM with one to many weight chunks per CTA, on every depth of its rings; rows of MXFP4 exponents
    too wide for FP16 operands; results repeat bit for bit, from L2 and from HBM."""
    _, Linear = _mods()
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    wide = fmt.endswith("wide")
    fmt = fmt.split()[0]
    for N, K in ((130, 32), (260, 160), (100, 640), (513, 1504), (128, 3136), (1030, 4704)):
        W = Weight(fmt, N, K, seed=K + T, **({"e_lo": 100, "e_hi": 140} if wide else {}))
        lin = Linear(fmt, *W.args)
        x, xd, _ = _x(np.random.default_rng(K), T, K, "bf16")
        first = lin.forward(xd)
        _check(first, x, W)
        for i in range(6):
            if i % 2:
                flush.fill_(i)
            assert torch.equal(lin.forward(xd), first)
        lin.sync()
        lin.free()
