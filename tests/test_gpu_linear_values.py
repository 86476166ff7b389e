"""Every value of moe_linear_forward on the GPU: none unwritten, none NaN that is not one, none lost at the ends of
the formats or to long sums.

Tolerances are those of test_gpu_linear (FP32 accumulation of exact products); a
value that is not a number is outside them, and outputs start as NaN.

F32 rows are also held to an error of 1.5e-5 of the output's norm: an MMA's sum
loses at most half a last place on average (2^-24, times 0.72 over the mantissas),
always towards zero; a random walk's running sum is 2/3 of its last on average, and
a chain has at most 512 MMAs: 512 * 0.72 * 2^-24 * 2/3 = 1.5e-5.  (1152 with MXFP4
weights, whose products of 10 bits fit the accumulator's last places until the sum
has grown: the same bound.)
"""
import inspect

import numpy as np
import pytest
import torch

import test_gpu_linear as base
from test_gpu_linear import Weight, _x

pytestmark = pytest.mark.gpu


def close(got, x, W, out_bf16=False, base=None):
    got = got.float().cpu().numpy().astype(np.float64)
    sick = np.isnan(x).any(1)  # (E4M3 rows of randn * 100 hold a NaN where a value passes 448)
    assert np.isnan(got[sick]).all()
    got, x, base = got[~sick], x[~sick], None if base is None else base[~sick]
    ref = x @ W.w.T
    tol = (W.K / 16 + 32) * 2.0 ** -23 * (np.abs(x) @ W.terms.T)
    if base is not None:
        ref = ref + base
        tol = tol + 2.0 ** -23 * np.abs(ref)
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.isfinite(ref).all() and np.isfinite(tol).all()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def nan_out(lin, T, dtype=torch.float32):
    return torch.full((T, lin.N), float("nan"), dtype=dtype, device="cuda")


def value_tests():
    """The tests of test_gpu_linear that compare values, with each of their parameters."""
    for name, f in sorted(vars(base).items()):
        if name.startswith("test_") and "_check(" in inspect.getsource(f):
            sets = [{}]
            for m in getattr(f, "pytestmark", []):
                if m.name == "parametrize":
                    keys = [k.strip() for k in m.args[0].split(",")]
                    sets = [{**s, **dict(zip(keys, v if len(keys) > 1 else (v,)))} for s in sets for v in m.args[1]]
            for s in sets:
                yield pytest.param(f, s, id="-".join([name[5:]] + [str(v) for v in s.values()]))


@pytest.mark.parametrize("test,args", list(value_tests()))
def test_values_are_written_and_numbers(test, args, monkeypatch):
    """The value tests of test_gpu_linear, whose own comparison lets a NaN pass, with one that does not and with
    outputs that start as NaN."""
    B, Linear = base._mods()

    class Filled(Linear):
        def forward(self, x, x_scales=None, out=None, **kw):
            if out is None and not kw:
                out = nan_out(self, x.shape[0])
            return super().forward(x, x_scales, out=out, **kw)

    monkeypatch.setattr(base, "_check", close)
    monkeypatch.setattr(base, "_mods", lambda: (B, Filled))
    test(**args)


def mx_weight(codes, scales):
    W = Weight.__new__(Weight)
    W.fmt, (W.N, W.K) = "mxfp4", (codes.shape[0], codes.shape[1] * 2)
    W.args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    W.w = base.E2M1[base._nibbles(codes)] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
    W.terms = np.abs(W.w)
    return W


def same_rows(T, row):
    """T equal tokens, as values and as BF16 (which holds them exactly)."""
    x = np.tile(row, (T, 1))
    t = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(t.double().numpy(), x)
    return x, t.cuda()


@pytest.mark.parametrize("T,N", [(1, 64), (8, 64), (9, 64), (200, 10240)])
def test_mxfp4_powers_of_row_and_token_leave_the_range(T, N):
    """The row's power of two times the token's lies outside FP32's range; the sum times both does not.  With one tile
    per CTA and with K split over a cluster."""
    _, Linear = base._mods()
    K = 1024
    W = mx_weight(np.full((N, K // 2), 0x77, np.uint8), np.full((N, K // 32), 37, np.uint8))  # 6 * 2^-90 each
    lin = Linear("mxfp4", *W.args)
    x, xd = same_rows(T, np.full(K, 2.0 ** -46))
    close(lin.forward(xd, out=nan_out(lin, T)), x, W)
    half = nan_out(lin, T, torch.bfloat16)
    close(lin.forward(xd, out=half), x, W, out_bf16=True)
    lin.free()
    # the token's largest value meets weights of zero only; a row of zeros stays zero
    codes = np.full((N, K // 2), 0x11, np.uint8)  # 0.5 * 2^100
    codes[:, 0] = 0x10
    codes[N // 2] = 0
    W = mx_weight(codes, np.full((N, K // 32), 227, np.uint8))
    lin = Linear("mxfp4", *W.args)
    row = np.full(K, 2.0 ** 15)
    row[0] = 2.0 ** 43
    x, xd = same_rows(T, row)
    got = lin.forward(xd, out=nan_out(lin, T))
    close(got, x, W)
    assert torch.all(got[:, N // 2] == 0)
    lin.sync()
    lin.free()


def check_scales(T, lo, hi, p):
    _, Linear = base._mods()
    W = Weight("mxfp4", 70, 512, seed=hi, e_lo=lo, e_hi=hi)
    lin = Linear("mxfp4", *W.args)
    t = torch.from_numpy(np.random.default_rng(hi).standard_normal((T, 512)).astype(np.float32)).to(torch.bfloat16)
    xs = (t.double() * 2.0 ** p).to(torch.bfloat16)
    close(lin.forward(xs.cuda(), out=nan_out(lin, T)), xs.double().numpy(), W)
    lin.sync()
    lin.free()


@pytest.mark.parametrize("T", [9, 40, 200])
@pytest.mark.parametrize("lo,hi,p", [(230, 240, -60), (245, 254, -60), (14, 20, 60), (0, 3, 100)])
def test_mxfp4_scales_at_the_ends(T, lo, hi, p):
    """Block scales far from one, undone by x: neither may leave FP32's range before the other is applied."""
    check_scales(T, lo, hi, p)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 8, 9, 200])
@pytest.mark.parametrize("lo,hi,p", [(230, 240, -60), (245, 254, -60), (0, 250, -30), (14, 20, 60), (0, 3, 100),
                                     (27, 227, 0), (26, 60, 0), (200, 228, -30)])
def test_mxfp4_scales_at_the_ends_few_tokens(T, lo, hi, p):
    """The same for few tokens, and with scales from end to end of the format in a row."""
    check_scales(T, lo, hi, p)


@pytest.mark.parametrize("T", [1, 5, 8])
def test_mxfp4_scales_at_the_ends_rows_and_outputs(T):
    """Few tokens with scales that the weight stream does not take: both types of x and y, strides, accumulation, a
    graph; the workspace that the call then needs is asked for."""
    B, Linear = base._mods()
    N, K = 203, 608
    W = Weight("mxfp4", N, K, seed=T, e_lo=228, e_hi=240)
    lin = Linear("mxfp4", *W.args)
    rng = np.random.default_rng(T)
    codes = torch.from_numpy(rng.standard_normal((T, K + 32)).astype(np.float32)).to(torch.float8_e4m3fn)
    sc = rng.integers(20, 26, (T, K // 32), dtype=np.uint8)
    v = codes[:, :K].float().numpy().astype(np.float64) * np.repeat(2.0 ** (sc.astype(np.float64) - 127), 32, 1)
    t = torch.from_numpy(rng.standard_normal((T, K + 32)) * 2.0 ** -104).to(torch.bfloat16)
    for x, xd, xs in ((v, codes.cuda()[:, :K], torch.from_numpy(sc).cuda()), (t.double().numpy()[:, :K], t.cuda()[:, :K], None)):
        buf = torch.full((T, N + 3), float("nan"), device="cuda")
        close(lin.forward(xd, xs, out=buf[:, :N]), x, W)
        assert torch.isnan(buf[:, N:]).all()
        close(lin.forward(xd, xs, out=nan_out(lin, T, torch.bfloat16)), x, W, out_bf16=True)
        acc = torch.randn((T, N), device="cuda")
        before = acc.cpu().numpy().astype(np.float64)
        close(lin.forward(xd, xs, out=acc, accumulate=True), x, W, base=before)
        out = nan_out(lin, T)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.forward(xd, xs, out=out)
        g.replay()
        torch.cuda.synchronize()
        close(out, x, W)
    assert B.moe_linear_workspace_bytes(lin.handle, T) > 0 and B.moe_linear_workspace_bytes(lin.handle, 0) == 0
    with pytest.raises(B.MoeError) as e:
        B.moe_linear_forward(lin.handle, t.cuda()[:, :K], None, out)
    assert e.value.status == B.MOE_EWORKSPACE
    lin.sync()
    lin.free()


def i4_weight(N, K, large, small, seed):
    """Random codes and zero points; every row's first block has the large scale, the others small ones."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    zeros = rng.integers(0, 16, (N, K // 32), dtype=np.uint8)
    scales = (small * (1 + rng.random((N, K // 32)))).astype(np.float16)
    scales[::2, 0] = large  # (every other row: rows with and without one in a tile)
    W = Weight.__new__(Weight)
    W.fmt, W.N, W.K = "int4g32", N, K
    W.args = tuple(torch.from_numpy(a).cuda() for a in (codes, scales, zeros))
    s, z = (np.repeat(a.astype(np.float64), 32, 1) for a in (scales, zeros))
    W.w, W.terms = s * (base._nibbles(codes) - z), np.abs(s) * (base._nibbles(codes) + z)
    return W


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16, 17, 40, 200])
@pytest.mark.parametrize("large,small", [(65504.0, 2.0 ** -24), (60000.0, 1e-5), (8192.0, 6e-8), (4096.0, 6e-8), (4094.0, 6e-8)])
def test_int4_scales_far_apart_in_a_row(T, large, small):
    """FP16's largest and smallest group scales in one row; x is zero where the large one is, so that only the blocks
    with small ones count."""
    _, Linear = base._mods()
    N, K = 133, 320
    W = i4_weight(N, K, large, small, T)
    lin = Linear("int4g32", *W.args)
    rng = np.random.default_rng(T)
    for xt in ("bf16", "mxfp8"):
        x, xd, sc = _x(rng, T, K, xt, 32)
        xd[:, :32] = 0
        x[:, :32] = 0
        close(lin.forward(xd, sc, out=nan_out(lin, T)), x, W)
        buf = torch.full((T, N + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
        close(lin.forward(xd, sc, out=buf[:, :N]), x, W, out_bf16=True)
        assert torch.isnan(buf[:, N:].float()).all()
        acc = torch.randn((T, N), device="cuda")
        before = acc.cpu().numpy().astype(np.float64)
        close(lin.forward(xd, sc, out=acc, accumulate=True), x, W, base=before)
    lin.sync()
    lin.free()


@pytest.mark.parametrize("fmt", ["mxfp4", "int4g32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(640, 4096, 18432), (9, 512, 18432), (130, 20480, 7168), (640, 4096, 65536)])
def test_f32_rows_of_long_sums(fmt, T, N, K):
    """Long K with so many tiles that nothing else splits it (and with few)."""
    if K == 65536 and fmt == "int4g32":
        pytest.skip("1024 MMAs a chain: a cluster of 8 is the most")
    _, Linear = base._mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(K + T)
    if fmt == "bf16":
        args = ((0.02 * torch.randn((N, K), generator=g, device="cuda")).bfloat16(),)
        w = args[0].double()
    else:
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        w = torch.stack((codes & 15, codes >> 4), -1).view(N, K).long()
        if fmt == "mxfp4":
            sc = torch.randint(117, 122, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
            args = (codes, sc)
            w = torch.from_numpy(base.E2M1).cuda()[w] * torch.exp2(sc.double() - 127).repeat_interleave(32, 1)
        else:
            sc = torch.exp2(torch.rand((N, K // 32), generator=g, device="cuda") * 4 - 11).half()
            z = torch.randint(6, 11, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
            args = (codes, sc, z)
            w = (w - z.double().repeat_interleave(32, 1)) * sc.double().repeat_interleave(32, 1)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    lin = Linear(fmt, *args)
    ref = x.double() @ w.T
    got = lin.forward(x, out=nan_out(lin, T)).double()
    err = float((got - ref).norm() / ref.norm())
    assert err <= 1.5e-5, err
    lin.sync()
    lin.free()


@pytest.mark.parametrize("T", [1, 9, 300])
def test_bf16_weights_on_bf16_rows_use_no_workspace(T):
    B, Linear = base._mods()
    N, K = 130, 224
    W = Weight("bf16", N, K, seed=T)
    lin = Linear("bf16", *W.args)
    x, xd, _ = _x(np.random.default_rng(T), T, K, "bf16", 8)
    out = nan_out(lin, T)
    B.moe_linear_forward(lin.handle, xd, None, out)
    close(out, x, W)
    q, qd, sc = _x(np.random.default_rng(T), T, K, "mxfp8")
    if T > 8:  # rows that are converted need it
        with pytest.raises(B.MoeError) as e:
            B.moe_linear_forward(lin.handle, qd, sc, out)
        assert e.value.status == B.MOE_EWORKSPACE
    close(lin.forward(qd, sc, out=out), q, W)
    lin.sync()
    lin.free()
