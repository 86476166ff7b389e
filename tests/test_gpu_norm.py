"""moe_add_rmsnorm on the GPU against a plain NumPy form in 64 bits.

Tolerances.  The sum is one FP32 addition and one rounding: equal bit for bit.
n = s * rinv * g in FP32: the sum of squares adds positive terms (at most 8 * VPT
+ 5 + 32 <= 101 additions deep, a relative 101 * 2^-24, halved by the root),
rsqrtf is within 2 ulp and two products round: below 2^-18 of n in all.  BF16
rounds by 2^-8 of the value more; E4M3 by 2^-4 of the value, or by half of its
smallest step, 2^-10 in units of the block's scale.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _B():
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


def _rows(rng, T, H, pad, dtype, scale=1.0):
    buf = torch.from_numpy((rng.standard_normal((T, H + pad)) * scale).astype(np.float32)).to(dtype).cuda()
    return buf[:, :H]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _expected(residual, delta, gain, eps):
    s = residual.float().cpu()
    if delta is not None:
        s = s + delta.float().cpu()
    s = s.to(residual.dtype)
    v = _np(s)
    n = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return s, n * (1.0 if gain is None else _np(gain)[None, :])


def _check(n, y, q, q_scales):
    n = np.asarray(n)
    if y is not None:
        assert np.all(np.abs(_np(y) - n) <= np.abs(n) * (2.0 ** -8 + 2.0 ** -18))
    if q is not None:
        p = q_scales.cpu().numpy().astype(np.float64) - 127
        unit = np.repeat(2.0 ** p, 32, axis=1)
        got = _np(q) * unit
        bound = np.maximum(np.abs(n) * 2.0 ** -4, 2.0 ** -10 * unit) + np.abs(n) * 2.0 ** -18
        assert np.all(np.abs(got - n) <= bound)
        amax = np.abs(n).reshape(n.shape[0], -1, 32).max(2)
        assert np.all(amax <= 448.0 * 2.0 ** p * (1 + 2.0 ** -18))
        assert np.all((p == -127) | (amax >= 448.0 * 2.0 ** (p - 1) * (1 - 2.0 ** -18)))


def _run(T, H, rt, dt, gt, pads=(0, 0, 0, 0, 0), eps=1e-6, seed=0, scale=2.0, stream=None):
    B = _B()
    rng = np.random.default_rng(seed)
    res = _rows(rng, T, H, pads[0], TYPES[rt], scale)
    delta = None if dt is None else _rows(rng, T, H, pads[1], TYPES[dt])
    gain = None if gt is None else torch.from_numpy(1 + 0.2 * rng.standard_normal(H)).to(TYPES[gt]).cuda()
    s = torch.full((T, H + pads[2]), 7.0, dtype=TYPES[rt], device="cuda")
    y = torch.full((T, H + pads[3]), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((T, H + pads[4]), 7.0, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.zeros((T, H // 32), dtype=torch.uint8, device="cuda")
    B.moe_add_rmsnorm(res, delta, gain, eps, s[:, :H], y[:, :H], q[:, :H], sc, stream=stream)
    torch.cuda.synchronize()
    es, n = _expected(res, delta, gain, eps)
    assert torch.equal(s[:, :H].cpu(), es)
    _check(n, y[:, :H], q[:, :H], sc)
    for buf in (s, y, q):  # what lies between the rows stays
        assert torch.all(buf[:, H:].float() == 7.0)


@pytest.mark.parametrize("rt", ["bf16", "f32"])
@pytest.mark.parametrize("dt", [None, "bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (5, 96), (7, 544), (2, 7168), (33, 2080), (4, 8224), (3, 20000 - 32),
                                 (2, 40000), (1, 65536)])
def test_norm_matches_64_bits(T, H, rt, dt):
    _run(T, H, rt, dt, "f32" if (T + H // 32) % 2 else "bf16", seed=T + H)


@pytest.mark.parametrize("T", [152, 153, 1000, 2049])
@pytest.mark.parametrize("H", [64, 288, 1024, 7168])
def test_norm_many_rows(T, H):
    _run(T, H, "f32", "bf16", None, seed=T)


def test_norm_strided_rows():
    _run(9, 416, "bf16", "f32", "bf16", pads=(8, 12, 264, 16, 32), seed=4)
    _run(9, 416, "f32", "bf16", "f32", pads=(4, 24, 8, 8, 48), seed=5)


def test_norm_in_place_and_each_output_alone():
    B = _B()
    rng = np.random.default_rng(7)
    T, H = 11, 320
    for rt in ("bf16", "f32"):
        res, delta = _rows(rng, T, H, 0, TYPES[rt], 3.0), _rows(rng, T, H, 0, TYPES[rt])
        es, n = _expected(res, delta, None, 1e-5)
        keep, keep_d = res.clone(), delta.clone()
        y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
        B.moe_add_rmsnorm(res, delta, None, 1e-5, None, y, None, None)
        _check(n, y, None, None)
        B.moe_add_rmsnorm(res, delta, None, 1e-5, None, None, q, sc)
        _check(n, None, q, sc)
        assert torch.equal(res, keep) and torch.equal(delta, keep_d)
        B.moe_add_rmsnorm(res, delta, None, 1e-5, delta, y, None, None)  # in place of delta
        assert torch.equal(delta.cpu(), es)
        _check(n, y, None, None)
        B.moe_add_rmsnorm(res, keep_d, None, 1e-5, res, y, q, sc)        # in place of the residual
        assert torch.equal(res.cpu(), es)
        _check(n, y, q, sc)
        s = torch.empty_like(keep)
        B.moe_add_rmsnorm(keep, keep_d, None, 1e-5, s)
        assert torch.equal(s.cpu(), es)


def test_norm_zero_rows_small_values_and_scale_borders():
    B = _B()
    H = 128
    res = torch.zeros((4, H), device="cuda")
    res[1, :] = 2.0 ** -70                                       # eps dominates: n far below one
    res[2, 0], res[2, 32], res[2, 64] = 448.0, 449.0, 224.0      # blocks at, above and below a border
    gain = torch.full((H,), 1.0, device="cuda")
    y = torch.empty((4, H), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((4, H), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((4, H // 32), dtype=torch.uint8, device="cuda")
    B.moe_add_rmsnorm(res, None, gain, 1.0, None, y, q, sc)
    torch.cuda.synchronize()
    _, n = _expected(res, None, gain, 1.0)
    _check(n, y, q, sc)
    assert torch.all(sc[0] == 0) and torch.all(q[0].float() == 0) and torch.all(y[0] == 0)
    # eps = 0 on a row of zeros: 0 * inf, as in the formula
    B.moe_add_rmsnorm(res[:1], None, None, 0.0, None, y[:1], q[:1], sc[:1])
    assert torch.all(torch.isnan(y[0])) and torch.all(torch.isnan(q[0].float()))


def test_norm_non_finite_rows_stay_their_own():
    B = _B()
    rng = np.random.default_rng(3)
    T, H = 5, 96
    res = _rows(rng, T, H, 0, torch.float32)
    clean = res.clone()
    res[1, 5] = float("nan")
    res[3, 40] = float("inf")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    B.moe_add_rmsnorm(res, None, None, 1e-6, None, y, q, sc)
    _, n = _expected(clean, None, None, 1e-6)
    rows = [0, 2, 4]
    _check(n[rows], y[rows], q[rows], sc[rows])
    assert torch.all(torch.isnan(y[1])) and torch.all(torch.isnan(q[1].float()))
    assert torch.isnan(y[3, 40]) and torch.isnan(q[3, 40].float()) and int(torch.isnan(y[3]).sum()) == 1
    # an infinity made by the gain: the E4M3 NaN, its neighbours finite
    gain = torch.ones(H, device="cuda")
    gain[7] = float("inf")
    B.moe_add_rmsnorm(clean, None, gain, 1e-6, None, None, q, sc)
    assert torch.all(torch.isnan(q[:, 7].float())) and int(torch.isnan(q.float()).sum()) == T


def test_norm_on_a_side_stream_and_in_a_graph():
    B = _B()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _run(6, 256, "bf16", "bf16", "f32", seed=9, stream=side)
    x = torch.randn((4, 512), device="cuda")
    y = torch.empty((4, 512), dtype=torch.bfloat16, device="cuda")
    B.moe_add_rmsnorm(x, None, None, 1e-6, None, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_add_rmsnorm(x, None, None, 1e-6, None, y)
    x.copy_(torch.randn((4, 512), device="cuda") * 5)
    g.replay()
    torch.cuda.synchronize()
    _check(_expected(x, None, None, 1e-6)[1], y, None, None)


def test_norm_no_rows():
    B = _B()
    e = torch.empty((0, 64), device="cuda")
    B.moe_add_rmsnorm(e, None, None, 1e-6, e)
