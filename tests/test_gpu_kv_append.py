"""moe_kv_append on the GPU against its definition in 64 bits.

BF16 results: FP32 arithmetic (two products and their sum, 2^-23 of |a| + |b| at most) and one rounding, half a step or
2^-8 of the value.  MXFP8 results round once from the exact value and are compared for equality: the kernel's turned
value is within 2^-48 of the terms before it is rounded to odd.
"""
import numpy as np
import pytest
import torch

from attention_util import e4m3_blocks

pytestmark = pytest.mark.gpu


def _case(T, heads, kv, D, page, fmt, rot, seed, extra_pages=2, pad=0):
    from mxfp4_routed_expert_router_gb300 import attention as A
    rng = np.random.default_rng(seed)
    n_pages = -(-T // page) + extra_pages
    c = A.KvCache.empty(n_pages, kv, page, D, fmt)
    for t in (c.k, c.v):  # (what lies there stays where no token goes)
        t.view(torch.uint8).fill_(0x33)
    w = (heads + 2 * kv) * D
    x = torch.from_numpy(rng.standard_normal((T, w + pad)).astype(np.float32)).bfloat16().cuda()[:, :w]
    slots = torch.from_numpy(rng.permutation(n_pages * page)[:T].astype(np.int32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32)).cuda()
    rope = A.rope_table(5000, rot) if rot else None
    return c, x, slots, pos, rope


def _turned(x, pos, rope, pairs):
    """[T, heads, D] float64 -> turned."""
    if rope is None:
        return x
    rot = rope.shape[1]
    t = rope.double().cpu().numpy()[pos.cpu().numpy()][:, None]
    cos, sin = t[..., :rot // 2], t[..., rot // 2:]
    y = x.copy()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def _near(got, want, scale):
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * scale + 1e-38), err.max()


@pytest.mark.parametrize("T,heads,kv,D,page,fmt,rot,pairs,pad", [
    (1, 56, 8, 128, 64, "bf16", 128, False, 0), (1, 4, 4, 64, 16, "mxfp8", 64, False, 0),
    (3, 7, 1, 64, 32, "bf16", 32, False, 8), (17, 5, 5, 128, 16, "mxfp8", 48, False, 24),
    (33, 16, 1, 128, 256, "bf16", 64, True, 0), (176, 64, 8, 128, 64, "mxfp8", 64, True, 0),
    (129, 12, 4, 64, 128, "mxfp8", 16, True, 0), (300, 8, 2, 64, 64, "bf16", 0, False, 0),
    (257, 3, 3, 128, 64, "mxfp8", 0, False, 0), (2100, 40, 8, 128, 64, "bf16", 128, False, 0),
    (1500, 48, 16, 128, 64, "mxfp8", 128, False, 0), (1000, 24, 8, 64, 32, "mxfp8", 64, True, 8),
])
def test_append_matches_its_definition(T, heads, kv, D, page, fmt, rot, pairs, pad):
    c, x, slots, pos, rope = _case(T, heads, kv, D, page, fmt, rot, T + D + rot, pad=pad)
    k_out = torch.zeros((T, kv, D), dtype=torch.bfloat16, device="cuda") if T % 2 else None
    before = x.clone()
    q = c.append(x, heads, slots, pos, rope, pairs, k_out=k_out)
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    x64 = x.double().cpu().numpy().reshape(T, -1, D)
    turned = _turned(x64[:, :heads + kv], pos, rope, pairs)
    size = np.abs(x64).max()
    _near(q, turned[:, :heads], size)
    if k_out is not None:
        _near(k_out, turned[:, heads:], size)
    at = slots.cpu().numpy()
    pg, row = at // page, at % page
    free = np.ones((c.k.shape[0], page), bool)
    free[pg, row] = False
    for t, s, want in ((c.k, c.k_scales, turned[:, heads:]), (c.v, c.v_scales, x64[:, heads + kv:])):
        raw = t.view(torch.uint8).cpu().numpy()
        assert np.all(raw.transpose(0, 2, 1, 3)[free] == 0x33)
        if fmt == "bf16":
            _near(t[pg, :, row], want, size)
            continue
        val, byte = e4m3_blocks(want)
        assert np.array_equal(s.cpu().numpy()[pg, :, row], byte)
        got = t.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float().double().cpu().numpy()
        got = got * np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, -1)
        assert np.array_equal(got, val), (np.abs(got - val).max(), (got != val).sum())


def test_values_that_are_not_finite_and_blocks_of_zeros():
    c, x, slots, pos, rope = _case(6, 2, 2, 64, 16, "mxfp8", 0, 5)
    x[0, 128] = float("nan")
    x[1, 130] = float("inf")
    x[2, 256:320] = 0
    x[3, 260] = 3e38
    c.append(x, 2, slots)
    x64 = x.double().cpu().numpy().reshape(6, -1, 64)
    at = slots.cpu().numpy()
    for t, s, want in ((c.k, c.k_scales, x64[:, 2:4]), (c.v, c.v_scales, x64[:, 4:])):
        val, byte = e4m3_blocks(want)
        assert np.array_equal(s.cpu().numpy()[at // 16, :, at % 16], byte)
        got = t.view(torch.uint8)[at // 16, :, at % 16].view(torch.float8_e4m3fn).float().double().cpu().numpy()
        got = got * np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, -1)
        assert np.array_equal(got, val, equal_nan=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_padding_and_rows_out_of_range(fmt):
    from mxfp4_routed_expert_router_gb300 import attention as A, binding as B
    A.sync()
    c, x, slots, pos, rope = _case(40, 4, 2, 64, 16, fmt, 64, 9)
    full = c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    nowhere = torch.full_like(slots, -1)
    c.append(x, 4, nowhere, torch.full_like(pos, -7), rope)  # padding may have any position
    A.sync()
    assert torch.equal(c.k.view(torch.uint8), full[0]) and torch.equal(c.v.view(torch.uint8), full[1])
    for bad in (-2, c.k.shape[0] * 16, 2 ** 31 - 1, -2 ** 31):
        c.append(x, 4, torch.full_like(slots, bad), pos, rope)
        with pytest.raises(B.MoeError) as e:
            A.sync()
        assert e.value.status == B.MOE_EDEVICE
        A.sync()  # reported once
        assert torch.equal(c.k.view(torch.uint8), full[0]) and torch.equal(c.v.view(torch.uint8), full[1])
    for bad in (-1, 5000, 2 ** 31 - 1):
        p = pos.clone()
        p[7] = bad
        q = c.append(x, 4, slots, p, rope)
        with pytest.raises(B.MoeError):
            A.sync()
        assert torch.isnan(q[7]).all() and torch.isfinite(q[:7]).all() and torch.isfinite(q[8:]).all()


def test_in_place_on_streams_and_in_a_graph():
    c, x, slots, pos, rope = _case(50, 8, 2, 128, 64, "bf16", 128, 11)
    k_out = torch.empty((50, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = c.append(x, 8, slots, pos, rope, k_out=k_out)
    kc, vc = c.k.clone(), c.v.clone()
    y = x.clone()
    rows = y.view(50, 12, 128)
    c.k.zero_(), c.v.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.append(y, 8, slots, pos, rope, q_out=rows[:, :8], k_out=rows[:, 8:10], stream=side)
    side.synchronize()
    assert torch.equal(rows[:, :8], q) and torch.equal(rows[:, 8:10], k_out)
    assert torch.equal(rows[:, 10:], x.view(50, 12, 128)[:, 10:])
    at = (slots // 64).long(), (slots % 64).long()
    assert torch.equal(c.k[at[0], :, at[1]], kc[at[0], :, at[1]])
    assert torch.equal(c.v[at[0], :, at[1]], vc[at[0], :, at[1]])
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(g):
        c.append(x, 8, slots, pos, rope, q_out=out)
    x.copy_(x.flip(0)), pos.copy_(pos.flip(0)), slots.copy_(slots.flip(0))
    c.k.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, q.flip(0))
    assert torch.equal(c.k[at[0], :, at[1]], kc[at[0], :, at[1]])


def test_no_tokens():
    c, x, slots, pos, rope = _case(4, 4, 2, 64, 16, "bf16", 64, 12)
    q = c.append(x[:0], 4, slots[:0], pos[:0], rope)
    assert q.shape == (0, 4, 64)
