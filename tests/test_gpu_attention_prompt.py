"""moe_attention_prompt on the GPU against its definition in 64 bits; the tolerance is derived in attention_util."""
import numpy as np
import pytest
import torch

from attention_util import attend, tolerance

pytestmark = pytest.mark.gpu


def make(lens, heads, kv, D, seed, before=0, behind=0, pad=0, q_scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = before + sum(lens) + behind
    x = torch.randn((T, (heads + 2 * kv + pad) * D), generator=g, device="cuda").bfloat16()
    x = x.view(T, -1, D)
    x[:, :heads] *= q_scale
    off = torch.tensor(np.cumsum([before] + list(lens)), dtype=torch.int32, device="cuda")
    return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:heads + 2 * kv], off


def expected(q, k, v, lens, scale, before=0):
    heads, D = q.shape[1:]
    kv = k.shape[1]
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64,
                                                                                    device="cuda")
    a = before
    for n in lens:
        if n:
            rows = slice(a, a + n)
            kk, vv = (x[rows].double().transpose(0, 1).repeat_interleave(heads // kv, 0) for x in (k, v))
            see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
            o, pv, mag = attend(q[rows].double().transpose(0, 1), kk, vv, scale, see)
            out[rows], tol[rows] = o.transpose(0, 1), tolerance(o, pv, mag, D).transpose(0, 1)
        a += n
    return out, tol


def check(got, want):
    out, tol = want
    err = (got.double() - out).abs()
    assert torch.all(err <= tol), (err / tol.clamp_min(1e-30)).max()


CASES = [
    ([1], 1, 1, 64), ([1], 8, 1, 128), ([2], 64, 1, 128), ([16, 17], 8, 1, 128), ([127, 128, 129], 1, 1, 128),
    ([128], 2, 2, 64), ([255, 256, 257], 4, 4, 64), ([1, 0, 3, 0, 0, 200, 1], 7, 1, 128), ([513], 64, 8, 128),
    ([1000, 24], 12, 4, 64), ([1025], 6, 6, 128), ([1] * 70, 16, 2, 64), ([300, 1, 700], 40, 8, 128),
    ([640, 513], 48, 1, 64), ([2500], 2, 1, 128), ([40 * i % 300 for i in range(30)], 5, 1, 64), ([37] * 400, 2, 1, 64),
    ([130 * i % 777 for i in range(60)], 14, 2, 128), ([1 + 211 * i % 1500 for i in range(15)], 56, 8, 128),
    ([90 * i % 400 for i in range(200)], 8, 8, 64),
    ([i % 41 for i in range(1500)], 8, 1, 64), ([3] * 3000, 4, 2, 128), ([2] * 200 + [900] + [0, 50] * 100, 16, 2, 64),
]


@pytest.mark.parametrize("lens,heads,kv,D", CASES)
def test_prompt_matches_its_definition(lens, heads, kv, D):
    from mxfp4_routed_expert_router_gb300 import attention as A
    q, k, v, off = make(lens, heads, kv, D, sum(lens) + heads)
    got = A.prompt(q, k, v, off)
    A.sync()
    check(got, expected(q, k, v, lens, D ** -0.5))
    assert torch.equal(A.prompt(q, k, v, off), got)


def test_rows_of_no_sequence_stay():
    from mxfp4_routed_expert_router_gb300 import attention as A
    lens = [100, 30]
    q, k, v, off = make(lens, 8, 2, 64, 3, before=20, behind=50, pad=1)
    buf = torch.full((200, 9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf.view(200, -1)[:, :512].view(200, 8, 64)
    A.prompt(q, k, v, off, scale=0.3, out=out)
    want, tol = expected(q, k, v, lens, 0.3, before=20)
    check(out[20:150], (want[20:150], tol[20:150]))
    assert torch.all(out[:20] == 5.0) and torch.all(out[150:] == 5.0) and torch.all(buf[:, 8] == 5.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[70, 200, 90], [400, 129]])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(lens, D):
    from mxfp4_routed_expert_router_gb300 import attention as A
    q, k, v, off = make(lens, 8, 2, D, 21)
    good = A.prompt(q, k, v, off)
    check(good, expected(q, k, v, lens, D ** -0.5))
    for at in (0, 33, lens[0] - 1, lens[0], lens[0] + 128, sum(lens) - 1):
        end = int(off[(off > at).nonzero()[0, 0]])
        for bad in (float("inf"), float("-inf"), float("nan")):
            v2 = v.clone()
            v2[at, 1, 5] = bad
            got = A.prompt(q, k, v2, off)
            hit = got[at:end, 4:, 5].float()
            assert torch.all(torch.isnan(hit) if bad != bad else (hit == bad) | torch.isnan(hit))
            if bad == bad:  # (where no probability is zero the formula's infinity)
                assert torch.all(hit == bad)
            keep = torch.ones_like(got, dtype=torch.bool)
            keep[at:end, 4:, 5] = False
            assert torch.equal(got[keep], good[keep])
            k2 = k.clone()
            k2[at, 0] = bad
            got = A.prompt(q, k2, v, off)
            keep = torch.ones_like(got, dtype=torch.bool)
            keep[at:end, :4] = False
            assert torch.equal(got[keep], good[keep])
            if bad != bad:
                assert torch.isnan(got[at:end, :4]).all()
    A.sync()


def test_growing_and_large_scores():
    """Maxima that grow from key tile to key tile (O is rescaled each time), and rows of one large score."""
    from mxfp4_routed_expert_router_gb300 import attention as A
    for heads, kv, D in ((4, 1, 128), (3, 3, 64)):
        q, k, v, off = make([900], heads, kv, D, 31, q_scale=4.0)
        ramp = torch.linspace(0.1, 6.0, 900, device="cuda").view(-1, 1, 1)
        k = (k.float() * ramp).bfloat16()
        check(A.prompt(q, k, v, off), expected(q, k, v, [900], D ** -0.5))
        q, k = -q.abs(), k.abs()  # every score far below zero, falling
        check(A.prompt(q, k, v, off), expected(q, k, v, [900], D ** -0.5))
        k = k.flip(0)
        check(A.prompt(q, k, v, off), expected(q, k, v, [900], D ** -0.5))


def test_streams_and_graphs():
    from mxfp4_routed_expert_router_gb300 import attention as A
    lens = [300, 5, 0, 700]
    q, k, v, off = make(lens, 16, 2, 128, 41)
    want = A.prompt(q, k, v, off)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        with torch.cuda.stream(side):
            got.append(A.prompt(q, k, v, off))
        got.append(A.prompt(q, k, v, off, stream=side))
        got.append(A.prompt(q, k, v, off))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(g):
        A.prompt(q, k, v, off, out=out)
    lens = [1, 800, 100, 104]
    off.copy_(torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check(out, expected(q, k, v, lens, 128 ** -0.5))


def test_offsets_that_do_not_fit_stay_in_bounds():
    """Offsets beyond the rows are cut; ones that do not ascend leave rows out, and touch nothing else."""
    from mxfp4_routed_expert_router_gb300 import attention as A
    q, k, v, off = make([200], 4, 2, 64, 51, behind=40)
    want = A.prompt(q, k, v, torch.tensor([0, 200, 240], dtype=torch.int32, device="cuda"))
    got = A.prompt(q, k, v, torch.tensor([-5, 200, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)
    for bad in ([0, 240] * 150, [200, 100, 50], [0, 2 ** 31 - 1, -2 ** 31, 100], [-1, -1], [240, 240], [500, 600]):
        out = torch.full_like(q, 3.0, memory_format=torch.contiguous_format)
        A.prompt(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()


def test_no_rows_and_no_sequences():
    from mxfp4_routed_expert_router_gb300 import attention as A
    q, k, v, off = make([20], 4, 2, 64, 61)
    assert A.prompt(q[:0], k[:0], v[:0], off).shape == (0, 4, 64)
    out = torch.full_like(q, 3.0, memory_format=torch.contiguous_format)
    A.prompt(q, k, v, off[:1], out=out)
    assert torch.all(out == 3.0)


def test_rows_whose_offsets_pass_32_bits():
    """More than 2^31 values before the prompts: only their rows are read and written."""
    from mxfp4_routed_expert_router_gb300 import attention as A
    heads, kv, D, T = 64, 8, 128, 270000
    assert T * heads * D > 2 ** 31
    x = torch.zeros((T, heads + 2 * kv, D), dtype=torch.bfloat16, device="cuda")
    lens = [300, 5]
    first = T - 310
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x[first:] = torch.randn((310, heads + 2 * kv, D), generator=g, device="cuda").bfloat16()
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    out = torch.full((T, heads, D), 2.0, dtype=torch.bfloat16, device="cuda")
    A.prompt(q, k, v, torch.tensor([first, first + 300, first + 305], dtype=torch.int32, device="cuda"), out=out)
    A.sync()
    want = expected(q[first:], k[first:], v[first:], lens, D ** -0.5)
    check(out[first:first + 305], (want[0][:305], want[1][:305]))
    assert torch.all(out[first - 1000:first] == 2.0) and torch.all(out[first + 305:] == 2.0)
