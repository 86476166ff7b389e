"""moe_attention_decode over MXFP8 caches whose blocks have unlike powers of two: a sequence's powers stay its own.

Many sequences and key heads lie on each of the kernel's workers, one behind the other.
"""
import pytest
import torch

from attention_util import attend, cache_values, paged, random_cache

pytestmark = pytest.mark.gpu


def bound(o, pv, mag, D, v_sum, steps):
    """The kernel's error against ``attend``, value by value:
    * the output rounds to BF16, half a step: 2^-8 of it;
    * a probability, 2^12 for the largest, rounds to FP16: 2^-11 of sum p |v|, and where it (or its product with a power
      of two, 2^-4 at least) lies below FP16's normal range 2^-25 and 2^4 * 2^-25, or 2^-37 and 2^-33 of the largest,
      times the token's own |v|;
    * scores, exponentials and the quotient as in attention_util;
    * FP32 sums of the products, truncated at worst: 2^-22 at each of a warp's steps of 16 tokens of 64."""
    ds = 2 * ((D / 16 + 2) * 2.0 ** -22 * mag * 1.45 + 2.0 ** -21)
    return 2.0 ** -8 * o.abs() + (2.0 ** -11 + ds + (2 + steps) * 2.0 ** -22) * pv * 1.01 + 17 * 2.0 ** -37 * v_sum + 1e-30


def expected(c, q, table, lens, scale):
    """(output, bound) [B, heads, D]; NaN where a value that is not finite reaches the output."""
    k, v = cache_values(c)
    B, heads, D = q.shape
    out, tol = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = table[b, :-(-n // c.page_size)].long()
        kb, vb = (x[at].transpose(0, 1).reshape(c.n_kv_heads, -1, D)[:, :n] for x in (k, v))
        o, pv, mag = attend(q[b].double().view(c.n_kv_heads, -1, D), kb, vb, scale)
        v_sum = torch.nan_to_num(vb.abs()).sum(1, keepdim=True)
        out[b], tol[b] = (x.reshape(heads, D) for x in (o, bound(o, pv, mag, D, v_sum, n / 64 + 1)))
    return out, tol


def check(got, want):
    out, tol = want
    finite = torch.isfinite(out)
    assert torch.equal(torch.isnan(got), ~finite)
    err = torch.where(finite, got.double() - out, 0.0).abs()
    tol = torch.where(finite, tol, 1.0)
    assert torch.all(err <= tol), (err / tol).max()


def make(lens, heads, kv, D, page, seed, spread=1):
    held = sum(-(-n // page) for n in lens)
    c = random_cache(held + 2, kv, page, D, "mxfp8", seed, spread)
    table = paged(lens, page, held + 2, max(1, max(-(-n // page) for n in lens)), seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    q = (torch.randn((len(lens), heads, D), generator=g, device="cuda") * 1.5).bfloat16()
    return c, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


# tables of at most 512 tokens, and of more: sequences then go over from one worker to the next
MANY = [([1 + 53 * i % 150 for i in range(700)], 4, 4, 128, 32), ([1 + 53 * i % 150 for i in range(700)], 16, 4, 64, 16),
        ([1 + 97 * i % 640 for i in range(500)], 12, 4, 64, 64), ([1 + 97 * i % 640 for i in range(400)], 48, 4, 128, 64)]


@pytest.mark.parametrize("byte,code", [(247, 0x7F), (255, None), (160, None), (200, 0x38)])
@pytest.mark.parametrize("lens,heads,kv,D,page", MANY)
def test_powers_of_one_sequence_reach_no_other(lens, heads, kv, D, page, byte, code):
    """One token of some sequences has, in one block of one key head, the power that an infinity gets (beside the code of
    NaN), the NaN of the powers, or a large one: all else stays as it was, bit for bit."""
    c, q, table, n = make(lens, heads, kv, D, page, 5)
    clean = c.decode(q, table, n)
    hit = list(range(3, len(lens), 11))
    for b in hit:
        at, off, h, block = table[b, (lens[b] - 1) // page].item(), (lens[b] - 1) % page, b % kv, b % (D // 32)
        c.v_scales[at, h, off, block] = byte
        c.v.view(torch.uint8)[at, h, off, 32 * block + 1:32 * block + 32] = 0
        if code is not None:
            c.v.view(torch.uint8)[at, h, off, 32 * block] = code
    got = c.decode(q, table, n)
    same = torch.ones((len(lens), kv), dtype=torch.bool, device="cuda")
    for b in hit:
        same[b, b % kv] = False
    same = same.repeat_interleave(heads // kv, 1)
    assert torch.equal(got[same], clean[same])
    check(got, expected(c, q, table, lens, D ** -0.5))


@pytest.mark.parametrize("spread", [3, 12, 40])
@pytest.mark.parametrize("lens,heads,kv,D,page", MANY)
def test_powers_far_apart_with_many_sequences(lens, heads, kv, D, page, spread):
    """Powers that differ from block to block, and from sequence to sequence by 2^60: each value's bound is its own."""
    c, q, table, n = make(lens, heads, kv, D, page, 6, spread)
    for b in range(len(lens)):
        at = table[b, :-(-lens[b] // page)].long()
        c.v_scales[at] = (c.v_scales[at].int() + 40 * b % 61 - 30).to(torch.uint8)
    check(c.decode(q, table, n), expected(c, q, table, lens, D ** -0.5))


@pytest.mark.parametrize("lens,heads,kv,D,page", MANY)
def test_an_infinity_through_the_cache_s_writer(lens, heads, kv, D, page):
    """An infinite value, appended, is NaN where it stands; the other values of its block keep the other tokens' sum."""
    c, q, table, n = make(lens, heads, kv, D, page, 7)
    clean = c.decode(q, table, n)
    hit = list(range(2, len(lens), 17))
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rows = torch.randn((len(hit), (heads + 2 * kv) * D), generator=g, device="cuda").bfloat16()
    v = rows.view(len(hit), -1, D)[:, heads + kv:]
    slots = []
    for i, b in enumerate(hit):
        v[i, b % kv, b % D] = float("inf")
        slots.append(table[b, 0].item() * page)
    c.append(rows, heads, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    got = c.decode(q, table, n)
    others = torch.ones(len(lens), dtype=torch.bool, device="cuda")
    others[hit] = False
    assert torch.equal(got[others], clean[others])
    check(got, expected(c, q, table, lens, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_zeros_beside_others(D):
    """A head whose upper half is padding (blocks of zeros: power byte 0) and one that is zero in some tokens only."""
    lens = [1, 40, 700, 0, 333]
    c, q, table, n = make(lens, 8, 4, D, 32, 8)
    raw = c.v.view(torch.uint8)
    raw[:, 1, :, D // 2:] = 0
    c.v_scales[:, 1, :, D // 64:] = 0
    raw[:, 2, ::3] = 0
    c.v_scales[:, 2, ::3] = 0
    c.v_scales[:, 3] = 0  # (values of 2^-127)
    check(c.decode(q, table, n), expected(c, q, table, lens, D ** -0.5))


@pytest.mark.parametrize("top", [[0], [0, 16, 32, 48]])
@pytest.mark.parametrize("D", [64, 128])
def test_a_long_rest_far_below_a_maximum(D, top):
    """A few tokens 16 above the mean of 131,072 others, which have a share of 2 % together and values with powers 2^4
    below the largest: their sum must not get lost.  A sequence for each worker, all over the same pages, so that a warp
    sees 32,768 tokens."""
    from mxfp4_routed_expert_router_gb300.attention import KvCache
    n, page, heads = 131072, 256, 8
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    q = torch.randn((1, 1, D), generator=g, device="cuda")
    k = torch.randn((n, D), generator=g, device="cuda")
    k[top] = q[0] * (16 / (q[0].square().sum() * D ** -0.5))
    v = torch.rand((n, D), generator=g, device="cuda") * 8 + 4
    power = torch.full((n, D // 32), 123, dtype=torch.uint8, device="cuda")
    power[::16] = 127
    v[::16] = 2.0 ** -9
    one = torch.full_like(power, 127)
    shape = (n // page, 1, page, -1)
    c = KvCache(*[x.to(torch.float8_e4m3fn).view(shape) for x in (k, v)], *[x.view(shape) for x in (one, power)])
    q = (q * (1 + 0.02 * torch.randn((1, heads, D), generator=g, device="cuda"))).bfloat16()
    table = torch.arange(n // page, device="cuda", dtype=torch.int32).view(1, -1)
    want = expected(c, q, table, [n], D ** -0.5)
    got = c.decode(q.repeat(B, 1, 1), table.repeat(B, 1), torch.full((B,), n, dtype=torch.int32, device="cuda"))
    check(got, [x.expand(B, -1, -1) for x in want])
    check(c.decode(q, table, torch.tensor([n], dtype=torch.int32, device="cuda")), want)  # (one, over all workers)
