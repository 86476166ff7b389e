"""moe_attention_decode over BF16 caches: probabilities enter the product with v as two BF16 numbers, so that a result is
within little more than its own rounding of the 64-bit form."""
import pytest
import torch

from attention_util import attend, cache_values
from test_gpu_attention_decode import make

pytestmark = pytest.mark.gpu


def bound(o, pv, mag, D, steps):
    """The kernel's error against ``attend``, value by value:
    * the output rounds to BF16, half a step: 2^-8 of it;
    * a probability is the sum of two BF16 numbers, the second (what lies below the first's 8 bits) below 2^-7 of it and
      off by 2^-8 of itself, or 2^-17 of it where nothing lies there: 2^-15 of sum p |v|;
    * a score is D exact products added in FP32, truncated at worst 2^-22 of the sum of magnitudes at each of D / 16
      steps, and one multiplication by scale * log2 e; the exponential is good to 2^-21: twice that for the quotient;
    * FP32 sums of the products, truncated at worst: 2^-22 at each of a warp's steps of 16 tokens, two products each."""
    ds = 2 * ((D / 16 + 2) * 2.0 ** -22 * mag * 1.45 + 2.0 ** -21)
    return 2.0 ** -8 * o.abs() + (2.0 ** -15 + ds + (2 + 2 * steps) * 2.0 ** -22) * pv * 1.01 + 1e-30


@pytest.mark.parametrize("lens,heads,kv,D,page", [
    ([1000], 56, 8, 128, 64), ([1, 2, 17, 64, 65, 300, 0, 511], 12, 4, 64, 16), ([20000, 3], 32, 4, 128, 64),
    ([333, 100], 48, 2, 64, 32), ([700] * 40, 40, 8, 128, 64), ([4097, 900], 16, 1, 128, 256), ([30000], 40, 1, 64, 256),
])
@pytest.mark.parametrize("q_scale", [0.05, 1.5, 8.0])
def test_decode_is_as_good_as_its_output_s_rounding(lens, heads, kv, D, page, q_scale):
    c, q, table, n = make(lens, heads, kv, D, page, "bf16", 17, q_scale=q_scale)
    got = c.decode(q, table, n)
    k, v = cache_values(c)
    for b, L in enumerate(lens):
        if L == 0:
            assert not got[b].any()
            continue
        at = table[b, :-(-L // page)].long()
        kb, vb = (x[at].transpose(0, 1).reshape(kv, -1, D)[:, :L] for x in (k, v))
        o, pv, mag = attend(q[b].double().view(kv, -1, D), kb, vb, D ** -0.5)
        err, tol = (got[b].double().view(kv, -1, D) - o).abs(), bound(o, pv, mag, D, L / 64 + 1)
        assert torch.all(err <= tol), (b, (err / tol).max())


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_all_the_same_come_back(D):
    """Weights sum to one: v of a constant per place gives it, to the bit (2^-13 or so is less than half a step)."""
    c, q, table, n = make([1, 30, 500, 3000], 24, 2, D, 32, "bf16", 19)
    row = torch.linspace(-3, 5, D, device="cuda").bfloat16()
    c.v.copy_(row.expand_as(c.v))
    assert torch.equal(c.decode(q, table, n), row.expand(4, 24, D))


def test_an_infinite_value_gives_the_formula_s_infinity():
    """No probability is zero here: an infinite value of a token that a sequence holds is its output, and no other's."""
    lens = [1, 40, 900, 64]
    c, q, table, n = make(lens, 8, 2, 64, 32, "bf16", 23, q_scale=0.5)
    good = c.decode(q, table, n)
    for b, at in ((0, 0), (1, 39), (2, 0), (2, 517), (3, 33)):
        for bad in (float("inf"), float("-inf")):
            was = c.v[table[b, at // 32].item(), 1, at % 32, 9].item()
            c.v[table[b, at // 32].item(), 1, at % 32, 9] = bad
            got = c.decode(q, table, n)
            c.v[table[b, at // 32].item(), 1, at % 32, 9] = was
            assert torch.all(got[b, 4:, 9] == bad)
            got[b, 4:, 9] = good[b, 4:, 9]
            assert torch.equal(got, good)
