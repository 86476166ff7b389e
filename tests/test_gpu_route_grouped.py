"""moe_route_grouped on the GPU against a plain NumPy form in 64 bits.

Ids are equal.  Weights: an FP32 evaluation of exp has an argument error of
|l - max| * 2^-24 (below 40 * 2^-24 here), 2 ulp of the function, a sum of at
most 1024 positive terms taken pairwise (10 * 2^-24) and two divisions: below
2^-18 of the weight.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

W_TOL = 2.0 ** -18


def _B():
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


def expected(logits, bias, k, n_groups, k_groups, score, group_score, renorm, scale):
    """One token at a time, by the definition: Python sorting with the order rules, doubles throughout."""
    T, E = logits.shape
    gs = E // n_groups
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))

    def rank(v, i):  # larger first, NaN after every number, equal values by the lower index
        return (1, 0.0, i) if np.isnan(v) else (0, -v, i)

    for t in range(T):
        l = logits[t].astype(np.float64)
        on = [e for e in range(E) if not (np.isinf(l[e]) and l[e] < 0)]
        if not on:
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                s = np.exp(l - np.fmax.reduce(l))
                s = s / s[on].sum()
        c = s + (0.0 if bias is None else bias.astype(np.float64))
        tops = []
        for g in range(n_groups):
            mine = sorted((rank(c[e], e) for e in on if e // gs == g))
            vals = [c[r[2]] for r in mine[:2]]
            if not vals:
                tops.append((2, 0.0, g))
            else:
                v = vals[0] + vals[1] if group_score == "top2" and len(vals) > 1 else vals[0]
                tops.append(rank(v, g))
        kept = {r[2] for r in sorted(tops)[:k_groups]}
        sel = [r[2] for r in sorted(rank(c[e], e) for e in on if e // gs in kept)[:k]]
        ids[t, :len(sel)] = sel
        v = s[sel]
        if renorm:
            tot = v.sum()
            v = np.zeros_like(v) if tot == 0 else v / tot
        w[t, :len(sel)] = scale * v
    return ids, w


def _run(logits, bias, k, n_groups, k_groups, score, group_score, renorm, scale, stream=None):
    B = _B()
    T, E = logits.shape
    ids = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 99.0, device="cuda")
    B.moe_route_grouped(torch.from_numpy(logits).cuda(), None if bias is None else torch.from_numpy(bias).cuda(), T, E,
                        k, n_groups, k_groups, B.MOE_SCORE_SIGMOID if score == "sigmoid" else B.MOE_SCORE_SOFTMAX,
                        B.MOE_GROUP_TOP2 if group_score == "top2" else B.MOE_GROUP_MAX, renorm, scale, ids, w, stream)
    torch.cuda.synchronize()
    eids, ew = expected(logits, bias, k, n_groups, k_groups, score, group_score, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), eids)
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ew))
    fin = ~np.isnan(ew)
    assert np.all(np.abs(got[fin] - ew[fin]) <= W_TOL * np.abs(ew[fin]) + 1e-37)
    return eids


SHAPES = [  # T, E, k, n_groups, k_groups
    (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (65, 256, 8, 8, 4), (7, 256, 8, 1, 1), (5, 250, 6, 5, 3), (9, 96, 32, 3, 3),
    (4, 1024, 16, 16, 5), (6, 1020, 9, 17, 2), (5, 992, 7, 31, 30), (3, 1024, 32, 32, 1), (8, 33, 4, 11, 7),
    (5, 24, 3, 24, 3), (4, 1023, 12, 1, 1), (130, 64, 6, 2, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("T,E,k,n_groups,k_groups", SHAPES)
def test_route_matches_64_bits(T, E, k, n_groups, k_groups, score, group_score):
    rng = np.random.default_rng(T * 1000 + E + n_groups)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32)
    _run(logits, bias, k, n_groups, k_groups, score, group_score, True, 2.5)
    _run(logits, None, k, n_groups, k_groups, score, group_score, False, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_values_next_to_a_border(score, group_score):
    """Keys that agree to FP32 and beyond: the order is that of 64 bits, equal keys go to the lower index."""
    rng = np.random.default_rng(11)
    T, E = 200, 64
    base = np.float32(0.7)
    ulps = rng.integers(-3, 4, (T, E))  # logits a few FP32 steps around one value, many of them equal
    logits = (np.full((T, E), base).view(np.int32) + ulps).astype(np.int32).view(np.float32)
    _run(logits, None, 8, 8, 3, score, group_score, True, 1.0)
    _run(logits, None, 8, 1, 1, score, group_score, True, 1.0)
    # biases that all but cancel what the scores differ by
    logits = rng.choice(np.array([0.25, 0.5, 0.75, 1.0], np.float32), (T, E))
    s = 1.0 / (1.0 + np.exp(-np.array([0.25, 0.5, 0.75, 1.0])))
    bias = rng.choice((s[3] - s), E).astype(np.float32)
    _run(logits, bias, 6, 4, 2, score, group_score, True, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("n_groups,gs,k_groups", [(8, 16, 4), (4, 24, 1), (16, 5, 9), (32, 32, 16), (3, 2, 2)])
def test_route_groups_next_to_a_border(score, group_score, n_groups, gs, k_groups):
    """Group scores a few FP32 steps apart, or equal, around the last that stays: the groups are those of 64 bits.
    A group's largest logit lies 0 to 3 steps above one value, its second is the same in all, so that scores are
    equal or differ by an FP32 step of a key; the rest is far below."""
    rng = np.random.default_rng(100 * n_groups + gs)
    T, E = 150, n_groups * gs
    logits = (rng.standard_normal((T, E)) - 6.0).astype(np.float32)
    for t in range(T):
        for g in range(n_groups):
            at = g * gs + rng.permutation(gs)[:2]
            far = rng.choice([0.0, 0.0, 0.0, 0.5, -0.5])  # some groups are out of the question, or in it for sure
            logits[t, at[0]] = (np.float32(0.7 + far).view(np.int32) + rng.integers(0, 4)).astype(np.int32).view(np.float32)
            logits[t, at[1]] = np.float32(0.4 + far)
    bias = np.full(E, 0.125, np.float32)
    _run(logits, bias, min(4, k_groups * gs), n_groups, k_groups, score, group_score, True, 1.0)
    _run(logits, None, min(4, k_groups * gs), n_groups, k_groups, score, group_score, False, 1.0)


def test_route_wide_logits_and_saturated_scores():
    rng = np.random.default_rng(12)
    logits = (rng.standard_normal((40, 128)) * 30).astype(np.float32)  # many sigmoids equal to 1 or near 0
    _run(logits, None, 8, 8, 4, "sigmoid", "top2", True, 1.0)
    _run((logits - 200).astype(np.float32), None, 8, 8, 4, "sigmoid", "max", False, 1.0)
    _run((rng.standard_normal((40, 128)) * 10).astype(np.float32), None, 8, 8, 4, "softmax", "top2", True, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_experts_switched_off(score, group_score):
    rng = np.random.default_rng(13)
    T, E = 60, 48
    logits = rng.standard_normal((T, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
    logits[rng.random((T, E)) < 0.6] = -np.inf
    logits[0, :] = -np.inf                      # nothing is left
    logits[1, :] = -np.inf
    logits[1, 17] = 0.5                         # one expert is left
    logits[2, :40] = -np.inf                    # whole groups are off
    logits[3, :] = np.finfo(np.float32).min     # the type's lowest value is a number
    ids = _run(logits, bias, 10, 6, 2, score, group_score, True, 1.5)
    assert np.all(ids[0] == -1) and ids[1, 0] == 17 and np.all(ids[1, 1:] == -1) and np.all(ids[3] >= 0)
    _run(logits, None, 10, 6, 6, score, group_score, False, 1.5)
    _run(logits, bias, 10, 1, 1, score, group_score, True, 1.5)


def test_route_nan_ranks_last():
    rng = np.random.default_rng(14)
    logits = rng.choice(np.array([0.0, -0.0, 0.5, -1.0, np.nan, 2.0, -np.inf], np.float32), (80, 24))
    for gsc in ("max", "top2"):
        _run(logits, None, 6, 4, 2, "sigmoid", gsc, True, 1.0)
        _run(logits, None, 12, 1, 1, "sigmoid", gsc, False, 1.0)
    _run(np.full((3, 24), np.nan, np.float32), None, 6, 4, 2, "sigmoid", "max", True, 1.0)


def test_route_feeds_the_layer():
    """The ids and weights, empty slots among them, are what moe_forward_routed takes."""
    import oracle
    from mxfp4_routed_expert_router_gb300 import layer, workloads as wl
    from parity_util import TOL, oracle_weights, rel_err
    cfg = wl.custom("grouped", 9, 256, 128, 16, 1, 6, 21)
    rng = np.random.default_rng(21)
    logits = rng.standard_normal((cfg.T, 16)).astype(np.float32)
    logits[:, rng.permutation(16)[:9]] = -np.inf
    B = _B()
    ids = torch.empty((cfg.T, 6), dtype=torch.int32, device="cuda")
    w = torch.empty((cfg.T, 6), device="cuda")
    B.moe_route_grouped(torch.from_numpy(logits).cuda(), None, cfg.T, 16, 6, 4, 2, B.MOE_SCORE_SIGMOID,
                        B.MOE_GROUP_TOP2, True, 2.0, ids, w)
    L = layer.MoeLayer(cfg)
    x_bits = wl.tokens(cfg)
    out = L.forward_routed(layer.bf16_tensor(x_bits), ids, w)
    L.sync()
    eids, ew = expected(logits, None, 6, 4, 2, "sigmoid", "top2", True, 2.0)
    assert (eids == -1).any()
    ref = oracle.moe_layer_routed(oracle_weights(cfg, range(16)), x_bits, eids, ew.astype(np.float32))
    assert rel_err(out.cpu().numpy(), ref) <= TOL
    L.free()


def test_route_on_a_side_stream_and_in_a_graph():
    B = _B()
    rng = np.random.default_rng(15)
    logits = rng.standard_normal((20, 64)).astype(np.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _run(logits, None, 4, 4, 2, "sigmoid", "max", True, 1.0, stream=side)
    lg = torch.zeros((20, 64), device="cuda")
    ids = torch.empty((20, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((20, 4), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_route_grouped(lg, None, 20, 64, 4, 4, 2, B.MOE_SCORE_SOFTMAX, B.MOE_GROUP_MAX, True, 1.0, ids, w)
    lg.copy_(torch.from_numpy(logits))
    g.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(ids.cpu().numpy(), expected(logits, None, 4, 4, 2, "softmax", "max", True, 1.0)[0])
