"""The scored-routing oracle against independent statements of it, and the
entry points' refusals (nothing here needs a GPU)."""
import ctypes
import itertools

import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import scored_route as S
from routing_grouped_expert_gb300 import binding

CONFIGS = [  # score, biased, groups, keep, group_top, renormalize, scale
    ("softmax", False, 1, 1, 1, True, 1.0), ("softmax", False, 4, 2, 1, False, 16.0),
    ("softmax", True, 2, 1, 2, True, 1.0), ("sigmoid", True, 4, 2, 2, True, 2.5),
    ("sigmoid", False, 2, 2, 2, False, 1.0), ("sigmoid", True, 1, 1, 1, False, 0.5),
]


def test_softmax_without_bias_is_the_plain_routing():
    l = np.random.default_rng(0).standard_normal((64, 16)).astype(np.float32)
    l[3] = np.round(l[3])                               # ties
    idx = S.choose(l, 4)
    ref_idx, ref_w = O.route_topk(l, 4)
    np.testing.assert_array_equal(idx, ref_idx)
    np.testing.assert_allclose(S.weights(l, idx), ref_w, rtol=0, atol=1e-7)


@pytest.mark.parametrize("cfg", CONFIGS)
def test_choice_is_the_best_set_of_all(cfg):
    """Brute force: over all sets of `keep` groups, then over all k-subsets of
    their experts, none has a larger sum."""
    score, biased, G, keep, top, _, _ = cfg
    rng = np.random.default_rng(1)
    E, k = 8, 2
    l = rng.standard_normal((30, E))
    b = 0.3 * rng.standard_normal(E) if biased else None
    idx = S.choose(l, k, b, score, G, keep, top)
    rank, mask, group = S.ranking(l, b, score, G, keep, top)
    size = E // G
    for t in range(len(l)):
        kept = {e // size for e in range(E) if mask[t, e]}
        best = max(itertools.combinations(range(G), keep), key=lambda c: group[t, list(c)].sum())
        assert kept == set(best)
        cand = [e for e in range(E) if e // size in kept]
        best = max(itertools.combinations(cand, k), key=lambda c: rank[t, list(c)].sum())
        assert set(idx[t].tolist()) == set(best)
        assert rank[t, idx[t, 0]] >= rank[t, idx[t, 1]]


@pytest.mark.parametrize("cfg", CONFIGS)
def test_gradient_equals_differences(cfg):
    score, biased, G, keep, top, renorm, scale = cfg
    rng = np.random.default_rng(2)
    l = rng.standard_normal((5, 8))
    b = 0.3 * rng.standard_normal(8) if biased else None
    if biased:
        b[2] = -np.inf
    idx = S.choose(l, 3, b, score, G, keep, top)
    dw = rng.standard_normal(idx.shape)
    f = lambda x: (dw * S.weights(x, idx, b, score, renorm, scale)).sum()  # noqa: E731
    num = np.zeros_like(l)
    h = 1e-5
    for i in np.ndindex(l.shape):
        d = np.zeros_like(l)
        d[i] = h
        num[i] = (f(l + d) - f(l - d)) / (2 * h)
    # second-order remainder h^2 |f'''| / 6 and cancellation 2^-53 |f| / h
    np.testing.assert_allclose(S.backward(dw, l, idx, b, score, renorm, scale), num, rtol=0,
                               atol=1e-8 * max(1.0, scale))


def test_switched_off_experts():
    l = np.zeros((1, 4))
    b = np.array([-np.inf, 0.0, -np.inf, -np.inf])
    idx = S.choose(l, 3, b, "sigmoid")
    assert idx.tolist() == [[1, 0, 2]]
    np.testing.assert_array_equal(S.weights(l, idx, b, "sigmoid"), [[1.0, 0.0, 0.0]])
    off = np.full(4, -np.inf)
    idx = S.choose(l, 2, off, "sigmoid")
    np.testing.assert_array_equal(S.weights(l, idx, off, "sigmoid"), [[0.0, 0.0]])
    np.testing.assert_array_equal(S.backward(np.ones((1, 2)), l, idx, off, "sigmoid"),
                                  np.zeros((1, 4)))


def test_refusals():
    lib = binding.load_library()
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4100)    # never dereferenced
    good = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)
    INVALID, WS, OK = 1, 4, 0

    def route(T=16, E=16, k=4, logits=p, bias=p, idx=p, w=p, ws=p, nbytes=256, **kw):
        c = binding.RouteConfig(**{**good, **kw})
        return lib.moe_route_scored(logits, bias, c._ptr, T, E, k, idx, w, ws, nbytes, None)

    for bad in (dict(n_group=3), dict(n_group=0), dict(topk_group=0), dict(topk_group=5),
                dict(group_top=0), dict(group_top=3), dict(n_group=16, topk_group=4),
                dict(k=9), dict(k=0), dict(k=17), dict(E=0), dict(E=1028), dict(T=-1),
                dict(logits=None), dict(idx=None), dict(w=None), dict(logits=odd), dict(bias=odd),
                dict(scale=float("inf")), dict(scale=float("nan")),
                dict(E=66, n_group=33, topk_group=33)):
        assert route(**bad) == INVALID, bad
    assert route(ws=None) == WS and route(nbytes=255) == WS
    assert route(ws=ctypes.c_void_p(4096 + 16)) == WS
    assert route(T=0, logits=None, idx=None, w=None, ws=None, nbytes=0) == OK
    assert lib.moe_route_scored(p, p, None, 16, 16, 4, p, p, p, 256, None) == INVALID
    c = binding.RouteConfig(**good)
    bwd = lib.moe_route_scored_backward
    assert bwd(None, p, p, p, c._ptr, 16, 16, 4, p, p, 256, None) == INVALID
    assert bwd(p, p, p, p, c._ptr, 16, 16, 4, None, p, 256, None) == INVALID
    assert bwd(p, p, p, p, None, 16, 16, 4, p, p, 256, None) == INVALID
    assert bwd(p, p, p, p, c._ptr, 16, 16, 4, p, p, 8, None) == WS
    assert bwd(None, None, None, None, c._ptr, 0, 16, 4, None, None, 0, None) == OK
    big = 1 << 40
    fwd = lib.moe_forward_scored
    assert fwd(p, p, odd, c._ptr, p, p, p, 16, 512, 1024, 16, 4, p, p, big, None) == INVALID
    assert fwd(p, p, p, None, p, p, p, 16, 512, 1024, 16, 4, p, p, big, None) == INVALID
    assert fwd(p, p, None, c._ptr, p, p, p, 16, 512, 1024, 16, 4, p, p, 64, None) == WS
    assert lib.moe_forward_scored_train(p, p, None, c._ptr, p, p, p, 16, 512, 1024, 16, 9, p, p,
                                        big, None) == INVALID
    assert lib.moe_backward_scored(p, p, None, c._ptr, p, p, p, 16, 512, 1024, 16, 4, p, None, p,
                                   p, p, p, big, None) == INVALID
    with pytest.raises(ValueError):
        binding.RouteConfig(score="relu")
