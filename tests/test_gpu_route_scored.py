"""Scored routing on the GPU against the 64-bit oracle.

The choice is an integer decision on fp32 values: it must equal the oracle's
on every token whose decision does not hang on less than TIE of a difference
(fp32 scores are within 4 ulp of the exact ones, 2^-22 of values up to one;
sums of two such values twice that).  Exactly equal values on both sides are
ties and follow the rule.  Weights: expf is within 2 ulp, l - max is rounded
once (an error of 2^-24 |l - max| in the exponent), the sum of at most 32
terms adds 5 roundings and the division, the score's own division and the
scale one each: 2^-24 (16 + 2 |l - max|) of the weight covers them.
The gradient multiplies weights by a difference of dw and a weighted mean:
2^-18 of the sum of the absolute terms."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import moe_oracle as O
from oracle import scored_route as S
from routing_grouped_expert_gb300 import inputs as I
from tests.helpers import assert_moe_close, backward_mismatches, to_np

pytestmark = pytest.mark.gpu

TIE = 2.0 ** -20

CASES = [  # T, E, k, score, biased, groups, keep, group_top, renormalize, scale
    (1, 1, 1, "softmax", False, 1, 1, 1, True, 1.0),
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (7, 5, 5, "sigmoid", True, 1, 1, 1, True, 1.0),
    (128, 8, 2, "softmax", False, 1, 1, 1, True, 1.0),
    (333, 8, 2, "softmax", True, 4, 1, 2, False, 1.0),
    (1000, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (257, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (129, 37, 5, "sigmoid", False, 1, 1, 1, True, 1.0),
    (65, 66, 7, "softmax", True, 22, 5, 2, True, 1.0),
    (65, 96, 3, "sigmoid", False, 32, 2, 2, True, 1.0),
    (200, 64, 32, "sigmoid", True, 2, 1, 1, False, 1.0),
    (64, 1024, 32, "softmax", True, 32, 8, 2, True, 1.0),
    (64, 1000, 8, "sigmoid", True, 8, 2, 2, True, 1.0),
    (40, 512, 16, "softmax", False, 16, 4, 2, False, 1.0),
    (4097, 128, 6, "sigmoid", True, 4, 4, 1, True, 1.0),
]


def make(case, kind="normal", spread=1.0):
    T, E, k, score, biased, G, keep, top, renorm, scale = case
    g = torch.Generator().manual_seed(T * 7919 + E * 31 + k)
    if kind == "ties":
        l = torch.tensor([-1.0, -0.0, 0.0, 0.5, 2.0])[torch.randint(0, 5, (T, E), generator=g)]
        b = torch.full((E,), 0.25)   # one value: equal sums then have equal terms
    else:
        l = spread * torch.randn(T, E, generator=g)
        b = 0.1 * torch.randn(E, generator=g)
    cfg = moe.RouteConfig(score, G, keep, top, renorm, scale)
    return l, (b if biased else None), cfg


def near(values, count):
    """Rows whose `count` largest values hang on a difference below TIE (equal
    values are ties, not near ties)."""
    v = -np.sort(-values, axis=1)[:, :count + 1]
    with np.errstate(invalid="ignore"):
        gap = v[:, :-1] - v[:, 1:]
    return ((gap > 0) & (gap < TIE * (1 + np.abs(v[:, :-1])))).any(axis=1)


def check(case, l, b, cfg, idx, w):
    T, E, k, score, _, G, keep, top, renorm, scale = case
    ln, bn = l.numpy(), None if b is None else b.numpy()
    ref = S.choose(ln, k, bn, score, G, keep, top)
    rank, mask, group = S.ranking(ln, bn, score, G, keep, top)
    close = near(np.where(mask, rank, -np.inf), k) | (near(group, keep) if G > 1 else False)
    idx = to_np(idx)
    differ = (idx != ref).any(axis=1)
    assert not (differ & ~close).any(), np.nonzero(differ & ~close)[0][:8]
    assert close.sum() <= 2 + T // 50
    assert idx.min() >= 0 and idx.max() < E
    assert all(len(set(r)) == k for r in idx.tolist())
    want = S.weights(ln, idx, bn, score, renorm, scale)
    far = np.abs(ln).max() * 2
    assert (np.abs(to_np(w) - want) <= 2.0 ** -24 * (16 + 2 * far) * want + 1e-30).all()


@pytest.mark.parametrize("kind", ["normal", "ties"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_route(case, kind):
    l, b, cfg = make(case, kind)
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(l.cuda(), case[2], cfg, bias=None if b is None else b.cuda(),
                                  ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    check(case, l, b, cfg, idx, w)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    T, E, k, score, _, G, keep, top, renorm, scale = case
    l, b, cfg = make(case)
    if b is not None and k < keep * (E // G):
        b[E // 2] = -float("inf")
    dev_b = None if b is None else b.cuda()
    idx, _ = moe.moe_route_scored(l.cuda(), k, cfg, bias=dev_b)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(5))
    ws = moe.Workspace()
    got = to_np(moe.moe_route_scored_backward(dw.cuda(), idx, l.cuda(), cfg, bias=dev_b, ws=ws))
    assert moe.moe_get_device_status(ws) == 0
    i, bn = to_np(idx), None if b is None else b.numpy()
    ref = S.backward(dw.numpy(), l.numpy(), i, bn, score, renorm, scale)
    w = np.abs(S.weights(l.numpy(), i, bn, score, renorm, scale))
    g = np.abs(dw.numpy())
    size = np.zeros_like(ref)
    mean = (w * g).sum(axis=1, keepdims=True) / (scale if renorm else 1.0)
    np.put_along_axis(size, i.astype(np.int64), w * (g + mean), axis=1)
    if score == "softmax" and not renorm:
        size += S.scores(l.numpy(), score) * mean
    assert (np.abs(got - ref) <= 2.0 ** -18 * size + 1e-30).all()
    dense = score == "softmax" and not renorm
    if not dense:
        chosen = np.zeros(ref.shape, bool)
        np.put_along_axis(chosen, i.astype(np.int64), True, axis=1)
        assert (got[~chosen] == 0).all()


def test_backward_equals_differences():
    """The GPU's gradient against central differences of its own 64-bit
    definition, on one token per configuration."""
    for case in CASES[5:8]:
        T, E, k, score, _, G, keep, top, renorm, scale = case
        l, b, cfg = make(case)
        l = l[:3].contiguous()
        dev_b = None if b is None else b.cuda()
        idx, _ = moe.moe_route_scored(l.cuda(), k, cfg, bias=dev_b)
        dw = torch.randn(3, k, generator=torch.Generator().manual_seed(6))
        got = to_np(moe.moe_route_scored_backward(dw.cuda(), idx, l.cuda(), cfg, bias=dev_b))
        bn = None if b is None else b.numpy()
        f = lambda x: (dw.numpy() * S.weights(x, to_np(idx), bn, score, renorm, scale)  # noqa: E731
                       ).sum(axis=1)
        x, h = l.numpy().astype(np.float64), 1e-5
        for e in range(E):
            d = np.zeros_like(x)
            d[:, e] = h
            num = (f(x + d) - f(x - d)) / (2 * h)
            np.testing.assert_allclose(got[:, e], num, rtol=0, atol=2e-6 * scale)


@pytest.mark.parametrize("offset", [-30.0, -70.0, -300.0, 60.0])
def test_extreme_logits_keep_renormalised_weights(offset):
    """Scores near the ends of the range: the weights are ratios, which stay
    finite and sum to the scale though every score underflows."""
    for score in ("sigmoid", "softmax"):
        case = (50, 32, 4, score, False, 1, 1, 1, True, 2.0)
        l, b, cfg = make(case)
        l = l + offset
        idx, w = moe.moe_route_scored(l.cuda(), 4, cfg)
        np.testing.assert_array_equal(to_np(idx), S.choose(l.numpy(), 4, None, score))
        # in 64 bits sigmoid(-300) is still a normal number
        want = S.weights(l.numpy(), to_np(idx), None, score, True, 2.0)
        # as above, the score's own error twice (in the sum as well)
        np.testing.assert_allclose(to_np(w), want, rtol=2.0 ** -19, atol=0)


def test_switched_off_experts():
    case = (300, 64, 6, "sigmoid", True, 8, 3, 2, True, 1.0)
    l, b, cfg = make(case)
    off = torch.arange(64) % 3 != 0
    b[off] = -float("inf")
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(l.cuda(), 6, cfg, bias=b.cuda(), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    check(case, l, b, cfg, idx, w)
    assert not off[to_np(idx).astype(int)].any()
    # fewer experts on than slots: the rest carry no weight
    b[:] = -float("inf")
    b[9] = 0.0
    idx, w = moe.moe_route_scored(l.cuda(), 6, cfg, bias=b.cuda())
    check(case, l, b, cfg, idx, w)
    on = to_np(idx) == 9
    np.testing.assert_array_equal(to_np(w), on.astype(np.float32))
    # no expert on
    b[9] = -float("inf")
    idx, w = moe.moe_route_scored(l.cuda(), 6, cfg, bias=b.cuda(), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    assert (to_np(w) == 0).all() and to_np(idx).min() >= 0
    d = moe.moe_route_scored_backward(torch.ones_like(w), idx, l.cuda(), cfg, bias=b.cuda())
    assert (to_np(d) == 0).all()


def test_plain_softmax_is_moe_route_topk():
    for T, E, k in ((300, 8, 2), (513, 256, 8), (64, 1024, 8)):
        l = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).cuda()
        idx, w = moe.moe_route_scored(l, k, moe.RouteConfig())
        ref_idx, ref_w = moe.moe_route_topk(l, k)
        assert torch.equal(idx, ref_idx)
        torch.testing.assert_close(w, ref_w, rtol=0, atol=2e-6)


def test_nonfinite_values_are_reported():
    case = (100, 32, 4, "sigmoid", True, 4, 2, 2, True, 1.0)
    for score in ("sigmoid", "softmax"):
        for what in ("logit", "bias"):
            for value in (float("nan"), float("inf")):
                l, b, _ = make(case)
                cfg = moe.RouteConfig(score, 4, 2, 2)
                if what == "logit":
                    l[37, 5] = value
                else:
                    b[5] = value
                ws = moe.Workspace()
                idx, w = moe.moe_route_scored(l.cuda(), 4, cfg, bias=b.cuda(), ws=ws)
                assert moe.moe_get_device_status(ws) == 2
                i = to_np(idx)
                assert i.min() >= 0 and i.max() < 32
                assert all(len(set(r)) == 4 for r in i.tolist())
                # the next call on the workspace starts clean
                l, b, _ = make(case)
                moe.moe_route_scored(l.cuda(), 4, cfg, bias=b.cuda(), ws=ws)
                assert moe.moe_get_device_status(ws) == 0


def test_backward_skips_and_reports_bad_indices():
    l = torch.randn(20, 16, generator=torch.Generator().manual_seed(1))
    cfg = moe.RouteConfig("sigmoid")
    idx, _ = moe.moe_route_scored(l.cuda(), 4, cfg)
    dw = torch.randn(20, 4, generator=torch.Generator().manual_seed(2)).cuda()
    good = moe.moe_route_scored_backward(dw, idx, l.cuda(), cfg)
    bad = idx.clone()
    bad[7, 2], bad[9, 0] = -1, 16
    ws = moe.Workspace()
    got = moe.moe_route_scored_backward(dw, bad, l.cuda(), cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 1
    rows = [t for t in range(20) if t not in (7, 9)]
    assert torch.equal(got[rows], good[rows])
    assert int((got[7] != 0).sum()) <= 3 and int((got[9] != 0).sum()) <= 3


def test_empty_batch_and_another_stream():
    cfg = moe.RouteConfig("sigmoid", 4, 2, 2)
    idx, w = moe.moe_route_scored(torch.empty(0, 16, device="cuda"), 4, cfg)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    l = torch.randn(500, 16, generator=torch.Generator().manual_seed(3)).cuda()
    want = moe.moe_route_scored(l, 4, cfg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = moe.Workspace()
        got = moe.moe_route_scored(l, 4, cfg, ws=ws)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


LAYERS = {  # T, H, F, E, k, score, biased, groups, keep, group_top, renormalize, scale
    "sigmoid_groups": (150, 256, 128, 32, 6, "sigmoid", True, 8, 4, 2, True, 2.5),
    "softmax_dense": (300, 256, 256, 4, 2, "softmax", True, 1, 1, 1, False, 4.0),
    "softmax_small": (64, 256, 384, 8, 2, "softmax", False, 2, 1, 1, True, 1.0),
}


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_forward_and_backward(name, monkeypatch):
    """The whole layer on scored routing, against the oracle's layer with the
    oracle's routing replaced by the scored one; gradients likewise, the logit
    gradient by the scored formula from the oracle's weight gradients."""
    T, H, F, E, k, score, biased, G, keep, top, renorm, scale = LAYERS[name]
    d = I.make_inputs(I.small(name, T=T, H=H, F=F, E=E, k=k), "cpu")
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(8)) if biased else None
    cfg = moe.RouteConfig(score, G, keep, top, renorm, scale)
    dev = {n: t.cuda() for n, t in d.items()}
    dev_b = None if b is None else b.cuda()
    args = (dev["x"], dev["logits"], dev["W1"], dev["W3"], dev["W2"], k, cfg)
    ws, wst = moe.Workspace(), moe.Workspace()
    out = moe.moe_forward_scored(*args, bias=dev_b, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    routing = moe.moe_forward_routing(ws, T, H, F, E, k)
    alone = moe.moe_route_scored(dev["logits"], k, cfg, bias=dev_b)
    assert torch.equal(routing[0], alone[0]) and torch.equal(routing[1], alone[1])
    ln, bn = d["logits"].numpy(), None if b is None else b.numpy()
    idx, w = to_np(alone[0]), to_np(alone[1])
    check((T, E, k, score, biased, G, keep, top, renorm, scale), d["logits"], b, cfg, *alone)
    monkeypatch.setattr(O, "route_topk", lambda *_: (idx, w))
    ref = O.forward_perm(d["x"], ln, d["W1"], d["W3"], d["W2"], k)
    big = max(1.0, float(np.abs(w).max()))
    assert_moe_close(out / big, ref["out"] / big, f"{name} out")
    trained = moe.moe_forward_scored_train(*args, ws=wst, bias=dev_b)
    assert torch.equal(trained, out)
    dout = torch.randn(T, H, generator=torch.Generator().manual_seed(31)).to(torch.bfloat16)
    dx, dl, dW1, dW3, dW2 = moe.moe_backward_scored(dout.cuda(), *args[1:], ws=wst, bias=dev_b)
    assert moe.moe_get_device_status(wst) == 0
    ref = O.backward(d["x"], ln, d["W1"], d["W3"], d["W2"], k, dout, magnitudes=True)
    msgs = []
    for key, got in (("dx", dx), ("dW1", dW1), ("dW3", dW3), ("dW2", dW2)):
        msgs += backward_mismatches(name, got, ref, key)
    assert not msgs, msgs
    want = S.backward(ref["dw"], ln, idx, bn, score, renorm, scale)
    # dw comes from bf16 expert outputs: normwise, as the other gradients
    assert np.linalg.norm(to_np(dl) - want) <= 2.0 ** -5 * np.linalg.norm(want) + 1e-6 * T * E


def test_layer_empty_batch_and_other_workspaces():
    d = I.make_inputs(I.small("tiny", T=32, H=128, F=128, E=8, k=2), "cuda")
    cfg = moe.RouteConfig("sigmoid", 2, 1, 2)
    a = moe.moe_forward_scored(d["x"], d["logits"], d["W1"], d["W3"], d["W2"], 2, cfg)
    # the plain layer on the same default workspace is what it was
    plain = moe.moe_forward(d["x"], d["logits"], d["W1"], d["W3"], d["W2"], 2)
    again = moe.moe_forward_scored(d["x"], d["logits"], d["W1"], d["W3"], d["W2"], 2, cfg)
    assert torch.equal(a, again)
    assert torch.equal(plain, moe.moe_forward(d["x"], d["logits"], d["W1"], d["W3"], d["W2"], 2))
    empty = moe.moe_forward_scored(d["x"][:0], d["logits"][:0], d["W1"], d["W3"], d["W2"], 2, cfg)
    assert empty.shape == (0, 128)


LARGE = [  # several tokens per warp, chunks of four and single experts
    (2049, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (3001, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (2500, 100, 8, "sigmoid", True, 5, 2, 2, True, 1.0),
    (5000, 64, 8, "softmax", True, 1, 1, 1, True, 1.0),
    (2050, 24, 16, "softmax", True, 2, 2, 2, False, 1.0),
    (2700, 250, 12, "sigmoid", False, 10, 7, 2, True, 1.0),
    (4111, 12, 3, "sigmoid", True, 3, 2, 1, True, 1.0),
    (2100, 16, 9, "softmax", False, 16, 9, 1, True, 1.0),
    (2048, 384, 6, "softmax", True, 8, 3, 2, True, 1.0),
    (20000, 32, 4, "sigmoid", True, 4, 2, 1, True, 1.0),
]


@pytest.mark.parametrize("kind", ["normal", "ties"])
@pytest.mark.parametrize("case", LARGE, ids=str)
def test_route_large_batches(case, kind):
    l, b, cfg = make(case, kind)
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(l.cuda(), case[2], cfg, bias=None if b is None else b.cuda(),
                                  ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    check(case, l, b, cfg, idx, w)
    # the first tokens of the batch, one per warp: the same bits
    few = moe.moe_route_scored(l[:70].cuda(), case[2], cfg, bias=None if b is None else b.cuda())
    assert torch.equal(few[0], idx[:70])
    torch.testing.assert_close(few[1], w[:70], rtol=2.0 ** -20, atol=0)


def test_outputs_given_and_refused():
    l = torch.randn(40, 16, generator=torch.Generator().manual_seed(3)).cuda()
    cfg = moe.RouteConfig("sigmoid")
    idx, w = moe.moe_route_scored(l, 4, cfg)
    i2 = torch.empty(40, 4, dtype=torch.int32, device="cuda")
    w2 = torch.empty(40, 4, device="cuda")
    got = moe.moe_route_scored(l, 4, cfg, topk_idx=i2, topk_w=w2)
    assert got[0] is i2 and got[1] is w2 and torch.equal(i2, idx) and torch.equal(w2, w)
    with pytest.raises(ValueError):
        moe.moe_route_scored(l, 4, cfg, topk_idx=i2[:, :3])
    with pytest.raises(TypeError):
        moe.moe_route_scored(l, 4, cfg, bias=torch.zeros(16, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        moe.moe_route_scored(l.half(), 4, cfg)
    with pytest.raises(ValueError):
        moe.moe_route_scored(l.t(), 4, cfg)
    with pytest.raises(ValueError):
        moe.moe_route_scored_backward(w[:, :3].contiguous(), idx, l, cfg)
    with pytest.raises(moe.MoeError):
        moe.moe_route_scored(l, 17, cfg)


def test_captured_in_a_graph():
    """Route and gradient replayed from a CUDA graph on refilled inputs."""
    cfg = moe.RouteConfig("sigmoid", 8, 4, 2, True, 2.5)
    l = torch.zeros(300, 64, device="cuda")
    dw = torch.randn(300, 6, generator=torch.Generator().manual_seed(4)).cuda()
    ws = moe.Workspace()
    moe.moe_route_scored(l, 6, cfg, ws=ws)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        idx, w = moe.moe_route_scored(l, 6, cfg, ws=ws)
        d = moe.moe_route_scored_backward(dw, idx, l, cfg, ws=ws)
    for seed in (1, 2):
        l.copy_(torch.randn(300, 64, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        ref = moe.moe_route_scored(l, 6, cfg)
        assert torch.equal(idx, ref[0]) and torch.equal(w, ref[1])
        assert torch.equal(d, moe.moe_route_scored_backward(dw, idx, l, cfg))


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_status_of_a_reused_workspace(T):
    """A report of the last token; the next call clears it, whatever the
    workspace held before."""
    cfg = moe.RouteConfig("sigmoid", 8, 4, 2, True, 2.5)
    dense = moe.RouteConfig("softmax", renormalize=False)   # its gradient reads every logit
    ws = moe.Workspace()
    ws.ensure(256).fill_(0xff)
    good = torch.randn(T, 64, generator=torch.Generator().manual_seed(6)).cuda()
    bad = good.clone()
    bad[T - 1, 63] = float("nan")
    dw = torch.randn(T, 6, generator=torch.Generator().manual_seed(7)).cuda()
    idx, _ = moe.moe_route_scored(good, 6, cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    for _ in range(3):
        moe.moe_route_scored(bad, 6, cfg, ws=ws)
        assert moe.moe_get_device_status(ws) == 2
        moe.moe_route_scored_backward(dw, idx, good, dense, ws=ws)
        assert moe.moe_get_device_status(ws) == 0
        moe.moe_route_scored_backward(dw, idx, bad, dense, ws=ws)
        assert moe.moe_get_device_status(ws) == 2
        moe.moe_route_scored(good, 6, cfg, ws=ws)
        assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_renormalised_slot_has_no_gradient(score):
    """Its weight is the constant scale."""
    cfg = moe.RouteConfig(score, scale=2.5)
    l = torch.randn(37, 24, generator=torch.Generator().manual_seed(8)).cuda()
    dw = torch.randn(37, 1, generator=torch.Generator().manual_seed(9)).cuda()
    idx, w = moe.moe_route_scored(l, 1, cfg)
    assert torch.equal(w, torch.full_like(w, 2.5))
    assert not moe.moe_route_scored_backward(dw, idx, l, cfg).any()


DENSE = [  # softmax without renormalisation: 1, 2, 4, 8, 16 and 32 logits per lane
    (70, 20, 3, "softmax", False, 1, 1, 1, False, 1.0),
    (300, 64, 6, "softmax", False, 1, 1, 1, False, 1.0),
    (131, 33, 4, "softmax", True, 1, 1, 1, False, 2.5),
    (257, 100, 5, "softmax", True, 5, 2, 2, False, 1.0),
    (90, 128, 8, "softmax", False, 4, 2, 1, False, 1.0),
    (75, 250, 7, "softmax", True, 10, 4, 2, False, 1.0),
    (60, 511, 8, "softmax", False, 7, 3, 1, False, 16.0),
    (50, 1000, 8, "softmax", True, 8, 2, 2, False, 1.0),
    (33, 1024, 32, "softmax", False, 32, 8, 1, False, 1.0),
]


@pytest.mark.parametrize("case", DENSE, ids=str)
def test_dense_gradient(case):
    test_backward(case)


MANY_TOKENS = [  # more tokens than the grid takes at once; more than 8 logits per lane but in the last
    (40001, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (20011, 250, 12, "sigmoid", True, 10, 4, 2, True, 1.0),
    (24001, 160, 4, "sigmoid", True, 1, 1, 1, True, 2.5),
    (6007, 384, 6, "softmax", True, 8, 3, 2, True, 1.0),
    (2501, 1000, 8, "sigmoid", True, 8, 2, 2, True, 1.0),
    (12011, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
]


@pytest.mark.parametrize("case", MANY_TOKENS, ids=str)
def test_route_and_gradient_of_many_tokens(case):
    """Every warp routes several tokens one after the other.  The choice is
    checked against the oracle at tokens of every pass, and all of it against
    the same tokens routed in batches that the grid takes at once."""
    T, E, k = case[:3]
    l, b, cfg = make(case)
    dev_l, dev_b = l.cuda(), None if b is None else b.cuda()
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(dev_l, k, cfg, bias=dev_b, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    rows = torch.arange(0, T, max(1, T // 1500))
    rows = torch.cat([rows, torch.arange(T - 40, T)]).unique()
    check((len(rows), *case[1:]), l[rows], b, cfg, idx[rows.cuda()], w[rows.cuda()])
    for t0 in range(0, T, 1000):
        part = moe.moe_route_scored(dev_l[t0:t0 + 1000], k, cfg, bias=dev_b)
        assert torch.equal(part[0], idx[t0:t0 + 1000])
        torch.testing.assert_close(part[1], w[t0:t0 + 1000], rtol=2.0 ** -20, atol=0)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(5)).cuda()
    d = moe.moe_route_scored_backward(dw, idx, dev_l, cfg, bias=dev_b, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    i, wn = to_np(idx[rows.cuda()]), np.abs(to_np(w[rows.cuda()])).astype(np.float64)
    g = np.abs(to_np(dw[rows.cuda()])).astype(np.float64)
    bn = None if b is None else b.numpy()
    score, renorm, scale = case[3], case[8], case[9]
    ref = S.backward(to_np(dw[rows.cuda()]), l[rows].numpy(), i, bn, score, renorm, scale)
    size = np.zeros_like(ref)
    mean = (wn * g).sum(axis=1, keepdims=True) / (scale if renorm else 1.0)
    np.put_along_axis(size, i.astype(np.int64), wn * (g + mean), axis=1)
    if score == "softmax" and not renorm:
        size += S.scores(l[rows].numpy(), score) * mean
    assert (np.abs(to_np(d[rows.cuda()]) - ref) <= 2.0 ** -18 * size + 1e-30).all()


@pytest.mark.parametrize("T", [60, 2100])     # a token per warp, several tokens per warp
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_masked_by_the_lowest_logit(score, T):
    """Logits of the type's lowest value, which some routers mask with: never
    chosen while others are left, no weight and no gradient, and finite where a
    whole row is masked."""
    low = torch.finfo(torch.float32).min
    l, _, _ = make((T, 64, 6, score, False, 1, 1, 1, True, 1.0))
    masked = torch.arange(64) % 4 == 1
    l[:, masked] = low
    l[3, :] = low                      # a row whose mask leaves nothing
    l[5, 4:] = low                     # fewer experts than slots
    for renorm in (True, False):
        cfg = moe.RouteConfig(score, 8, 8, 1, renorm)
        ws = moe.Workspace()
        idx, w = moe.moe_route_scored(l.cuda(), 6, cfg, ws=ws)
        assert moe.moe_get_device_status(ws) == 0
        i, ln = to_np(idx), l.numpy()
        np.testing.assert_array_equal(i, S.choose(ln, 6, None, score, 8, 8, 1))
        want = S.weights(ln, i, None, score, renorm, 1.0)
        dw = torch.randn(T, 6, generator=torch.Generator().manual_seed(5))
        ref = S.backward(dw.numpy(), ln, i, None, score, renorm, 1.0)
        if score == "sigmoid" and renorm:
            # sigmoid(low) is zero in 64 bits too, but the ratio of equal scores
            # is one: each of the six has a sixth, and 1 - s is one
            want[3] = 1 / 6
            g3 = dw[3].double().numpy()
            np.put(ref[3], i[3], (g3 - g3.mean()) / 6)
        # as above; the logits that are left are at most 8 apart
        np.testing.assert_allclose(to_np(w), want, rtol=2.0 ** -18, atol=1e-30)
        d = to_np(moe.moe_route_scored_backward(dw.cuda(), idx, l.cuda(), cfg, ws=ws))
        assert moe.moe_get_device_status(ws) == 0 and np.isfinite(d).all()
        rows = np.delete(np.arange(T), 3)
        assert (d[rows][:, masked.numpy()] == 0).all()
        size = np.zeros_like(ref)
        g = np.abs(dw.numpy()).astype(np.float64)
        mean = (want * g).sum(axis=1, keepdims=True)
        np.put_along_axis(size, i.astype(np.int64), want * (g + mean), axis=1)
        if score == "softmax" and not renorm:
            size += S.scores(ln, score) * mean
        assert (np.abs(d - ref) <= 2.0 ** -18 * size + 1e-30).all()


@pytest.mark.parametrize("scored", [False, True])
def test_layer_gradients_of_an_empty_batch_are_zero(scored):
    d = I.make_inputs(I.small("tiny", T=32, H=128, F=256, E=8, k=2), "cuda")
    weights = (d["W1"], d["W3"], d["W2"])
    empty = d["x"][:0], d["logits"][:0], *weights, 2
    ws = moe.Workspace()
    # what the allocator hands out next is not zero
    leftovers = [torch.full_like(w, float("nan")) for w in (*weights, *weights)]
    del leftovers
    if scored:
        cfg = moe.RouteConfig("sigmoid", 2, 1, 2)
        moe.moe_forward_scored_train(*empty, cfg, ws)
        dx, dl, *dW = moe.moe_backward_scored(d["x"][:0], *empty[1:], cfg, ws)
    else:
        moe.moe_forward_train(*empty, ws)
        dx, dl, *dW = moe.moe_backward(d["x"][:0], *empty[1:], ws)
    assert dx.shape == (0, 128) and dl.shape == (0, 8)
    for got, w in zip(dW, weights):
        assert got.shape == w.shape and (got == 0).all()
