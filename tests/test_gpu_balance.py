"""The balance loss, its counts and its gradient on the GPU against the 64-bit oracle.

Counts and tokens are equal.  U = 2^-24.  With R the largest |l - max l| of a row:
exp is within 4 ulp and rounds its argument (R U of the result), a row's sum adds 10
levels and up to 32 values, the division two roundings: a probability is within
U (64 + 2 R) of itself (R at most 80 here: smaller probabilities than exp(-80) are
compared on an absolute scale of 1e-30).  The loss sums positive terms over tokens
(at most 300 in a warp here) and experts: relative U (512 + 2 R).  The gradient
multiplies such a probability by a difference of loads whose terms have those errors:
U (160 + 6 R) of the sum of its absolute terms; added onto dlogits, one rounding of
the result more."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import training as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA = 0.03

CASES = [  # T, E, k, seq_offsets, masked
    (1, 1, 1, None, False),
    (1, 8, 2, None, False),
    (15, 3, 3, None, True),
    (129, 8, 2, None, False),
    (301, 64, 6, None, True),
    (1000, 256, 8, None, False),
    (2049, 37, 5, None, False),
    (5000, 160, 6, None, True),
    (700, 1024, 32, None, False),
    (333, 1000, 8, None, True),
    (600, 513, 4, None, False),
    (300, 68, 2, None, False),
    (40, 16, 4, [0, 40], False),
    (500, 32, 4, [0, 1, 1, 2, 300, 300, 500], True),
    (3000, 256, 8, [0, 100, 100, 1517, 2900], True),       # rows behind the last sequence
    (900, 12, 3, [17, 400, 850], False),                   # and ahead of the first
    (640, 64, 2, list(range(0, 641, 5)), True),            # many short ones
    (50, 8, 2, [50, 50, 50], False),                       # none has a token
]


def make(case, score, seed=0, spread=1.0):
    T, E, k, offsets, masked = case
    g = torch.Generator().manual_seed(seed + T * 7919 + E)
    l = spread * torch.randn(T, E, generator=g) + 0.5 * torch.randn(1, E, generator=g)
    idx = torch.topk(l + torch.randn(T, E, generator=g), k, dim=1).indices.to(torch.int32)
    kw = dict(score=score, seq_offsets=None if offsets is None else
              torch.tensor(offsets, dtype=torch.int32),
              mask=torch.rand(T, generator=g) > 0.3 if masked else None)
    return l, idx, kw


def cuda(kw):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}


def reach(l):
    return float((l.max(dim=1, keepdim=True).values - l).max()) if l.numel() else 0.0


def check(case, l, idx, kw, rows=slice(None)):
    T, E, k, offsets, _ = case
    dev = cuda(kw)
    ws = moe.Workspace()
    loss, counts, tokens = moe.moe_balance_loss(l.cuda(), idx.cuda(), ALPHA, ws=ws, **dev)
    assert moe.moe_get_device_status(ws) == 0
    ref = {n: v.numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    want, c, n = R.balance(l.numpy(), idx.numpy(), ALPHA, **ref)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    far = min(reach(l), 80.0)
    assert abs(float(loss) - want) <= U * (512 + 2 * far) * want + 1e-30
    dloss = torch.tensor(1.75, device="cuda")
    got = moe.moe_balance_loss_backward(dloss, counts, tokens, l.cuda(), k, ALPHA, **dev)
    grad, size = R.balance_backward(1.75, l.numpy(), c, k, ALPHA, **ref)
    tol = U * (160 + 6 * far) * size
    assert (np.abs(got.cpu().double().numpy() - grad) <= tol + 1e-30).all()
    base = torch.randn(T, E, generator=torch.Generator().manual_seed(3)) * ALPHA / max(T, 1)
    onto = base.cuda()
    out = moe.moe_balance_loss_backward(dloss, counts, tokens, l.cuda(), k, ALPHA, onto=onto, **dev)
    assert out is onto
    both = base.double().numpy() + grad
    assert (np.abs(onto.cpu().double().numpy() - both) <= tol + U * np.abs(both) + 1e-30).all()
    off = np.ones(T, bool)
    for rows in R.members(T, ref["seq_offsets"], ref["mask"]):
        off[rows] = False
    assert (got.cpu().numpy()[off] == 0).all()
    assert torch.equal(onto.cpu()[off], base[off])
    # None stands for 1, a gradient may lie anywhere,
    inside = moe.moe_balance_loss_backward(torch.full((4,), 1.75, device="cuda")[1], counts, tokens,
                                           l.cuda(), k, ALPHA, **dev)
    assert torch.equal(inside, got)
    # and 2 dloss for twice the gradient, bit for bit
    one = moe.moe_balance_loss_backward(None, counts, tokens, l.cuda(), k, ALPHA, **dev)
    two = moe.moe_balance_loss_backward(torch.tensor([2.0], device="cuda"), counts, tokens,
                                        l.cuda(), k, ALPHA, **dev)
    assert torch.equal(2 * one, two)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_balance(case, score):
    check(case, *make(case, score))


@pytest.mark.parametrize("E", [2, 9, 20, 33, 50, 77, 100, 128, 131, 333, 512, 516])
def test_every_way_to_hold_a_row(E):
    case = (1100, E, min(E, 5), [0, 3, 700, 1090], True)
    for score in ("softmax", "sigmoid"):
        check(case, *make(case, score))


@pytest.mark.parametrize("S", [600, 2000, 65536])
def test_many_sequences(S):
    """Most of them empty: more than a block keeps at hand, and all that are allowed."""
    T, E, k = 700, 8, 2
    r = np.random.default_rng(S)
    offsets = np.sort(r.integers(0, T + 1, S + 1))
    case = (T, E, k, offsets.tolist(), True)
    check(case, *make(case, "softmax"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-300.0, -60.0, 60.0, 300.0])
def test_far_logits(score, shift):
    """Scores that would vanish or saturate."""
    case = (200, 24, 4, [0, 90, 200], False)
    l, idx, kw = make(case, score, spread=4.0)
    l = l + shift
    far = min(reach(l), 80.0)
    loss, counts, tokens = moe.moe_balance_loss(l.cuda(), idx.cuda(), ALPHA, **cuda(kw))
    ref = {n: v.numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    want = R.balance(l.numpy(), idx.numpy(), ALPHA, **ref)[0]
    assert abs(float(loss) - want) <= U * (512 + 2 * far) * want
    got = moe.moe_balance_loss_backward(None, counts, tokens, l.cuda(), 4, ALPHA, **cuda(kw))
    grad, size = R.balance_backward(1.0, l.numpy(), counts.cpu().numpy(), 4, ALPHA, **ref)
    assert (np.abs(got.cpu().double().numpy() - grad) <= U * (160 + 6 * far) * size + 1e-30).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_lowest_values(score):
    """Experts switched off by the type's lowest value have probability zero."""
    case = (150, 8, 2, None, False)
    l, idx, kw = make(case, score)
    l[:, 5] = torch.finfo(torch.float32).min
    l[3] = torch.finfo(torch.float32).min      # all of them: equal
    idx = torch.randint(0, 5, (150, 2), dtype=torch.int32)
    ws = moe.Workspace()
    loss, counts, tokens = moe.moe_balance_loss(l.cuda(), idx.cuda(), ALPHA, ws=ws, **kw)
    assert moe.moe_get_device_status(ws) == 0
    p = R.probabilities(np.where(l.numpy() < -1e30, -1e4, l.numpy()), score)
    want = ALPHA * (8 * counts.cpu().numpy()[0] / 300 * p.mean(axis=0)).sum()
    assert abs(float(loss) - want) <= 1e-5 * want
    got = moe.moe_balance_loss_backward(None, counts, tokens, l.cuda(), 2, ALPHA, **kw)
    assert torch.isfinite(got).all() and (got[torch.arange(150) != 3, 5] == 0).all()


def test_even_loads_have_no_gradient():
    T, E = 512, 16
    l = torch.randn(T, E, device="cuda")
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 8) % E], dim=1).to(torch.int32)
    loss, counts, tokens = moe.moe_balance_loss(l, idx.cuda(), ALPHA)
    assert (counts == 64).all() and abs(float(loss) / ALPHA - 1) < 1e-5
    got = moe.moe_balance_loss_backward(None, counts, tokens, l, 2, ALPHA)
    assert (got == 0).all()


def test_masked_tokens_are_not_looked_at():
    case = (400, 32, 4, [0, 130, 390], True)
    l, idx, kw = make(case, "softmax")
    kw = cuda(kw)
    want = moe.moe_balance_loss(l.cuda(), idx.cuda(), ALPHA, **kw)
    grad = moe.moe_balance_loss_backward(None, *want[1:], l.cuda(), 4, ALPHA, **kw)
    off = torch.ones(400, dtype=torch.bool)
    off[:390] = ~kw["mask"][:390].cpu()
    l[off] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38] * 8)
    idx[off] = 77
    ws = moe.Workspace()
    got = moe.moe_balance_loss(l.cuda(), idx.cuda(), ALPHA, ws=ws, **kw)
    assert moe.moe_get_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(moe.moe_balance_loss_backward(None, *got[1:], l.cuda(), 4, ALPHA, **kw), grad)


@pytest.mark.parametrize("T", [100, 5000])
def test_status(T):
    """What only the device can see, at a small and a large batch; the next call is clean."""
    case = (T, 16, 2, None, False)
    l, idx, kw = make(case, "softmax")
    l, idx = l.cuda(), idx.cuda()
    ws = moe.Workspace()
    want = moe.moe_balance_loss(l, idx, ALPHA, ws=ws, **kw)
    for bad in (float("nan"), float("inf"), -float("inf")):
        m = l.clone()
        m[T - 3, 7] = bad
        moe.moe_balance_loss(m, idx, ALPHA, ws=ws, **kw)
        assert moe.moe_status_string(moe.moe_get_device_status(ws)).find("NaN") >= 0
    for bad in (-1, 16, 2 ** 30, -2 ** 31):
        i = idx.clone()
        i[T // 2, 1] = bad
        loss, counts, tokens = moe.moe_balance_loss(l, i, ALPHA, ws=ws, **kw)
        assert moe.moe_get_device_status(ws) == 1
        assert int(counts.sum()) == 2 * T - 1 and int(tokens) == T
    for offsets in ([0, T + 1], [-1, T], [0, 50, 20, T], [2 ** 31 - 1, -2 ** 31]):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        _, counts, tokens = moe.moe_balance_loss(l, idx, ALPHA, seq_offsets=o, ws=ws)
        assert moe.moe_get_device_status(ws) == 1
        moe.moe_balance_loss_backward(None, counts, tokens, l, 2, ALPHA, seq_offsets=o)
    got = moe.moe_balance_loss(l, idx, ALPHA, ws=ws, **kw)
    assert moe.moe_get_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_batch():
    l, idx = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, tokens = moe.moe_balance_loss(l, idx, ALPHA)
    assert float(loss) == 0 and (counts == 0).all() and int(tokens) == 0
    assert moe.moe_balance_loss_backward(None, counts, tokens, l, 2, ALPHA).shape == (0, 8)
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts, tokens = moe.moe_balance_loss(l, idx, ALPHA, seq_offsets=o)
    assert float(loss) == 0 and counts.shape == (3, 8) and (tokens == 0).all()


def test_counts_are_the_layers():
    """The counts are those of the permutation of the same routing."""
    l = torch.randn(3000, 64, device="cuda")
    idx, _ = moe.moe_route_topk(l, 6)
    _, counts, _ = moe.moe_balance_loss(l, idx, ALPHA)
    assert torch.equal(counts[0], moe.moe_permute(idx, 64)[0])


def test_streams_graphs_and_repeats():
    case = (6000, 128, 4, [0, 1000, 1003, 5900], True)
    sets = [make(case, "sigmoid", seed) for seed in (1, 2)]
    ws = moe.Workspace()

    def step(l, idx, kw):
        loss, counts, tokens = moe.moe_balance_loss(l, idx, ALPHA, ws=ws, **kw)
        return loss, counts, tokens, moe.moe_balance_loss_backward(loss, counts, tokens, l, 4,
                                                                   ALPHA, **kw)

    sets = [(l.cuda(), idx.cuda(), cuda(kw)) for l, idx, kw in sets]
    want = [step(*s) for s in sets]
    for _ in range(20):
        got = step(*sets[0])
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = step(*sets[1])
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    l, idx, kw = sets[0][0].clone(), sets[0][1].clone(), cuda(sets[0][2])
    kw = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    graphs, outs = [], []
    for _ in range(2):    # two graphs on one workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(l, idx, kw))
        graphs.append(graph)
    for i in (1, 0, 1):
        l.copy_(sets[i][0])
        idx.copy_(sets[i][1])
        for n in ("seq_offsets", "mask"):
            kw[n].copy_(sets[i][2][n])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_refusals():
    l, idx = torch.randn(10, 8, device="cuda"), torch.zeros(10, 2, dtype=torch.int32, device="cuda")
    o = torch.tensor([0, 10], device="cuda")
    with pytest.raises(TypeError):
        moe.moe_balance_loss(l, idx.long(), ALPHA)
    with pytest.raises(TypeError):
        moe.moe_balance_loss(l, idx, ALPHA, seq_offsets=o)
    with pytest.raises(TypeError):
        moe.moe_balance_loss(l, idx, ALPHA, mask=torch.ones(10, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_balance_loss(l, idx, ALPHA, mask=torch.ones(9, dtype=torch.bool, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, idx, float("inf"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, idx, ALPHA, seq_offsets=o[:1].int())
    loss, counts, tokens = moe.moe_balance_loss(l, idx, ALPHA)
    with pytest.raises(ValueError):
        moe.moe_balance_loss_backward(l, counts, tokens, l, 2, ALPHA)
    with pytest.raises(ValueError):
        moe.moe_balance_loss_backward(None, counts[:, :4], tokens, l, 2, ALPHA)
