"""Layer norm and its gradients on the GPU against the 64-bit oracle.

U = 2^-24 is half a step of fp32, relative; `half` that of the output's type
(bf16: 2^-8).  Sums over H or over tokens are trees of fp32 additions: a term
passes through at most 24 roundings in a sum over a row (8 to 64 values per
thread one after the other count once each, 10 levels of a block's tree), and
through at most 128 in a sum over T <= 10000 tokens (up to 66 rows of a block,
then the blocks).  So, with |.| the terms' absolute values:
  mean     32 U mean|h|;  rstd relative 64 U (its own and the mean's errors, rsqrtf 2 ulp)
  y        half |y| + U w (64 |xhat| + 32 mean|h| rstd) + 2 U (|xhat w| + |b|)
  dx       half |dx| + U (rstd (8 |w dy| + 40 mean|w dy| + 48 |xhat| mean|w dy xhat|) + |dh|)
  dw, db   half |dw| + 136 U sum_t |dy xhat|"""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import training as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32

# T, H: one value; below, at and above the widths at which the kernels' shapes change; odd ones
SIZES = [(1, 1), (3, 7), (5, 8), (1, 128), (33, 255), (64, 256), (7, 264), (300, 511), (9, 512),
         (129, 520), (4, 1000), (11, 1001), (2000, 1024), (3, 1025), (50, 1032), (301, 2048),
         (17, 4099), (160, 4096), (1, 7168), (700, 7168), (5, 8191), (6, 8192), (4, 8193),
         (9, 8200), (2, 12345), (310, 16384), (3, 16383)]
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


def to64(t):
    return t.detach().double().cpu().numpy()


def make(T, H, dtype, wtype, seed=0, offset=0.5, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + H)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=r(T, H).to(dtype), residual=(spread * r(T, H) + offset).to(dtype),
                weight=(1 + 0.3 * r(H)).to(wtype), bias=r(H).to(wtype), dy=r(T, H).to(dtype),
                dh=r(T, H).to(dtype))


def check_forward(d, y, h, stats, eps, bias=True):
    b = to64(d["bias"]) if bias else 0.0
    want, mean, rstd = R.norm(to64(h), to64(d["weight"]), None, eps)
    half = HALF[d["x"].dtype]
    size = np.abs(to64(h)).mean(axis=1)
    if stats is not None:
        s = to64(stats)
        assert (np.abs(s[:, 0] - mean) <= 32 * U * size + 1e-38).all()
        assert (np.abs(s[:, 1] / rstd - 1) <= 64 * U).all()
    w = np.abs(to64(d["weight"]))
    xhat = np.abs(to64(h) - mean[:, None]) * rstd[:, None]
    tol = half * np.abs(want + b) + U * w * (64 * xhat + (32 * size * rstd)[:, None]) + \
        2 * U * (xhat * w + np.abs(b))
    assert (np.abs(to64(y) - (want + b)) <= tol).all()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, types):
    d = make(*size, *types)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], 1e-5, residual=d["residual"])
    both = to64(d["x"]) + to64(d["residual"])
    # one rounding of the sum; the fp32 sum of two bf16 values may be rounded before
    assert (np.abs(to64(h) - both) <= HALF[types[0]] * np.abs(both) * (1 + 2.0 ** -15)).all()
    check_forward(d, y, h, stats, 1e-5)
    # without a residual, a bias, statistics
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], want_stats=False)
    assert h is d["x"] and stats is None
    check_forward(d, y, h, None, 1e-5, bias=False)


def check_backward(d, h, stats, got, dh=None):
    dx, dw, db = got
    s = to64(stats)
    args = [to64(d["dy"]), to64(h), s[:, 0], s[:, 1], to64(d["weight"])]
    want = R.norm_backward(*args, None if dh is None else to64(dh))
    half, whalf = HALF[dx.dtype], HALF[dw.dtype]
    x = np.abs(args[1] - args[2][:, None]) * args[3][:, None]
    g = np.abs(args[0] * args[4])
    tol = args[3][:, None] * (8 * g + 40 * g.mean(axis=1, keepdims=True) +
                              48 * x * (g * x).mean(axis=1, keepdims=True))
    tol = half * np.abs(want[0]) + U * (tol + (0 if dh is None else np.abs(to64(dh))))
    assert (np.abs(to64(dx) - want[0]) <= tol).all()
    a = np.abs(args[0])
    assert (np.abs(to64(dw) - want[1]) <= whalf * np.abs(want[1]) + 136 * U * (a * x).sum(0)).all()
    if db is not None:
        assert (np.abs(to64(db) - want[2]) <= whalf * np.abs(want[2]) + 136 * U * a.sum(0)).all()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, types):
    d = make(*size, *types)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], 1e-5, residual=d["residual"])
    got = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"])
    check_backward(d, h, stats, got, d["dh"])
    again = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))   # the same bits
    got = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], has_bias=False)
    assert got[2] is None
    check_backward(d, h, stats, got)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", [(5000, 33), (3000, 255), (2500, 500), (2000, 1001), (1300, 2047),
                                  (900, 4099), (500, 7170), (400, 9001), (320, 12002)], ids=str)
def test_many_rows_of_odd_widths(size, types):
    """Blocks that take several rows, none of which starts on a 16-byte boundary of its own."""
    d = make(*size, *types)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], 1e-5, residual=d["residual"])
    check_forward(d, y, h, stats, 1e-5)
    got = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"])
    check_backward(d, h, stats, got, d["dh"])


def test_gradient_equals_differences():
    """The GPU's gradients against central differences of the definition."""
    d = make(3, 40, F32, F32)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"])
    dx, dw, db = (to64(t) for t in moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"]))
    x, w, b, dy = (to64(d[n]) for n in ("x", "weight", "bias", "dy"))
    for grad, at, f in ((dx, x, lambda a: R.norm(a, w, b, 1e-5)[0]),
                        (dw, w, lambda a: R.norm(x, a, b, 1e-5)[0]),
                        (db, b, lambda a: R.norm(x, w, a, 1e-5)[0])):
        for i in np.ndindex(at.shape):
            up, down = at.copy(), at.copy()
            up[i] += 1e-5
            down[i] -= 1e-5
            slope = ((f(up) - f(down)) * dy).sum() / 2e-5
            assert abs(grad[i] - slope) <= 1e-5 * (1 + abs(slope))


def test_large_mean_small_spread():
    """The variance is taken around the mean: a spread of 1 around 3000 survives."""
    d = make(20, 2048, F32, F32, offset=3000.0, spread=1.0)
    d["x"].zero_()
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], residual=d["residual"])
    check_forward(d, y, h, stats, 1e-5)
    s = to64(stats)
    assert (np.abs(s[:, 1] - 1) < 0.1).all()


def test_constant_rows_and_empty_batches():
    w, b = torch.full((128,), 2.0, device="cuda"), torch.ones(128, device="cuda")
    x = torch.full((3, 128), 5.0, device="cuda")
    y, h, stats = moe.moe_layer_norm(x, w, b, 1e-4)
    assert (y == 1).all() and (stats[:, 0] == 5).all()
    assert (stats[:, 1] - 100).abs().max() < 1e-4
    dx, dw, db = moe.moe_layer_norm_backward(torch.ones_like(x), h, stats, w)
    assert (dx == 0).all() and (dw == 0).all() and (db == 3).all()
    none = torch.empty(0, 128, device="cuda")
    y, h, stats = moe.moe_layer_norm(none, w, b)
    assert y.shape == (0, 128) and stats.shape == (0, 2)
    dx, dw, db = moe.moe_layer_norm_backward(none, none, stats, w)
    assert dx.shape == (0, 128) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_token(bad):
    d = make(40, 2048, BF, BF)
    clean = moe.moe_layer_norm(d["x"], d["weight"], d["bias"])
    stats = clean[2].clone()
    want = moe.moe_layer_norm_backward(d["dy"], d["x"], stats, d["weight"])[0]
    d["x"][7, 100] = bad
    y, h, s = moe.moe_layer_norm(d["x"], d["weight"], d["bias"])
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(s[keep], stats[keep])
    assert not torch.isfinite(y[7].float()).all()
    dx = moe.moe_layer_norm_backward(d["dy"], h, s, d["weight"])[0]
    assert torch.equal(dx[keep], want[keep])


@pytest.mark.parametrize("H", [512, 1001, 7168])
def test_in_place(H):
    """The sum takes the residual's place, dx takes dy's or dh's."""
    d = make(333, H, BF, BF)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], residual=d["residual"])
    for name in ("x", "residual"):
        e = {k: v.clone() for k, v in d.items()}
        got = moe.moe_layer_norm(e["x"], e["weight"], e["bias"], residual=e["residual"], h=e[name])
        assert got[1] is e[name] and torch.equal(got[1], h) and torch.equal(got[0], y)
    e = d["x"].clone()
    assert torch.equal(moe.moe_layer_norm(e, d["weight"], y=e)[0],
                       moe.moe_layer_norm(d["x"], d["weight"])[0])
    want = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"])
    for name in ("dy", "dh"):
        e = {k: v.clone() for k, v in d.items()}
        got = moe.moe_layer_norm_backward(e["dy"], h, stats, d["weight"], dh=e["dh"], dx=e[name])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_graphs_and_workspaces():
    """Another stream, a captured call replayed on new values, two graphs that
    share a workspace, a workspace that other sizes used before."""
    d, e = make(600, 2048, BF, F32, 1), make(600, 2048, BF, F32, 2)
    ws = moe.Workspace()

    def step(v):
        y, h, stats = moe.moe_layer_norm(v["x"], v["weight"], v["bias"], residual=v["residual"])
        return (y, h, stats) + moe.moe_layer_norm_backward(v["dy"], h, stats, v["weight"],
                                                           dh=v["dh"], ws=ws)

    want = [step(d), step(e)]
    small = make(5, 64, F32, F32)
    _, h, stats = moe.moe_layer_norm(small["x"], small["weight"])
    moe.moe_layer_norm_backward(small["dy"], h, stats, small["weight"], ws=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step(d)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    held = {k: v.clone() for k, v in d.items()}
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(held))
        graphs.append(graph)
    for source, ref in ((e, want[1]), (d, want[0]), (e, want[1])):
        for k in held:
            held[k].copy_(source[k])
        for graph, out in zip(graphs, outs):
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refusals():
    d = make(4, 64, BF, F32)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_layer_norm(d["x"].t().contiguous().t(), d["weight"])
    with pytest.raises(ValueError, match="shape"):
        moe.moe_layer_norm(d["x"], d["weight"][:32])
    with pytest.raises(TypeError):
        moe.moe_layer_norm(d["x"], d["weight"], d["bias"].to(BF))
    with pytest.raises(TypeError):
        moe.moe_layer_norm(d["x"].float(), d["weight"].to(BF))
    with pytest.raises(ValueError, match="h: x itself"):
        moe.moe_layer_norm(d["x"], d["weight"], h=d["dy"])
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm(d["x"], d["weight"], eps=0.0)
    odd = torch.empty(4 * 64 + 1, dtype=BF, device="cuda")[1:].view(4, 64)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm(odd, d["weight"])
