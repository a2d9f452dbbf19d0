"""AdamW steps on the GPU against the 64-bit oracle.

U = 2^-24, half a step of fp32 relative; half: that of the parameters' type (bf16 2^-8).
Written with fp32 factors (each rounded once) and at most 4 roundings:
  m   6 U (b1 |m| + (1 - b1) |g|),  v  8 U v
  p   U (3 |p| + 24 |step| + 8 |parts of the step|) and, rounded to the parameter, half |p|
where |parts| is the step with m replaced by b1 |m| + (1 - b1) |g| (the terms of m may
cancel).  8-bit moments: a value is at most half an e4m3 step from the fp32 one (and the
fp32 one as above from the oracle's), in units of its block's scale; the scale is the
largest magnitude over 448 to 12 U.  The oracle starts from what the GPU holds."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import training as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
BLOCK = moe.ADAMW_BLOCK
KINDS = [(BF, True), (BF, False), (F32, False)]      # parameters, masters


def to64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, dtype, gtype, bits, master, seed=0, decay=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    shapes = [n if isinstance(n, tuple) else (n,) for n in sizes]
    params = [(0.1 * r(n)).to(dtype) for n in shapes]
    st = moe.AdamWState(params, bits=bits, master=master, decay=decay)
    size = [10.0 ** -(i % 6) for i in range(len(shapes))]
    grads = [(s * r(n)).to(gtype) for s, n in zip(size, shapes)]
    return st, grads, g


def moments(st, i):
    """(m, v) that the state holds for parameter i, flat, in 64 bits."""
    a, n = st.starts[i], st.params[i].numel()
    m, v = to64(st.exp_avg)[a:a + n], to64(st.exp_avg_sq)[a:a + n]
    if st.bits == 32:
        return m, v
    block = (a + np.arange(n)) // BLOCK
    # a root that is held as zero counts as 2^-11 of its block's unit
    v = np.maximum(v, 2.0 ** -11)
    return m * to64(st.exp_avg_scale)[block], (v * to64(st.exp_avg_sq_scale)[block]) ** 2


def held(st):
    p = st.params if st.master is None else [st.of(st.master, i) for i in range(len(st.params))]
    return [(to64(q).ravel(),) + moments(st, i) for i, q in enumerate(p)]


def check_step(st, grads, c, t, before, lr=None, scale=1.0):
    lr = c.lr if lr is None else lr
    for i, (p, m, v) in enumerate(before):
        g = to64(grads[i]).ravel()
        if not len(g):
            continue
        wd = c.weight_decay * st.decay[i]
        want, wm, wv = R.adamw(p, g, m, v, t, lr, c.beta1, c.beta2, c.eps, wd, scale)
        root = np.sqrt(wv / (1 - c.beta2 ** t)) + c.eps
        parts = c.beta1 * np.abs(m) + (1 - c.beta1) * np.abs(g * scale)
        rate = lr / (1 - c.beta1 ** t) / root
        tol = U * (3 * np.abs(p) + 24 * rate * np.abs(wm) + 8 * rate * parts) + 1e-44
        got = to64(st.params[i]).ravel()
        if st.master is not None:
            master = st.of(st.master, i)
            assert (np.abs(to64(master).ravel() - want) <= tol + U * np.abs(want)).all()
            assert torch.equal(st.params[i], master.to(st.params[i].dtype))
        else:
            half = 2.0 ** -8 if st.params[i].dtype is BF else U
            assert (np.abs(got - want) <= tol + half * np.abs(want)).all()
        gm, gv = moments(st, i)
        if st.bits == 32:
            assert (np.abs(gm - wm) <= 6 * U * parts + 1e-44).all()
            assert (np.abs(gv - wv) <= 8 * U * wv + 1e-44).all()
            continue
        a, n = st.starts[i], len(g)
        for x, err, flat, scales in ((wm, 6 * U * parts, st.exp_avg, st.exp_avg_scale),
                                     (np.sqrt(wv), 8 * U * np.sqrt(wv), st.exp_avg_sq,
                                      st.exp_avg_sq_scale)):
            most = np.array([np.abs(x[b:b + BLOCK]).max() for b in range(0, n, BLOCK)])
            s = to64(scales)[a // BLOCK:a // BLOCK + len(most)]
            assert (np.abs(s - most / 448) <= 20 * U * most / 448 + 1e-44).all()
            unit = s[np.arange(n) // BLOCK]
            q = to64(flat)[a:a + n]
            half = R.e4m3_step(np.minimum(np.abs(x) / np.where(unit > 0, unit, 1), 448)) / 2
            assert (np.abs(q * unit - x) <= unit * half * (1 + 1e-5) + err + 1e-44).all()
            assert (to64(flat)[a + n:a + -(-n // BLOCK) * BLOCK] == 0).all()


SIZES = [
    [1],
    [7, 256, 255, 257, 8, 4095, 4096, 4097, 1],
    [(3, 5, 64), (128, 128), 100003],
    [0, 5, 0, 300, 0],
    [2, 3] * 20,                                    # more than the smaller table holds
    list(range(1, 560, 2)),                         # more than one launch holds
]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gtype", [BF, F32], ids=str)
@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[-1]}")
def test_steps(sizes, kind, gtype, bits):
    """The first steps from empty moments, each against one of the oracle."""
    st, grads, g = make(sizes, kind[0], gtype, bits, kind[1],
                        decay=[float(i % 3 != 1) for i in range(len(sizes))])
    c = moe.AdamWConfig(lr=0.01, beta1=0.9, beta2=0.97, eps=1e-8, weight_decay=0.1)
    ws = moe.Workspace()
    for t in (1, 2, 3, 50):
        before = held(st)
        moe.moe_adamw_step(st, grads, c, t, ws=ws)
        assert moe.moe_get_device_status(ws) == 0
        check_step(st, grads, c, t, before)
        for x in grads:
            x.copy_(x.roll(1) * 0.7 if x.numel() > 1 else -x)


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_and_a_captured_step(bits):
    """step, lr and grad_scale read on the device: a captured step that counts."""
    st, grads, _ = make([1000, 3], BF, F32, bits, True)
    other = make([1000, 3], BF, F32, bits, True)[0]
    c = moe.AdamWConfig(lr=123.0, beta2=0.99)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr, scale = torch.tensor(0.0, device="cuda"), torch.tensor([1.0], device="cuda")
    ws = moe.Workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        moe.moe_adamw_step(st, grads, c, step, lr=lr, grad_scale=scale, ws=ws)
    for t in range(1, 6):
        lr.fill_(0.01 / t)
        scale.fill_(0.5 + t)
        before = held(st)
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == t and moe.moe_get_device_status(ws) == 0
        check_step(st, grads, c, t, before, lr=float(lr), scale=float(scale))
        # the same step by the host's numbers, the gradients scaled before
        now = moe.AdamWConfig(lr=float(lr), beta2=0.99)
        moe.moe_adamw_step(other, [g * scale for g in grads], now, t)
    for a, b in zip(st.params, other.params):
        torch.testing.assert_close(a, b, rtol=2 ** -6, atol=1e-3)


def test_a_captured_step_of_many_tensors():
    """More tensors than one launch takes, replayed: the bits of the same steps called."""
    sizes = [1 + 37 * (i % 9) for i in range(600)]
    c = moe.AdamWConfig(lr=0.01)
    sets = [make(sizes, BF, F32, 8, True) for _ in range(2)]
    (a, ga, _), (b, gb, _) = sets
    steps = [torch.full((1,), t, device="cuda") for t in (1, 2, 3)]
    at = steps[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adamw_step(a, ga, c, at)
    for t in steps:
        at.copy_(t)
        graph.replay()
        moe.moe_adamw_step(b, gb, c, t)
    torch.cuda.synchronize()
    for x, y in ((a.master, b.master), (a.exp_avg, b.exp_avg), (a.exp_avg_sq, b.exp_avg_sq),
                 (a.exp_avg_scale, b.exp_avg_scale)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    # a number below 1 counts as 1
    (a, ga, _), (b, gb, _) = [make([300], F32, F32, 32, False) for _ in range(2)]
    moe.moe_adamw_step(a, ga, c, torch.zeros(1, dtype=torch.int64, device="cuda"))
    moe.moe_adamw_step(b, gb, c, torch.ones(1, dtype=torch.int64, device="cuda"))
    assert torch.equal(a.params[0], b.params[0])


def test_long_run_of_steps_is_torchs():
    """fp32 parameters and moments: a hundred steps beside torch's own optimizer."""
    g = torch.Generator(device="cuda").manual_seed(1)
    p = [torch.randn(n, generator=g, device="cuda") for n in (1000, 257)]
    q = [x.clone().requires_grad_(True) for x in p]
    st = moe.AdamWState(p)
    opt = torch.optim.AdamW(q, lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.05)
    c = moe.AdamWConfig(3e-3, 0.9, 0.95, 1e-8, 0.05)
    for t in range(1, 101):
        grads = [torch.randn(x.shape, generator=g, device="cuda") for x in p]
        moe.moe_adamw_step(st, grads, c, t)
        for x, d in zip(q, grads):
            x.grad = d
        opt.step()
    # 100 steps of at most lr 10, each within 40 U of itself and 3 U of the parameter
    for a, b in zip(p, q):
        assert ((a - b.detach()).abs() <= 100 * U * (0.03 * 40 + 3 * (a.abs() + 3))).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_elements_that_are_not_finite_stay_as_they_were(bits, bad):
    sizes, at = [700, 300], 511
    st, grads, _ = make(sizes, F32, F32, bits, False)
    c = moe.AdamWConfig(lr=0.01)
    moe.moe_adamw_step(st, grads, c, 1)
    before = held(st)
    ref_state, ref_grads, _ = make(sizes, F32, F32, bits, False)
    moe.moe_adamw_step(ref_state, ref_grads, c, 1)
    grads[0][at] = bad
    ws = moe.Workspace()
    moe.moe_adamw_step(st, grads, c, 2, ws=ws)
    assert moe.moe_get_device_status(ws) == 2
    moe.moe_adamw_step(ref_state, ref_grads, c, 2)
    after = held(st)
    assert after[0][0][at] == before[0][0][at]
    if bits == 32:
        assert after[0][1][at] == before[0][1][at] and after[0][2][at] == before[0][2][at]
    else:   # rounded again by its block's new scale
        unit = to64(st.exp_avg_scale)[at // BLOCK]
        q = abs(before[0][1][at]) / unit
        assert abs(after[0][1][at] - before[0][1][at]) <= R.e4m3_step(q) * unit
    keep = np.arange(700) != at
    assert np.array_equal(after[0][0][keep], to64(ref_state.params[0])[keep])
    assert np.array_equal(after[1][0], to64(ref_state.params[1]))
    assert np.isfinite(after[0][1]).all() and np.isfinite(after[0][2]).all()
    moe.moe_adamw_step(st, ref_grads, c, 3, ws=ws)
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_a_scale_that_is_not_finite_skips_the_step(bits):
    st, grads, _ = make([5000, 33], BF, BF, bits, True)
    c = moe.AdamWConfig(lr=0.01)
    moe.moe_adamw_step(st, grads, c, 1)
    flats = [t for t in (st.master, st.exp_avg, st.exp_avg_sq, st.exp_avg_scale,
                         st.exp_avg_sq_scale, *st.params) if t is not None]
    before = [t.clone() for t in flats]
    ws = moe.Workspace()
    moe.moe_adamw_step(st, grads, c, 2, grad_scale=torch.tensor(float("inf"), device="cuda"), ws=ws)
    assert moe.moe_get_device_status(ws) == 2
    for a, b in zip(flats, before):
        if bits == 8 and a.dtype == F32 and a is not st.master:
            torch.testing.assert_close(a, b, rtol=4 * U, atol=0)
        else:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_roots_held_as_zero_do_not_let_a_step_run_away():
    """Gradients 2^18.3 below their block's largest: the root is rounded to zero, the first
    moment is not.  When their gradient is exactly zero then, they move by no more than a
    few rates, not by the moment over eps."""
    p = [torch.zeros(256, device="cuda")]
    st = moe.AdamWState(p, bits=8)
    c = moe.AdamWConfig(lr=0.01, beta1=0.9, beta2=0.97, eps=1e-12, weight_decay=0.0)
    g = torch.full((256,), 100.0 * 2.0 ** -18.9, device="cuda")
    g[0] = 100.0
    moe.moe_adamw_step(st, [g], c, 1)
    # m keeps 2^-18.9 of its largest as its smallest value only with a larger gradient
    st.exp_avg.view(torch.uint8)[1:] = 1
    assert (st.exp_avg_sq.float()[1:] == 0).all() and (st.exp_avg.float()[1:] > 0).all()
    before, held_before = p[0].clone(), held(st)
    moe.moe_adamw_step(st, [torch.zeros_like(g)], c, 2)
    check_step(st, [torch.zeros_like(g)], c, 2, held_before)
    assert ((p[0] - before).abs()[1:] < 20 * 0.01).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-38, 0.0])
def test_tiny_blocks(scale):
    """Blocks whose magnitudes leave the normal range become zero, not NaN."""
    p = [torch.ones(600, device="cuda")]
    st = moe.AdamWState(p, bits=8)
    g = torch.full((600,), scale, device="cuda")
    for t in (1, 2):
        moe.moe_adamw_step(st, [g], moe.AdamWConfig(lr=0.1, weight_decay=0.0), t)
    assert torch.isfinite(p[0]).all()
    assert torch.isfinite(st.exp_avg.float()).all() and torch.isfinite(st.exp_avg_sq_scale).all()
    if scale == 0.0:
        assert (p[0] == 1).all() and (st.exp_avg.float() == 0).all()


def test_extreme_betas():
    for b1, b2 in ((0.0, 0.0), (0.0, 0.999), (0.999999, 0.9999999)):
        st, grads, _ = make([300], F32, F32, 32, False)
        c = moe.AdamWConfig(0.01, b1, b2, 1e-8, 0.0)
        step = torch.ones((), dtype=torch.int64, device="cuda")
        before = held(st)
        moe.moe_adamw_step(st, grads, c, 1)
        check_step(st, grads, c, 1, before)
        again = make([300], F32, F32, 32, False)[0]
        moe.moe_adamw_step(again, grads, c, step)
        torch.testing.assert_close(again.params[0], st.params[0], rtol=1e-5, atol=1e-7)


def test_bytes_around_the_tensors_are_left_alone():
    """Parameters inside a larger buffer, gaps of one value between them."""
    flat = torch.randn(5000, device="cuda")
    keep = flat.clone()
    spans = [(0, 1), (4, 7), (12, 260), (276, 300), (1000, 4096)]
    params = [flat[a:b] for a, b in spans]
    st = moe.AdamWState(params, bits=8)
    moe.moe_adamw_step(st, [torch.ones_like(p) for p in params], moe.AdamWConfig(lr=0.5), 1)
    inside = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for a, b in spans:
        inside[a:b] = True
    assert torch.equal(flat[~inside], keep[~inside]) and (flat[inside] != keep[inside]).all()


def test_streams_and_repeats():
    c = moe.AdamWConfig(lr=0.01)
    done = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        st, grads, _ = make([100003, 77, 4096], BF, BF, 8, True)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for t in range(1, 5):
                moe.moe_adamw_step(st, grads, c, t)
        torch.cuda.synchronize()
        done.append([st.master, st.exp_avg, st.exp_avg_sq, st.exp_avg_scale, *st.params])
    for other in done[1:]:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(done[0], other))


def test_refusals():
    st, grads, _ = make([100, (4, 8)], BF, BF, 8, False)
    c = moe.AdamWConfig()
    step = lambda g, s=st, t=1, **kw: moe.moe_adamw_step(s, g, c, t, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="1 for 2"):
        step(grads[:1])
    with pytest.raises(ValueError, match="shape"):
        step([grads[0], grads[1].view(8, 4)])
    with pytest.raises(ValueError, match="contiguous"):
        step([grads[0], grads[1].t().contiguous().t()])
    with pytest.raises(TypeError):
        step([grads[0], grads[1].float()])
    with pytest.raises(TypeError):
        step([g.half() for g in grads])
    with pytest.raises(ValueError):
        step([grads[0], grads[1].cpu()])
    with pytest.raises(moe.MoeError):
        step(grads, t=0)
    with pytest.raises(ValueError):
        step(grads, t=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError):
        step(grads, lr=torch.ones(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_adamw_step(st, grads, moe.AdamWConfig(beta1=1.0), 1)
    odd = torch.empty(101, dtype=BF, device="cuda")[1:]
    with pytest.raises(ValueError, match="aligned"):
        moe.AdamWState([odd])
    with pytest.raises(moe.MoeError):
        step([odd, grads[1]])
    keep = st.exp_avg
    st.exp_avg = keep[:256]
    with pytest.raises(ValueError, match="exp_avg"):
        step(grads)
    st.exp_avg = keep
    st.params[0].data = st.params[0].data.clone()
    with pytest.raises(ValueError, match="elsewhere"):
        step(grads)
