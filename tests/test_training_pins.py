"""Pins of the training step's 64-bit oracle, and the refusals of its entry points
(nothing here needs a GPU)."""
import copy
import ctypes

import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import training as R
from routing_grouped_expert_gb300 import binding


def differences(f, x, h=1e-6):
    """Central differences of f over every element of x."""
    grad = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        grad[i] = (f(a) - f(b)) / (2 * h)
    return grad


# ------------------------------------------------------------------ layer norm
def test_norm_is_torchs():
    r = np.random.default_rng(1)
    h, w, b = r.normal(2, 3, (7, 33)), r.normal(1, 0.1, 33), r.normal(0, 1, 33)
    y, mean, rstd = R.norm(h, w, b, 1e-5)
    want = torch.nn.functional.layer_norm(torch.tensor(h), (33,), torch.tensor(w), torch.tensor(b))
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(mean, h.mean(axis=1), rtol=1e-14)
    np.testing.assert_allclose(rstd, 1 / np.sqrt(h.var(axis=1) + 1e-5), rtol=1e-13)


def test_norm_gradient_equals_differences():
    r = np.random.default_rng(2)
    h, w, dy, dh = (r.normal(size=s) for s in ((3, 6), 6, (3, 6), (3, 6)))
    loss = lambda h, w, b: (R.norm(h, w, b, 1e-5)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = R.norm(h, w, None, 1e-5)
    dx, dw, db = R.norm_backward(dy, h, mean, rstd, w, dh)
    np.testing.assert_allclose(dx, differences(lambda a: loss(a, w, None), h) + dh, atol=1e-7)
    np.testing.assert_allclose(dw, differences(lambda a: loss(h, a, None), w), atol=1e-7)
    np.testing.assert_allclose(db, differences(lambda a: loss(h, w, a), np.zeros(6)), atol=1e-7)


# ---------------------------------------------------------------- balance loss
def case(score, seed=3):
    r = np.random.default_rng(seed)
    l = r.normal(size=(11, 5))
    idx = np.argsort(-l, axis=1)[:, :2]
    return l, idx, dict(alpha=0.3, score=score, seq_offsets=[0, 4, 4, 9],
                        mask=np.array([1, 0, 1, 1, 1, 1, 1, 0, 1, 1, 1], bool))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_by_hand(score):
    l, idx, kw = case(score)
    loss, counts, tokens = R.balance(l, idx, **kw)
    assert tokens.tolist() == [3, 0, 4] and counts.sum(axis=1).tolist() == [6, 0, 8]
    want = 0.0
    for rows in ([0, 2, 3], [4, 5, 6, 8]):
        for e in range(5):
            f = sum(int(e in idx[t]) for t in rows) * 5 / (2 * len(rows))
            mass = 0.0
            for t in rows:
                s = [1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x) for x in l[t]]
                mass += s[e] / sum(s)
            want += f * mass / len(rows)
    assert abs(loss - 0.3 * want / 3) < 1e-14
    # even loads: the loss is alpha
    even = np.array([[t % 5, (t + 1) % 5] for t in range(10)])
    assert abs(R.balance(l[:10], even, 0.3, score)[0] - 0.3) < 1e-14


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_equals_differences(score):
    l, idx, kw = case(score)
    _, counts, _ = R.balance(l, idx, **kw)
    grad, size = R.balance_backward(1.7, l, counts, 2, kw["alpha"], score, kw["seq_offsets"],
                                    kw["mask"])
    want = differences(lambda a: 1.7 * R.balance(a, idx, **kw)[0], l)
    np.testing.assert_allclose(grad, want, atol=1e-9)
    assert (np.abs(grad) <= size + 1e-15).all()
    for t in (1, 7, 9, 10):
        assert (grad[t] == 0).all()


def test_scores_that_vanish_keep_their_ratios():
    p = R.probabilities([[-800.0, -800.0, -801.0]], "sigmoid")
    e = np.exp([0.0, 0.0, -1.0])
    np.testing.assert_allclose(p[0], e / e.sum(), rtol=1e-12)
    np.testing.assert_allclose(R.probabilities([[800.0, 900.0]], "sigmoid")[0], [0.5, 0.5])


# ------------------------------------------------------------------------ AdamW
def test_adamw_is_torchs():
    r = np.random.default_rng(4)
    p0, grads = r.normal(size=9), r.normal(size=(5, 9))
    p = torch.tensor(p0, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.02, betas=(0.8, 0.97), eps=1e-6, weight_decay=0.1)
    q, m, v = p0, np.zeros(9), np.zeros(9)
    for t, g in enumerate(grads, 1):
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = R.adamw(q, g, m, v, t, 0.02, 0.8, 0.97, 1e-6, 0.1)
    np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12)


def test_e4m3_values_and_steps():
    x = torch.tensor(R.E4M3)
    assert len(R.E4M3) == 253    # both zeros are one
    assert torch.equal(x.to(torch.float8_e4m3fn).double(), x)
    pos = np.array([v for v in R.E4M3 if v >= 0])
    np.testing.assert_array_equal(R.e4m3_step(pos[:-1]), np.diff(pos))


# -------------------------------------------------------------------- refusals
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)   # never read
BIG = 1 << 40
INVALID, WS, OK = 1, 4, 0


def test_norm_refuses():
    f = binding.load_library().moe_layer_norm
    good = dict(x=P, r=P, w=P, b=P, eps=1e-5, T=4, H=128, t=0, wt=0, y=P, h=P, s=P)
    call = lambda **kw: f(*{**good, **kw}.values(), None)  # noqa: E731
    for bad in (dict(x=None), dict(x=ODD), dict(w=None), dict(b=ODD), dict(y=None), dict(h=None),
                dict(r=None), dict(s=ODD), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(T=-1), dict(H=0), dict(H=16385), dict(t=2),
                dict(t=1, wt=0), dict(wt=2), dict(wt=-1)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, w=None, y=None, h=None) == OK
    size = binding.moe_layer_norm_workspace_size
    assert size(-1, 128) == 0 and size(1, 0) == 0 and size(1, 16385) == 0
    assert 0 < size(0, 128) <= size(1, 128) < size(10 ** 6, 128)
    b = binding.load_library().moe_layer_norm_backward
    good = dict(dy=P, h=P, s=P, w=P, dh=P, T=4, H=128, t=0, wt=0, dx=P, dw=P, db=P, ws=P, n=BIG)
    call = lambda **kw: b(*{**good, **kw}.values(), None)  # noqa: E731
    for bad in (dict(dy=None), dict(h=None), dict(s=None), dict(w=None), dict(dh=ODD),
                dict(dx=None), dict(dw=None), dict(db=ODD), dict(T=-1), dict(H=16385),
                dict(t=1, wt=0), dict(T=0, dw=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(n=1024), dict(ws=ctypes.c_void_p(4096 + 16))):
        assert call(**bad) == WS, bad


def test_balance_refuses():
    lib = binding.load_library()
    good = dict(l=P, i=P, sc=0, al=0.1, o=P, m=P, T=4, E=8, k=2, S=3, loss=P, c=P, n=P, ws=P,
                size=BIG)
    call = lambda **kw: lib.moe_balance_loss(*{**good, **kw}.values(), None)  # noqa: E731
    for bad in (dict(l=None), dict(i=ODD), dict(sc=2), dict(al=float("nan")), dict(o=None),
                dict(o=ODD), dict(m=ODD), dict(T=-1), dict(E=0), dict(E=1025), dict(k=9),
                dict(k=0), dict(S=0), dict(S=65537), dict(loss=None), dict(c=None), dict(n=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(size=256)):
        assert call(**bad) == WS, bad
    good = dict(d=P, c=P, n=P, l=P, sc=0, al=0.1, o=P, m=P, T=4, E=8, k=2, S=3, acc=0, out=P)
    call = lambda **kw: lib.moe_balance_loss_backward(*{**good, **kw}.values(), None)  # noqa: E731
    for bad in (dict(d=ctypes.c_void_p(4098)), dict(c=None), dict(n=None), dict(l=None), dict(sc=-1), dict(o=None),
                dict(m=ODD), dict(S=0), dict(k=33, E=64), dict(out=None)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, c=None, n=None, l=None, out=None) == OK
    size = moe.moe_balance_workspace_size
    assert size(-1, 8) == 0 and size(4, 0) == 0 and size(4, 8, 0) == 0 and size(4, 8, 65537) == 0
    assert 0 < size(0, 8) <= size(4, 8) < size(4, 8, 9)


def test_adamw_refuses():
    lib = binding.load_library()
    Tensor, Config = binding._AdamWTensor, binding._AdamWConfigStruct
    good = dict(param=4096, n=10, start=256, decay=1.0, grad=4096, count=1, pt=0, gt=0, lr=1e-3,
                b1=0.9, b2=0.99, eps=1e-8, wd=0.1, bits=32, step=1, at=None, lr_at=None, gs=None,
                master=P, m=P, v=P, ms=None, vs=None, ws=P, size=256)

    def call(**kw):
        a = {**good, **kw}
        tensors = (Tensor * 1)((a["param"], a["n"], a["start"], a["decay"]))
        grads = (ctypes.c_void_p * 1)(a["grad"])
        config = Config(a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["bits"])
        return lib.moe_adamw_step(tensors, grads, a["count"], a["pt"], a["gt"],
                                  ctypes.byref(config), a["step"], a["at"], a["lr_at"], a["gs"],
                                  a["master"], a["m"], a["v"], a["ms"], a["vs"], a["ws"],
                                  a["size"], None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(param=0), dict(param=4104), dict(grad=0), dict(grad=4104), dict(n=-1),
                dict(start=100), dict(start=-256), dict(decay=nan), dict(count=-1), dict(pt=2),
                dict(gt=-1), dict(pt=1), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
                dict(b2=nan), dict(eps=0.0), dict(eps=inf), dict(wd=nan), dict(bits=16),
                dict(step=0), dict(at=ODD), dict(lr_at=ctypes.c_void_p(4098)), dict(m=None),
                dict(v=None), dict(m=ctypes.c_void_p(4112)), dict(master=ctypes.c_void_p(4112)),
                dict(bits=8), dict(bits=8, ms=P), dict(bits=8, ms=P, vs=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(size=255)):
        assert call(**bad) == WS, bad


def test_bindings_refuse():
    """Checks that come before anything of CUDA."""
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(16)
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x.half(), w)
    with pytest.raises(TypeError):
        moe.moe_layer_norm_backward(x, x, torch.zeros(4, 2), w.double())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w)            # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 0.1, "max")
    for params, kw in (([], {}), ([w], dict(bits=16)), ([w], dict(master=True)), ([w.half()], {}),
                       ([w], dict(decay=[1.0, 1.0]))):
        with pytest.raises((ValueError, TypeError)):
            moe.AdamWState(params, **kw)


def test_adamw_state_layout(monkeypatch):
    """Every parameter on blocks of its own; shared memory refused; copies keep
    parameters and places of their own."""
    def need(t, dtype, shape, name, cuda=True):
        return _need(t, dtype, shape, name, cuda=False)
    _need = binding._need
    monkeypatch.setattr(binding, "_need", need)
    params = [torch.randn(n) for n in (1, 256, 0, 257)]
    st = moe.AdamWState(params, bits=8, decay=[1, 0, 1, 0.5])
    assert st.starts == [0, 256, 512, 512] and st.size == 1024
    assert st.exp_avg.dtype == torch.float8_e4m3fn and st.exp_avg_scale.shape == (4,)
    assert st.of(st.exp_avg, 3).shape == (257,) and st.master is None
    b = [torch.randn(4, 5).to(torch.bfloat16), torch.randn(300).to(torch.bfloat16)]
    st = moe.AdamWState(b, master=True)
    assert torch.equal(st.of(st.master, 0), b[0].float())
    assert torch.equal(st.of(st.master, 1), b[1].float())
    # leaves of a graph: the masters are none
    leaf = torch.randn(8).to(torch.bfloat16).requires_grad_(True)
    masters = moe.AdamWState([leaf], master=True).master
    assert not masters.requires_grad and masters.grad_fn is None
    flat = torch.zeros(64)
    with pytest.raises(ValueError, match="share memory"):
        moe.AdamWState([flat[32:], flat[:36]])
    with pytest.raises(ValueError, match="share memory"):
        moe.AdamWState([flat, flat])
    with pytest.raises(TypeError):
        moe.AdamWState([flat, flat.to(torch.bfloat16)])
    with pytest.raises(ValueError, match="contiguous"):
        moe.AdamWState([torch.zeros(4, 8).t()])
    other = copy.deepcopy(st)
    assert other._ptrs == [p.data_ptr() for p in other.params] != st._ptrs
    assert [t.param for t in other._table] == other._ptrs and other.starts == st.starts


def test_adamw_config_is_a_plain_value():
    c = moe.AdamWConfig(lr=0.1, beta2=0.95)
    assert copy.deepcopy(c) == c and c.beta1 == 0.9
