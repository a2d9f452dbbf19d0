"""What an AdamW step rounds, and where: what many steps would add up."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import training as R
from tests import test_gpu_adamw as A

pytestmark = pytest.mark.gpu

U = A.U


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", [(A.BF, True), (A.F32, False)], ids=str)
@pytest.mark.parametrize("rate", [2e-8, 5e-8, 1e-7])
def test_a_small_decay_is_not_lost(rate, kind, bits):
    """Weights from 1 to 2 that decay by less than their rounding in a step, lr * decay of
    2e-8 to 1e-7: over elements and steps the decay has to come out in the mean.  Each step is
    compared with the oracle's from what the GPU held before.  A weight's rounding is off by at most
    2^-24, evenly spread while the update (17 units of the last place and more) is random: over
    N = 2^16 elements and 20 steps the mean of the sums deviates by 2^-24 sqrt(20 / 3) / 2^8 =
    6.0e-10; six of those, and the steps' own error of 32 U times 2e-6 each, of either sign:
    3.6e-9 + 20 * 3.8e-12.  Twice that is allowed; the decay lost is 20 * 1.5 * 2e-8 = 6e-7."""
    g = torch.Generator(device="cuda").manual_seed(7)
    n, lr = 1 << 16, 2e-6
    r = lambda: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    p = (1 + torch.rand(n, generator=g, device="cuda")).to(kind[0])
    st = moe.AdamWState([p], bits=bits, master=kind[1])
    c = moe.AdamWConfig(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=rate / lr)
    for t in (1, 2, 3):
        moe.moe_adamw_step(st, [r()], moe.AdamWConfig(lr=1e-3, beta2=0.95, weight_decay=0.0), t)
    if kind[1]:     # the masters fill the range, not bf16 values alone
        st.master.copy_(1 + torch.rand(n, generator=g, device="cuda"))
    total = np.zeros(n)
    for t in range(4, 24):
        (w, m, v), = A.held(st)
        grad = r()
        moe.moe_adamw_step(st, [grad], c, t)
        want = R.adamw(w, A.to64(grad), m, v, t, lr, c.beta1, c.beta2, c.eps, c.weight_decay)[0]
        total += A.held(st)[0][0] - want
    assert abs(total.mean()) <= 2 * (3.6e-9 + 20 * 3.8e-12)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", A.KINDS, ids=str)
@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_a_skipped_step_writes_nothing(scale, kind, bits):
    """With a scale that is not finite nothing changes, nor do 8-bit moments' scales, which a
    rounding of 448 scale / 448 would move: blocks whose largest value is not 448 (a state from
    elsewhere), and ones that end within a tensor's last block, among them."""
    sizes = [5000, 33, 256, 4096]
    st, grads, g = A.make(sizes, kind[0], A.F32, bits, kind[1])
    c = moe.AdamWConfig(lr=0.01)
    moe.moe_adamw_step(st, grads, c, 1)
    if bits == 8:
        for s in (st.exp_avg_scale, st.exp_avg_sq_scale):
            s.mul_(1 + torch.rand(s.shape, generator=g, device="cuda"))
        st.exp_avg[:256] = (st.exp_avg[:256].float() / 4).to(st.exp_avg.dtype)
    flats = [t for t in (st.master, st.exp_avg, st.exp_avg_sq, st.exp_avg_scale,
                         st.exp_avg_sq_scale, *st.params) if t is not None]
    before = [t.clone() for t in flats]
    ws = moe.Workspace()
    for t in range(2, 12):
        moe.moe_adamw_step(st, grads, c, t, grad_scale=torch.tensor(scale, device="cuda"), ws=ws)
        assert moe.moe_get_device_status(ws) == 2
    for a, b in zip(flats, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_small_roots():
    """Second moments down to the smallest subnormal, with an eps below their roots: the step
    stays that of the moments.  Their own rounding, up to 2^-150 in the product with beta2 and
    8 U of it, moves a root by what it moves v; the rest of the step is 24 U."""
    n = 1 << 14
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    v = (10.0 ** (-44.5 + 20 * u)).float()
    m = v.double().sqrt().float() * torch.randn(n, generator=g, device="cuda")
    p = torch.zeros(n, device="cuda")
    st = moe.AdamWState([p])
    st.exp_avg.copy_(m)
    st.exp_avg_sq.copy_(v)
    c = moe.AdamWConfig(lr=0.01, beta1=0.9, beta2=0.99, eps=1e-30, weight_decay=0.0)
    (_, m, v), = A.held(st)
    moe.moe_adamw_step(st, [torch.zeros(n, device="cuda")], c, 100)
    m, v, inv = c.beta1 * m, c.beta2 * v, c.lr / (1 - c.beta1 ** 100)
    error = 8 * U * v + 2.0 ** -150
    low, high = (inv * np.abs(m) / (np.sqrt(np.maximum(x, 0) / (1 - c.beta2 ** 100)) + c.eps)
                 for x in (v + error, v - error))
    got = np.abs(A.to64(p))
    assert (got >= low * (1 - 24 * U) - 1e-44).all() and (got <= high * (1 + 24 * U) + 1e-44).all()


def test_small_roots_in_8_bits():
    """The same of roots held in 8 bits: a block's largest, of v = 1e-40, decays by the root of
    beta2.  v is off by 2^-150 a product, four of them: 3e-5 of v."""
    p = [torch.zeros(256, device="cuda")]
    st = moe.AdamWState(p, bits=8)
    codes = torch.linspace(64, 448, 256, device="cuda").to(st.exp_avg_sq.dtype)
    st.exp_avg_sq.copy_(codes)
    st.exp_avg_sq_scale.fill_(1e-20 / 448)
    c = moe.AdamWConfig(lr=0.01, beta1=0.9, beta2=0.99, eps=1e-30, weight_decay=0.0)
    moe.moe_adamw_step(st, [torch.zeros(256, device="cuda")], c, 100)
    want = 1e-20 / 448 * 0.99 ** 0.5
    assert abs(float(st.exp_avg_sq_scale) / want - 1) <= 3e-5
    assert torch.equal(st.exp_avg_sq.view(torch.uint8), codes.view(torch.uint8))


@pytest.mark.parametrize("kind", A.KINDS, ids=str)
@pytest.mark.parametrize("size", [1.0, 1e-6, 1e-13, 1e6])
def test_moments_are_those_of_elementary_operations(size, kind):
    """m, v, the root, the scale and the quotient in fp32, each operation rounded to nearest and
    none fused: fp32 moments, 8-bit codes and scales are equal bit for bit.  Gradients of `size`
    down to 1e-8 of it in a block, some zero; betas and a gradient scale that round."""
    f = np.float32
    for bits in (32, 8):
        st, grads, g = A.make([1 << 17, 4099, 255], kind[0], A.F32, bits, kind[1], seed=11)
        c = moe.AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8)
        scale = torch.tensor(0.37, device="cuda")
        b1, b2, o1, o2 = f(c.beta1), f(c.beta2), f(1 - c.beta1), f(1 - c.beta2)
        for t in (1, 2, 3):
            spread = [10.0 ** (-8 * torch.rand(x.shape, generator=g, device="cuda") ** 4) for x in grads]
            grads = [size * s * torch.randn(s.shape, generator=g, device="cuda") for s in spread]
            for x in grads:
                x[torch.rand(x.shape, generator=g, device="cuda") < 0.05] = 0.0
            all_of = lambda x: x.float().cpu().numpy()  # noqa: E731
            m, v = all_of(st.exp_avg), all_of(st.exp_avg_sq)
            if bits == 8:
                m = m * np.repeat(all_of(st.exp_avg_scale), A.BLOCK)
                v = np.maximum(v, f(2.0 ** -11)) * np.repeat(all_of(st.exp_avg_sq_scale), A.BLOCK)
                v = v * v
            moe.moe_adamw_step(st, grads, c, t, grad_scale=scale)
            for i, x in enumerate(grads):
                a = st.starts[i]
                x = all_of(x) * f(0.37)
                pad = -len(x) % A.BLOCK
                x = np.concatenate([x, np.zeros(pad, f)])
                at = slice(a, a + len(x))
                m[at] = m[at] * b1 + x * o1
                v[at] = v[at] * b2 + (x * o2) * x
            assert m.dtype == v.dtype == f
            if bits == 32:
                assert np.array_equal(m, all_of(st.exp_avg)) and np.array_equal(v, all_of(st.exp_avg_sq))
                continue
            for x, flat, scales in ((m, st.exp_avg, st.exp_avg_scale),
                                    (np.sqrt(v), st.exp_avg_sq, st.exp_avg_sq_scale)):
                x = x.reshape(-1, A.BLOCK)
                unit = np.abs(x).max(axis=1) * f(1 / 448)
                assert np.array_equal(unit, all_of(scales))
                with np.errstate(divide="ignore", invalid="ignore"):
                    q = np.where(unit[:, None] > 0, x / unit[:, None], f(0))
                codes = torch.from_numpy(q.reshape(-1)).to(torch.float8_e4m3fn)
                assert torch.equal(codes.view(torch.uint8), flat.cpu().view(torch.uint8))


@pytest.mark.parametrize("kind", A.KINDS, ids=str)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_weights_stay_infinite(decay, bits, kind):
    """A weight held at -inf, as a mask is, is no less by a step; its neighbours step as ever, and
    the status is clean."""
    sizes = [700, 300]
    sets = [A.make(sizes, kind[0], A.F32, bits, kind[1]) for _ in range(2)]
    c = moe.AdamWConfig(lr=0.01, weight_decay=decay)
    at = [(0, 3, float("inf")), (0, 699, -float("inf")), (1, 100, -float("inf"))]
    (st, grads, _), (ref, same, _) = sets
    for i, j, v in at:
        st.params[i][j] = v
        if kind[1]:
            st.of(st.master, i)[j] = v
    ws = moe.Workspace()
    for t in (1, 2, 3):
        moe.moe_adamw_step(st, grads, c, t, ws=ws)
        assert moe.moe_get_device_status(ws) == 0
        moe.moe_adamw_step(ref, same, c, t)
    for i, j, v in at:
        assert float(st.params[i][j]) == v
        ref.params[i][j] = v
    assert all(torch.equal(a, b) for a, b in zip(st.params, ref.params))
    assert torch.equal(st.exp_avg.view(torch.uint8), ref.exp_avg.view(torch.uint8))
