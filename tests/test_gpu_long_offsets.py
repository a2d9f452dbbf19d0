"""Batches whose tensors hold more than 2^32 elements: the last tokens against
the same tokens in a call of their own and against the oracle."""
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import adapter as P
from tests.test_gpu_adapter import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_route():
    T, E, k = 4_200_003, 1024, 8
    cfg = moe.RouteConfig("softmax", 8, 4, 2, False, 1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.empty(T, E, device="cuda")
    l[:4] = torch.randn(4, E, generator=g, device="cuda")
    l[4:].copy_(l[3])
    l[T - 500:] = torch.randn(500, E, generator=g, device="cuda")
    assert l.numel() > 1 << 32
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(l, k, cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    tail = l[T - 500:].clone()
    want = moe.moe_route_scored(tail, k, cfg)
    assert torch.equal(idx[T - 500:], want[0])
    torch.testing.assert_close(w[T - 500:], want[1], rtol=2.0 ** -20, atol=0)
    assert (idx[4:T - 500] == idx[3]).all()
    dw = torch.ones(T, k, device="cuda")
    dw[T - 500:] = torch.randn(500, k, generator=g, device="cuda")
    d = moe.moe_route_scored_backward(dw, idx, l, cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    part = moe.moe_route_scored_backward(dw[T - 500:].clone(), want[0], tail, cfg)
    assert torch.equal(d[T - 500:], part)
    assert torch.equal(d[T - 501], d[3])


@pytest.mark.parametrize("H,N", [(128, 16384), (16384, 128)])
def test_adapters(H, N):
    T, n, R = 300_000, 5, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x, dy = torch.zeros(T, H, dtype=bf, device="cuda"), torch.zeros(T, N, dtype=bf, device="cuda")
    assert max(x.numel(), dy.numel()) > 1 << 32
    idx = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    own = torch.cat([torch.arange(0, 70), torch.arange(T - 300, T)])
    at = own.cuda()
    x[at], dy[at] = r(len(own), H).to(bf), r(len(own), N).to(bf)
    idx[at] = torch.randint(-1, n, (len(own),), generator=g, device="cuda").to(torch.int32)
    W = (r(H, N) / H ** 0.5).to(bf)
    A, B = (r(n, R, H) / H ** 0.5).to(bf), (r(n, R, N) / R ** 0.5).to(bf)
    s = r(n)
    ws = moe.Workspace()
    y = moe.moe_adapter_project(x, W, A, B, s, idx, ws=ws)
    dx, dA, dB = moe.moe_adapter_project_backward(dy, x, W, A, B, s, idx, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    few = [t.cpu() for t in (x[at], W, A, B, s, idx[at])]
    ref, mag = P.project(*few, magnitudes=True)
    assert_close(y[at], ref, mag, "y")
    assert (y[70:T - 300] == 0).all() and (dx[70:T - 300] == 0).all()
    ref, mag = P.backward(dy[at].cpu(), *few, magnitudes=True)
    for key, got in (("dx", dx[at]), ("dA", dA), ("dB", dB)):
        assert_close(got, ref[key], mag[key], key)


def test_route_the_most_tokens_that_are_accepted():
    T = 2 ** 31 - 1                    # T * k < 2^31
    l = torch.randn(1, device="cuda").expand(T).reshape(T, 1).contiguous()
    l[-1, 0], l[-2, 0] = 0.5, -1.5
    cfg = moe.RouteConfig("sigmoid", renormalize=False)
    ws = moe.Workspace()
    idx, w = moe.moe_route_scored(l, 1, cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    want = torch.sigmoid(l[[0, 5, T // 2, T - 2, T - 1], 0].double())
    rows = torch.tensor([0, 5, T // 2, T - 2, T - 1], device="cuda")
    torch.testing.assert_close(w[rows, 0].double(), want, rtol=2.0 ** -20, atol=0)
    assert int(idx.max()) == 0 and int(idx.min()) == 0 and torch.equal(w[3], w[T - 3])
    d = moe.moe_route_scored_backward(torch.ones_like(w), idx, l, cfg, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    torch.testing.assert_close(d[rows, 0].double(), want * (1 - want), rtol=2.0 ** -18, atol=0)
