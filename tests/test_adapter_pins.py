"""The adapter oracle against plain loops, automatic differentiation and
differences, and the entry points' refusals (nothing here needs a GPU)."""
import ctypes

import torch

from oracle import adapter as P
from routing_grouped_expert_gb300 import binding


def small(T=9, H=5, N=4, n=3, R=2, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    idx = torch.tensor([0, 2, -1, 2, 0, -1, 2, 2, 0], dtype=torch.int32)[:T]
    return r(T, H), r(H, N), r(n, R, H), r(n, R, N), r(n), idx, r(T, N)


def test_projection_is_the_loop():
    x, W, A, B, s, idx, _ = small()
    y = P.project(x, W, A, B, s, idx)
    for t in range(9):
        for c in range(4):
            want = sum(float(x[t, h]) * float(W[h, c]) for h in range(5))
            a = int(idx[t])
            if a >= 0:
                for r in range(2):
                    z = sum(float(x[t, h]) * float(A[a, r, h]) for h in range(5))
                    want += float(s[a]) * z * float(B[a, r, c])
            assert abs(float(y[t, c]) - want) < 1e-12


def test_gradients_are_autograd_and_differences():
    x, W, A, B, s, idx, dy = small()
    leaves = [v.clone().requires_grad_(True) for v in (x, A, B)]
    z = torch.stack([s[a] * leaves[1][a] @ leaves[0][t] if a >= 0 else x.new_zeros(2)
                     for t, a in enumerate(idx.tolist())])
    up = torch.stack([z[t] @ leaves[2][a] if a >= 0 else x.new_zeros(4)
                      for t, a in enumerate(idx.tolist())])
    grads = torch.autograd.grad(((leaves[0] @ W + up) * dy).sum(), leaves)
    g = P.backward(dy, x, W, A, B, s, idx)
    for want, key in zip(grads, ("dx", "dA", "dB")):
        torch.testing.assert_close(g[key], want, rtol=0, atol=1e-12)
    assert (g["dA"][1] == 0).all() and (g["dB"][1] == 0).all()   # an adapter without a token
    h = 1e-6
    for which, key in ((0, "dx"), (1, "dA"), (2, "dB")):
        args = [x, A, B]
        flat = args[which].reshape(-1)
        for i in range(flat.numel()):
            f = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign * h
                v = list(args)
                v[which] = moved.view_as(args[which])
                f.append(float((P.project(v[0], W, v[1], v[2], s, idx) * dy).sum()))
            # y is at most quadratic in the three: central differences are exact
            # but for cancellation, 2^-53 |f| / h
            assert abs((f[0] - f[1]) / (2 * h) - float(g[key].reshape(-1)[i])) < 1e-7


def test_refusals():
    lib = binding.load_library()
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4100)    # never dereferenced
    big = 1 << 40
    INVALID, WS, OK = 1, 4, 0
    ws = lib.moe_adapter_workspace_size
    wsb = lib.moe_adapter_workspace_size_backward
    assert 0 < ws(16, 512, 1024, 4, 16) < wsb(16, 512, 1024, 4, 16)
    assert ws(0, 512, 1024, 4, 16) > 0
    for bad in ((-1, 512, 1024, 4, 16), (16, 500, 1024, 4, 16), (16, 512, 1000, 4, 16),
                (16, 0, 1024, 4, 16), (16, 512, 1024, 0, 16), (16, 512, 1024, 1025, 16),
                (16, 512, 1024, 4, 0), (16, 512, 1024, 4, 12), (16, 512, 1024, 4, 136),
                (1 << 30, 512, 1024, 4, 16)):
        assert ws(*bad) == 0 and wsb(*bad) == 0
        assert lib.moe_adapter_project(p, p, p, p, p, p, *bad, p, p, big, None) == INVALID
        assert lib.moe_adapter_project_backward(p, p, p, p, p, p, p, *bad, p, p, p, p, big,
                                                None) == INVALID
    size = (16, 512, 1024, 4, 16)
    for i in range(7):
        for q in (None, odd):
            a = [p] * 7
            a[i] = q
            assert lib.moe_adapter_project(*a[:6], *size, a[6], p, big, None) == INVALID
    for i in range(10):
        a = [p] * 10
        a[i] = None
        assert lib.moe_adapter_project_backward(*a[:7], *size, *a[7:], p, big, None) == INVALID
    need = ws(*size)
    assert lib.moe_adapter_project(*[p] * 6, *size, p, p, need - 1, None) == WS
    assert lib.moe_adapter_project(*[p] * 6, *size, p, None, need, None) == WS
    assert lib.moe_adapter_project(*[p] * 6, *size, p, ctypes.c_void_p(4096 + 16), need,
                                   None) == WS
    assert lib.moe_adapter_project_backward(*[p] * 7, *size, p, p, p, p, need, None) == WS
    assert lib.moe_adapter_project(None, p, p, p, p, None, 0, 512, 1024, 4, 16, None, None, 0,
                                   None) == OK
