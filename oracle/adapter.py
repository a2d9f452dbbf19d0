"""CPU oracle of the adapter projection and its gradients -- TEST
INFRASTRUCTURE.  The definition in fp64, adapter by adapter, sharing no code
with the library:

    y[t]  = x[t] W + s_a (x[t] A_a^T) B_a,  a = adapter_idx[t]; y[t] = x[t] W for a = -1
    dx[t] = dy[t] W^T + dz[t] A_a,  dz[t] = s_a (dy[t] B_a^T)
    dA_a  = sum_t dz[t]^T x[t],     dB_a = sum_t (s_a x[t] A_a^T)^T dy[t]

`magnitudes=True` also returns, per result, the sums of absolute values that
bound what rounding does: "low" follows the rounding of z (or dz), the one
stored intermediate, and "sum" the fp32 accumulation of every product.
"""
from __future__ import annotations

import torch


def _f64(t):
    return t.detach().to("cpu", torch.float64)


def _low(x, A, scale, idx, magnitude=False):
    """z [T, R]: s_a x A_a^T of each token's own adapter, zero without one."""
    z = x.new_zeros(x.shape[0], A.shape[1])
    for a in range(A.shape[0]):
        t = (idx == a).nonzero()[:, 0]
        z[t] = scale[a] * (x[t].abs() @ A[a].abs().t() if magnitude else x[t] @ A[a].t())
    return z


def _up(z, B, idx):
    out = z.new_zeros(z.shape[0], B.shape[2])
    for a in range(B.shape[0]):
        t = (idx == a).nonzero()[:, 0]
        out[t] = z[t] @ B[a]
    return out


def _outer(z, v, n, idx):
    """[n, R, D]: the adapters' sums of z[t]^T v[t]."""
    out = z.new_zeros(n, z.shape[1], v.shape[1])
    for a in range(n):
        t = (idx == a).nonzero()[:, 0]
        out[a] = z[t].t() @ v[t]
    return out


def project(x, W, A, B, scale, idx, magnitudes=False):
    x, W, A, B, scale = (_f64(t) for t in (x, W, A, B, scale))
    idx = idx.cpu()
    z = _low(x, A, scale, idx)
    y = x @ W + _up(z, B, idx)
    if not magnitudes:
        return y
    zm = _low(x, A, scale.abs(), idx, True)
    return y, dict(low=_up(z.abs(), B.abs(), idx),
                   sum=x.abs() @ W.abs() + _up(zm, B.abs(), idx))


def backward(dy, x, W, A, B, scale, idx, magnitudes=False):
    dy, x, W, A, B, scale = (_f64(t) for t in (dy, x, W, A, B, scale))
    idx = idx.cpu()
    n = A.shape[0]
    dx = project(dy, W.t(), B, A, scale, idx)
    z, dz = _low(x, A, scale, idx), _low(dy, B, scale, idx)
    g = dict(dx=dx, dA=_outer(dz, x, n, idx), dB=_outer(z, dy, n, idx))
    if not magnitudes:
        return g
    zm, dzm = _low(x, A, scale.abs(), idx, True), _low(dy, B, scale.abs(), idx, True)
    mags = dict(dx=project(dy, W.t(), B, A, scale, idx, True)[1],
                dA=dict(low=_outer(dz.abs(), x.abs(), n, idx), sum=_outer(dzm, x.abs(), n, idx)),
                dB=dict(low=_outer(z.abs(), dy.abs(), n, idx), sum=_outer(zm, dy.abs(), n, idx)))
    return g, mags
