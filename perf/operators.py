"""Measured cases of the scored router and of the adapter projection.

Four operators of an expert layer that is trained and served with many
fine-tuned variants at once:

  route             logits [T, E] -> (topk_idx, topk_w): softmax or sigmoid
                    scores, a balance bias that steers the choice only, groups
                    of experts, the k best, renormalised weights;
  route_backward    the gradient of topk_w with respect to the logits;
  adapter           y = x W + s_a (x A_a^T) B_a: one projection W shared by all
                    tokens and a low-rank adapter a of each token's request;
  adapter_backward  dx, dA and dB of the same (W is frozen).

`run` computes them in plain torch operations in fp32, rounded once at the
end, or, where `own` is true, by the library's calls.  `exact` is the
definition in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def _route(name, op, T, E, k, score, bias, groups, keep, group_top, renorm, scale):
    c = dict(op=op, T=T, E=E, k=k, score=score, bias=bias, groups=groups, keep=keep,
             group_top=group_top, renorm=renorm, scale=scale)
    return dict(c, name=name) if name else c


def _adapter(name, op, T, H, N, n, R, order):
    c = dict(op=op, T=T, H=H, N=N, n=n, R=R, order=order)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a chat being decoded: pure latency
        _route("route_token", "route", 1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # a decode batch on a layer of few experts
        _route("route_decode_E8", "route", 128, 8, 2, "softmax", False, 1, 1, 1, True, 1.0),
        # the fine-grained layer's batch: sigmoid scores, balance bias, 4 of 8 groups
        _route("route_fine_grained", "route", 8192, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # a long training batch, an odd token count and a group size that is no power
        # of two, scores not renormalised
        _route("route_long_odd", "route", 40001, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
        # the training step of the fine-grained layer
        _route("route_bwd_fine_grained", "route_backward", 8192, 256, 8, "sigmoid", True, 8, 4, 2,
               True, 2.5),
        # scores not renormalised: every expert's logit has a gradient
        _route("route_bwd_dense", "route_backward", 40001, 64, 6, "softmax", False, 1, 1, 1,
               False, 1.0),
        # one token of one request through a small projection: pure latency
        _adapter("adapter_token", "adapter", 1, 512, 1024, 4, 8, "shuffled"),
        # a decode batch, each token from some request, up-projection of the decode layer
        _adapter("adapter_decode", "adapter", 128, 6144, 16384, 32, 16, "shuffled"),
        # an odd batch of decode tokens in any order, wide ranks, fine-grained shape
        _adapter("adapter_mixed", "adapter", 777, 7168, 2048, 24, 64, "shuffled"),
        # a prefill chunk of whole requests
        _adapter("adapter_prefill", "adapter", 4096, 6144, 10752, 16, 16, "segments"),
        # fine-tuning a few adapters at once, short odd batch
        _adapter("adapter_bwd_short", "adapter_backward", 301, 2048, 1024, 3, 8, "segments"),
        # fine-tuning adapters of the fine-grained layer's projection
        _adapter("adapter_bwd_long", "adapter_backward", 8192, 7168, 2048, 8, 16, "segments"),
    ]


_MOST = 4096 * 6144 * 10752          # multiply-adds of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "adapter", "adapter_backward"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        per = max(2, _log(rng, 8, 512) // groups)
        E = groups * per
        T = _log(rng, 1, 40001)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(8, keep * per))
        return _route(None, op, T, E, k, rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, keep, rng.choice([1, 2]),
                      rng.random() < 0.7, rng.choice([1.0, 2.5]))
    H, N = 128 * _log(rng, 2, 64), 128 * _log(rng, 2, 84)
    n, R = _log(rng, 1, 32), rng.choice([8, 16, 24, 32, 64, 128])
    # the plain form multiplies every token by every adapter: that counts too
    most = _MOST // (H * N + n * R * (H + N)) // (3 if op == "adapter_backward" else 1)
    T = min(_log(rng, 1, 8192), max(1, most))
    return _adapter(None, op, T, H, N, n, R, rng.choice(["shuffled", "segments"]))


def work(case):
    """Bytes: each input read once, each output written once.  A shuffled batch
    of T tokens meets n (1 - (1 - 0.9 / n)^T) of the n adapters on average."""
    c, T = case, case["T"]
    if c["op"] == "route":
        return dict(bytes=T * c["E"] * 4 + T * c["k"] * 8 + c["E"] * 4 * c["bias"],
                    flops=6 * T * c["E"])
    if c["op"] == "route_backward":
        dense = c["score"] == "softmax" and not c["renorm"]
        read = T * c["k"] * 8 + T * (c["E"] if dense else c["k"]) * 4
        return dict(bytes=read + T * c["E"] * 4, flops=6 * T * (c["E"] if dense else c["k"]))
    H, N, n, R = c["H"], c["N"], c["n"], c["R"]
    met = n * (1 - (1 - 0.9 / n) ** T)
    flops = 2 * T * H * N + 0.9 * 2 * T * R * (H + N)
    data = 2 * (T * H + H * N + T * N + met * R * (H + N)) + 4 * T
    if c["op"] == "adapter":
        return dict(bytes=data, flops=flops)
    # x, dy, W, A, B read; dx, dA, dB written; x A, dy B, their products, dA, dB
    return dict(bytes=data + 2 * (T * H + n * R * (H + N)), flops=flops + 0.9 * 4 * T * R * (H + N))


# ----------------------------------------------------------------- the inputs
def _normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _adapter_idx(case, g):
    """int32 [T]: every token's adapter, -1 (no adapter) for one request in ten.
    "shuffled": each token of a request of its own; "segments": whole requests
    of ragged lengths one after the other."""
    T, n = case["T"], case["n"]
    if case["order"] == "shuffled":
        of = torch.randint(0, n, (T,), generator=g, device="cuda")
        none = torch.rand(T, generator=g, device="cuda") < 0.1
        return torch.where(none, -1, of).to(torch.int32)
    requests = max(1, min(T, 2 * n))
    cuts = torch.randint(0, T, (requests,), generator=g, device="cuda")
    request = (cuts[None, :] <= torch.arange(T, device="cuda")[:, None]).sum(1)
    of = torch.randint(0, n, (requests + 1,), generator=g, device="cuda")
    none = torch.rand(requests + 1, generator=g, device="cuda") < 0.1
    return torch.where(none, -1, of)[request].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, T = case, case["T"]
    s = dict(case=dict(case))
    if c["op"].startswith("route"):
        s["logits"] = _normal((T, c["E"]), 1.0, g)
        # the balance bias of a router in training: small beside the scores' spread
        s["bias"] = _normal((c["E"],), 0.02, g) if c["bias"] else None
        if c["op"] == "route_backward":
            s["topk_idx"] = _plain_route(c, s["logits"], s["bias"])[0]
            s["dtopk_w"] = _normal((T, c["k"]), 1.0, g)
        if own:
            import routing_grouped_expert_gb300 as moe
            s["config"] = moe.RouteConfig(score=c["score"], n_group=c["groups"],
                                          topk_group=c["keep"], group_top=c["group_top"],
                                          renormalize=c["renorm"], scale=c["scale"])
            s["ws"] = moe.Workspace()
        return s
    H, N, n, R = c["H"], c["N"], c["n"], c["R"]
    bf = torch.bfloat16
    s["x"] = _normal((T, H), 1.0, g, bf)
    s["W"] = _normal((H, N), 1 / math.sqrt(H), g, bf)
    s["A"] = _normal((n, R, H), 1 / math.sqrt(H), g, bf)
    s["B"] = _normal((n, R, N), 0.5 / math.sqrt(R), g, bf)
    s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    s["adapter_idx"] = _adapter_idx(c, g)
    if c["op"] == "adapter_backward":
        s["dy"] = _normal((T, N), 1.0, g, bf)
    if own:
        import routing_grouped_expert_gb300 as moe
        s["ws"] = moe.Workspace()
    return s


# ------------------------------------------------------------- the plain forms
def _scores(c, logits):
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    # the sum is rounded once: the scores do not depend on its order
    return e / e.double().sum(dim=1, keepdim=True).float()


def _plain_route(c, logits, bias):
    """Choice by score + bias (by the logit itself where there is no bias: the
    score rises with it); equal values go to the lower index."""
    T, E, groups = c["T"], c["E"], c["groups"]
    s = _scores(c, logits)
    biased = s if bias is None else s + bias
    rank = logits if bias is None else biased
    if groups > 1:
        per = (biased if c["group_top"] == 2 else rank).view(T, groups, E // groups)
        best = torch.sort(per, dim=2, descending=True).values
        group = best[:, :, 0] + best[:, :, 1] if c["group_top"] == 2 else best[:, :, 0]
        order = torch.sort(group, dim=1, descending=True, stable=True).indices
        kept = torch.zeros(T, groups, dtype=torch.bool, device=logits.device)
        kept.scatter_(1, order[:, :c["keep"]], True)
        kept = kept[:, :, None].expand(T, groups, E // groups).reshape(T, E)
        rank = torch.where(kept, rank, -math.inf)
    idx = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(s, 1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), w * c["scale"]


def _plain_route_backward(c, logits, idx, dw):
    """w_j = scale s_j / (sum of the chosen s, or 1); s' = s (1 - s) for the
    sigmoid, the softmax Jacobian over all experts for the softmax."""
    idx = idx.long()
    s = _scores(c, logits)
    sel = torch.gather(s, 1, idx)
    dw = dw * c["scale"]
    if c["renorm"]:
        total = sel.sum(dim=1, keepdim=True)
        dw = (dw - (dw * sel).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dw)
    if c["score"] == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(dim=1, keepdim=True))


def _mask(idx, n, scale):
    """[T, n]: the token's adapter scale at its adapter, zero elsewhere."""
    own_one = idx.long()[:, None] == torch.arange(n, device=idx.device)
    return own_one * scale


def _low(x, A, mask):
    """[T, n R]: s_a (x A_a^T) at each token's own adapter, zero elsewhere."""
    n, R, H = A.shape
    z = (x @ A.reshape(n * R, H).t()).view(x.shape[0], n, R)
    return (z * mask[:, :, None]).reshape(x.shape[0], n * R)


def _plain_adapter(s):
    x, W, A, B = (s[k].float() for k in ("x", "W", "A", "B"))
    n, R, N = B.shape
    z = _low(x, A, _mask(s["adapter_idx"], n, s["scale"]))
    return (x @ W + z @ B.reshape(n * R, N)).to(torch.bfloat16)


def _plain_adapter_backward(s):
    x, W, A, B, dy = (s[k].float() for k in ("x", "W", "A", "B", "dy"))
    n, R, H = A.shape
    mask = _mask(s["adapter_idx"], n, s["scale"])
    z, dz = _low(x, A, mask), _low(dy, B, mask)
    dx = dy @ W.t() + dz @ A.reshape(n * R, H)
    dA, dB = (dz.t() @ x).view_as(A), (z.t() @ dy).view_as(B)
    return tuple(t.to(torch.bfloat16) for t in (dx, dA, dB))


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        import routing_grouped_expert_gb300 as moe
        if c["op"] == "route":
            return moe.moe_route_scored(s["logits"], c["k"], s["config"], bias=s["bias"],
                                        ws=s["ws"])
        if c["op"] == "route_backward":
            return moe.moe_route_scored_backward(s["dtopk_w"], s["topk_idx"], s["logits"],
                                                 s["config"], bias=s["bias"], ws=s["ws"])
        if c["op"] == "adapter":
            return moe.moe_adapter_project(s["x"], s["W"], s["A"], s["B"], s["scale"],
                                           s["adapter_idx"], ws=s["ws"])
        return moe.moe_adapter_project_backward(s["dy"], s["x"], s["W"], s["A"], s["B"],
                                                s["scale"], s["adapter_idx"], ws=s["ws"])
    if c["op"] == "route":
        return _plain_route(c, s["logits"], s["bias"])
    if c["op"] == "route_backward":
        return _plain_route_backward(c, s["logits"], s["topk_idx"], s["dtopk_w"])
    return _plain_adapter(s) if c["op"] == "adapter" else _plain_adapter_backward(s)


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("route"):
        l = s["logits"].double()
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
        if c["op"] == "route":
            v = p if s["bias"] is None else p + s["bias"].double()
            if c["groups"] > 1:
                g = v.view(c["T"], c["groups"], -1).topk(c["group_top"], dim=2).values.sum(2)
                drop = g.argsort(dim=1, descending=True, stable=True)[:, c["keep"]:]
                v = v.view(c["T"], c["groups"], -1).scatter(
                    1, drop[:, :, None].expand(-1, -1, c["E"] // c["groups"]), -math.inf)
                v = v.reshape(c["T"], c["E"])
            idx = v.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
            w = p.gather(1, idx)
            w = w / w.sum(1, keepdim=True) if c["renorm"] else w
            return None, w * c["scale"]
        # dL/dlogits of L = <dw, w>, by automatic differentiation of the definition
        l.requires_grad_(True)
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
        w = p.gather(1, s["topk_idx"].long())
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        return torch.autograd.grad((w * c["scale"] * s["dtopk_w"].double()).sum(), l)[0]
    x, W, A, B = (s[k].double() for k in ("x", "W", "A", "B"))
    forward = c["op"] == "adapter"
    out = x @ W if forward else s["dy"].double() @ W.t()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(c["n"]):
        t = (s["adapter_idx"] == a).nonzero()[:, 0]
        f = s["scale"][a].double()
        if forward:
            out[t] += f * (x[t] @ A[a].t()) @ B[a]
        else:
            dy = s["dy"][t].double()
            dz = f * (dy @ B[a].t())
            out[t] += dz @ A[a]
            dA[a] = dz.t() @ x[t]
            dB[a] = f * (x[t] @ A[a].t()).t() @ dy
    return out if forward else (out, dA, dB)
