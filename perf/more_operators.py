"""Measured cases of what a training step runs around the expert layer.

  norm, norm_backward        layer norm of h = x + residual, ahead of the router and the
                             experts; dx (with the residual branch's gradient added),
                             dweight and dbias;
  balance, balance_backward  the loss that keeps the experts' loads even, per sequence,
                             with the per-expert counts; its gradient in the logits,
                             by itself or added onto the layer's;
  adamw                      one optimizer step over many tensors, both moments in fp32
                             or in 8 bits, with or without fp32 master weights.

`run` computes them in plain torch operations in fp32, rounded once at the
end, or, where `own` is true, by the library's calls.  `exact` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ the cases
def _norm(name, op, T, H, dtype, wtype, bias, residual):
    c = dict(op=op, T=T, H=H, dtype=dtype, wtype=wtype, bias=bias, residual=residual)
    return dict(c, name=name) if name else c


def _balance(name, op, T, E, k, score, S, onto):
    """S sequences of ragged lengths, with masked tokens and rows behind the last
    sequence; S = 0: the whole batch counts as one.  onto: added onto dlogits."""
    c = dict(op=op, T=T, E=E, k=k, score=score, S=S, onto=onto)
    return dict(c, name=name) if name else c


def _adamw(name, bits, master, dtype, gtype, count, most, mix, E=0, H=0, F=0):
    """`count` tensors of ragged lengths up to `most`, drawn by `mix`; or, with E,
    the weights [E, H, F], [E, H, F], [E, F, H] of E experts."""
    c = dict(op="adamw", bits=bits, master=master, dtype=dtype, gtype=gtype, count=count,
             most=most, mix=mix, E=E, H=H, F=F)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a chat being decoded: pure latency
        _norm("norm_token", "norm", 1, 7168, "bf16", "bf16", False, True),
        # the fine-grained layer's batch, with the residual add
        _norm("norm_fine_grained", "norm", 8192, 7168, "bf16", "bf16", True, True),
        # a short odd batch of an odd width in fp32
        _norm("norm_bwd_odd", "norm_backward", 1237, 1001, "fp32", "fp32", True, False),
        # the training step of the fine-grained layer
        _norm("norm_bwd_fine_grained", "norm_backward", 8192, 7168, "bf16", "bf16", True, True),
        # a short odd batch on few experts: pure latency
        _balance("balance_short", "balance", 301, 8, 2, "softmax", 0, False),
        # a long batch of packed sequences on fine-grained experts, masked tokens, padding
        _balance("balance_sequences", "balance", 40001, 256, 8, "sigmoid", 24, False),
        # the gradient of one batch's loss by itself
        _balance("balance_bwd", "balance_backward", 8192, 64, 6, "softmax", 0, False),
        # the packed batch's gradient, added onto the layer's own dlogits
        _balance("balance_bwd_sequences", "balance_backward", 40001, 256, 8, "sigmoid", 24, True),
        # norms, routers and adapters of a model: many small ragged tensors
        _adamw("adamw_ragged", 32, True, "bf16", "bf16", 150, 2000000, 1),
        # sixteen experts of the fine-grained layer
        _adamw("adamw_experts", 32, True, "bf16", "bf16", 0, 0, 0, 16, 7168, 2048),
        # the ragged tensors with 8-bit moments and fp32 gradients
        _adamw("adamw8_ragged", 8, False, "bf16", "fp32", 150, 2000000, 2),
        # sixteen experts with 8-bit moments
        _adamw("adamw8_experts", 8, False, "bf16", "bf16", 0, 0, 0, 16, 7168, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "balance", "balance_backward", "adamw", "adamw"])
    if op.startswith("norm"):
        H = _log(rng, 8, 16384)
        if rng.random() < 0.5:
            H = max(8, H // 8 * 8)
        T = min(_log(rng, 1, 40001), 8192 * 7168 // H)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        wtype = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
        return _norm(None, op, T, H, dtype, wtype, rng.random() < 0.7, rng.random() < 0.7)
    if op.startswith("balance"):
        E, T = _log(rng, 2, 512), _log(rng, 1, 40001)
        return _balance(None, op, T, E, rng.randint(1, min(8, E)),
                        rng.choice(["softmax", "sigmoid"]),
                        rng.choice([0, 0, 1, 2, 7, 24, 64]) if T > 64 else 0,
                        op == "balance_backward" and rng.random() < 0.5)
    bits = rng.choice([32, 8])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    master = dtype == "bf16" and rng.random() < 0.5
    gtype = rng.choice(["bf16", "fp32"])
    if rng.random() < 0.3:
        return _adamw(None, bits, master, dtype, gtype, 0, 0, 0, rng.randint(1, 8),
                      128 * _log(rng, 1, 56), 128 * _log(rng, 1, 16))
    return _adamw(None, bits, master, dtype, gtype, _log(rng, 1, 200), _log(rng, 2, 2000000),
                  rng.randint(3, 1 << 20))


_BYTES = {"bf16": 2, "fp32": 4}
_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BLOCK = 256     # elements that share one scale of an 8-bit moment; tensors start on one
_ALPHA = 1e-2    # the balance loss's factor


def _sizes(c):
    if c["E"]:
        return [c["E"] * c["H"] * c["F"]] * 3
    r = random.Random(c["mix"])
    return [int(math.exp(r.uniform(0.0, math.log(c["most"])))) | 1 for _ in range(c["count"])]


def work(case):
    """Bytes: each input read once, each output written once."""
    c = case
    if c["op"].startswith("norm"):
        n, b, w = c["T"] * c["H"], _BYTES[c["dtype"]], c["H"] * _BYTES[c["wtype"]] * (1 + c["bias"])
        if c["op"] == "norm":   # x, y (and residual, h), the statistics, the weights
            return dict(bytes=n * b * (4 if c["residual"] else 2) + 8 * c["T"] + w, flops=9 * n)
        # dy, h, dx (and dh), the statistics, the weight, dweight and dbias
        return dict(bytes=n * b * (4 if c["residual"] else 3) + 8 * c["T"] +
                    c["H"] * _BYTES[c["wtype"]] + w, flops=16 * n)
    if c["op"].startswith("balance"):
        T, E, S = c["T"], c["E"], max(1, c["S"])
        if c["op"] == "balance":
            return dict(bytes=4 * T * E + 4 * T * c["k"] + 4 * S * E + (T if c["S"] else 0),
                        flops=6 * T * E)
        return dict(bytes=4 * T * E * (3 if c["onto"] else 2) + 4 * S * E + (T if c["S"] else 0),
                    flops=10 * T * E)
    n = sum(_sizes(c))
    per = _BYTES[c["gtype"]] + (8 + _BYTES[c["dtype"]] if c["master"] else 2 * _BYTES[c["dtype"]])
    per += 16 if c["bits"] == 32 else 4 + 16 / _BLOCK
    return dict(bytes=n * per, flops=16 * n)


# ----------------------------------------------------------------- the inputs
def _normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _prepare_norm(s, c, g):
    T, H, dt, wt = c["T"], c["H"], _TYPE[c["dtype"]], _TYPE[c["wtype"]]
    s["weight"] = 1 + _normal((H,), 0.1, g)
    s["weight"] = s["weight"].to(wt)
    s["bias"] = _normal((H,), 0.1, g, wt) if c["bias"] else None
    if c["op"] == "norm":
        s["x"] = _normal((T, H), 1.0, g, dt)
        # the residual stream: larger than what a block adds, and off zero
        s["residual"] = (3 * torch.randn(T, H, generator=g, device="cuda") + 0.5).to(dt) \
            if c["residual"] else None
        return
    s["h"] = (3 * torch.randn(T, H, generator=g, device="cuda") + 0.5).to(dt)
    h = s["h"].double()
    mean = h.mean(dim=1)
    rstd = ((h - mean[:, None]).square().mean(dim=1) + 1e-5).rsqrt()
    s["stats"] = torch.stack([mean, rstd], dim=1).float()
    s["dy"] = _normal((T, H), 1.0, g, dt)
    s["dh"] = _normal((T, H), 1.0, g, dt) if c["residual"] else None


def _prepare_balance(s, c, g):
    T, E, S = c["T"], c["E"], c["S"]
    # a router in training: some experts are liked more than others
    s["logits"] = _normal((T, E), 1.0, g) + _normal((1, E), 0.3, g)
    s["topk_idx"] = torch.topk(s["logits"], c["k"], dim=1).indices.to(torch.int32)
    s["seq_offsets"] = s["mask"] = None
    if S:
        # ragged sequences, empty ones among them, and rows behind the last one
        cuts = torch.randint(0, T - T // 50, (S,), generator=g, device="cuda").sort().values
        s["seq_offsets"] = torch.cat([torch.zeros(1, device="cuda"), cuts[1:],
                                      torch.tensor([T - T // 50], device="cuda")]).to(torch.int32)
        s["mask"] = torch.rand(T, generator=g, device="cuda") > 0.05
    if c["op"] == "balance_backward":
        _, s["counts"], s["tokens"] = _plain_balance(s)
        s["dloss"] = torch.ones((), device="cuda")
        if c["onto"]:
            s["dlogits"] = _normal((T, E), _ALPHA / T, g)


def _quantised(x):
    """(values in e4m3, one scale per block) of a flat fp32 tensor."""
    x = x.view(-1, _BLOCK)
    scale = x.abs().amax(dim=1) / 448.0
    q = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0)
    return q.to(torch.float8_e4m3fn).view(-1), scale


def _prepare_adamw(s, c, g):
    sizes = _sizes(c)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // _BLOCK) * _BLOCK
    flat = {name: torch.zeros(at, device="cuda") for name in ("p", "g", "m", "v")}
    for i, (o, n) in enumerate(zip(starts, sizes)):
        size = 10.0 ** (-2 - 3 * ((i * 7) % 10) / 10)   # each tensor's gradients have a size of their own
        flat["p"][o:o + n].normal_(0, 0.02, generator=g)
        flat["g"][o:o + n].normal_(0, size, generator=g)
        flat["m"][o:o + n].normal_(0, 0.3 * size, generator=g)
        flat["v"][o:o + n].uniform_(0.2, 1.8, generator=g).mul_(size * size)
    s["t"] = 10
    s["master"] = flat["p"] if c["master"] else None
    s["p"] = flat["p"].to(_TYPE[c["dtype"]]).clone()
    s["g"] = flat["g"].to(_TYPE[c["gtype"]])
    if c["bits"] == 32:
        s["m"], s["v"] = flat["m"], flat["v"]
    else:
        s["m"], s["m_scale"] = _quantised(flat["m"])
        s["v"], s["v_scale"] = _quantised(flat["v"].sqrt())
    if own:
        import routing_grouped_expert_gb300 as moe
        # the tensors as a model has them: one after the other in a larger buffer
        shapes = [(c["E"], c["H"], c["F"])] * 2 + [(c["E"], c["F"], c["H"])] if c["E"] else \
            [(n,) for n in sizes]
        view = lambda f: [f[o:o + n].view(z) for o, n, z in zip(starts, sizes, shapes)]  # noqa: E731
        s["state"] = st = moe.AdamWState(view(s["p"]), bits=c["bits"], master=c["master"])
        # the moments of the steps before, as from a checkpoint
        for name, to in (("m", st.exp_avg), ("v", st.exp_avg_sq), ("m_scale", st.exp_avg_scale),
                         ("v_scale", st.exp_avg_sq_scale), ("master", st.master)):
            if to is not None:
                to.copy_(s[name])
                s[name] = to
        s["grads"] = view(s["g"])
        s["config"] = moe.AdamWConfig(*_HYPER)
        s["ws"] = moe.Workspace()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    (_prepare_norm if op.startswith("norm") else _prepare_balance if op.startswith("balance")
     else _prepare_adamw)(s, s["case"], g)
    return s


# ------------------------------------------------------------- the plain forms
_EPS = 1e-5


def _plain_norm(s):
    x = s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    mean = f.mean(dim=1, keepdim=True)
    d = f - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + _EPS)
    y = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(x.dtype), h, torch.cat([mean, rstd], dim=1)


def _plain_norm_backward(s):
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    dy, w = s["dy"].float(), s["weight"].float()
    xhat = (s["h"].float() - mean) * rstd
    wdy = dy * w
    dx = rstd * (wdy - wdy.mean(dim=1, keepdim=True) - xhat * (wdy * xhat).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * xhat).sum(dim=0)
    db = dy.sum(dim=0).to(s["weight"].dtype) if s["bias"] is not None else None
    return dx.to(s["dy"].dtype), dw.to(s["weight"].dtype), db


def _probabilities(logits, score):
    """(p, dp factor): softmax, or sigmoid scores over their sum; dp_i/dl_e is
    p_i (delta_ie - p_e) factor_e."""
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
        return s / s.sum(dim=1, keepdim=True), 1.0 / (1.0 + torch.exp(logits))
    e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True), 1.0


def _members(s):
    """[S, T] of the counted tokens of each sequence, as fp32 zeros and ones."""
    T = s["case"]["T"]
    if s["seq_offsets"] is None:
        return torch.ones(1, T, device="cuda")
    t, o = torch.arange(T, device="cuda"), s["seq_offsets"]
    return ((t >= o[:-1, None]) & (t < o[1:, None]) & s["mask"]).float()


def _plain_balance(s):
    c = s["case"]
    of = _members(s)
    p, _ = _probabilities(s["logits"], c["score"])
    chosen = torch.zeros_like(p).scatter_(1, s["topk_idx"].long(), 1.0)
    n, counts, mass = of.sum(dim=1), of @ chosen, of @ p
    per = (counts * mass).sum(dim=1) * c["E"] / (c["k"] * n.clamp(min=1) ** 2)
    return per.sum() * (_ALPHA / of.shape[0]), counts.to(torch.int32), n.to(torch.int32)


def _plain_balance_backward(s):
    c = s["case"]
    of = _members(s)
    p, factor = _probabilities(s["logits"], c["score"])
    n = s["tokens"].float().clamp(min=1)[:, None]
    # a sequence's loads over their mean, less one: the probabilities' sum has no gradient
    load = s["counts"].float() * c["E"] / (c["k"] * n) - 1.0
    load = of.t() @ (load / n) * (s["dloss"] * (_ALPHA / of.shape[0]))
    grad = p * factor * (load - (p * load).sum(dim=1, keepdim=True))
    if not c["onto"]:
        return grad
    s["dlogits"].add_(grad)
    return s["dlogits"]


_HYPER = (1e-3, 0.9, 0.95, 1e-8, 0.1)     # lr, beta1, beta2, eps, weight decay


def _plain_adamw(s):
    lr, b1, b2, eps, wd = _HYPER
    c, t = s["case"], s["t"]
    g = s["g"].float()
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, _BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, _BLOCK) * s["v_scale"][:, None]).view(-1).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = s["p"].float() if s["master"] is None else s["master"]
    p = p * (1 - lr * wd) - lr / (1 - b1 ** t) * m / (v.sqrt() / math.sqrt(1 - b2 ** t) + eps)
    if s["master"] is not None:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            q, scale = _quantised(x)
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)


def _adamw_outputs(s):
    """The state's own buffers: parameters, masters, moments (8-bit ones as they
    are held, with their scales)."""
    return {n: s[n] for n in ("p", "master", "m", "v", "m_scale", "v_scale")
            if s.get(n) is not None}


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "adamw":
        s["t"] += 1
    if own:
        import routing_grouped_expert_gb300 as moe
        if op == "norm":
            return moe.moe_layer_norm(s["x"], s["weight"], s["bias"], _EPS, residual=s["residual"])
        if op == "norm_backward":
            return moe.moe_layer_norm_backward(s["dy"], s["h"], s["stats"], s["weight"],
                                               has_bias=s["bias"] is not None, dh=s["dh"])
        if op == "balance":
            return moe.moe_balance_loss(s["logits"], s["topk_idx"], _ALPHA, c["score"],
                                        seq_offsets=s["seq_offsets"], mask=s["mask"])
        if op == "balance_backward":
            return moe.moe_balance_loss_backward(s["dloss"], s["counts"], s["tokens"], s["logits"],
                                                 c["k"], _ALPHA, c["score"],
                                                 seq_offsets=s["seq_offsets"], mask=s["mask"],
                                                 onto=s.get("dlogits"))
        moe.moe_adamw_step(s["state"], s["grads"], s["config"], s["t"], ws=s["ws"])
        return _adamw_outputs(s)
    if op == "adamw":
        _plain_adamw(s)
        return _adamw_outputs(s)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "balance": _plain_balance,
            "balance_backward": _plain_balance_backward}[op](s)


# ------------------------------------------------------------- in 64 bits
def _exact_norm(s, c):
    w = s["weight"].double()
    if c["op"] == "norm":
        total = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        h = total.to(s["x"].dtype).double()      # what is normalised is what is stored
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        rstd = (var + _EPS) ** -0.5
        y = (h - mean) * rstd * w
        return (y if s["bias"] is None else y + s["bias"].double()), total, torch.cat([mean, rstd], 1)
    # the gradient of <dy, y> by automatic differentiation, with the statistics as functions of h
    h = s["h"].double().requires_grad_(True)
    w.requires_grad_(True)
    var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
    y = (h - mean) * (var + _EPS) ** -0.5 * w
    dx, dw = torch.autograd.grad((y * s["dy"].double()).sum(), (h, w))
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return dx, dw, s["dy"].double().sum(dim=0) if s["bias"] is not None else None


def _exact_balance(s, c):
    T, E, k = c["T"], c["E"], c["k"]
    ends = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    logits = s["logits"].double().requires_grad_(True)
    losses = []
    for a, b in zip(ends, ends[1:]):
        rows = torch.arange(a, b, device="cuda")
        if s["mask"] is not None:
            rows = rows[s["mask"][a:b]]
        n = rows.numel()
        if n == 0:
            continue
        l = logits[rows]
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
        p = p / p.sum(dim=1, keepdim=True)
        f = torch.bincount(s["topk_idx"][rows].view(-1).long(), minlength=E).double() * (E / (k * n))
        losses.append((f * p.mean(dim=0)).sum())
    loss = sum(losses) * (_ALPHA / (len(ends) - 1)) if losses else logits.sum() * 0
    if c["op"] == "balance":
        return loss.detach(), None, None
    grad = torch.autograd.grad(loss, logits)[0]
    return grad + s["dlogits"].double() if c["onto"] else grad


def _exact_adamw(s, c):
    lr, b1, b2, eps, wd = _HYPER
    t, g = s["t"] + 1, s["g"].double()
    m, r = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = m * s["m_scale"].double().repeat_interleave(_BLOCK)
        r = (r * s["v_scale"].double().repeat_interleave(_BLOCK)) ** 2
    m.lerp_(g, 1 - b1)
    r.mul_(b2).addcmul_(g, g, value=1 - b2)
    step = (m / (1 - b1 ** t)).div_((r / (1 - b2 ** t)).sqrt_().add_(eps))
    p = (s["p"] if s["master"] is None else s["master"]).double()
    p = p - lr * (step + wd * p)
    out = {"p": p}
    if s["master"] is not None:
        out["master"] = p
    if c["bits"] == 32:
        out.update(m=m, v=r)
    else:     # the values ahead of their rounding to 8 bits
        for name, x in (("m", m), ("v", r.sqrt())):
            x = x.view(-1, _BLOCK)
            scale = x.abs().amax(dim=1) / 448
            out[name] = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0).view(-1)
            out[name + "_scale"] = scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_norm if op.startswith("norm") else _exact_balance if op.startswith("balance")
            else _exact_adamw)(s, s["case"])
