"""A pre-norm expert block trained step by step.

    python examples/trained_block.py

out = x + layer(norm(x)): the norm (moe_layer_norm), the router's projection and
choice (moe_router_logits, moe_route_topk inside moe_forward_train), the expert layer,
and the residual.  The loss is a squared error plus the experts' balance loss per
sequence (moe_balance_loss); its gradient is added onto the layer's own in the
router's logits, and one AdamW step (moe_adamw_step) moves the bf16 weights by fp32
masters, and the norm's fp32 weights by themselves.  `train(captured=True)` replays
the whole step from a CUDA graph; the step's number and the learning rate are read on
the device.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routing_grouped_expert_gb300 as moe  # noqa: E402

T, H, F, E, K = 512, 256, 384, 16, 2
EPS, ALPHA = 1e-5, 0.05
CONFIG = moe.AdamWConfig(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.05)


class Block:
    """Parameters, optimizer states and workspaces of a block."""

    def __init__(self, seed: int, bits: int = 32):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.params = dict(
            norm_w=torch.ones(H, device="cuda"), norm_b=torch.zeros(H, device="cuda"),
            Wg=normal(H, E, std=H ** -0.5), W1=normal(E, H, F, std=H ** -0.5),
            W3=normal(E, H, F, std=H ** -0.5), W2=normal(E, F, H, std=F ** -0.5))
        p = self.params
        # one state for each type of parameter; the norm is not decayed
        self.states = [moe.AdamWState([p["Wg"], p["W1"], p["W3"], p["W2"]], bits=bits, master=True),
                       moe.AdamWState([p["norm_w"], p["norm_b"]], decay=[0.0, 0.0])]
        self.ws = [moe.Workspace() for _ in range(5)]
        self.topk_idx = None

    def check(self):
        for ws in self.ws:
            status = moe.moe_get_device_status(ws)
            if status:
                raise RuntimeError(moe.moe_status_string(status))


def make(seed: int = 0, bits: int = 32):
    """A block, and tokens of three sequences with targets for them."""
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    target = (x.float() + torch.randn(T, H, generator=g, device="cuda")).to(torch.bfloat16)
    offsets = torch.tensor([0, 100, 101, T], dtype=torch.int32, device="cuda")
    return Block(seed, bits), x, target, offsets


def gradients(m: Block, x, target, offsets):
    """(loss, the parameters' gradients by name)."""
    p, (layer_ws, norm_ws, balance_ws, gate_ws, _) = m.params, m.ws
    y, h, stats = moe.moe_layer_norm(x, p["norm_w"], p["norm_b"], EPS)
    logits = moe.moe_router_logits(y, p["Wg"], ws=gate_ws)
    layer = (p["W1"], p["W3"], p["W2"], K, layer_ws)
    out = moe.moe_forward_train(y, logits, *layer)
    m.topk_idx = moe.moe_forward_routing(layer_ws, T, H, F, E, K)[0]
    balance, counts, tokens = moe.moe_balance_loss(logits, m.topk_idx, ALPHA, seq_offsets=offsets,
                                                   ws=balance_ws)
    diff = h.float() + out.float() - target.float()
    loss = diff.square().sum() / T + balance
    dout = (2.0 / T * diff).to(torch.bfloat16)
    dy, dlogits, dW1, dW3, dW2 = moe.moe_backward(dout, logits, *layer)
    moe.moe_balance_loss_backward(None, counts, tokens, logits, K, ALPHA, seq_offsets=offsets,
                                  onto=dlogits)
    dWg = (y.float().t() @ dlogits).to(torch.bfloat16)
    dy = (dy.float() + dlogits @ p["Wg"].float().t()).to(torch.bfloat16)
    _, dw, db = moe.moe_layer_norm_backward(dy, h, stats, p["norm_w"], dh=dout, ws=norm_ws)
    return loss, dict(norm_w=dw, norm_b=db, Wg=dWg, W1=dW1, W3=dW3, W2=dW2)


def step(m: Block, x, target, offsets, number, lr=None):
    """One step, the number-th; returns its loss on the device."""
    loss, g = gradients(m, x, target, offsets)
    grads = [[g["Wg"], g["W1"], g["W3"], g["W2"]], [g["norm_w"], g["norm_b"]]]
    for state, of in zip(m.states, grads):
        moe.moe_adamw_step(state, of, CONFIG, number, lr=lr, ws=m.ws[4])
    return loss


def train(steps: int = 30, seed: int = 0, bits: int = 32, captured: bool = False) -> Block:
    """A block after some steps; its losses are in `losses`."""
    m, x, target, offsets = make(seed, bits)
    number = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.full((), CONFIG.lr, device="cuda")
    losses = []
    if captured:
        # the workspaces grow before the capture; what the step changes is put back
        kept = [t.clone() for t in _state_of(m)]
        step(m, x, target, offsets, 1, lr)
        for t, k in zip(_state_of(m), kept):
            t.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            number += 1
            loss = step(m, x, target, offsets, number, lr)
        for _ in range(steps):
            graph.replay()
            losses.append(float(loss))
    else:
        for _ in range(steps):
            number += 1
            losses.append(float(step(m, x, target, offsets, number, lr)))
    m.check()
    m.losses = losses
    return m


def _state_of(m: Block):
    flats = [t for s in m.states for t in (s.exp_avg, s.exp_avg_sq, s.exp_avg_scale,
                                           s.exp_avg_sq_scale, s.master) if t is not None]
    return list(m.params.values()) + flats


if __name__ == "__main__":
    for bits in (32, 8):
        losses = train(bits=bits, captured=True).losses
        print("moments in %2d bits: loss per token  first %.4f  last %.4f" % (bits, losses[0], losses[-1]))
