"""A layer served and fine-tuned for several requests at once.

    python examples/adapted_layer.py

Every token belongs to a request with a low-rank adapter of its own, or none.  A
step runs the shared projection with the requests' adapters
(moe_adapter_project), the router projection, and the expert layer on scored
routing: sigmoid scores, a balance bias, groups of experts, renormalised weights
(moe_forward_scored).  `serve` is one such step for tokens being decoded;
`finetune` trains the adapters of all requests together on frozen layer weights
(moe_forward_scored_train, moe_backward_scored, moe_adapter_project_backward) and
moves the balance bias towards even loads, as a router is trained without an
auxiliary loss.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routing_grouped_expert_gb300 as moe  # noqa: E402

H, F, E, K, RANK, ADAPTERS = 256, 384, 32, 4, 16, 6
CONFIG = moe.RouteConfig(score="sigmoid", n_group=8, topk_group=4, group_top=2, renormalize=True,
                         scale=1.5)


def make_model(seed: int = 0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    return dict(W=normal(H, H, std=H ** -0.5), A=normal(ADAPTERS, RANK, H, std=H ** -0.5),
                B=normal(ADAPTERS, RANK, H, std=0.01),
                scale=torch.ones(ADAPTERS, device="cuda"),
                Wg=normal(H, E, std=H ** -0.5), bias=torch.zeros(E, device="cuda"),
                W1=normal(E, H, F, std=H ** -0.5), W3=normal(E, H, F, std=H ** -0.5),
                W2=normal(E, F, H, std=F ** -0.5))


def project(m, x, adapter_idx, ws=None):
    return moe.moe_adapter_project(x, m["W"], m["A"], m["B"], m["scale"], adapter_idx, ws=ws)


def serve(m, x, adapter_idx):
    """One step for a batch of tokens, each of some request."""
    h = project(m, x, adapter_idx)
    logits = moe.moe_router_logits(h, m["Wg"])
    return moe.moe_forward_scored(h, logits, m["W1"], m["W3"], m["W2"], K, CONFIG, bias=m["bias"])


def finetune(m, x, adapter_idx, target, steps: int = 20, lr: float = 0.3, balance: float = 1e-3):
    """Trains A and B of every adapter on |layer(x) - target|^2 / T; returns the
    losses and the largest load over the mean, per step."""
    ws, ws_a = moe.Workspace(), moe.Workspace()
    T = x.shape[0]
    losses, loads = [], []
    for _ in range(steps):
        h = project(m, x, adapter_idx, ws=ws_a)
        logits = moe.moe_router_logits(h, m["Wg"])
        layer = (m["W1"], m["W3"], m["W2"], K, CONFIG, ws)
        out = moe.moe_forward_scored_train(h, logits, *layer, bias=m["bias"])
        counts = moe.moe_forward_routing(ws, T, H, F, E, K)[2].float()
        diff = out.float() - target.float()
        losses.append(float(diff.square().sum() / T))
        loads.append(float(counts.max() / counts.mean()))
        dout = (2.0 / T * diff).to(torch.bfloat16)
        dh, dlogits, *_ = moe.moe_backward_scored(dout, logits, *layer, bias=m["bias"])
        dh = (dh.float() + dlogits @ m["Wg"].float().t()).to(torch.bfloat16)
        _, dA, dB = moe.moe_adapter_project_backward(dh, x, m["W"], m["A"], m["B"], m["scale"],
                                                     adapter_idx, ws=ws_a)
        m["A"] = (m["A"].float() - lr * dA.float()).to(torch.bfloat16)
        m["B"] = (m["B"].float() - lr * dB.float()).to(torch.bfloat16)
        m["bias"] += balance * torch.sign(counts.mean() - counts)
    for w in (ws, ws_a):
        status = moe.moe_get_device_status(w)
        if status:
            raise RuntimeError(moe.moe_status_string(status))
    return losses, loads


def main(T: int = 768, steps: int = 20):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    # whole requests one after the other; the last tokens have no adapter
    adapter_idx = (torch.arange(T, device="cuda") * (ADAPTERS + 1) // T).to(torch.int32)
    adapter_idx[adapter_idx == ADAPTERS] = -1
    teacher, m = make_model(), make_model()
    teacher["B"] = (teacher["B"].float() * 10).to(torch.bfloat16)
    target = serve(teacher, x, adapter_idx)
    losses, loads = finetune(m, x, adapter_idx, target, steps)
    # tokens being decoded: one of each request
    pick = torch.arange(0, T, T // 8, device="cuda")
    out = serve(m, x[pick].contiguous(), adapter_idx[pick].contiguous())
    error = float((out.float() - target[pick].float()).square().sum(1).mean())
    return losses, loads, error


if __name__ == "__main__":
    losses, loads, error = main()
    print("loss per token  first %.4f  last %.4f" % (losses[0], losses[-1]))
    print("largest load / mean  first %.3f  last %.3f" % (loads[0], loads[-1]))
    print("decoded tokens' error %.4f" % error)
