"""A training step of a block -- norm, router, balance loss, expert layer, their
gradients, and the optimizer -- run together as a user would: against the same step
in torch, captured into a graph, and on a second stream."""
import importlib.util
import os

import pytest
import torch

import routing_grouped_expert_gb300 as moe

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                       "trained_block.py")


def load_example():
    spec = importlib.util.spec_from_file_location("trained_block", EXAMPLE)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def reference(ex, m, x, target, offsets):
    """Gradients of the block's loss by torch's automatic differentiation, in fp64, with the
    choice of experts as the block made it."""
    p = {n: t.detach().double().requires_grad_(True) for n, t in m.params.items()}
    h = x.double()
    y = torch.nn.functional.layer_norm(h, (ex.H,), p["norm_w"], p["norm_b"], ex.EPS)
    logits = y @ p["Wg"]
    w = torch.softmax(logits.gather(1, m.topk_idx.long()), dim=1)
    out = h.clone()
    for j in range(ex.K):
        for e in range(ex.E):
            rows = (m.topk_idx[:, j] == e).nonzero()[:, 0]
            if rows.numel():
                a = y[rows]
                f = (torch.nn.functional.silu(a @ p["W1"][e]) * (a @ p["W3"][e])) @ p["W2"][e]
                out = out.index_add(0, rows, w[rows, j:j + 1] * f)
    prob = torch.softmax(logits, dim=1)
    balance = 0.0
    for a, b in zip(offsets.tolist(), offsets.tolist()[1:]):
        if b > a:
            f = torch.bincount(m.topk_idx[a:b].reshape(-1).long(), minlength=ex.E).double()
            balance = balance + (f * ex.E / (ex.K * (b - a)) * prob[a:b].mean(dim=0)).sum()
    loss = (out - target.double()).square().sum() / x.shape[0] + \
        ex.ALPHA * balance / (offsets.numel() - 1)
    names = list(p)
    return loss.item(), dict(zip(names, torch.autograd.grad(loss, [p[n] for n in names])))


def test_gradients_are_torchs():
    """Every gradient within 5% of its norm.  The layer keeps pre-activations, activations
    and gradients in bf16, about eight roundings of 2^-8 / sqrt(3) on average each in a
    chain: 0.65%; the weights' gradients sum them over tokens.  5% leaves more than 7x; a
    term left out (the balance loss, the residual, a bias) moves a norm by far more."""
    ex = load_example()
    m, x, target, offsets = ex.make(3)
    loss, grads = ex.gradients(m, x, target, offsets)
    want, ref = reference(ex, m, x, target, offsets)
    assert abs(float(loss) - want) < 0.02 * abs(want)
    assert set(grads) == set(ref)
    for n in ref:
        a, b = grads[n].double(), ref[n]
        assert float((a - b).norm()) <= 0.05 * float(b.norm()), n


@pytest.mark.parametrize("bits", [32, 8])
def test_example_trains_and_equals_its_graph(bits):
    """The example's steps run; replayed from a graph they leave the same bits; the
    status of every workspace is clean."""
    ex = load_example()
    eager = ex.train(steps=4, bits=bits)
    graph = ex.train(steps=4, bits=bits, captured=True)
    assert len(eager.losses) == 4 and all(l == l for l in eager.losses)
    assert eager.losses == graph.losses
    for n in eager.params:
        assert torch.equal(eager.params[n], graph.params[n]), n
    for flat in ("exp_avg", "exp_avg_sq"):
        for a, b in zip(eager.states, graph.states):
            assert torch.equal(getattr(a, flat).view(torch.uint8), getattr(b, flat).view(torch.uint8))


def test_two_streams_at_once():
    """Two blocks trained on two streams at once: the bits of each alone."""
    ex = load_example()
    want = [ex.train(steps=3, seed=s) for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for s, stream in zip((1, 2), streams):
        with torch.cuda.stream(stream):
            sets.append(ex.make(s))
    # as train() does, the number and the rate on the device
    numbers = [torch.full((1,), step, device="cuda") for step in range(1, 4)]
    lr = torch.full((), ex.CONFIG.lr, device="cuda")
    torch.cuda.synchronize()
    for number in numbers:
        for (m, x, target, offsets), stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                ex.step(m, x, target, offsets, number, lr)
    torch.cuda.synchronize()
    for (m, *_), w in zip(sets, want):
        for n in w.params:
            assert torch.equal(m.params[n], w.params[n]), n


def test_beside_a_layer_that_fills_the_device():
    """The operators on one stream while the expert layer, which takes every SM for
    as long as it runs, runs on another: the bits of each alone, no wait that ran out."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    E, H, F, k = 32, 2048, 1024, 4
    x, logits = r(8192, H).to(bf), r(8192, E)
    W = [(r(E, H, F) / H ** 0.5).to(bf), (r(E, H, F) / H ** 0.5).to(bf), (r(E, F, H) / F ** 0.5).to(bf)]
    l, idx = r(30000, 256), torch.randint(0, 256, (30000, 8), generator=g, device="cuda").int()
    offsets = torch.arange(0, 30001, 500, device="cuda", dtype=torch.int32)
    w, dy = 1 + 0.1 * r(H), r(8192, H).to(bf)
    ws = [moe.Workspace() for _ in range(3)]

    def operators():
        loss, counts, tokens = moe.moe_balance_loss(l, idx, 0.01, seq_offsets=offsets, ws=ws[0])
        dl = moe.moe_balance_loss_backward(loss, counts, tokens, l, 8, 0.01, seq_offsets=offsets)
        y, h, stats = moe.moe_layer_norm(x, w)
        return (loss, counts, tokens, dl, y, stats) + \
            moe.moe_layer_norm_backward(dy, h, stats, w, has_bias=False, ws=ws[1])[:2]

    def layer():
        return moe.moe_forward(x, logits, *W, k, ws=ws[2])

    want, out = operators(), layer()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got, outs = [], []
    for _ in range(20):
        with torch.cuda.stream(a):
            outs.append(layer())
        with torch.cuda.stream(b):
            got.append(operators())
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out)
    for some in got:
        assert all(torch.equal(p, q) for p, q in zip(some, want))
    for v in ws:
        assert moe.moe_get_device_status(v) == 0
