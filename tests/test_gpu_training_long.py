"""The training step's operators on tensors of more than 2^32 elements: their ends
against the same rows or elements in a call of their own."""
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from tests.test_gpu_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [16384, 16385 - 8 - 4])   # rows on 16-byte boundaries, and not
def test_norm(H):
    T, n = (1 << 32) // H + 1000, 300
    g = torch.Generator(device="cuda").manual_seed(H)
    w = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[T - n:] = torch.randn(n, H, generator=g, device="cuda")
    assert x.numel() > 1 << 32
    y, h, stats = moe.moe_layer_norm(x, w, residual=x, h=x)   # doubled in place
    # (not bit for bit against a call on these rows alone: where rows do not start on
    # 16-byte boundaries, the order of a row's sums goes by its place between them)
    d = dict(x=x[T - n:], weight=w)
    check_forward(d, y[T - n:], h[T - n:], stats[T - n:], 1e-5, bias=False)
    assert (y[:T - n].view(torch.int16) & 0x7fff).max() == 0
    # only the last rows have a gradient: adding the others' zeros rounds nothing
    y.zero_()
    y[T - n:] = torch.randn(n, H, generator=g, device="cuda")
    d["dy"] = y[T - n:].clone()
    dx, dw, db = moe.moe_layer_norm_backward(y, x, stats, w, dx=y)
    assert (dx[:T - n].view(torch.int16) & 0x7fff).max() == 0
    check_backward(d, h[T - n:], stats[T - n:], (dx[T - n:], dw, db))


def test_balance():
    T, E, k, n = (1 << 32) // 1024 + 5000, 1024, 2, 500
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.zeros(T, E, device="cuda")
    l[T - n:] = torch.randn(n, E, generator=g, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    o = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    loss, counts, tokens = moe.moe_balance_loss(l, idx, 0.01, seq_offsets=o)
    assert tokens.tolist() == [T - n, n]
    assert torch.equal(counts[0], torch.bincount(idx[:T - n].view(-1), minlength=E).int())
    tail = l[T - n:].clone()
    two = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
    part, c, m = moe.moe_balance_loss(tail, idx[T - n:].clone(), 0.01, seq_offsets=two)
    assert torch.equal(counts[1], c[1])
    # equal logits: the first sequence's loss is 0.01 / 2 whatever its loads
    assert abs(float(loss) - float(part) - 0.005) < 1e-7
    got = moe.moe_balance_loss_backward(None, counts, tokens, l, k, 0.01, seq_offsets=o)
    want = moe.moe_balance_loss_backward(None, c, m, tail, k, 0.01, seq_offsets=two)
    torch.testing.assert_close(got[T - n:], want, rtol=1e-5, atol=0)
    assert torch.isfinite(got[-n - 5000::997]).all()


def test_balance_of_the_most_tokens():
    """2^31 - 1 tokens of one expert: token numbers end with the type."""
    T = 2 ** 31 - 1
    l = torch.full((T, 1), 0.5, device="cuda")
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    loss, counts, tokens = moe.moe_balance_loss(l, idx, 0.25)
    assert int(counts) == T and int(tokens) == T and abs(float(loss) - 0.25) < 1e-6
    del idx
    onto = torch.ones(T, 1, device="cuda")
    moe.moe_balance_loss_backward(None, counts, tokens, l, 1, 0.25, onto=onto)
    assert (onto == 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    """One tensor of more than 2^32 elements, and one behind it in the state."""
    n, m = (1 << 32) + 5003, 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(m, dtype=torch.bfloat16, device="cuda")
    dp = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    dp[n - m:] = 0.5
    dp[7] = -2.0
    dq = torch.full((m,), 0.25, dtype=torch.bfloat16, device="cuda")
    st = moe.AdamWState([p, q], bits=bits)
    c = moe.AdamWConfig(lr=0.125, weight_decay=0.0)
    moe.moe_adamw_step(st, [dp, dq], c, 1)
    # the first step moves by lr against the gradient's sign
    assert (p[n - m:] == -0.125).all() and p[7] == 0.125 and (q == 0.875).all()
    p[7] = 0
    p[n - m:] = 0
    assert (p.view(torch.int16) & 0x7fff).max() == 0
    tail = st.of(st.exp_avg, 1).float()
    assert (tail > 0).all() and (st.exp_avg.view(torch.uint8)[-4:] == 0).all()
