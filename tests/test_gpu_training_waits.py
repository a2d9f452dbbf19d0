"""Waits of the training operators that run out: a part that is waited for comes late, the waits are
short, MOE_ERR_TIMEOUT is reported, and later calls on the same workspace are right.  Nothing
hangs: what is late comes after a few hundredths of a second."""
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from tests import test_gpu_balance as B
from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

TIMEOUT = 3
LIMIT = 10_000_000      # ns
CASE = (3000, 40, 4, [0, 700, 1500, 2990], True)


@pytest.fixture
def hold():
    """A device word that holds the first block up, with short waits."""
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    moe.moe_diag_hold(at, LIMIT)
    yield at
    moe.moe_diag_hold()


def balance(case=CASE, seed=0):
    l, idx, kw = B.make(case, "softmax", seed)
    return l.cuda(), idx.cuda(), B.cuda(kw)


@pytest.mark.parametrize("T", [40, 3000, 60000])
def test_balance_block_that_is_late(hold, T):
    l, idx, kw = balance((T, 40, 4, [0, T // 3, T], True))
    ws = moe.Workspace()
    call = lambda: moe.moe_balance_loss(l, idx, 0.01, ws=ws, **kw)  # noqa: E731
    want = call()
    assert moe.moe_get_device_status(ws) == 0
    hold.fill_(LIMIT // 4)          # within the limit
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert moe.moe_get_device_status(ws) == 0
    hold.fill_(5 * LIMIT)
    call()
    assert moe.moe_get_device_status(ws) == TIMEOUT
    hold.zero_()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("types", N.TYPES, ids=str)
@pytest.mark.parametrize("size", [(5, 1024), (2000, 1001), (700, 7168), (9, 4099), (400, 9001),
                                  (320, 7000)], ids=str)
def test_norm_rows_that_are_late(hold, size, types):
    """One row a block and many, blocks that fetch few ahead and all that fit."""
    d = N.make(*size, *types)
    y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"])
    ws = moe.Workspace()
    call = lambda: moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"], ws=ws)  # noqa: E731
    want = call()
    assert moe.moe_get_device_status(ws) == 0
    hold.fill_(5 * LIMIT)
    call()
    assert moe.moe_get_device_status(ws) == TIMEOUT
    hold.zero_()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert moe.moe_get_device_status(ws) == 0


def test_limits_are_checked_and_put_back():
    with pytest.raises(moe.MoeError):
        moe.moe_diag_hold(None, 10)
    with pytest.raises(moe.MoeError):
        moe.moe_diag_hold(None, 3_000_000_000)
    for word in (torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32, device="cuda")):
        with pytest.raises((TypeError, ValueError)):     # on the host, of another type
            moe.moe_diag_hold(word, LIMIT)
    moe.moe_diag_hold(torch.full((1,), 5 * LIMIT, device="cuda"), LIMIT)
    moe.moe_diag_hold()
    l, idx, kw = balance()
    ws = moe.Workspace()
    moe.moe_balance_loss(l, idx, 0.01, ws=ws, **kw)
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T", [40, 3000, 60000])
def test_replay_after_a_late_one(hold, T):
    """A replay in which a block came late, after the others had given up, and then one with
    other inputs in which it comes last, but in time: that one is right, its status clean."""
    case = (T, 40, 4, [0, T // 3, T], True)
    (l, idx, kw), (l2, idx2, kw2) = balance(case), balance(case, seed=5)
    ws = moe.Workspace()
    call = lambda: moe.moe_balance_loss(l, idx, 0.01, ws=ws, **kw)  # noqa: E731
    want = moe.moe_balance_loss(l2, idx2, 0.01, **kw2)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    hold.fill_(5 * LIMIT)
    graph.replay()
    assert moe.moe_get_device_status(ws) == TIMEOUT
    for a, b in ((l, l2), (idx, idx2), (kw["mask"], kw2["mask"])):
        a.copy_(b)
    hold.fill_(LIMIT // 4)
    graph.replay()
    assert moe.moe_get_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(out, want))
