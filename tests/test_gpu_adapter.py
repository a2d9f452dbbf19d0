"""The adapter projection and its gradients on the GPU against the fp64
oracle, elementwise.  What is rounded: the result, once to bf16 (8 significant
bits: at most 2^-8 of it); the low-rank activation z (or dz), once to bf16
(2^-8 of the sum of |z| |B| that it enters); and fp32 sums on the tensor core,
taken as 2^-17 of the sum of the absolute products (2^7 roundings of 2^-24)."""
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from oracle import adapter as P

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8
ACC = 2.0 ** -17

CASES = [  # T, H, N, n, R, order
    (1, 128, 128, 1, 8, "one"),
    (1, 512, 1024, 4, 8, "shuffled"),
    (1, 2048, 128, 3, 128, "one"),
    (1, 7168, 256, 2, 40, "one"),
    (1, 512, 128, 2, 16, "none"),
    (2, 640, 384, 4, 16, "distinct"),
    (3, 1152, 256, 5, 8, "distinct"),
    (4, 2048, 640, 3, 128, "shuffled"),
    (1, 16384, 128, 3, 16, "one"),
    (1, 128, 20480, 3, 8, "one"),
    (7, 256, 384, 5, 24, "shuffled"),
    (31, 2048, 256, 40, 16, "distinct"),
    (32, 384, 128, 32, 40, "distinct"),
    (33, 128, 256, 2, 72, "shuffled"),
    (64, 1024, 256, 9, 8, "segments"),
    (65, 256, 128, 300, 16, "distinct"),
    (128, 2048, 512, 7, 128, "shuffled"),
    (129, 384, 256, 3, 64, "segments"),
    (200, 512, 256, 4, 16, "none"),
    (256, 256, 256, 1, 32, "one"),
    (257, 256, 128, 64, 8, "distinct"),
    (300, 128, 384, 1024, 8, "shuffled"),
    (777, 640, 256, 6, 48, "shuffled"),
    (1000, 256, 512, 5, 16, "segments"),
    (1300, 7168, 128, 4, 16, "segments"),
    (2600, 256, 2048, 5, 24, "shuffled"),      # more tiles than SMs: persistent CTAs
    (2563, 2048, 1920, 3, 16, "segments"),
    (700, 128, 256, 200, 128, "distinct"),     # several units of rank rows per block
    (600, 512, 256, 24, 64, "shuffled"),       # units of few tokens each: gathered rows
    (300, 2048, 128, 100, 24, "distinct"),
    (128, 1024, 128, 40, 40, "shuffled"),
    (515, 7168, 128, 24, 64, "shuffled"),
    (2049, 512, 2432, 8, 16, "shuffled"),      # an odd number of feature tiles in pairs
    (1025, 256, 5120, 9, 8, "segments"),       # blocks that are no multiple of 64 tokens
    (140, 512, 128, 20, 32, "distinct"),
    (777, 1024, 128, 24, 64, "shuffled"),      # three CTAs per unit of rank rows
    (1000, 128, 256, 1, 8, "one"),             # the tokens of a gradient split by 2, 4 and 8
    (2100, 256, 128, 1, 40, "one"),
    (4100, 128, 128, 1, 128, "shuffled"),
    (2100, 128, 128, 2, 72, "none"),
]


def make(case, seed=0):
    T, H, N, n, R, order = case
    g = torch.Generator().manual_seed(seed + T * 101 + H + n)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = torch.bfloat16
    x, dy = r(T, H).to(bf), r(T, N).to(bf)
    W = (r(H, N) / H ** 0.5).to(bf)
    A, B = (r(n, R, H) / H ** 0.5).to(bf), (r(n, R, N) / R ** 0.5).to(bf)
    scale = r(n)
    if order == "one":
        idx = torch.full((T,), n - 1)
    elif order == "none":
        idx = torch.full((T,), -1)
    elif order == "distinct":
        idx = (torch.arange(T) * 7 + 3) % n
    elif order == "shuffled":
        idx = torch.randint(-1, n, (T,), generator=g)
    else:
        cuts = torch.randint(0, T, (6,), generator=g)
        idx = torch.randint(-1, n, (7,), generator=g)[(cuts[None] <= torch.arange(T)[:, None])
                                                      .sum(1)]
    return dict(x=x, W=W, A=A, B=B, scale=scale, adapter_idx=idx.to(torch.int32)), dy


def dev(d):
    return {k: v.cuda() for k, v in d.items()}


def assert_close(got, ref, mag, what):
    g = got.detach().cpu().double()
    tol = EPS * ref.abs() + EPS * mag["low"] + ACC * mag["sum"] + 1e-30
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), [tuple(i) for i in bad.nonzero()[:4].tolist()],
                           float(((g - ref).abs() / tol).max()))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_project(case):
    d, _ = make(case)
    ws = moe.Workspace()
    y = moe.moe_adapter_project(**dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    ref, mag = P.project(*d.values(), magnitudes=True)
    assert_close(y, ref, mag, "y")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    d, dy = make(case)
    ws = moe.Workspace()
    got = moe.moe_adapter_project_backward(dy.cuda(), **dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    ref, mag = P.backward(dy, *d.values(), magnitudes=True)
    for key, g in zip(("dx", "dA", "dB"), got):
        assert_close(g, ref[key], mag[key], key)
    for a in range(case[3]):
        if not (d["adapter_idx"] == a).any():
            assert (got[1][a] == 0).all() and (got[2][a] == 0).all()
            break


def test_repeated_calls_give_the_same_bits_on_any_workspace():
    ws = moe.Workspace()
    first = {}
    for rep in range(3):
        for case in (CASES[9], CASES[16], CASES[4], CASES[15]):
            d, dy = make(case)
            v = dev(d)
            ws.ensure(256)
            ws.buf.fill_(255)                       # NaN patterns in every leftover
            y = moe.moe_adapter_project(**v, ws=ws)
            g = moe.moe_adapter_project_backward(dy.cuda(), **v, ws=ws)
            now = [t.cpu() for t in (y, *g)]
            for a, b in zip(now, first.setdefault(case, now)):
                assert torch.equal(a, b)


def test_bad_index_counts_as_none_and_is_reported():
    d, dy = make((100, 256, 128, 4, 16, "shuffled"))
    d["adapter_idx"][17], d["adapter_idx"][60] = 4, -5
    ws = moe.Workspace()
    y = moe.moe_adapter_project(**dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 1
    g = moe.moe_adapter_project_backward(dy.cuda(), **dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 1
    d["adapter_idx"][17] = d["adapter_idx"][60] = -1
    assert torch.equal(y, moe.moe_adapter_project(**dev(d), ws=ws))
    assert moe.moe_get_device_status(ws) == 0
    for a, b in zip(g, moe.moe_adapter_project_backward(dy.cuda(), **dev(d))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,N", [(100, 256), (700, 256), (2600, 2048)])   # split, split, persistent
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_other_requests_do_not_see_nonfinite_values(T, N, value):
    """A non-finite weight of one adapter, or value of one token, stays with the
    requests it belongs to, forward and backward."""
    d, dy = make((T, 256, N, 4, 16, "shuffled"))
    idx = d["adapter_idx"]
    clean = moe.moe_adapter_project(**dev(d))
    grads = moe.moe_adapter_project_backward(dy.cuda(), **dev(d))
    others = idx != 2
    for key, status in (("A", 0), ("B", 2)):
        bad = {**d, key: d[key].clone()}
        bad[key][2, 5, 77] = value
        ws = moe.Workspace()
        y = moe.moe_adapter_project(**dev(bad), ws=ws)
        assert moe.moe_get_device_status(ws) == status
        assert torch.equal(y.cpu()[others], clean.cpu()[others])
        dx, dA, dB = moe.moe_adapter_project_backward(dy.cuda(), **dev(bad), ws=ws)
        assert torch.equal(dx.cpu()[others], grads[0].cpu()[others])
        for a in (0, 1, 3):
            assert torch.equal(dA[a], grads[1][a]) and torch.equal(dB[a], grads[2][a])
    t = int((idx == 2).nonzero()[3, 0])
    bad = {**d, "x": d["x"].clone()}
    bad["x"][t, 9] = value
    ws = moe.Workspace()
    y = moe.moe_adapter_project(**dev(bad), ws=ws)
    keep = torch.arange(T) != t
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    bad_dy = dy.clone()
    bad_dy[t, 3] = value
    dx, dA, dB = moe.moe_adapter_project_backward(bad_dy.cuda(), **dev(bad), ws=ws)
    assert torch.equal(dx.cpu()[keep], grads[0].cpu()[keep])
    for a in (0, 1, 3):
        assert torch.equal(dA[a], grads[1][a]) and torch.equal(dB[a], grads[2][a])


def test_tokens_do_not_depend_on_their_neighbours():
    """A token of a batch of other requests and the same token alone in its
    block: the same sums, up to the order in which K is split."""
    d, _ = make((256, 512, 256, 5, 16, "shuffled"))
    y = moe.moe_adapter_project(**dev(d))
    one = {k: (v[37:38] if k in ("x", "adapter_idx") else v) for k, v in d.items()}
    alone = moe.moe_adapter_project(**dev(one))
    ref, mag = P.project(*one.values(), magnitudes=True)
    assert_close(alone, ref, mag, "alone")
    assert_close(y[37:38], ref, mag, "in a batch")


def test_empty_batch_and_another_stream():
    d, dy = make((50, 256, 128, 3, 16, "shuffled"))
    v = dev(d)
    e = {**v, "x": v["x"][:0], "adapter_idx": v["adapter_idx"][:0]}
    assert moe.moe_adapter_project(**e).shape == (0, 128)
    dx, dA, dB = moe.moe_adapter_project_backward(dy[:0].cuda(), **e)
    assert dx.shape == (0, 256) and (dA == 0).all() and (dB == 0).all()
    want = moe.moe_adapter_project(**v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = moe.moe_adapter_project(**v, ws=moe.Workspace())
    s.synchronize()
    assert torch.equal(got, want)


def test_binding_checks_types_and_shapes():
    good = dev(make((4, 128, 256, 2, 8, "one"))[0])
    A = good["A"]
    for key, bad, err in (("x", good["x"].float(), TypeError), ("x", good["x"].cpu(), ValueError),
                          ("W", good["W"].t(), ValueError),
                          ("A", A.transpose(1, 2), ValueError),
                          ("A", A.repeat(1, 1, 2)[:, :, ::2], ValueError),
                          ("B", good["B"][:1], ValueError),
                          ("scale", good["scale"].double(), TypeError),
                          ("adapter_idx", good["adapter_idx"].long(), TypeError),
                          ("adapter_idx", good["adapter_idx"][:3], ValueError)):
        with pytest.raises(err):
            moe.moe_adapter_project(**{**good, key: bad})


def test_output_given_and_default_workspace():
    v = dev(make((70, 256, 128, 3, 16, "shuffled"))[0])
    y = torch.empty(70, 128, dtype=torch.bfloat16, device="cuda")
    assert moe.moe_adapter_project(**v, y=y) is y
    assert torch.equal(y, moe.moe_adapter_project(**v, ws=moe.Workspace()))
    with pytest.raises(ValueError):
        moe.moe_adapter_project(**v, y=y[:69])
    with pytest.raises(moe.MoeError):     # a rank that is no multiple of 8
        moe.moe_adapter_project(v["x"], v["W"], v["A"][:, :12].contiguous(),
                                v["B"][:, :12].contiguous(), v["scale"], v["adapter_idx"])


@pytest.mark.parametrize("T,N", [(1, 256), (40, 256), (2600, 2048)])   # one token, split tiles, pairs
def test_captured_in_a_graph(T, N):
    d, dy = make((T, 256, N, 4, 16, "shuffled"))
    v, dy = dev(d), dy.cuda()
    ws = moe.Workspace()
    moe.moe_adapter_project(**v, ws=ws)
    moe.moe_adapter_project_backward(dy, **v, ws=ws)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        y = moe.moe_adapter_project(**v, ws=ws)
        grads = moe.moe_adapter_project_backward(dy, **v, ws=ws)
    other, _ = make((T, 256, N, 4, 16, "shuffled"), seed=9)
    for k in ("x", "adapter_idx", "scale"):
        v[k].copy_(other[k])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, moe.moe_adapter_project(**v))
    for a, b in zip(grads, moe.moe_adapter_project_backward(dy, **v)):
        assert torch.equal(a, b)


def test_operands_of_the_layers_own_calls_share_a_workspace():
    """An adapter projection between two layer calls on one workspace changes
    neither."""
    from routing_grouped_expert_gb300 import inputs as I
    d = I.make_inputs(I.small("tiny", T=64, H=256, F=128, E=8, k=2), "cuda")
    args = (d["x"], d["logits"], d["W1"], d["W3"], d["W2"], 2)
    ws = moe.Workspace()
    want = moe.moe_forward(*args, ws=ws)
    v = dev(make((64, 256, 128, 3, 16, "shuffled"))[0])
    y = moe.moe_adapter_project(**v, ws=ws)
    assert torch.equal(want, moe.moe_forward(*args, ws=ws))
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(y, moe.moe_adapter_project(**v, ws=ws))


@pytest.mark.parametrize("T", [1, 2, 3])
def test_few_tokens_keep_to_themselves_and_report(T):
    """Non-finite values, bad indices and a status left by an
    earlier call."""
    d, _ = make((T, 256, 384, 5, 16, "distinct"))
    d["adapter_idx"] = torch.arange(T, dtype=torch.int32)
    ws = moe.Workspace()
    ws.ensure(1 << 16).fill_(0xff)
    clean = moe.moe_adapter_project(**dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    last = T - 1
    others = torch.arange(T) != last
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = {**d, "B": d["B"].clone()}
        bad["B"][last, 3, 200] = value
        zeroed = {**d, "B": d["B"].clone()}
        zeroed["B"][last, 3, 200] = 0.
        y = moe.moe_adapter_project(**dev(bad), ws=ws)
        assert moe.moe_get_device_status(ws) == 2
        assert torch.equal(y, moe.moe_adapter_project(**dev(zeroed), ws=ws))
        assert moe.moe_get_device_status(ws) == 0
        for key in ("A", "x"):
            bad = {**d, key: d[key].clone()}
            bad[key][(last, 5, 77) if key == "A" else (last, 77)] = value
            y = moe.moe_adapter_project(**dev(bad), ws=ws)
            assert moe.moe_get_device_status(ws) == 0
            assert torch.equal(y.cpu()[others], clean.cpu()[others])
            assert not y.cpu()[last].isfinite().all()
    none = {**d, "adapter_idx": d["adapter_idx"].clone()}
    for index in (5, -2):
        none["adapter_idx"][last] = index
        y = moe.moe_adapter_project(**dev(none), ws=ws)
        assert moe.moe_get_device_status(ws) == 1
    none["adapter_idx"][last] = -1
    assert torch.equal(y, moe.moe_adapter_project(**dev(none), ws=ws))
    assert moe.moe_get_device_status(ws) == 0


def test_gradients_of_changing_requests_repeat_bit_for_bit():
    """Long gradients whose weight-gradient launch starts while the one before it
    runs, on one workspace that still holds the last call's rows, masks and plan:
    each call's results are those of a workspace of its own."""
    T, H, N, n, R = 4096, 2048, 2048, 6, 16
    base, dy = make((T, H, N, n, R, "segments"))
    v, dy = dev(base), dy.cuda()
    orders = []
    for seed in range(3):
        g = torch.Generator().manual_seed(100 + seed)
        cuts = torch.randint(0, T, (2 + 5 * seed,), generator=g)
        of = torch.randint(-1, n, (len(cuts) + 1,), generator=g)
        orders.append(of[(cuts[None] <= torch.arange(T)[:, None]).sum(1)].to(torch.int32).cuda())
    want = [moe.moe_adapter_project_backward(dy, **{**v, "adapter_idx": i}, ws=moe.Workspace())
            for i in orders]
    ws = moe.Workspace()
    for rep in range(20):
        i = (rep * 2) % 3
        got = moe.moe_adapter_project_backward(dy, **{**v, "adapter_idx": orders[i]}, ws=ws)
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b), rep
    assert moe.moe_get_device_status(ws) == 0


PAIRS = [  # persistent pairs of CTAs in both directions, every box of rank rows
    (3000, 384, 2176, 7, 8, "shuffled"),
    (2333, 640, 2432, 4, 128, "shuffled"),
    (2200, 2176, 384, 5, 24, "segments"),
    (2117, 2432, 640, 3, 64, "shuffled"),
    (2500, 2304, 2304, 200, 16, "distinct"),     # many entries per block
]
# more than 32 token blocks: the weight gradients look at blocks 32 at a time
MANY_BLOCKS = [  # T, H, N, n, R: one adapter (its tokens split over a cluster) and several
    (9001, 128, 128, 1, 16),
    (9001, 128, 128, 10, 24),
    (8700, 256, 128, 4, 128),
    (17000, 128, 128, 20, 8),
]


@pytest.mark.parametrize("case", PAIRS, ids=str)
def test_pairs_of_ctas(case):
    test_project(case)
    test_backward(case)


@pytest.mark.parametrize("case", MANY_BLOCKS, ids=str)
def test_gradients_over_many_blocks(case):
    """Adapters with tokens on both sides of the 32nd block (of up to 256
    tokens), only before it, only after it, and none."""
    T, H, N, n, R = case
    d, dy = make((*case, "none"))
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-1, n, (T,), generator=g) if n == 1 else torch.full((T,), n - 1)
    if n > 1:
        idx[:5000] = torch.randint(0, max(1, n // 3), (5000,), generator=g)     # only before
        idx[3000:3400] = -1
        idx[T - 300:] = n // 2                                                  # only after
        if n > 4:
            idx[100], idx[T - 1] = n // 3 + 1, n // 3 + 1                       # one token on each side
    d["adapter_idx"] = idx.to(torch.int32)
    ws = moe.Workspace()
    got = moe.moe_adapter_project_backward(dy.cuda(), **dev(d), ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    ref, mag = P.backward(dy, *d.values(), magnitudes=True)
    for key, v in zip(("dx", "dA", "dB"), got):
        assert_close(v, ref[key], mag[key], key)
    for a in range(n):
        if not (idx == a).any():
            assert (got[1][a] == 0).all() and (got[2][a] == 0).all()
    y = moe.moe_adapter_project(**dev(d), ws=ws)
    ref, mag = P.project(*d.values(), magnitudes=True)
    assert_close(y, ref, mag, "y")
