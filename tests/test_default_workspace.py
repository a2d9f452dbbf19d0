"""The workspace of calls that are given none: one per thread and stream."""
import threading

import pytest
import torch

import routing_grouped_expert_gb300 as moe
from routing_grouped_expert_gb300 import binding


class FakeWorkspace:
    def __init__(self, device):
        self.device, self.sizes = device, []

    def ensure(self, nbytes):
        self.sizes.append(nbytes)


def test_one_per_stream_and_thread(monkeypatch):
    """Calls that may overlap share no workspace (no GPU is touched here)."""
    at = {"device": 0, "stream": 11, "capturing": False}
    monkeypatch.setattr(binding, "Workspace", FakeWorkspace)
    monkeypatch.setattr(binding, "_stream", lambda: at["stream"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at["device"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at["capturing"])
    first = binding._ws(None, 100)
    assert binding._ws(None, 50) is first and first.sizes == [100, 50]
    at["stream"] = 12
    second = binding._ws(None, 100)
    assert second is not first
    at["device"] = 1
    assert binding._ws(None, 1) not in (first, second)
    at.update(device=0, stream=11)
    assert binding._ws(None, 1) is first
    found = []
    t = threading.Thread(target=lambda: found.append(binding._ws(None, 1)))
    t.start()
    t.join()
    assert found[0] is not first and found[0] is not second
    # a captured call's workspace is the graph's: no later call may share it
    at["capturing"] = True
    captured = binding._ws(None, 1)
    assert captured is not first and binding._ws(None, 1) is not captured
    at["capturing"] = False
    assert binding._ws(None, 1) is first
    own = FakeWorkspace("cuda")
    assert binding._ws(own, 7) is own and own.sizes == [7]


def adapters(seed, T=1024, H=1024, N=512, n=40, R=16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = torch.bfloat16
    return dict(x=r(T, H).to(bf).cuda(), W=(r(H, N) / H ** 0.5).to(bf).cuda(),
                A=(r(n, R, H) / H ** 0.5).to(bf).cuda(), B=(r(n, R, N) / R ** 0.5).to(bf).cuda(),
                scale=r(n).cuda(),
                adapter_idx=torch.randint(-1, n, (T,), generator=g).to(torch.int32).cuda())


@pytest.mark.gpu
def test_two_streams_without_a_workspace():
    """Calls in flight on two streams, and from two threads: the bits of calls
    made one after the other."""
    cases = [adapters(1), adapters(2, T=900, n=7, R=32)]
    dy = [torch.randn(c["x"].shape[0], c["W"].shape[1], device="cuda").to(torch.bfloat16)
          for c in cases]

    def calls(i):
        return (moe.moe_adapter_project(**cases[i]),
                *moe.moe_adapter_project_backward(dy[i], **cases[i]))

    want = []
    for i in range(2):
        want.append(calls(i))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(i))
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(streams[i]):
            for rep in range(10):
                got[i].append(calls(i))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for result in got[i]:
            for a, b in zip(result, want[i]):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_without_a_workspace():
    """Replays of a captured call beside calls on the stream it was captured on."""
    a, b = adapters(3), adapters(4)
    want_a, want_b = moe.moe_adapter_project(**a), moe.moe_adapter_project(**b)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        y = moe.moe_adapter_project(**a)
    other = torch.cuda.Stream()
    for rep in range(5):
        with torch.cuda.stream(other):
            g.replay()
        with torch.cuda.stream(s):
            got = moe.moe_adapter_project(**b)
    torch.cuda.synchronize()
    assert torch.equal(y, want_a) and torch.equal(got, want_b)


@pytest.mark.gpu
def test_a_workspace_that_grows_on_another_stream():
    """The memory it leaves is not reused while that stream's calls run."""
    small, large = adapters(5, T=300), adapters(6, T=4000)
    want = moe.moe_adapter_project(**large)
    ws = moe.Workspace()
    moe.moe_adapter_project(**small, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = moe.moe_adapter_project(**small, ws=ws)
        got = moe.moe_adapter_project(**large, ws=ws)
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(first, moe.moe_adapter_project(**small))
