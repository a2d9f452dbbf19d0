"""Kernels whose dynamic shared memory, with what they hold statically, is just over the 48 KB
that a kernel has without asking.  A larger call before would have asked for them too, so each
operator's sizes run in a process of their own."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import routing_grouped_expert_gb300 as moe
from tests import test_gpu_balance as B
from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_alone(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def test_norm_gradients():
    """Rings of 48,561 to 49,152 bytes."""
    run_alone("""
from tests import test_gpu_norm as N
import routing_grouped_expert_gb300 as moe
for dtype, dh, widths in ((N.BF, False, (1497, 1512, 1520, 2001, 2016, 2032)),
                          (N.BF, True, (1329, 1344, 1608, 1616, 2008, 2024)),
                          (N.F32, False, (1208, 1216, 1505, 1520, 2009, 2032)),
                          (N.F32, True, (1337, 1352, 2016, 2036))):
    for H in widths:
        d = N.make(7, H, dtype, dtype)
        y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"], 1e-5)
        extra = d["dh"] if dh else None
        N.check_backward(d, h, stats, moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=extra),
                         extra)
""")


def test_balance_loss():
    """Sums of 605 to 768 experts: 38,720 to 49,152 bytes beside 10,448."""
    run_alone("""
from tests import test_gpu_balance as B
for E in (605, 608, 640, 700, 767, 768):
    for score in ("softmax", "sigmoid"):
        case = (150, E, 6, [0, 70, 140], True)
        B.check(case, *B.make(case, score))
""")


def test_permutation():
    """Tables of counts of chunks x experts, 4 bytes each: 49,152 bytes beside 132."""
    run_alone("""
import numpy as np
import torch
import routing_grouped_expert_gb300 as moe
from oracle import moe_oracle as O
from tests.helpers import to_np
g = torch.Generator().manual_seed(1)
for T, E, k in ((3050, 256, 8), (16300, 64, 6), (6100, 128, 8), (1780, 438, 8)):
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    for a, b in zip(moe.moe_permute(idx.cuda(), E), O.permute(idx.numpy(), E)):
        np.testing.assert_array_equal(to_np(a), b)
""")


def test_two_threads():
    """Calls of two sizes of one kernel, by two threads on streams of their own."""
    def both(calls, times):
        failed = []

        def loop(call, stream):
            try:
                with torch.cuda.stream(stream):
                    for _ in range(times):
                        call()
                stream.synchronize()
            except Exception as e:   # noqa: BLE001
                failed.append(e)

        threads = [threading.Thread(target=loop, args=(c, torch.cuda.Stream())) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed, failed

    def norm(H):
        d = N.make(64, H, N.BF, N.BF)
        y, h, stats = moe.moe_layer_norm(d["x"], d["weight"], d["bias"])
        ws = moe.Workspace()
        ws.ensure(moe.moe_layer_norm_workspace_size(64, H))
        return lambda: moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=d["dh"], ws=ws)

    def balance(E):
        l, idx, kw = B.make((64, E, 4, None, False), "softmax")
        l, idx, ws = l.cuda(), idx.cuda(), moe.Workspace()
        ws.ensure(moe.moe_balance_workspace_size(64, E))
        return lambda: moe.moe_balance_loss(l, idx, 0.01, ws=ws, **kw)

    calls = [norm(H) for H in (4096, 2064, 2560, 3600)], [balance(E) for E in (1024, 800)]
    torch.cuda.synchronize()
    both(calls[0], 1500)
    both(calls[1], 1500)
