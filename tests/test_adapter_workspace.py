"""The adapters' workspace sizes (nothing here needs a GPU)."""
import os
import subprocess
import sys

import routing_grouped_expert_gb300 as moe
from tests.conftest import ROOT

SHAPES = [  # H, N, n, R
    (512, 1024, 4, 16), (6144, 10752, 16, 16), (256, 256, 300, 16), (4096, 4096, 1024, 64),
    (7168, 2048, 24, 64), (128, 128, 1, 8), (2048, 128, 1024, 128),
]


def test_sizes_and_refusals_on_a_host_without_a_device():
    """More tokens than one small block: sizes are given, and a call is refused,
    where there is no device at all (in a process of its own, with none)."""
    code = """
import ctypes
import routing_grouped_expert_gb300 as moe
from routing_grouped_expert_gb300 import binding
for T in (1, 128, 129, 300, 5000):
    for shape in %r:
        assert moe.moe_adapter_workspace_size(T, *shape) > 0
        assert moe.moe_adapter_workspace_size_backward(T, *shape) > 0
p = ctypes.c_void_p(4096)    # never dereferenced
lib = binding.load_library()
size = (300, 512, 1024, 4, 16)
assert lib.moe_adapter_project(*[p] * 6, *size, p, p, 1 << 40, None) == 6
assert lib.moe_adapter_project_backward(*[p] * 7, *size, p, p, p, p, 1 << 40, None) == 6
print("done")
""" % SHAPES
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": ""}
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True,
                       text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", (r.returncode, r.stderr[-2000:])


def test_a_workspace_for_a_batch_serves_smaller_ones():
    for H, N, n, R in SHAPES:
        for size in (moe.moe_adapter_workspace_size, moe.moe_adapter_workspace_size_backward):
            last = 0
            for T in [*range(0, 1200), *range(1200, 20000, 37), 1 << 20]:
                now = size(T, H, N, n, R)
                assert now >= last, (size.__name__, H, N, n, R, T)
                last = now
            # a number of adapters or a rank that grows needs no less either
            assert size(700, H, N, n, R) >= size(700, H, N, max(1, n - 1), R)
            assert size(700, H, N, n, R) >= size(700, H, N, n, max(8, R - 8))
        for T in (0, 1, 200, 5000):
            assert (moe.moe_adapter_workspace_size_backward(T, H, N, n, R) >=
                    moe.moe_adapter_workspace_size(T, H, N, n, R))
