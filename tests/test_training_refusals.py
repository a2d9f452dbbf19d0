"""What the training operators refuse on the host: factors that are finite in 64 bits and not in
the fp32 that the kernels work with."""
import ctypes

import pytest

from routing_grouped_expert_gb300 import binding

P = ctypes.c_void_p(4096)   # never read
INVALID = 1


@pytest.mark.parametrize("bad", [dict(lr=1e39), dict(lr=-1e39), dict(eps=1e39), dict(wd=1e39),
                                 dict(decay=-1e39), dict(wd=1e30, decay=1e30)], ids=str)
def test_adamw_refuses_factors_that_leave_fp32(bad):
    a = {**dict(lr=1e-3, eps=1e-8, wd=0.1, decay=1.0), **bad}
    tensors = (binding._AdamWTensor * 1)((4096, 10, 0, a["decay"]))
    grads = (ctypes.c_void_p * 1)(4096)
    config = binding._AdamWConfigStruct(a["lr"], 0.9, 0.99, a["eps"], a["wd"], 32)
    assert binding.load_library().moe_adamw_step(
        tensors, grads, 1, 0, 0, ctypes.byref(config), 1, None, None, None, P, P, P, None, None, P,
        256, None) == INVALID


def test_balance_refuses_factors_that_leave_fp32():
    """alpha E / (S k) is what the sums are multiplied by."""
    lib = binding.load_library()
    assert lib.moe_balance_loss(P, P, 0, 3e38, None, None, 4, 8, 2, 1, P, P, P, P, 1 << 40,
                                None) == INVALID
    assert lib.moe_balance_loss_backward(None, P, P, P, 0, -3e38, None, None, 4, 8, 2, 1, 0, P,
                                         None) == INVALID
