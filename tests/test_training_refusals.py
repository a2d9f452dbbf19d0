"""What the training operators refuse on the host: factors that are finite in 64 bits and not in
the fp32 that the kernels work with; tensors that are not 16-byte aligned, by name."""
import ctypes

import pytest
import torch

import routing_grouped_expert_gb300 as moe
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


@pytest.mark.gpu
def test_misaligned_tensors_are_named():
    """Views cut out of a buffer at odd places."""
    cut = lambda n, dtype, at=1: torch.zeros(n + at, dtype=dtype, device="cuda")[at:]  # noqa: E731
    whole = lambda *n: torch.zeros(n, device="cuda")  # noqa: E731

    def names(name, call, *args, **kw):
        with pytest.raises(moe.MoeError, match=name + " is not 16-byte aligned"):
            call(*args, **kw)

    st = moe.AdamWState([whole(5), whole(0), whole(100)])
    names(r"grads\[2\]", moe.moe_adamw_step, st, [whole(5), whole(0), cut(100, torch.float32)],
          moe.AdamWConfig(), 1)
    x = whole(4, 16)
    names("weight", moe.moe_layer_norm, x, cut(16, torch.float32))
    names("x", moe.moe_layer_norm, cut(64, torch.float32).view(4, 16), whole(16))
    names("dh", moe.moe_layer_norm_backward, x, x, whole(4, 2), whole(16),
          dh=cut(64, torch.float32).view(4, 16))
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets = cut(2, torch.int32)
    names("mask", moe.moe_balance_loss, x, idx, 0.1, mask=cut(4, torch.bool))
    names("seq_offsets", moe.moe_balance_loss, x, idx, 0.1, seq_offsets=offsets)
    _, counts, tokens = moe.moe_balance_loss(x, idx, 0.1)
    names("mask", moe.moe_balance_loss_backward, None, counts, tokens, x, 2, 0.1,
          mask=cut(4, torch.bool))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["lr", "grad_scale"])
def test_numbers_in_the_place_of_device_scalars(name):
    st = moe.AdamWState([torch.zeros(5, device="cuda")])
    with pytest.raises(ValueError, match=name):
        moe.moe_adamw_step(st, [torch.zeros(5, device="cuda")], moe.AdamWConfig(), 1, **{name: 0.1})
