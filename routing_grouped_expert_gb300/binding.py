"""ctypes binding of libmoe.so: the same entry points as include/moe.h, taking
torch tensors.  This layer only checks shapes, dtypes and devices and passes
raw pointers, sizes and the current CUDA stream; all computation runs in the
library's kernels.  A missing or unloadable library raises MoeError: there is
no CPU or PyTorch fallback.

Every call takes a Workspace, `ws`.  Without one it uses a default that belongs
to the calling thread and the current stream, so such calls may run beside each
other; calls that are given one must not overlap on it.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import threading
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_NONFINITE",
                3: "MOE_ERR_TIMEOUT", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA",
                6: "MOE_ERR_UNSUPPORTED"}

# Every symbol include/moe.h declares, with its ctypes signature.
_VP, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "moe_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_route_topk": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP]),
    "moe_route_scored": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP]),
    "moe_route_scored_backward": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "moe_forward_scored": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP,
                                _SZ, _VP]),
    "moe_forward_scored_train": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP,
                                      _VP, _SZ, _VP]),
    "moe_backward_scored": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP,
                                 _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_permute": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_permute_noalloc": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP]),
    "moe_grouped_ffn": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ,
                             _VP]),
    "moe_combine": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP, _VP]),
    "moe_forward": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "moe_forward_host": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ,
                              _VP]),
    "moe_forward_events": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ,
                                _VP, _VP]),
    "moe_forward_stage_name": (ctypes.c_char_p, [_I]),
    "moe_get_device_status": (_I, [_VP, _VP]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_diag_wait_timeout": (_I, [_VP, _SZ, ctypes.c_longlong, _VP]),
    "moe_diag_count_wait_timeout": (_I, [_VP, _SZ, ctypes.c_longlong, _VP]),
    "moe_diag_hold": (_I, [_VP, ctypes.c_longlong]),
    "moe_workspace_size_train": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_forward_train": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "moe_backward": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP,
                          _VP, _SZ, _VP]),
    "moe_router_logits": (_I, [_VP, _VP, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "moe_workspace_size_gated": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moe_forward_gated": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                               _VP, _VP, _SZ, _VP]),
    "moe_forward_f32": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "moe_forward_graph_create": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ,
                                      _VP, ctypes.POINTER(ctypes.c_void_p)]),
    "moe_graph_launch": (_I, [_VP, _VP]),
    "moe_graph_destroy": (_I, [_VP]),
    "moe_cast_bf16": (_I, [_VP, _VP, _SZ, _VP]),
    "moe_forward_routing": (_I, [_VP, _SZ, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP,
                                 _VP]),
    "moe_adapter_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_adapter_workspace_size_backward": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_adapter_project": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _SZ,
                                 _VP]),
    "moe_adapter_project_backward": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                          _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_layer_norm": (_I, [_VP, _VP, _VP, _VP, ctypes.c_float, _I, _I, _I, _I, _VP, _VP, _VP,
                            _VP]),
    "moe_layer_norm_workspace_size": (_SZ, [_I, _I]),
    "moe_layer_norm_backward": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _VP,
                                     _SZ, _VP]),
    "moe_balance_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_balance_loss": (_I, [_VP, _VP, _I, ctypes.c_float, _VP, _VP, _I, _I, _I, _I, _VP, _VP,
                              _VP, _VP, _SZ, _VP]),
    "moe_balance_loss_backward": (_I, [_VP, _VP, _VP, _VP, _I, ctypes.c_float, _VP, _VP, _I, _I,
                                       _I, _I, _I, _VP, _VP]),
    "moe_adamw_step": (_I, [_VP, _VP, _I, _I, _I, _VP, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP,
                            _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_plan_workspace_size": (_SZ, [_I, _I]),
    "moe_plan_replicas": (_I, [_VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
}


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        name = STATUS_NAMES.get(code, str(code))
        super().__init__(f"{what}: {name}")


_lib = None


def load_library(path: str | None = None):
    """Load libmoe.so once and declare its signatures."""
    global _lib
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise MoeError(-1, f"libmoe.so is not built ({p}); run "
                               "`python -m routing_grouped_expert_gb300.build`")
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _check(code: int, what: str):
    if code != MOE_OK:
        raise MoeError(code, what)


def _refused(code: int, what: str, **tensors):
    """_check of a call that failed, naming a tensor that is not 16-byte aligned."""
    if code == 1:
        for name, t in tensors.items():
            if t is not None and t.data_ptr() % 16:
                raise MoeError(code, f"{what}: {name} is not 16-byte aligned")
    _check(code, what)


def _p(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream():
    # the raw handle: building a torch.cuda.Stream object costs 3 us per call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor, dtype, shape, name: str, cuda: bool = True):
    if t.dtype is dtype and t.shape == shape and (t.is_cuda or not cuda) and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _out(t: torch.Tensor | None, dtype, shape, like: torch.Tensor, name: str) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one on `like`'s device."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(t, dtype, shape, name)
    return t


class Workspace:
    """A reusable device workspace (grows on demand, 256-byte aligned).  Calls
    on one workspace must not overlap in time: a stream or a thread that runs
    beside others takes one of its own."""

    def __init__(self, device=None):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.buf = torch.empty(0, dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> torch.Tensor:
        if self.buf.numel() < nbytes:
            if self.buf.numel():
                # calls on this stream may still use it when it is freed
                self.buf.record_stream(torch.cuda.current_stream(self.device))
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.buf

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


# The calling thread's own workspaces, by (device, stream): calls without one on
# other streams or in other threads may overlap in time.
_default_ws = threading.local()


def _ws(ws: Workspace | None, nbytes: int) -> Workspace:
    """`ws`, or without one the default of this thread and stream, with room for
    `nbytes`.  A call that is being captured into a CUDA graph without a
    workspace gets one in the graph's own memory, as its outputs do."""
    if ws is None:
        dev = torch.cuda.current_device()
        if torch.cuda.is_current_stream_capturing():
            ws = Workspace(torch.device("cuda", dev))
        else:
            key = (dev, _stream())
            ws = _default_ws.__dict__.get(key)
            if ws is None:
                ws = _default_ws.__dict__[key] = Workspace(torch.device("cuda", dev))
    ws.ensure(nbytes)
    return ws


# ------------------------------------------------------------ entry points
def moe_workspace_size(T: int, H: int, F: int, E: int, k: int) -> int:
    return int(load_library().moe_workspace_size(T, H, F, E, k))


def moe_status_string(code: int) -> str:
    return load_library().moe_status_string(code).decode()


def moe_get_device_status(ws: Workspace) -> int:
    """Synchronises the current stream; returns the device status word."""
    return int(load_library().moe_get_device_status(ws.ptr, _stream()))


def moe_diag_wait_timeout(ws: Workspace, limit_ns: int) -> None:
    """Make a bounded device wait run out (see include/moe.h)."""
    _check(load_library().moe_diag_wait_timeout(ws.ptr, ws.nbytes, limit_ns, _stream()),
           "moe_diag_wait_timeout")


def moe_diag_count_wait_timeout(ws: Workspace, limit_ns: int) -> None:
    """Make the bounded token-block counter wait run out (see include/moe.h)."""
    _check(load_library().moe_diag_count_wait_timeout(ws.ptr, ws.nbytes, limit_ns, _stream()),
           "moe_diag_count_wait_timeout")


def moe_diag_hold(hold_at: torch.Tensor | None = None, limit_ns: int = 0) -> None:
    """Shorten bounded waits of this thread's calls, and hold up a part that is waited for (see
    include/moe.h)."""
    if hold_at is not None:
        _need(hold_at, torch.int64, (1,), "hold_at")
    _check(load_library().moe_diag_hold(_p(hold_at), limit_ns), "moe_diag_hold")


def moe_route_topk(logits: torch.Tensor, k: int, topk_idx=None, topk_w=None,
                   ws: Workspace | None = None):
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    topk_idx = torch.empty(T, k, dtype=torch.int32, device=logits.device) \
        if topk_idx is None else topk_idx
    topk_w = torch.empty(T, k, dtype=torch.float32, device=logits.device) \
        if topk_w is None else topk_w
    _need(topk_idx, torch.int32, (T, k), "topk_idx")
    _need(topk_w, torch.float32, (T, k), "topk_w")
    ws = _ws(ws, 256)
    _check(load_library().moe_route_topk(_p(logits), T, E, k, _p(topk_idx), _p(topk_w), ws.ptr,
                                         ws.nbytes, _stream()), "moe_route_topk")
    return topk_idx, topk_w


class _RouteConfigStruct(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}


@dataclass(frozen=True)
class RouteConfig:
    """How moe_route_scored routes (see moe_route_config in include/moe.h)."""
    score: str = "softmax"      # or "sigmoid"
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in ROUTE_SCORES:
            raise ValueError(f"score: expected one of {sorted(ROUTE_SCORES)}, got {self.score!r}")
        c = _RouteConfigStruct(ROUTE_SCORES[self.score], self.n_group, self.topk_group,
                               self.group_top, int(self.renormalize), self.scale)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ptr", ctypes.c_void_p(ctypes.addressof(c)))

    def __reduce__(self):   # copies and pickles are made from the fields
        return type(self), (self.score, self.n_group, self.topk_group, self.group_top,
                            self.renormalize, self.scale)


def _need_bias(bias, E: int):
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")


def moe_route_scored(logits: torch.Tensor, k: int, config: RouteConfig, bias=None, topk_idx=None,
                     topk_w=None, ws: Workspace | None = None):
    """(topk_idx [T, k], topk_w [T, k]) by scores, balance bias and groups."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    _need_bias(bias, E)
    topk_idx = _out(topk_idx, torch.int32, (T, k), logits, "topk_idx")
    topk_w = _out(topk_w, torch.float32, (T, k), logits, "topk_w")
    buf = _ws(ws, 256).buf
    _check(load_library().moe_route_scored(_p(logits), _p(bias), config._ptr, T, E, k,
                                           _p(topk_idx), _p(topk_w), _p(buf), buf.numel(),
                                           _stream()), "moe_route_scored")
    return topk_idx, topk_w


def moe_route_scored_backward(dtopk_w: torch.Tensor, topk_idx: torch.Tensor, logits: torch.Tensor,
                              config: RouteConfig, bias=None, dlogits=None,
                              ws: Workspace | None = None):
    """dlogits [T, E] of moe_route_scored's weights, given their gradient."""
    T, E = logits.shape
    k = dtopk_w.shape[1]
    _need(logits, torch.float32, (T, E), "logits")
    _need(dtopk_w, torch.float32, (T, k), "dtopk_w")
    _need(topk_idx, torch.int32, (T, k), "topk_idx")
    _need_bias(bias, E)
    dlogits = _out(dlogits, torch.float32, (T, E), logits, "dlogits")
    buf = _ws(ws, 256).buf
    _check(load_library().moe_route_scored_backward(_p(dtopk_w), _p(topk_idx), _p(logits),
                                                    _p(bias), config._ptr, T, E, k, _p(dlogits),
                                                    _p(buf), buf.numel(), _stream()),
           "moe_route_scored_backward")
    return dlogits


def moe_permute(topk_idx: torch.Tensor, E: int, ws: Workspace | None = None, out=None):
    T, k = topk_idx.shape
    _need(topk_idx, torch.int32, (T, k), "topk_idx")
    dev = topk_idx.device
    if out is None:
        out = (torch.empty(E, dtype=torch.int32, device=dev),
               torch.empty(E + 1, dtype=torch.int32, device=dev),
               torch.empty(T * k, dtype=torch.int32, device=dev),
               torch.empty(T * k, dtype=torch.int32, device=dev))
    counts, offsets, sorted_src, dest_of = out
    need = moe_workspace_size(T, 128, 128, E, k)
    ws = _ws(ws, need)
    _check(load_library().moe_permute(_p(topk_idx), T, E, k, _p(counts), _p(offsets),
                                      _p(sorted_src), _p(dest_of), ws.ptr, ws.nbytes, _stream()),
           "moe_permute")
    return counts, offsets, sorted_src, dest_of


def moe_grouped_ffn(x, sorted_src, offsets, W1, W3, W2, k: int, y_sorted=None,
                    ws: Workspace | None = None):
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    _need(sorted_src, torch.int32, (T * k,), "sorted_src")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    y_sorted = torch.empty(T * k, H, dtype=torch.bfloat16, device=x.device) \
        if y_sorted is None else y_sorted
    _need(y_sorted, torch.bfloat16, (T * k, H), "y_sorted")
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    _check(load_library().moe_grouped_ffn(_p(x), _p(sorted_src), _p(offsets), _p(W1), _p(W3),
                                          _p(W2), T, H, F, E, k, _p(y_sorted), ws.ptr, ws.nbytes,
                                          _stream()), "moe_grouped_ffn")
    return y_sorted


def moe_combine(y_sorted, dest_of, topk_w, out=None):
    T, k = topk_w.shape
    H = y_sorted.shape[1]
    _need(y_sorted, torch.bfloat16, (y_sorted.shape[0], H), "y_sorted")
    _need(dest_of, torch.int32, (T * k,), "dest_of")
    _need(topk_w, torch.float32, (T, k), "topk_w")
    out = torch.empty(T, H, dtype=torch.bfloat16, device=y_sorted.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    _check(load_library().moe_combine(_p(y_sorted), _p(dest_of), _p(topk_w), T, H, k, _p(out),
                                      _stream()), "moe_combine")
    return out


def moe_forward(x, router_logits, W1, W3, W2, k: int, out=None, ws: Workspace | None = None):
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(router_logits, torch.float32, (T, E), "router_logits")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    _check(load_library().moe_forward(_p(x), _p(router_logits), _p(W1), _p(W3), _p(W2), T, H, F,
                                      E, k, _p(out), ws.ptr, ws.nbytes, _stream()),
           "moe_forward")
    return out


def _need_layer(x, router_logits, W1, W3, W2):
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(router_logits, torch.float32, (T, E), "router_logits")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    return T, H, F, E


def moe_forward_scored(x, router_logits, W1, W3, W2, k: int, config: RouteConfig, bias=None,
                       out=None, ws: Workspace | None = None):
    """moe_forward routed by moe_route_scored."""
    T, H, F, E = _need_layer(x, router_logits, W1, W3, W2)
    _need_bias(bias, E)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    _check(load_library().moe_forward_scored(_p(x), _p(router_logits), _p(bias), config._ptr,
                                             _p(W1), _p(W3), _p(W2), T, H, F, E, k, _p(out),
                                             ws.ptr, ws.nbytes, _stream()), "moe_forward_scored")
    return out


FORWARD_STAGES = 7


class ForwardGraph:
    """moe_forward captured once into a CUDA graph on the current stream (which
    must not be the legacy default stream): launch() runs the whole layer on
    the current stream, reading x and router_logits and writing out as they
    are then.  The tensors given here, and the workspace memory captured (a
    private workspace unless one is given), are kept alive by this object;
    refill x and router_logits in place between launches."""

    def __init__(self, x, router_logits, W1, W3, W2, k: int, out=None,
                 ws: Workspace | None = None):
        T, H = x.shape
        E, _, F = W1.shape
        _need(x, torch.bfloat16, (T, H), "x")
        _need(router_logits, torch.float32, (T, E), "router_logits")
        _need(W1, torch.bfloat16, (E, H, F), "W1")
        _need(W3, torch.bfloat16, (E, H, F), "W3")
        _need(W2, torch.bfloat16, (E, F, H), "W2")
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
        _need(out, torch.bfloat16, (T, H), "out")
        if ws is None:
            ws = Workspace(x.device)
        ws.ensure(moe_workspace_size(T, H, F, E, k))
        # the captured pointers: kept alive even if `ws` later grows elsewhere
        self.tensors = (x, router_logits, W1, W3, W2, out, ws.buf)
        self.ws, self.out = ws, out
        self._h = ctypes.c_void_p()
        _check(load_library().moe_forward_graph_create(
            _p(x), _p(router_logits), _p(W1), _p(W3), _p(W2), T, H, F, E, k, _p(out), ws.ptr,
            ws.nbytes, _stream(), ctypes.byref(self._h)), "moe_forward_graph_create")

    def launch(self):
        _check(load_library().moe_graph_launch(self._h, _stream()), "moe_graph_launch")
        return self.out

    def close(self):
        """Free the graph (after its last launch has completed)."""
        if self._h:
            _check(load_library().moe_graph_destroy(self._h), "moe_graph_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_forward_f32(x, router_logits, W1, W3, W2, k: int, out=None,
                    ws: Workspace | None = None):
    """The layer with its fp32 combine sum unrounded ([T, H] fp32): a partial
    output of a layer split over GPUs along the FFN features."""
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(router_logits, torch.float32, (T, E), "router_logits")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    out = torch.empty(T, H, dtype=torch.float32, device=x.device) if out is None else out
    _need(out, torch.float32, (T, H), "out")
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    _check(load_library().moe_forward_f32(_p(x), _p(router_logits), _p(W1), _p(W3), _p(W2), T,
                                          H, F, E, k, _p(out), ws.ptr, ws.nbytes, _stream()),
           "moe_forward_f32")
    return out


def moe_forward_routing(ws: Workspace, T: int, H: int, F: int, E: int, k: int):
    """The routing the last layer call on `ws` computed: (topk_idx, topk_w,
    counts, offsets, sorted_src, dest_of) copied out of the workspace."""
    dev = ws.device
    outs = (torch.empty(T, k, dtype=torch.int32, device=dev),
            torch.empty(T, k, dtype=torch.float32, device=dev),
            torch.empty(E, dtype=torch.int32, device=dev),
            torch.empty(E + 1, dtype=torch.int32, device=dev),
            torch.empty(T * k, dtype=torch.int32, device=dev),
            torch.empty(T * k, dtype=torch.int32, device=dev))
    _check(load_library().moe_forward_routing(ws.ptr, ws.nbytes, T, H, F, E, k,
                                              *[_p(t) for t in outs], _stream()),
           "moe_forward_routing")
    return outs


def moe_cast_bf16(x: torch.Tensor, out=None):
    """bf16 copy of an fp32 tensor (round to nearest even), on the GPU."""
    _need(x, torch.float32, tuple(x.shape), "x")
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, torch.bfloat16, tuple(x.shape), "out")
    _check(load_library().moe_cast_bf16(_p(x), _p(out), x.numel(), _stream()), "moe_cast_bf16")
    return out


def moe_forward_stage_name(i: int) -> str:
    r = load_library().moe_forward_stage_name(i)
    return None if r is None else r.decode()


def moe_forward_events(x, router_logits, W1, W3, W2, k: int, events, out=None,
                       ws: Workspace | None = None):
    """moe_forward that records events[0] before the first kernel and
    events[i] after stage i (torch.cuda.Event objects with timing)."""
    T, H = x.shape
    E, _, F = W1.shape
    if len(events) != FORWARD_STAGES + 1:
        raise ValueError(f"need {FORWARD_STAGES + 1} events")
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    for e in events:            # torch creates the CUDA event on its first record
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * (FORWARD_STAGES + 1))(*[e.cuda_event for e in events])
    _check(load_library().moe_forward_events(_p(x), _p(router_logits), _p(W1), _p(W3), _p(W2),
                                             T, H, F, E, k, _p(out), ws.ptr, ws.nbytes, arr,
                                             _stream()), "moe_forward_events")
    return out


def moe_forward_host(x_host, logits_host, W1, W3, W2, k: int, out_host=None,
                     ws: Workspace | None = None):
    """Host activations in (pinned CPU tensors), host result out; weights on
    the device.  The result is valid after the current stream synchronises."""
    T, H = x_host.shape
    E, _, F = W1.shape
    _need(x_host, torch.bfloat16, (T, H), "x_host", cuda=False)
    _need(logits_host, torch.float32, (T, E), "logits_host", cuda=False)
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    out_host = torch.empty(T, H, dtype=torch.bfloat16, pin_memory=True) \
        if out_host is None else out_host
    _need(out_host, torch.bfloat16, (T, H), "out_host", cuda=False)
    ws = _ws(ws, moe_workspace_size(T, H, F, E, k))
    _check(load_library().moe_forward_host(_p(x_host), _p(logits_host), _p(W1), _p(W3), _p(W2),
                                           T, H, F, E, k, _p(out_host), ws.ptr, ws.nbytes,
                                           _stream()), "moe_forward_host")
    return out_host


# ------------------------------------------ either side of the routed path
def moe_workspace_size_gated(T: int, H: int, F: int, Fs: int, E: int, k: int) -> int:
    return int(load_library().moe_workspace_size_gated(T, H, F, Fs, E, k))


def moe_router_logits(x, Wg, logits=None, ws: Workspace | None = None):
    """logits [T, E] fp32 = x [T, H] @ Wg [H, E] (bf16 in)."""
    T, H = x.shape
    E = Wg.shape[1]
    _need(x, torch.bfloat16, (T, H), "x")
    _need(Wg, torch.bfloat16, (H, E), "Wg")
    logits = torch.empty(T, E, dtype=torch.float32, device=x.device) if logits is None \
        else logits
    _need(logits, torch.float32, (T, E), "logits")
    ws = _ws(ws, 1024 + 4 * (T // 128 + 4))
    _check(load_library().moe_router_logits(_p(x), _p(Wg), T, H, E, _p(logits), ws.ptr,
                                            ws.nbytes, _stream()), "moe_router_logits")
    return logits


def moe_forward_gated(x, Wg, W1, W3, W2, k: int, shared=None, out=None,
                      ws: Workspace | None = None):
    """Router projection + routed experts (+ `shared` = (Ws1, Ws3, Ws2))."""
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(Wg, torch.bfloat16, (H, E), "Wg")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    Fs = 0
    if shared is not None:
        Ws1, Ws3, Ws2 = shared
        Fs = Ws1.shape[1]
        _need(Ws1, torch.bfloat16, (H, Fs), "Ws1")
        _need(Ws3, torch.bfloat16, (H, Fs), "Ws3")
        _need(Ws2, torch.bfloat16, (Fs, H), "Ws2")
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    ws = _ws(ws, moe_workspace_size_gated(T, H, F, Fs, E, k))
    sp = (None, None, None) if shared is None else tuple(_p(t) for t in shared)
    _check(load_library().moe_forward_gated(_p(x), _p(Wg), _p(W1), _p(W3), _p(W2), *sp, T, H,
                                            F, Fs, E, k, _p(out), ws.ptr, ws.nbytes, _stream()),
           "moe_forward_gated")
    return out


# --------------------------------------- adapters beside a shared projection
def moe_adapter_workspace_size(T: int, H: int, N: int, n: int, R: int) -> int:
    return int(load_library().moe_adapter_workspace_size(T, H, N, n, R))


def moe_adapter_workspace_size_backward(T: int, H: int, N: int, n: int, R: int) -> int:
    return int(load_library().moe_adapter_workspace_size_backward(T, H, N, n, R))


def _need_adapters(x, W, A, B, scale, adapter_idx):
    T, H = x.shape
    N = W.shape[1]
    n, R, _ = A.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(W, torch.bfloat16, (H, N), "W")
    _need(A, torch.bfloat16, (n, R, H), "A")
    _need(B, torch.bfloat16, (n, R, N), "B")
    _need(scale, torch.float32, (n,), "scale")
    _need(adapter_idx, torch.int32, (T,), "adapter_idx")
    return T, H, N, n, R


def moe_adapter_project(x, W, A, B, scale, adapter_idx, y=None, ws: Workspace | None = None):
    """y [T, N] = x W + scale_a (x A_a^T) B_a, a = adapter_idx[t] (-1: none);
    A [n, R, H], B [n, R, N]."""
    T, H, N, n, R = _need_adapters(x, W, A, B, scale, adapter_idx)
    y = _out(y, torch.bfloat16, (T, N), x, "y")
    lib = load_library()
    buf = _ws(ws, lib.moe_adapter_workspace_size(T, H, N, n, R)).buf
    _check(lib.moe_adapter_project(_p(x), _p(W), _p(A), _p(B), _p(scale), _p(adapter_idx), T, H,
                                   N, n, R, _p(y), _p(buf), buf.numel(), _stream()),
           "moe_adapter_project")
    return y


def moe_adapter_project_backward(dy, x, W, A, B, scale, adapter_idx,
                                 ws: Workspace | None = None):
    """(dx, dA, dB) of moe_adapter_project, given dy [T, N]."""
    T, H, N, n, R = _need_adapters(x, W, A, B, scale, adapter_idx)
    _need(dy, torch.bfloat16, (T, N), "dy")
    dx, dA, dB = torch.empty_like(x), torch.empty_like(A), torch.empty_like(B)
    lib = load_library()
    buf = _ws(ws, lib.moe_adapter_workspace_size_backward(T, H, N, n, R)).buf
    _check(lib.moe_adapter_project_backward(_p(dy), _p(x), _p(W), _p(A), _p(B), _p(scale),
                                            _p(adapter_idx), T, H, N, n, R, _p(dx), _p(dA),
                                            _p(dB), _p(buf), buf.numel(), _stream()),
           "moe_adapter_project_backward")
    return dx, dA, dB


# ------------------------------------------------------------- training
def moe_workspace_size_train(T: int, H: int, F: int, E: int, k: int) -> int:
    return int(load_library().moe_workspace_size_train(T, H, F, E, k))


def moe_forward_train(x, router_logits, W1, W3, W2, k: int, ws: Workspace, out=None):
    """moe_forward that keeps in `ws` what moe_backward needs."""
    T, H = x.shape
    E, _, F = W1.shape
    _need(x, torch.bfloat16, (T, H), "x")
    _need(router_logits, torch.float32, (T, E), "router_logits")
    _need(W1, torch.bfloat16, (E, H, F), "W1")
    _need(W3, torch.bfloat16, (E, H, F), "W3")
    _need(W2, torch.bfloat16, (E, F, H), "W2")
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    ws.ensure(moe_workspace_size_train(T, H, F, E, k))
    _check(load_library().moe_forward_train(_p(x), _p(router_logits), _p(W1), _p(W3), _p(W2),
                                            T, H, F, E, k, _p(out), ws.ptr, ws.nbytes,
                                            _stream()), "moe_forward_train")
    return out


def moe_backward(dout, router_logits, W1, W3, W2, k: int, ws: Workspace):
    """Gradients after moe_forward_train on the same ws: (dx, dlogits, dW1,
    dW3, dW2)."""
    T, H = dout.shape
    E, _, F = W1.shape
    _need(dout, torch.bfloat16, (T, H), "dout")
    _need(router_logits, torch.float32, (T, E), "router_logits")
    dev = dout.device
    dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    dl = torch.empty(T, E, dtype=torch.float32, device=dev)
    dW1 = torch.empty(E, H, F, dtype=torch.bfloat16, device=dev)
    dW3 = torch.empty(E, H, F, dtype=torch.bfloat16, device=dev)
    dW2 = torch.empty(E, F, H, dtype=torch.bfloat16, device=dev)
    _check(load_library().moe_backward(_p(dout), _p(router_logits), _p(W1), _p(W3), _p(W2), T, H,
                                       F, E, k, _p(dx), _p(dl), _p(dW1), _p(dW3), _p(dW2),
                                       ws.ptr, ws.nbytes, _stream()), "moe_backward")
    return dx, dl, dW1, dW3, dW2


def moe_forward_scored_train(x, router_logits, W1, W3, W2, k: int, config: RouteConfig,
                             ws: Workspace, bias=None, out=None):
    """moe_forward_scored that keeps in `ws` what moe_backward_scored needs."""
    T, H, F, E = _need_layer(x, router_logits, W1, W3, W2)
    _need_bias(bias, E)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    ws.ensure(moe_workspace_size_train(T, H, F, E, k))
    _check(load_library().moe_forward_scored_train(
        _p(x), _p(router_logits), _p(bias), config._ptr, _p(W1), _p(W3), _p(W2), T, H, F, E, k,
        _p(out), ws.ptr, ws.nbytes, _stream()), "moe_forward_scored_train")
    return out


def moe_backward_scored(dout, router_logits, W1, W3, W2, k: int, config: RouteConfig,
                        ws: Workspace, bias=None):
    """Gradients after moe_forward_scored_train on the same ws: (dx, dlogits,
    dW1, dW3, dW2)."""
    T, H, F, E = _need_layer(dout, router_logits, W1, W3, W2)
    _need_bias(bias, E)
    dx = torch.empty_like(dout)
    dl = torch.empty_like(router_logits)
    dW1, dW3, dW2 = torch.empty_like(W1), torch.empty_like(W3), torch.empty_like(W2)
    _check(load_library().moe_backward_scored(
        _p(dout), _p(router_logits), _p(bias), config._ptr, _p(W1), _p(W3), _p(W2), T, H, F, E, k,
        _p(dx), _p(dl), _p(dW1), _p(dW3), _p(dW2), ws.ptr, ws.nbytes, _stream()),
           "moe_backward_scored")
    return dx, dl, dW1, dW3, dW2


# --------------------------------- around the layer in a training step
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _dtype(t: torch.Tensor, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return d


def _beside(t: torch.Tensor, dtype, shape, dev: int, name: str):
    """_need, and on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    _need(t, dtype, shape, name)
    raise ValueError(f"{name}: on {t.device}, not on the current CUDA device of the other tensors")


def _device_of(t: torch.Tensor, name: str) -> int:
    """A call's device, that of its first tensor: it has to be the current one, on whose
    stream the call runs, and that of the other tensors."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if d != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, which is not the current CUDA device")
    return d


def _norm_types(x, weight, name):
    dt, wt = _dtype(x, name), _dtype(weight, "weight")
    if dt == 1 and wt == 0:
        raise TypeError("weight: expected torch.float32 beside float32 tensors")
    return dt, wt


def moe_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias=None, eps: float = 1e-5,
                   residual=None, y=None, h=None, stats=None, want_stats: bool = True):
    """(y [T, H], h, stats [T, 2]): layer norm of h = x + residual, or of x, which
    is then h.  stats (mean and 1 / std of each token, for the backward) is None
    unless wanted or given."""
    shape, dtype, wtype = x.shape, x.dtype, weight.dtype
    T, H = shape
    dt, wt = _norm_types(x, weight, "x")
    dev = _device_of(x, "x")
    _beside(x, dtype, shape, dev, "x")
    _beside(weight, wtype, (H,), dev, "weight")
    if bias is not None:
        _beside(bias, wtype, (H,), dev, "bias")
    if y is None:
        y = torch.empty_like(x)
    else:
        _beside(y, dtype, shape, dev, "y")
    if residual is not None:
        _beside(residual, dtype, shape, dev, "residual")
        if h is None:
            h = torch.empty_like(x)
        else:
            _beside(h, dtype, shape, dev, "h")
    elif h is not None and h is not x:
        raise ValueError("h: x itself without a residual")
    if stats is not None:
        _beside(stats, torch.float32, (T, 2), dev, "stats")
    elif want_stats:
        stats = torch.empty((T, 2), dtype=torch.float32, device=x.device)
    code = load_library().moe_layer_norm(_p(x), _p(residual), _p(weight), _p(bias), eps, T, H, dt,
                                         wt, _p(y), None if residual is None else _p(h), _p(stats),
                                         _stream())
    if code != MOE_OK:
        _refused(code, "moe_layer_norm", x=x, residual=residual, weight=weight, bias=bias, y=y,
                 h=h, stats=stats)
    return y, x if residual is None else h, stats


@functools.lru_cache(maxsize=1024)
def moe_layer_norm_workspace_size(T: int, H: int) -> int:
    return int(load_library().moe_layer_norm_workspace_size(T, H))


def moe_layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, stats: torch.Tensor,
                            weight: torch.Tensor, has_bias: bool = True, dh=None, dx=None,
                            ws: Workspace | None = None):
    """(dx, dweight, dbias) of moe_layer_norm, given dy and, where h is used past
    the norm too, its gradient dh; dx is x's and the residual's gradient.  dbias
    is None unless has_bias."""
    shape, dtype = dy.shape, dy.dtype
    T, H = shape
    dt, wt = _norm_types(dy, weight, "dy")
    dev = _device_of(dy, "dy")
    _beside(dy, dtype, shape, dev, "dy")
    _beside(h, dtype, shape, dev, "h")
    _beside(stats, torch.float32, (T, 2), dev, "stats")
    _beside(weight, weight.dtype, (H,), dev, "weight")
    if dh is not None:
        _beside(dh, dtype, shape, dev, "dh")
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _beside(dx, dtype, shape, dev, "dx")
    dw = torch.empty_like(weight)
    db = torch.empty_like(weight) if has_bias else None
    buf = _ws(ws, moe_layer_norm_workspace_size(T, H)).buf
    code = load_library().moe_layer_norm_backward(
        _p(dy), _p(h), _p(stats), _p(weight), _p(dh), T, H, dt, wt, _p(dx), _p(dw), _p(db),
        _p(buf), buf.numel(), _stream())
    if code != MOE_OK:
        _refused(code, "moe_layer_norm_backward", dy=dy, h=h, stats=stats, weight=weight, dh=dh,
                 dx=dx)
    return dx, dw, db


@functools.lru_cache(maxsize=1024)
def moe_balance_workspace_size(T: int, E: int, S: int = 1) -> int:
    return int(load_library().moe_balance_workspace_size(T, E, S))


def _balance_shape(logits, score, seq_offsets, mask):
    shape = logits.shape
    T, E = shape
    if score not in ROUTE_SCORES:
        raise ValueError(f"score: expected one of {sorted(ROUTE_SCORES)}, got {score!r}")
    dev = _device_of(logits, "logits")
    _beside(logits, torch.float32, shape, dev, "logits")
    S = 1
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        _beside(seq_offsets, torch.int32, (S + 1,), dev, "seq_offsets")
    if mask is not None:
        _beside(mask, torch.bool, (T,), dev, "mask")
    return T, E, S, dev


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, alpha: float,
                     score: str = "softmax", seq_offsets=None, mask=None,
                     ws: Workspace | None = None):
    """(loss [], counts [S, E], tokens [S]): the experts' balance loss of the
    sequences seq_offsets [S + 1] (without: all tokens are one), over the tokens
    whose mask [T] is set; the choices of each expert and the counted tokens."""
    T, E, S, dev = _balance_shape(logits, score, seq_offsets, mask)
    k = topk_idx.shape[1]
    _beside(topk_idx, torch.int32, (T, k), dev, "topk_idx")
    device = logits.device
    loss = torch.empty((), dtype=torch.float32, device=device)
    counts = torch.empty((S, E), dtype=torch.int32, device=device)
    tokens = torch.empty((S,), dtype=torch.int32, device=device)
    buf = _ws(ws, moe_balance_workspace_size(T, E, S)).buf
    code = load_library().moe_balance_loss(
        _p(logits), _p(topk_idx), ROUTE_SCORES[score], alpha, _p(seq_offsets), _p(mask), T, E, k, S,
        _p(loss), _p(counts), _p(tokens), _p(buf), buf.numel(), _stream())
    if code != MOE_OK:
        _refused(code, "moe_balance_loss", logits=logits, topk_idx=topk_idx,
                 seq_offsets=seq_offsets, mask=mask)
    return loss, counts, tokens


def moe_balance_loss_backward(dloss, counts: torch.Tensor, tokens: torch.Tensor,
                              logits: torch.Tensor, k: int, alpha: float, score: str = "softmax",
                              seq_offsets=None, mask=None, onto=None):
    """dlogits [T, E] of moe_balance_loss, given its counts and tokens and dloss
    (a device scalar, or None: 1); onto: dlogits to which it is added, in place."""
    T, E, S, dev = _balance_shape(logits, score, seq_offsets, mask)
    _beside(counts, torch.int32, (S, E), dev, "counts")
    _beside(tokens, torch.int32, (S,), dev, "tokens")
    if dloss is not None:
        if dloss.numel() != 1:
            raise ValueError("dloss: expected one float32 value")
        _beside(dloss, torch.float32, dloss.shape, dev, "dloss")
    if onto is None:
        dlogits = torch.empty_like(logits)
    else:
        _beside(onto, torch.float32, (T, E), dev, "onto")
        dlogits = onto
    code = load_library().moe_balance_loss_backward(
        _p(dloss), _p(counts), _p(tokens), _p(logits), ROUTE_SCORES[score], alpha,
        _p(seq_offsets), _p(mask), T, E, k, S, int(onto is not None), _p(dlogits), _stream())
    if code != MOE_OK:
        _refused(code, "moe_balance_loss_backward", counts=counts, tokens=tokens, logits=logits,
                 seq_offsets=seq_offsets, mask=mask, onto=onto)
    return dlogits


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("n", ctypes.c_int64), ("start", ctypes.c_int64),
                ("decay", ctypes.c_double)]


class _AdamWConfigStruct(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("state_bits", ctypes.c_int32)]


ADAMW_BLOCK = 256    # elements of a block that shares one scale of an 8-bit moment


@dataclass(frozen=True)
class AdamWConfig:
    """The factors of an AdamW step (see moe_adamw_step in include/moe.h)."""
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 1e-2


class AdamWState:
    """The moments of a list of parameters (all bf16 or all fp32, on one device),
    and their fp32 master weights where wanted: bits is 32 (fp32 moments) or 8
    (e4m3 in blocks of 256 elements with an fp32 scale each, the second moment as
    its square root).  decay: a factor on the weight decay for each parameter.

    exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale (8 bits; else None) and
    master (or None) are flat tensors that hold all parameters' values, each
    parameter's from a block of its own on: `of(flat, i)` is parameter i's part of
    a flat one of values.  To save a state, keep these; to load one, copy into
    them.  The parameters are kept alive and updated where they lie."""

    def __init__(self, params, bits: int = 32, master: bool = False, decay=None):
        self.params = list(params)
        if not self.params:
            raise ValueError("params: no tensor given")
        if bits not in (8, 32):
            raise ValueError(f"bits: expected 8 or 32, got {bits}")
        first = self.params[0]
        self.param_type = _dtype(first, "params[0]")
        if master and self.param_type == 1:
            raise ValueError("master: float32 parameters are their own")
        decay = [1.0] * len(self.params) if decay is None else [float(d) for d in decay]
        if len(decay) != len(self.params):
            raise ValueError("decay: one factor for each parameter")
        self.starts, at, spans = [], 0, []
        for i, p in enumerate(self.params):
            _need(p, first.dtype, p.shape, f"params[{i}]")
            if p.device != first.device:
                raise ValueError(f"params[{i}]: on {p.device}, not {first.device}")
            if p.data_ptr() % 16:
                raise ValueError(f"params[{i}]: must be 16-byte aligned")
            self.starts.append(at)
            at += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
            if p.numel():
                spans.append((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size(), i))
        spans.sort()
        for (_, end, i), (begin, _, j) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"params[{min(i, j)}] and params[{max(i, j)}] share memory")
        self.bits, self.size, dev = bits, at, first.device
        kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
        zeros = lambda n, dtype: torch.zeros(n, dtype=dtype, device=dev)  # noqa: E731
        self.exp_avg, self.exp_avg_sq = zeros(at, kind), zeros(at, kind)
        self.exp_avg_scale = self.exp_avg_sq_scale = self.master = None
        if bits == 8:
            self.exp_avg_scale = zeros(at // ADAMW_BLOCK, torch.float32)
            self.exp_avg_sq_scale = zeros(at // ADAMW_BLOCK, torch.float32)
        if master:
            self.master = zeros(at, torch.float32)
            for i, p in enumerate(self.params):
                self.of(self.master, i).copy_(p.detach())
        self.decay = tuple(decay)
        self._bind()

    def _bind(self):
        """What a step compares with and hands over, for all parameters at once."""
        first, count = self.params[0], len(self.params)
        # whatever becomes of a parameter, the memory that a step writes stays its own
        self._held = [p.detach() for p in self.params]
        self._shapes = [p.shape for p in self.params]
        self._ptrs = [p.data_ptr() for p in self.params]
        self._devices = [first.get_device()] * count
        self._table = (_AdamWTensor * count)(*[
            (p.data_ptr(), p.numel(), o, d)
            for p, o, d in zip(self.params, self.starts, self.decay)])

    def __getstate__(self):   # copies and pickles have parameters, and places, of their own
        return {k: v for k, v in self.__dict__.items()
                if k not in ("_table", "_ptrs", "_devices", "_shapes", "_held")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._bind()

    def of(self, flat: torch.Tensor, i: int) -> torch.Tensor:
        """Parameter i's part of a flat tensor of this state, in its shape."""
        p = self.params[i]
        return flat[self.starts[i]:self.starts[i] + p.numel()].view(p.shape)


def moe_adamw_step(state: AdamWState, grads, config: AdamWConfig, step, lr=None, grad_scale=None,
                   ws: Workspace | None = None) -> None:
    """One AdamW step on the state's parameters, in place, by gradients of their
    shapes (all bf16 or all fp32; 16-byte aligned).  step: its number (1 for the first), or an
    int64 tensor of one element that holds it on the device; lr, grad_scale:
    device scalars, in the place of config.lr and 1."""
    grads, n = list(grads), len(state.params)
    if len(grads) != n:
        raise ValueError(f"grads: {len(grads)} for {n} parameters")
    gt, dev = _dtype(grads[0], "grads[0]"), _device_of(state.exp_avg, "state")
    # all at once: per tensor it would cost the host more than the step costs the device
    dtype = grads[0].dtype
    if ([g.dtype for g in grads] != [dtype] * n or [g.shape for g in grads] != state._shapes or
            list(map(torch.Tensor.get_device, grads)) != state._devices or
            not all(map(torch.Tensor.is_contiguous, grads))):
        for i, (g, shape) in enumerate(zip(grads, state._shapes)):
            _need(g, dtype, shape, f"grads[{i}]")
        raise ValueError(f"grads: must be on {state.exp_avg.device}")
    if list(map(torch.Tensor.data_ptr, state.params)) != state._ptrs:
        raise ValueError("params: one lies elsewhere than where the state was made for it")
    table = array.array("Q", map(torch.Tensor.data_ptr, grads))
    kind = torch.float32 if state.bits == 32 else torch.float8_e4m3fn
    for name, dtype, size in (("exp_avg", kind, state.size), ("exp_avg_sq", kind, state.size),
                              ("exp_avg_scale", torch.float32, state.size // ADAMW_BLOCK),
                              ("exp_avg_sq_scale", torch.float32, state.size // ADAMW_BLOCK),
                              ("master", torch.float32, state.size)):
        t = getattr(state, name)
        if t is not None:
            _beside(t, dtype, (size,), dev, f"state.{name}")
    step_at = None
    if isinstance(step, torch.Tensor):
        if step.dtype != torch.int64 or step.numel() != 1 or step.get_device() != dev:
            raise ValueError("step: expected an int, or one int64 value on the device")
        step_at, step = step, 1
    for name, t in (("lr", lr), ("grad_scale", grad_scale)):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or
                              t.numel() != 1 or t.get_device() != dev):
            raise ValueError(f"{name}: expected one float32 value on the device")
    c = _AdamWConfigStruct(config.lr, config.beta1, config.beta2, config.eps, config.weight_decay,
                           state.bits)
    buf = _ws(ws, 256).buf
    code = load_library().moe_adamw_step(
        state._table, table.buffer_info()[0], n, state.param_type, gt,
        ctypes.byref(c), step, _p(step_at), _p(lr), _p(grad_scale), _p(state.master),
        _p(state.exp_avg), _p(state.exp_avg_sq), _p(state.exp_avg_scale),
        _p(state.exp_avg_sq_scale), _p(buf), buf.numel(), _stream())
    if code != MOE_OK:
        _refused(code, "moe_adamw_step", **{f"grads[{i}]": g for i, g in enumerate(grads) if g.numel()})


def moe_plan_workspace_size(E: int, G: int) -> int:
    return load_library().moe_plan_workspace_size(E, G)


def moe_plan_replicas(counts: torch.Tensor, G: int, beta: int, budget: int, rounds: int = -1,
                      lam: int = -1, ws: Workspace | None = None):
    """Replica plan of expert row counts [E] (int32, on the GPU) for G GPUs.
    Returns (blocks_per_gpu [E, G], row_ranges [E, G, 2], gpu_load [G], info [4]),
    int32 tensors on the counts' device; lam = -1: no reduction penalty."""
    E = counts.shape[0]
    _need(counts, torch.int32, (E,), "counts")
    dev = counts.device
    n = torch.empty(E, G, dtype=torch.int32, device=dev)
    rows = torch.empty(E, G, 2, dtype=torch.int32, device=dev)
    load = torch.empty(G, dtype=torch.int32, device=dev)
    info = torch.empty(4, dtype=torch.int32, device=dev)
    need = moe_plan_workspace_size(E, G)
    ws = _ws(ws, max(need, 256))
    _check(load_library().moe_plan_replicas(_p(counts), E, G, beta, budget, rounds, lam, _p(n),
                                            _p(rows), _p(load), _p(info), ws.ptr, ws.nbytes,
                                            _stream()), "moe_plan_replicas")
    return n, rows, load, info
