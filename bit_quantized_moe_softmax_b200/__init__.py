"""ds4 routed-MoE expert FFN on B200 (sm_100a): Python binding of libds4moe.so.

The functions below carry the names of the C ABI in ``include/ds4moe.h`` and
only marshal arguments: torch tensors become device pointers, the current
torch stream becomes the ``stream`` argument.  Every step of the layer runs in
the library's CUDA kernels; there is no CPU or PyTorch fallback, and loading
fails loudly when the library is missing.

``MoELayer`` is plumbing on top: it allocates the weight and workspace
buffers with torch, binds them and loads a layer.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libds4moe.so")
_lib = None

DS4MOE_ACT_F32 = 0
DS4MOE_ACT_BF16 = 1
DS4MOE_Q8_E4M3 = 0
DS4MOE_Q8_INT8 = 1

STATUS = {0: "OK", -1: "ERR_ARG", -2: "ERR_ALIGN", -3: "ERR_SHAPE", -4: "ERR_NOT_READY", -5: "ERR_CUDA",
          -6: "ERR_TIMEOUT", -7: "ERR_DEVICE"}

# Every symbol include/ds4moe.h declares.
EXPORTS = ("ds4moe_create", "ds4moe_destroy", "ds4moe_weight_bytes", "ds4moe_workspace_bytes", "ds4moe_bind",
           "ds4moe_pack_q2k", "ds4moe_pack_iq2xxs", "ds4moe_set_grid", "ds4moe_set_router", "ds4moe_set_expert",
           "ds4moe_set_shared", "ds4moe_forward", "ds4moe_forward_host", "ds4moe_route", "ds4moe_dequant",
           "ds4moe_get_device_error", "ds4moe_last_error", "ds4moe_plan_launches", "ds4moe_plan_kernel",
           "ds4moe_forward_profiled", "ds4moe_route_noalloc", "ds4moe_forward_residual",
           "ds4moe_forward_residual_profiled", "ds4moe_set_steering", "ds4moe_forward_host_async",
           "ds4moe_host_sync", "ds4moe_probe", "ds4moe_selftest_wait",
           "ds4moe_permutation", "ds4moe_pack_q4k", "ds4moe_forward_chain", "ds4moe_forward_routed",
           "ds4moe_combine_slots", "ds4moe_add_rmsnorm", "ds4moe_widen_rows", "ds4moe_project",
           "ds4moe_project_work_bytes", "ds4moe_get_project_error", "ds4moe_selftest_project_wait", "ds4moe_sample")


class ds4moe_shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("has_shared", ctypes.c_int32), ("has_bias", ctypes.c_int32), ("decode_max", ctypes.c_int32),
                ("expert_bits", ctypes.c_int32)]


class Ds4MoeError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__("%s: %s (%s)" % (where, msg, STATUS.get(status, status)))
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libds4moe.so from the package directory (built by build.py); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libds4moe.so not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "ds4moe_create": ([ctypes.POINTER(ds4moe_shape), ctypes.POINTER(vp)], i32),
            "ds4moe_destroy": ([vp], i32),
            "ds4moe_weight_bytes": ([vp], sz),
            "ds4moe_workspace_bytes": ([vp, i32], sz),
            "ds4moe_bind": ([vp, vp, sz, vp, sz, vp], i32),
            "ds4moe_pack_q2k": ([vp, i64, vp, vp], i32),
            "ds4moe_pack_q4k": ([vp, i64, vp, vp], i32),
            "ds4moe_pack_iq2xxs": ([vp, i64, vp, vp, vp], i32),
            "ds4moe_set_grid": ([vp, vp, vp], i32),
            "ds4moe_set_router": ([vp, vp, vp, vp], i32),
            "ds4moe_set_expert": ([vp, i32, vp, vp, vp, vp], i32),
            "ds4moe_set_shared": ([vp, vp, vp, vp, vp], i32),
            "ds4moe_forward": ([vp, vp, i32, vp, vp], i32),
            "ds4moe_forward_host": ([vp, vp, i32, vp, vp], i32),
            "ds4moe_forward_host_async": ([vp, vp, i32, vp, vp], i32),
            "ds4moe_host_sync": ([vp], i32),
            "ds4moe_route": ([vp, vp, i32, vp, vp, vp], i32),
            "ds4moe_dequant": ([vp, i32, i32, i32, vp, vp], i32),
            "ds4moe_probe": ([vp, i32, i32, i32, vp, i32, vp, vp], i32),
            "ds4moe_selftest_wait": ([vp, vp], i32),
            "ds4moe_permutation": ([vp, vp, i32, vp, vp, vp, vp], i32),
            "ds4moe_get_device_error": ([vp, vp, ctypes.POINTER(i32)], i32),
            "ds4moe_last_error": ([], ctypes.c_char_p),
            "ds4moe_plan_launches": ([vp, i32], i32),
            "ds4moe_plan_kernel": ([vp, i32, i32], ctypes.c_char_p),
            "ds4moe_forward_profiled": ([vp, vp, i32, vp, ctypes.POINTER(vp), vp], i32),
            "ds4moe_route_noalloc": ([vp, vp, i32, vp, vp, vp], i32),
            "ds4moe_forward_residual": ([vp, vp, i32, vp, vp], i32),
            "ds4moe_forward_chain": ([ctypes.POINTER(vp), i32, vp, i32, vp, vp, vp], i32),
            "ds4moe_forward_routed": ([vp, vp, i32, vp, vp, vp, vp], i32),
            "ds4moe_combine_slots": ([vp, vp, vp, i32, i32, i32, vp, vp], i32),
            "ds4moe_set_steering": ([vp, vp, ctypes.c_float, vp], i32),
            "ds4moe_forward_residual_profiled": ([vp, vp, i32, vp, ctypes.POINTER(vp), vp], i32),
            "ds4moe_add_rmsnorm": ([vp, i32, vp, i32, vp, ctypes.c_float, i32, i32, vp, vp, i32, vp, i32, i32, vp,
                                    vp], i32),
            "ds4moe_widen_rows": ([vp, i32, vp, i32, i32, i32, vp, i32, vp], i32),
            "ds4moe_project": ([vp, i32, vp, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp], i32),
            "ds4moe_project_work_bytes": ([i32, i32, i32, i32, i32], sz),
            "ds4moe_get_project_error": ([vp, ctypes.POINTER(i32)], i32),
            "ds4moe_selftest_project_wait": ([vp, i32, vp, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, sz, i32, vp], i32),
            "ds4moe_sample": ([vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def ds4moe_last_error() -> str:
    return lib().ds4moe_last_error().decode()


def _ok(status: int, where: str):
    if status != 0:
        raise Ds4MoeError(status, where, ds4moe_last_error())


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ C ABI names
def ds4moe_create(hidden, inter, n_experts, top_k, max_tokens, act_dtype=DS4MOE_ACT_F32, has_shared=1,
                  has_bias=0, decode_max=0, expert_bits=0) -> int:
    s = ds4moe_shape(hidden, inter, n_experts, top_k, max_tokens, act_dtype, has_shared, has_bias, decode_max,
                     expert_bits)
    h = ctypes.c_void_p()
    _ok(lib().ds4moe_create(ctypes.byref(s), ctypes.byref(h)), "ds4moe_create")
    return h.value


def ds4moe_destroy(h: int):
    _ok(lib().ds4moe_destroy(h), "ds4moe_destroy")


def ds4moe_weight_bytes(h: int) -> int:
    return lib().ds4moe_weight_bytes(h)


def ds4moe_workspace_bytes(h: int, n_tokens: int) -> int:
    return lib().ds4moe_workspace_bytes(h, n_tokens)


def ds4moe_bind(h: int, weights: torch.Tensor, workspace: torch.Tensor | None, stream=None):
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _ok(lib().ds4moe_bind(h, _ptr(weights), weights.numel() * weights.element_size(), _ptr(workspace), wsb,
                          _stream(stream)), "ds4moe_bind")


def ds4moe_pack_q2k(w: torch.Tensor, blocks: torch.Tensor, stream=None):
    _ok(lib().ds4moe_pack_q2k(_ptr(w), w.numel(), _ptr(blocks), _stream(stream)), "ds4moe_pack_q2k")


def ds4moe_pack_q4k(w: torch.Tensor, blocks: torch.Tensor, stream=None):
    _ok(lib().ds4moe_pack_q4k(_ptr(w), w.numel(), _ptr(blocks), _stream(stream)), "ds4moe_pack_q4k")


def ds4moe_pack_iq2xxs(w: torch.Tensor, grid: torch.Tensor, blocks: torch.Tensor, stream=None):
    _ok(lib().ds4moe_pack_iq2xxs(_ptr(w), w.numel(), _ptr(grid), _ptr(blocks), _stream(stream)),
        "ds4moe_pack_iq2xxs")


def ds4moe_set_grid(h: int, grid: torch.Tensor, stream=None):
    _ok(lib().ds4moe_set_grid(h, _ptr(grid), _stream(stream)), "ds4moe_set_grid")


def ds4moe_set_router(h: int, W: torch.Tensor, bias: torch.Tensor | None = None, stream=None):
    _ok(lib().ds4moe_set_router(h, _ptr(W), _ptr(bias), _stream(stream)), "ds4moe_set_router")


def ds4moe_set_expert(h: int, e: int, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, stream=None):
    _ok(lib().ds4moe_set_expert(h, e, _ptr(gate), _ptr(up), _ptr(down), _stream(stream)), "ds4moe_set_expert")


def ds4moe_set_shared(h: int, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, stream=None):
    _ok(lib().ds4moe_set_shared(h, _ptr(gate), _ptr(up), _ptr(down), _stream(stream)), "ds4moe_set_shared")


def ds4moe_forward(h: int, x: torch.Tensor, out: torch.Tensor, stream=None):
    _ok(lib().ds4moe_forward(h, _ptr(x), x.shape[0], _ptr(out), _stream(stream)), "ds4moe_forward")


def ds4moe_set_steering(h: int, v: torch.Tensor | None, F: float, stream=None):
    _ok(lib().ds4moe_set_steering(h, None if v is None else _ptr(v), ctypes.c_float(F), _stream(stream)),
        "ds4moe_set_steering")


def ds4moe_forward_routed(h: int, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, out: torch.Tensor,
                          stream=None):
    _ok(lib().ds4moe_forward_routed(h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _ptr(out), _stream(stream)),
        "ds4moe_forward_routed")


def ds4moe_combine_slots(y: torch.Tensor, w: torch.Tensor, base: torch.Tensor | None, out: torch.Tensor,
                         stream=None):
    n, k = w.shape
    _ok(lib().ds4moe_combine_slots(_ptr(y), _ptr(w), _ptr(base), n, k, out.shape[1], _ptr(out), _stream(stream)),
        "ds4moe_combine_slots")


def ds4moe_forward_chain(handles, x: torch.Tensor, out: torch.Tensor, work: torch.Tensor, stream=None):
    arr = (ctypes.c_void_p * len(handles))(*handles)
    _ok(lib().ds4moe_forward_chain(arr, len(handles), _ptr(x), x.shape[0], _ptr(out), _ptr(work), _stream(stream)),
        "ds4moe_forward_chain")


def ds4moe_forward_residual(h: int, x: torch.Tensor, out: torch.Tensor, stream=None):
    _ok(lib().ds4moe_forward_residual(h, _ptr(x), x.shape[0], _ptr(out), _stream(stream)), "ds4moe_forward_residual")


def ds4moe_forward_residual_profiled(h: int, x: torch.Tensor, out: torch.Tensor, events, stream=None):
    arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    _ok(lib().ds4moe_forward_residual_profiled(h, _ptr(x), x.shape[0], _ptr(out), arr, _stream(stream)),
        "ds4moe_forward_residual_profiled")


def ds4moe_plan_launches(h: int, n_tokens: int) -> int:
    return lib().ds4moe_plan_launches(h, n_tokens)


def ds4moe_plan_kernel(h: int, n_tokens: int, i: int) -> str | None:
    r = lib().ds4moe_plan_kernel(h, n_tokens, i)
    return None if r is None else r.decode()


def ds4moe_forward_profiled(h: int, x: torch.Tensor, out: torch.Tensor, events, stream=None):
    """events: a flat list of torch.cuda.Event(enable_timing=True), 2 per launch of the plan."""
    arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    _ok(lib().ds4moe_forward_profiled(h, _ptr(x), x.shape[0], _ptr(out), arr, _stream(stream)),
        "ds4moe_forward_profiled")


def ds4moe_forward_host(h: int, x_host: torch.Tensor, out_host: torch.Tensor, stream=None):
    _ok(lib().ds4moe_forward_host(h, _ptr(x_host), x_host.shape[0], _ptr(out_host), _stream(stream)),
        "ds4moe_forward_host")


def ds4moe_forward_host_async(h: int, x_host: torch.Tensor, out_host: torch.Tensor, stream=None):
    """Enqueue a host-buffer forward; out_host is valid after ds4moe_host_sync(h)."""
    _ok(lib().ds4moe_forward_host_async(h, _ptr(x_host), x_host.shape[0], _ptr(out_host), _stream(stream)),
        "ds4moe_forward_host_async")


def ds4moe_host_sync(h: int):
    _ok(lib().ds4moe_host_sync(h), "ds4moe_host_sync")


def ds4moe_route(h: int, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, stream=None):
    _ok(lib().ds4moe_route(h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _stream(stream)), "ds4moe_route")


def ds4moe_route_noalloc(h: int, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, stream=None):
    """Routing with the library's static device scratch instead of the bound workspace.

    For callers that cannot allocate device memory (a host that owns every
    device buffer through its own pool, or code that must not stall the device
    with a synchronizing allocation); the handle needs only its weight buffer
    bound.  Limit: n_tokens * n_experts <= 8192; calls that overlap on the GPU
    race on the shared scratch.
    """
    _ok(lib().ds4moe_route_noalloc(h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _stream(stream)),
        "ds4moe_route_noalloc")


def ds4moe_probe(h: int, plan: int, which: int, e: int, inp: torch.Tensor, out: torch.Tensor, stream=None):
    """Raw accumulators of one plan's projection kernels on caller rows, all routed to expert e (-1: shared)."""
    _ok(lib().ds4moe_probe(h, plan, which, e, _ptr(inp), inp.shape[0], _ptr(out), _stream(stream)), "ds4moe_probe")


def ds4moe_dequant(h: int, e: int, which: int, as_bf16: int, out: torch.Tensor, stream=None):
    _ok(lib().ds4moe_dequant(h, e, which, as_bf16, _ptr(out), _stream(stream)), "ds4moe_dequant")


def ds4moe_permutation(h: int, ids: torch.Tensor, counts: torch.Tensor, offsets: torch.Tensor,
                       pos_of_slot: torch.Tensor, stream=None):
    """The prefill plan's stable counting sort of the (token, slot) pairs of ids [n][k] by expert."""
    _ok(lib().ds4moe_permutation(h, _ptr(ids), ids.shape[0], _ptr(counts), _ptr(offsets), _ptr(pos_of_slot),
                                 _stream(stream)), "ds4moe_permutation")


def ds4moe_selftest_wait(h: int, stream=None):
    """A bounded wait on an mbarrier nothing arrives at: gives up after its limit and sets error bit 1."""
    _ok(lib().ds4moe_selftest_wait(h, _stream(stream)), "ds4moe_selftest_wait")


def ds4moe_get_device_error(h: int, stream=None) -> int:
    code = ctypes.c_int32(0)
    st = lib().ds4moe_get_device_error(h, _stream(stream), ctypes.byref(code))
    if st not in (0, -6, -7):
        _ok(st, "ds4moe_get_device_error")
    return code.value


# ------------------------------------------------------------------ around the layer
_ACT = {torch.float32: DS4MOE_ACT_F32, torch.bfloat16: DS4MOE_ACT_BF16}
_Q8 = {torch.float8_e4m3fn: DS4MOE_Q8_E4M3, torch.int8: DS4MOE_Q8_INT8}


class _NoFast:
    """In place of _fastcall where it was not built, or cannot be loaded: every call goes the long way."""
    add_rmsnorm = widen_rows = project = sample = staticmethod(lambda *args: False)


_fast = None


def _load_fast():
    """_fastcall: checks and call in one step for tensors of the current device on its current stream: True, or
    False (and nothing launched) where a call is not plainly in order, or the status of one that failed behind its
    checks and so is not made again."""
    global _fast
    from .build import fast_path

    path, found = fast_path(), _NoFast
    if os.path.exists(path):
        lib()  # the library that it calls
        try:
            spec = importlib.util.spec_from_file_location("_fastcall", path)
            found = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(found)
        except ImportError as e:
            warnings.warn("%s: %s; the calls that it shortens check in Python" % (os.path.basename(path), e))
            found = _NoFast
    _fast = found
    return _fast


def _refuse(where: str, msg: str):
    raise Ds4MoeError(-1, where, msg)


def _fits(*sizes: int) -> bool:
    """Whether the C entry points' 32-bit sizes hold these (ctypes would cut them off)."""
    return all(-1 << 31 <= s < 1 << 31 for s in sizes)


def _sizes(where: str, *sizes: int):
    if not _fits(*sizes):
        _refuse(where, "sizes %s: one is beyond 32 bits" % (sizes,))


def _tensors(where: str, dev: int, specs):
    """Each (name, tensor or None, shape, types): on CUDA device dev, contiguous, of that shape and one of the types."""
    for _, t, shape, types in specs:
        if t is not None and not (t.dtype in types and t.shape == shape and t.get_device() == dev
                                  and t.is_contiguous()) or dev < 0:
            break
    else:
        return
    given = [s for s in specs if s[1] is not None]
    for name, t, _, types in given:
        if t.dtype not in types:
            _refuse(where, "%s: unsupported type %s" % (name, t.dtype))
    for name, t, shape, _ in given:
        if t.shape != shape:
            _refuse(where, "%s: shape %s, expected %s" % (name, tuple(t.shape), shape))
    for name, t, _, _ in given:
        if dev < 0 or t.get_device() != dev:
            _refuse(where, "%s: on %s, expected one CUDA device for all" % (name, t.device))
    for name, t, _, _ in given:
        if not t.is_contiguous():
            _refuse(where, "%s: not contiguous" % name)


def _call(where: str, dev: int, stream, fn, *args):
    """fn(*args, stream) with device dev current; the default stream is dev's current one."""
    if dev < 0:
        _refuse(where, "expected CUDA tensors")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    else:
        stream = _stream(stream)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    else:
        status = fn(*args, stream)
    if status:
        _ok(status, where)


def _q8_groups(where: str, group: int, hidden: int) -> int:
    if group not in (0, 32, 64, 128):
        _refuse(where, "group %r (0, 32, 64 or 128)" % (group,))
    return -(-hidden // group) if group else 1


def ds4moe_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                       sum: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       q: torch.Tensor | None = None, scale: torch.Tensor | None = None, group: int = 128,
                       stream=None):
    """s = x + residual into ``sum``, its RMS norm times ``weight`` into ``out`` and, as 8-bit codes with one scale
    per ``group`` columns (0: per row), into ``q`` (float8_e4m3fn or int8) and ``scale`` [n, groups].

    x [n, H] and residual binary32 or bf16; ``sum`` of residual's type (it may be residual itself), ``out`` binary32
    or bf16.  Outputs that are None are not written; at least one is needed.
    """
    where = "ds4moe_add_rmsnorm"
    if stream is None:
        done = (_fast or _load_fast()).add_rmsnorm(x, weight, eps, residual, sum, out, q, scale, group)
        if done:
            return None if done is True else _ok(done, where)
    if x.dim() != 2:
        _refuse(where, "x: %d dimensions, expected [n, hidden]" % x.dim())
    n, H = x.shape
    _sizes(where, n, H)
    dev = x.get_device()
    shape = (n, H)
    groups = 1 if q is None and scale is None else _q8_groups(where, group, H)   # (group means nothing without codes)
    _tensors(where, dev, (
        ("x", x, shape, _ACT), ("weight", weight, (H,), (torch.float32,)), ("residual", residual, shape, _ACT),
        ("sum", sum, shape, _ACT if residual is None else (residual.dtype,)), ("out", out, shape, _ACT),
        ("q", q, shape, _Q8),
        ("scale", scale, (n, groups), (torch.float32,))))
    _call(where, dev, stream, lib().ds4moe_add_rmsnorm, x.data_ptr(), _ACT[x.dtype], _ptr(residual),
          0 if residual is None else _ACT[residual.dtype], weight.data_ptr(), eps, n, H, _ptr(sum), _ptr(out),
          0 if out is None else _ACT[out.dtype], _ptr(q), 0 if q is None else _Q8[q.dtype], 0 if q is None else group,
          _ptr(scale))


def ds4moe_widen_rows(q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, group: int = 128, stream=None):
    """out = q * scale: 8-bit rows of ds4moe_add_rmsnorm (codes [n, H], scales [n, groups]) as binary32 or bf16."""
    where = "ds4moe_widen_rows"
    if stream is None:
        done = (_fast or _load_fast()).widen_rows(q, scale, out, group)
        if done:
            return None if done is True else _ok(done, where)
    if q.dim() != 2:
        _refuse(where, "q: %d dimensions, expected [n, hidden]" % q.dim())
    n, H = q.shape
    _sizes(where, n, H)
    dev = q.get_device()
    _tensors(where, dev, (("q", q, (n, H), _Q8),
                               ("scale", scale, (n, _q8_groups(where, group, H)), (torch.float32,)),
                               ("out", out, (n, H), _ACT)))
    _call(where, dev, stream, lib().ds4moe_widen_rows, q.data_ptr(), _Q8[q.dtype], scale.data_ptr(), group, n, H,
          out.data_ptr(), _ACT[out.dtype])


def ds4moe_project_work_bytes(n: int, in_features: int, out_features: int, n_adapters: int, rank: int) -> int:
    sizes = (n, in_features, out_features, n_adapters, rank)
    return lib().ds4moe_project_work_bytes(*sizes) if _fits(*sizes) else 0


def ds4moe_project(x: torch.Tensor, W: torch.Tensor, out: torch.Tensor, A: torch.Tensor | None = None,
                   B: torch.Tensor | None = None, adapter_scale: torch.Tensor | None = None,
                   ids: torch.Tensor | None = None, work: torch.Tensor | None = None, stream=None):
    """out = x W^T, plus adapter_scale[a] B[a] (A[a] x_i) for each row i whose adapter is a = ids[i].

    bf16 x [n, in], W [out, in], A [adapters, rank, in], B [adapters, out, rank], out [n, out]; binary32
    adapter_scale [adapters]; int32 ids [n], -1 for none.  ``work``: uint8 scratch of ds4moe_project_work_bytes
    (allocated here by default).
    """
    where = "ds4moe_project"
    if stream is None and work is None:
        done = (_fast or _load_fast()).project(x, W, out, A, B, adapter_scale, ids)
        if done:
            return None if done is True else _ok(done, where)
    _project(where, lib().ds4moe_project, x, W, out, A, B, adapter_scale, ids, work, stream)


def _project(where, fn, x, W, out, A, B, adapter_scale, ids, work, stream, *more):
    if x.dim() != 2 or W.dim() != 2:
        _refuse(where, "x: expected [n, in], W: [out, in]")
    n, fin = x.shape
    dev = x.get_device()
    fout = W.shape[0]
    bf = (torch.bfloat16,)
    na = rank = wb = 0
    if A is not None:
        if B is None or adapter_scale is None or ids is None or A.dim() != 3:
            _refuse(where, "adapters need A [adapters, rank, in], B, adapter_scale and ids")
        na, rank = A.shape[0], A.shape[1]
    elif B is not None or adapter_scale is not None or ids is not None:
        _refuse(where, "B, adapter_scale and ids need A")
    _sizes(where, n, fin, fout, na, rank)
    _tensors(where, dev, (("x", x, (n, fin), bf), ("W", W, (fout, fin), bf), ("out", out, (n, fout), bf),
                               ("A", A, (na, rank, fin), bf), ("B", B, (na, fout, rank), bf),
                               ("adapter_scale", adapter_scale, (na,), (torch.float32,)),
                               ("ids", ids, (n,), (torch.int32,))))
    if na and n:
        if work is None:
            # of the stream that the call runs on: the allocator then hands it on only behind the call
            need = lib().ds4moe_project_work_bytes(n, fin, fout, na, rank)
            if stream is None:
                work = torch.empty(need, dtype=torch.uint8, device=x.device)
            else:
                with torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=x.device)):
                    work = torch.empty(need, dtype=torch.uint8, device=x.device)
        elif work.get_device() != dev or not work.is_contiguous():
            _refuse(where, "work: contiguous on %s expected" % x.device)
        wb = work.numel() * work.element_size()
    _call(where, dev, stream, fn, x.data_ptr(), n, W.data_ptr(), fin, fout, _ptr(A), _ptr(B), _ptr(adapter_scale), na, rank,
          _ptr(ids), out.data_ptr(), _ptr(work), wb, *more)


def ds4moe_get_project_error(stream=None) -> int:
    code = ctypes.c_int32(0)
    st = lib().ds4moe_get_project_error(_stream(stream), ctypes.byref(code))
    if st not in (0, -6):
        _ok(st, "ds4moe_get_project_error")
    return code.value


def ds4moe_selftest_project_wait(x, W, out, A=None, B=None, adapter_scale=None, ids=None, tiles: int = 0, stream=None):
    """ds4moe_project whose waits give up at once from each CTA's ``tiles``-th tile on: NaN there, and the error word."""
    _sizes("ds4moe_selftest_project_wait", tiles)
    _project("ds4moe_selftest_project_wait", lib().ds4moe_selftest_project_wait, x, W, out, A, B, adapter_scale, ids, None,
             stream, tiles)


def ds4moe_sample(logits: torch.Tensor, u: torch.Tensor, token: torch.Tensor, temperature: torch.Tensor | None = None,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, prob: torch.Tensor | None = None,
                  probs: torch.Tensor | None = None, stream=None):
    """The next token of each row of logits [n, vocab] (binary32 or bf16; rows may be strided) by the uniform
    numbers u [n], after temperature, top-k, top-p and min-p (one value per row each, None: off).

    token [n] int32; prob [n]: the token's probability; probs [n, vocab]: the filtered distribution.
    """
    where = "ds4moe_sample"
    if stream is None:
        done = (_fast or _load_fast()).sample(logits, u, token, temperature, top_k, top_p, min_p, prob, probs)
        if done:
            return None if done is True else _ok(done, where)
    if logits.dim() != 2:
        _refuse(where, "logits: %d dimensions, expected [n, vocab]" % logits.dim())
    n, V = logits.shape
    _sizes(where, n, V)
    dev = logits.get_device()
    if logits.dtype not in _ACT:
        _refuse(where, "logits: unsupported type %s" % logits.dtype)
    if V > 1 and logits.stride(1) != 1:
        _refuse(where, "logits: a row's elements must be next to each other")
    f, one = (torch.float32,), (n,)
    _tensors(where, dev, (("u", u, one, f), ("token", token, one, (torch.int32,)),
                                    ("temperature", temperature, one, f), ("top_k", top_k, one, (torch.int32,)),
                                    ("top_p", top_p, one, f), ("min_p", min_p, one, f), ("prob", prob, one, f),
                                    ("probs", probs, (n, V), f)))
    _call(where, dev, stream, lib().ds4moe_sample, logits.data_ptr(), _ACT[logits.dtype],
          logits.stride(0) if n > 1 else V, n, V, _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
          u.data_ptr(), token.data_ptr(), _ptr(prob), _ptr(probs))


# ------------------------------------------------------------------ plumbing
class MoELayer:
    """One layer's handle plus torch-allocated weight and workspace buffers.

    ``load`` takes a dict with H, I, E, k, W_r, b_r, grid and either packed
    blocks (gate, up: [E, I*H/256, 66] u8; down: [E, H*I/256, 84] u8) or float
    weights to pack on the device (gate_f, up_f: [E, I, H]; down_f: [E, H, I]),
    plus sh_gate/sh_up/sh_down bf16 when has_shared.  With expert_bits=4 all
    three expert matrices are Q4_K-style blocks ([E, n/256, 144] u8) and no
    grid is needed.
    """

    def __init__(self, H, I, E, k, max_tokens, act_dtype=DS4MOE_ACT_F32, has_shared=True, has_bias=False,
                 decode_max=0, device="cuda", expert_bits=0):
        self.H, self.I, self.E, self.k = H, I, E, k
        self.expert_bits = expert_bits
        self.max_tokens = max_tokens
        self.act_dtype = act_dtype
        self.device = torch.device(device)
        self.h = ds4moe_create(H, I, E, k, max_tokens, act_dtype, int(has_shared), int(has_bias), decode_max,
                               expert_bits)
        wb = ds4moe_weight_bytes(self.h)
        sb = ds4moe_workspace_bytes(self.h, max_tokens)
        self.weights = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(sb, dtype=torch.uint8, device=self.device)
        ds4moe_bind(self.h, self.weights, self.workspace)

    def __del__(self):
        h = getattr(self, "h", None)
        if h:
            try:
                ds4moe_destroy(h)
            except Exception:
                pass
            self.h = None

    def pack(self, layer: dict) -> dict:
        """Pack float expert weights with the device quantizers; returns gate/up/down blocks."""
        H, I, E = self.H, self.I, self.E
        dev = self.device
        nb = I * H // 256
        if self.expert_bits == 4:
            blocks = {}
            for name in ("gate", "up", "down"):
                t = torch.empty(E, nb, 144, dtype=torch.uint8, device=dev)
                for e in range(E):
                    ds4moe_pack_q4k(layer[name + "_f"][e].to(dev).contiguous(), t[e])
                blocks[name] = t
            return blocks
        grid = layer["grid"].to(dev).contiguous()
        gate = torch.empty(E, nb, 66, dtype=torch.uint8, device=dev)
        up = torch.empty(E, nb, 66, dtype=torch.uint8, device=dev)
        down = torch.empty(E, nb, 84, dtype=torch.uint8, device=dev)
        for e in range(E):
            ds4moe_pack_iq2xxs(layer["gate_f"][e].to(dev).contiguous(), grid, gate[e])
            ds4moe_pack_iq2xxs(layer["up_f"][e].to(dev).contiguous(), grid, up[e])
            ds4moe_pack_q2k(layer["down_f"][e].to(dev).contiguous(), down[e])
        return dict(gate=gate, up=up, down=down)

    def load(self, layer: dict):
        dev = self.device
        if "gate" not in layer:
            layer = {**layer, **self.pack(layer)}
        if layer.get("grid") is not None:
            ds4moe_set_grid(self.h, layer["grid"].to(dev).contiguous())
        b = layer.get("b_r")
        ds4moe_set_router(self.h, layer["W_r"].to(dev).contiguous(), None if b is None else b.to(dev).contiguous())
        for e in range(self.E):
            ds4moe_set_expert(self.h, e, layer["gate"][e].to(dev).contiguous(), layer["up"][e].to(dev).contiguous(),
                              layer["down"][e].to(dev).contiguous())
        if layer.get("sh_gate") is not None:
            ds4moe_set_shared(self.h, layer["sh_gate"].to(dev).contiguous(), layer["sh_up"].to(dev).contiguous(),
                              layer["sh_down"].to(dev).contiguous())
        torch.cuda.current_stream(dev).synchronize()
        return layer

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, residual: bool = False) -> torch.Tensor:
        """The layer on x; with residual=True, x + the layer (x and out must not overlap)."""
        if out is None:
            out = torch.empty(x.shape[0], self.H, dtype=torch.float32, device=x.device)
        (ds4moe_forward_residual if residual else ds4moe_forward)(self.h, x, out)
        return out

    def set_steering(self, v: torch.Tensor | None, F: float = 1.0):
        """Steer the layer output: y -= F v (v . y) (v: [H] binary32 on the device; None turns it off)."""
        ds4moe_set_steering(self.h, v, F)

    def route(self, x: torch.Tensor):
        ids = torch.empty(x.shape[0], self.k, dtype=torch.int32, device=x.device)
        w = torch.empty(x.shape[0], self.k, dtype=torch.float32, device=x.device)
        ds4moe_route(self.h, x, ids, w)
        return ids, w

    def dequant(self, e: int, which: int, as_bf16: bool = False) -> torch.Tensor:
        rows, cols = (self.H, self.I) if which == 2 else (self.I, self.H)
        out = torch.empty(rows, cols, dtype=torch.bfloat16 if as_bf16 else torch.float32, device=self.device)
        ds4moe_dequant(self.h, e, which, int(as_bf16), out)
        return out
