"""Thin Python binding of libq4moe (ctypes).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libq4moe.so``. PyTorch supplies device memory and the current
HIP stream. The library must have been built (``moe_experts_amd.build``);
importing this module fails loudly if it is missing - there is no fallback.

The functions carry the names of the C entry points in ``include/q4moe.h``.
Before any call reaches the library, the binding checks that every tensor is a
contiguous device tensor of the dtype and number of elements the shape
arguments imply, so a mismatched tensor can never be read or written out of
bounds by a kernel.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq4moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m moe_experts_amd.build` "
        "(the Q4_0 kernels have no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_lib.q4_strerror.restype = ctypes.c_char_p
_lib.q4_strerror.argtypes = [_I]
_lib.q4_0_gemv_workspace_bytes.restype = _Z
_lib.q4_0_gemv_workspace_bytes.argtypes = [_I, _I, _I]
_lib.q4_0_gemv.restype = _I
_lib.q4_0_gemv.argtypes = [_P, _P, _P, _I, _I, _I, _P, _Z, _P]
_lib.q4_0_gemv_noalloc.restype = _I
_lib.q4_0_gemv_noalloc.argtypes = [_P, _P, _P, _I, _I, _I, _P]
_lib.q8_0_gemv_workspace_bytes.restype = _Z
_lib.q8_0_gemv_workspace_bytes.argtypes = [_I, _I, _I]
_lib.q8_0_gemv.restype = _I
_lib.q8_0_gemv.argtypes = [_P, _P, _P, _I, _I, _I, _P, _Z, _P]
_lib.q4_0_gemm.restype = _I
_lib.q4_0_gemm.argtypes = [_P, _P, _P, _I, _I, _I, _P]
_lib.moe_q4_0_workspace_bytes.restype = _Z
_lib.moe_q4_0_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
_lib.moe_q4_0_decode.restype = _I
_lib.moe_q4_0_decode.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]
_lib.moe_q4_0_prefill_workspace_bytes.restype = _Z
_lib.moe_q4_0_prefill_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
_lib.moe_q4_0_prefill.restype = _I
_lib.moe_q4_0_prefill.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]
_lib.moe_router_workspace_bytes.restype = _Z
_lib.moe_router_workspace_bytes.argtypes = [_I, _I, _I]
_lib.moe_router_topk.restype = _I
_lib.moe_router_topk.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]
_lib.moe_q4_0_layer_workspace_bytes.restype = _Z
_lib.moe_q4_0_layer_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.moe_q4_0_layer.restype = _I
_lib.moe_q4_0_layer.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z, _P]

_lib.moe_q4_0_route_layout.restype = _I
_lib.moe_q4_0_route_layout.argtypes = [_I, _I, _I, _I, _I, ctypes.POINTER(_Z), ctypes.POINTER(_Z),
                                       ctypes.POINTER(_Z)]

_lib.moe_q4_0_prefill_route_layout.restype = _I
_lib.moe_q4_0_prefill_route_layout.argtypes = [_I, _I, _I, _I, _I] + [ctypes.POINTER(_Z)] * 4

for _name, _ints in (("q4_0_glu", 3), ("q4_0_glu_gemm", 3), ("q4_0_glu_backward", 3),
                     ("q4_0_gemm_backward", 3), ("q4_0_gemv_lora", 4), ("q4_0_gemm_lora", 4)):
    _f = getattr(_lib, _name + "_workspace_bytes")
    _f.restype = _Z
    _f.argtypes = [_I] * _ints
_lib.q4_0_glu.restype = _I
_lib.q4_0_glu.argtypes = [_P] * 4 + [_I] * 4 + [_P, _Z, _P]
_lib.q4_0_glu_gemm.restype = _I
_lib.q4_0_glu_gemm.argtypes = [_P] * 6 + [_I] * 4 + [_P, _Z, _P]
_lib.q4_0_glu_backward.restype = _I
_lib.q4_0_glu_backward.argtypes = [_P] * 6 + [_I] * 4 + [_P, _Z, _P]
_lib.q4_0_gemm_backward.restype = _I
_lib.q4_0_gemm_backward.argtypes = [_P] * 3 + [_I] * 3 + [_P, _Z, _P]
for _f in (_lib.q4_0_gemv_lora, _lib.q4_0_gemm_lora):
    _f.restype = _I
    _f.argtypes = [_P] * 7 + [_I] * 5 + [_P, _Z, _P]

_lib.q4_0_ffn_plan.restype = _I
_lib.q4_0_ffn_plan.argtypes = [_I] * 4 + [ctypes.POINTER(_I)] * 3

BLOCK_BYTES = 18
Q8_BLOCK_BYTES = 34


class Q4Error(RuntimeError):
    """A non-zero status returned by libq4moe."""

    def __init__(self, status: int):
        self.status = status
        super().__init__(f"libq4moe status {status}: {q4_strerror(status)}")


def q4_strerror(status: int) -> str:
    return _lib.q4_strerror(int(status)).decode()


def _check(rc: int):
    if rc != 0:
        raise Q4Error(rc)


def _raw_stream(index: int) -> int:
    """Handle of the current stream of a device, without building a Stream object."""
    return torch._C._cuda_getCurrentRawStream(index)


def _stream(device) -> int:
    return _raw_stream(device.index)


def _dev(t: torch.Tensor, name: str, dtype, numel: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


# Workspaces: one scratch buffer per host thread, device and stream, grown on
# demand. The calls of one thread on one stream run in order, so they can share
# it; two threads cannot, even on one stream: a call enqueues several kernels that
# hand partial sums over, without the interpreter's lock, and another thread's
# kernels may come between them. A thread's buffers go when it ends; the memory
# belongs to the stream it was taken on, so kernels still in flight there keep it. A
# call that is being captured takes memory of its own from the graph's pool
# instead: graphs that are replayed at the same time must not share scratch memory,
# and a graph must not depend on a buffer that a later, larger call replaces.
class _Workspaces(threading.local):
    def __init__(self):
        self.buffers: dict = {}  # (device index, stream handle): tensor


_workspaces = _Workspaces()

# A capture that was not begun through torch (hipStreamBeginCapture) gets ordinary
# memory, which torch would give to others while the graph still writes to it, and
# nothing says when that graph ends: such workspaces are kept until the process
# ends. A caller that minds passes ws.
_captured: list = []


def _of_a_graph_pool(address: int, index: int) -> bool:
    """Whether torch's allocator has this memory in a pool of its own, as it has a graph's."""
    for s in torch.cuda.memory_snapshot():
        if s["device"] == index and s["address"] <= address < s["address"] + s["total_size"]:
            return tuple(s["segment_pool_id"]) != (0, 0)
    return False


def workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    index = torch.device(device).index
    if index is not None and index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return workspace(nbytes, device)
    if index is None:
        index = torch.cuda.current_device()
    return _workspace(nbytes, index, _raw_stream(index))


def _workspace(nbytes: int, index: int, stream: int) -> torch.Tensor:
    """`index` is the current device: what is asked is whether its stream is being captured."""
    if torch._C._cuda_isCurrentStreamCapturing():
        buf = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
        if not _of_a_graph_pool(buf.data_ptr(), index):
            _captured.append(buf)
        return buf
    buffers = _workspaces.buffers
    key = (index, stream)
    buf = buffers.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = buffers[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8,
                                         device=torch.device("cuda", index))
    return buf


def q4_0_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_0_gemv_workspace_bytes(M, N, K))


def moe_q4_0_workspace_bytes(T: int, H: int, I: int, E: int, topk: int) -> int:
    return int(_lib.moe_q4_0_workspace_bytes(T, H, I, E, topk))


def q4_0_gemv(x: torch.Tensor, B: torch.Tensor, N: int, y: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = x[M, K] . deq(B) for a Q4_0 matrix B (uint8, K*(N/32)*18 bytes)."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    if N <= 0 or N % 32:
        raise ValueError("N must be a positive multiple of 32")
    px = _dev(x, "x", torch.float32, M * K)
    pb = _dev(B, "B", torch.uint8, K * (N // 32) * BLOCK_BYTES)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    py = _dev(y, "y", torch.float32, M * N)
    need = q4_0_gemv_workspace_bytes(M, N, K)
    if ws is None:
        ws = workspace(need, x.device)
    pw, nw = (None, 0) if ws is None else (_dev(ws, "ws", torch.uint8, ws.numel()), ws.numel())
    _check(_lib.q4_0_gemv(px, pb, py, M, N, K, pw, nw, _stream(x.device)))
    return y


# Largest q4_0_gemv workspace q4_0_gemv_noalloc serves from its static array.
GEMV_NOALLOC_MAX_WS = 16 << 20


def q4_0_gemv_noalloc(x: torch.Tensor, B: torch.Tensor, N: int,
                      y: torch.Tensor) -> torch.Tensor:
    """q4_0_gemv into a caller-provided y without any device allocation: the
    K-split partials live in the library's static per-GPU array."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    if N <= 0 or N % 32:
        raise ValueError("N must be a positive multiple of 32")
    px = _dev(x, "x", torch.float32, M * K)
    pb = _dev(B, "B", torch.uint8, K * (N // 32) * BLOCK_BYTES)
    py = _dev(y, "y", torch.float32, M * N)
    _check(_lib.q4_0_gemv_noalloc(px, pb, py, M, N, K, _stream(x.device)))
    return y


def q8_0_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q8_0_gemv_workspace_bytes(M, N, K))


def q8_0_gemv(x: torch.Tensor, B: torch.Tensor, N: int, y: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = x[M, K] . deq(B) for a Q8_0 matrix B (uint8, K*(N/32)*34 bytes)."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    if N <= 0 or N % 32:
        raise ValueError("N must be a positive multiple of 32")
    px = _dev(x, "x", torch.float32, M * K)
    pb = _dev(B, "B", torch.uint8, K * (N // 32) * Q8_BLOCK_BYTES)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    py = _dev(y, "y", torch.float32, M * N)
    pw, nw = _ws_arg(ws, q8_0_gemv_workspace_bytes(M, N, K), x.device)
    _check(_lib.q8_0_gemv(px, pb, py, M, N, K, pw, nw, _stream(x.device)))
    return y


def q4_0_gemm(X: torch.Tensor, B: torch.Tensor, N: int, Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[M, N] = X[M, K] (float16) . deq(B) with fp32 accumulation, on MFMA."""
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M, K = X.shape
    if N <= 0 or N % 32:
        raise ValueError("N must be a positive multiple of 32")
    px = _dev(X, "X", torch.float16, M * K)
    pb = _dev(B, "B", torch.uint8, K * (N // 32) * BLOCK_BYTES)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    py = _dev(Y, "Y", torch.float32, M * N)
    _check(_lib.q4_0_gemm(px, pb, py, M, N, K, _stream(X.device)))
    return Y


def moe_q4_0_decode(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
                    topk_ids: torch.Tensor, topk_w: torch.Tensor, I: int, E: int,
                    out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Routed-expert MoE decode; x [T, H] fp32, ids/weights [T, topk]."""
    if x.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("x must be [T, H] and topk_ids [T, topk]")
    T, H = x.shape
    topk = topk_ids.shape[1]
    mat = H * (I // 32) * BLOCK_BYTES
    px = _dev(x, "x", torch.float32, T * H)
    pg = _dev(Wg, "Wg", torch.uint8, E * mat)
    pu = _dev(Wu, "Wu", torch.uint8, E * mat)
    pd = _dev(Wd, "Wd", torch.uint8, E * mat)
    pi = _dev(topk_ids, "topk_ids", torch.int32, T * topk)
    pw_ = _dev(topk_w, "topk_w", torch.float32, T * topk)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=x.device)
    po = _dev(out, "out", torch.float32, T * H)
    need = moe_q4_0_workspace_bytes(T, H, I, E, topk)
    if ws is None:
        ws = workspace(need, x.device)
    pws, nws = (None, 0) if ws is None else (_dev(ws, "ws", torch.uint8, ws.numel()), ws.numel())
    _check(_lib.moe_q4_0_decode(px, pg, pu, pd, pi, pw_, po, T, H, I, E, topk, pws, nws,
                                _stream(x.device)))
    return out


def moe_q4_0_route_layout(T: int, H: int, I: int, E: int, topk: int):
    """Byte offsets (items, counts, mitems) of the routing table that
    moe_q4_0_decode leaves in its workspace (T >= 2)."""
    a, b, c = _Z(), _Z(), _Z()
    _check(_lib.moe_q4_0_route_layout(T, H, I, E, topk, ctypes.byref(a), ctypes.byref(b),
                                      ctypes.byref(c)))
    return a.value, b.value, c.value


def moe_q4_0_prefill_route_layout(T: int, H: int, I: int, E: int, topk: int):
    """Byte offsets (src, pos, tiles, counts) of the routing that
    moe_q4_0_prefill leaves in its workspace."""
    o = [_Z() for _ in range(4)]
    _check(_lib.moe_q4_0_prefill_route_layout(T, H, I, E, topk, *[ctypes.byref(v) for v in o]))
    return tuple(v.value for v in o)


def moe_router_workspace_bytes(T: int, H: int, E: int) -> int:
    return int(_lib.moe_router_workspace_bytes(T, H, E))


def moe_q4_0_layer_workspace_bytes(T: int, H: int, I: int, E: int, topk: int,
                                   n_shared: int) -> int:
    return int(_lib.moe_q4_0_layer_workspace_bytes(T, H, I, E, topk, n_shared))


def _ws_arg(ws, need: int, device):
    if ws is None:
        ws = workspace(need, device)
    return (None, 0) if ws is None else (_dev(ws, "ws", torch.uint8, ws.numel()), ws.numel())


def moe_router_topk(x: torch.Tensor, Wr: torch.Tensor, topk: int, n_shared: int = 0,
                    ws: torch.Tensor | None = None, logits: torch.Tensor | None = None,
                    ids: torch.Tensor | None = None, w: torch.Tensor | None = None):
    """MoE router: x [T, H] fp32, Wr [E, H] fp32. Returns (logits [T, E],
    topk_ids int32 [T, topk + n_shared], topk_w fp32 [T, topk + n_shared]),
    written into the given tensors when passed."""
    if x.dim() != 2 or Wr.dim() != 2:
        raise ValueError("x must be [T, H] and Wr [E, H]")
    T, H = x.shape
    E = Wr.shape[0]
    px = _dev(x, "x", torch.float32, T * H)
    pr = _dev(Wr, "Wr", torch.float32, E * H)
    slots = topk + n_shared
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    if ids is None:
        ids = torch.empty((T, slots), dtype=torch.int32, device=x.device)
    if w is None:
        w = torch.empty((T, slots), dtype=torch.float32, device=x.device)
    pl = _dev(logits, "logits", torch.float32, T * E)
    pi = _dev(ids, "ids", torch.int32, T * slots)
    pwt = _dev(w, "w", torch.float32, T * slots)
    pws, nws = _ws_arg(ws, moe_router_workspace_bytes(T, H, E), x.device)
    _check(_lib.moe_router_topk(px, pr, pl, pi, pwt, T, H, E, topk, n_shared, pws, nws,
                                _stream(x.device)))
    return logits, ids, w


def moe_q4_0_layer(x: torch.Tensor, Wr: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                   Wd: torch.Tensor, I: int, topk: int, n_shared: int = 0,
                   out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Router, then routed and shared experts: x [T, H] fp32, Wr [E, H] fp32, and
    Wg/Wu/Wd holding E + n_shared Q4_0 expert matrices (routed, then shared)."""
    if x.dim() != 2 or Wr.dim() != 2:
        raise ValueError("x must be [T, H] and Wr [E, H]")
    T, H = x.shape
    E = Wr.shape[0]
    mat = H * (I // 32) * BLOCK_BYTES
    px = _dev(x, "x", torch.float32, T * H)
    pr = _dev(Wr, "Wr", torch.float32, E * H)
    pg = _dev(Wg, "Wg", torch.uint8, (E + n_shared) * mat)
    pu = _dev(Wu, "Wu", torch.uint8, (E + n_shared) * mat)
    pd = _dev(Wd, "Wd", torch.uint8, (E + n_shared) * mat)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=x.device)
    po = _dev(out, "out", torch.float32, T * H)
    pws, nws = _ws_arg(ws, moe_q4_0_layer_workspace_bytes(T, H, I, E, topk, n_shared), x.device)
    _check(_lib.moe_q4_0_layer(px, pr, pg, pu, pd, po, T, H, I, E, topk, n_shared, pws, nws,
                               _stream(x.device)))
    return out


def moe_q4_0_prefill_workspace_bytes(T: int, H: int, I: int, E: int, topk: int) -> int:
    return int(_lib.moe_q4_0_prefill_workspace_bytes(T, H, I, E, topk))


def moe_q4_0_prefill(x16: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
                     topk_ids: torch.Tensor, topk_w: torch.Tensor, I: int, E: int,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Routed-expert MoE at prefill on the matrix cores; x16 [T, H] float16,
    ids/weights [T, topk]."""
    if x16.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("x16 must be [T, H] and topk_ids [T, topk]")
    T, H = x16.shape
    topk = topk_ids.shape[1]
    mat = H * (I // 32) * BLOCK_BYTES
    px = _dev(x16, "x16", torch.float16, T * H)
    pg = _dev(Wg, "Wg", torch.uint8, E * mat)
    pu = _dev(Wu, "Wu", torch.uint8, E * mat)
    pd = _dev(Wd, "Wd", torch.uint8, E * mat)
    pi = _dev(topk_ids, "topk_ids", torch.int32, T * topk)
    pw_ = _dev(topk_w, "topk_w", torch.float32, T * topk)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=x16.device)
    po = _dev(out, "out", torch.float32, T * H)
    pws, nws = _ws_arg(ws, moe_q4_0_prefill_workspace_bytes(T, H, I, E, topk), x16.device)
    _check(_lib.moe_q4_0_prefill(px, pg, pu, pd, pi, pw_, po, T, H, I, E, topk, pws, nws,
                                 _stream(x16.device)))
    return out


# ---------------------------------------------------------------------------
# Dense feed-forward over frozen Q4_0 weights. These calls take a few
# microseconds of GPU time at decode, so their host side is kept short: one
# check per tensor, workspace sizes remembered by shape. Gradients are calls of
# their own; torch's autograd sees none of them.
# ---------------------------------------------------------------------------
ACTIVATIONS = {"silu": 0, "gelu": 1}


def _act(act: str) -> int:
    a = ACTIVATIONS.get(act)
    if a is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)} (got {act!r})")
    return a


def _ptr(t, name: str, dtype, numel: int, index: int) -> int:
    """Address of a contiguous tensor of this type and size on device `index`. These calls record
    nothing for torch's autograd: on a tensor that requires a gradient their results would
    quietly have none, so that is refused while torch records."""
    if (isinstance(t, torch.Tensor) and t.get_device() == index >= 0 and t.dtype is dtype
            and t.numel() == numel and t.is_contiguous() and not t.requires_grad):
        return t.data_ptr()
    if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: call it "
                         "under torch.no_grad(), or in the forward or backward of a "
                         "torch.autograd.Function")
    p = _dev(t, name, dtype, numel)
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the first argument on device {index}")
    return p


def _columns(N: int, block: int):
    if N <= 0 or N % block:
        raise ValueError(f"N must be a positive multiple of {block}")


def _run(f, need: int, ws, index: int, *args):
    """Call f(*args, workspace, its size, stream) on device `index`, which need not be the
    current one."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _run(f, need, ws, index, *args)
    stream = _raw_stream(index)
    p, n = None, 0
    if ws is not None:
        n = ws.numel()
        p = _ptr(ws, "ws", torch.uint8, n, index)
    elif need:
        ws = _workspace(need, index, stream)
        p, n = ws.data_ptr(), ws.numel()
    rc = f(*args, p, n, stream)
    if rc != 0:
        raise Q4Error(rc)


@functools.lru_cache(maxsize=1024)
def q4_0_glu_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_0_glu_workspace_bytes(M, N, K))


@functools.lru_cache(maxsize=1024)
def q4_0_glu_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_0_glu_gemm_workspace_bytes(M, N, K))


@functools.lru_cache(maxsize=1024)
def q4_0_glu_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_0_glu_backward_workspace_bytes(M, N, K))


@functools.lru_cache(maxsize=1024)
def q4_0_gemm_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_0_gemm_backward_workspace_bytes(M, N, K))


@functools.lru_cache(maxsize=1024)
def q4_0_gemv_lora_workspace_bytes(M: int, N: int, K: int, R: int) -> int:
    return int(_lib.q4_0_gemv_lora_workspace_bytes(M, N, K, R))


@functools.lru_cache(maxsize=1024)
def q4_0_gemm_lora_workspace_bytes(M: int, N: int, K: int, R: int) -> int:
    return int(_lib.q4_0_gemm_lora_workspace_bytes(M, N, K, R))


#: Calls whose kernel q4_0_ffn_plan tells.
FFN_FORMS = {"q4_0_glu_gemm": 0, "q4_0_glu_backward": 1, "q4_0_gemm_backward": 2,
             "q4_0_gemm_lora": 3}


def q4_0_ffn_plan(form: str, M: int, N: int, K: int):
    """(rows of a GEMM tile, or 0 for the strips of few rows; splits of the contraction; K steps
    of a split) by which the call `form` serves a shape."""
    if form not in FFN_FORMS:
        raise ValueError(f"form must be one of {sorted(FFN_FORMS)} (got {form!r})")
    rows, splits, steps = _I(), _I(), _I()
    _check(_lib.q4_0_ffn_plan(FFN_FORMS[form], M, N, K, ctypes.byref(rows), ctypes.byref(splits),
                              ctypes.byref(steps)))
    return rows.value, splits.value, steps.value


def q4_0_glu(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, N: int, act: str = "silu",
             h: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """h[M, N] = act(x . deq(Wg)) * (x . deq(Wu)) for x [M, K] fp32, M <= 8, and two Q4_0
    matrices; act "silu" or "gelu" (tanh form)."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    _columns(N, 32)
    mat = K * (N // 32) * BLOCK_BYTES
    a = _act(act)
    i = x.get_device()
    px = _ptr(x, "x", torch.float32, M * K, i)
    pg = _ptr(Wg, "Wg", torch.uint8, mat, i)
    pu = _ptr(Wu, "Wu", torch.uint8, mat, i)
    if h is None:
        h = x.new_empty((M, N), dtype=torch.float32)
    ph = _ptr(h, "h", torch.float32, M * N, i)
    _run(_lib.q4_0_glu, q4_0_glu_workspace_bytes(M, N, K), ws, i, px, pg, pu, ph, M, N, K, a)
    return h


def q4_0_glu_gemm(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, N: int, act: str = "silu",
                  H: torch.Tensor | None = None, G: torch.Tensor | None = None,
                  U: torch.Tensor | None = None, save: bool = False,
                  ws: torch.Tensor | None = None):
    """H[M, N] = act(X . deq(Wg)) * (X . deq(Wu)), fp16 in and out, any M; K and N multiples of
    64. With save, or with G and U given, also returns g = X . deq(Wg) and u = X . deq(Wu) as
    fp16: (H, G, U), what q4_0_glu_backward reads."""
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M, K = X.shape
    _columns(N, 64)
    mat = K * (N // 32) * BLOCK_BYTES
    a = _act(act)
    if (G is None) != (U is None):
        raise ValueError("G and U are given together")
    i = X.get_device()
    px = _ptr(X, "X", torch.float16, M * K, i)
    pg = _ptr(Wg, "Wg", torch.uint8, mat, i)
    pu = _ptr(Wu, "Wu", torch.uint8, mat, i)
    if H is None:
        H = X.new_empty((M, N), dtype=torch.float16)
    if save and G is None:
        G = X.new_empty((M, N), dtype=torch.float16)
        U = X.new_empty((M, N), dtype=torch.float16)
    ph = _ptr(H, "H", torch.float16, M * N, i)
    pG = pU = None
    if G is not None:
        pG = _ptr(G, "G", torch.float16, M * N, i)
        pU = _ptr(U, "U", torch.float16, M * N, i)
    _run(_lib.q4_0_glu_gemm, q4_0_glu_gemm_workspace_bytes(M, N, K), ws, i, px, pg, pu, ph, pG, pU,
         M, N, K, a)
    return H if G is None else (H, G, U)


def q4_0_glu_backward(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor, Wg: torch.Tensor,
                      Wu: torch.Tensor, K: int, act: str = "silu",
                      dX: torch.Tensor | None = None,
                      ws: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of q4_0_glu_gemm with respect to X: dX [M, K] bf16 from dH [M, N] bf16 and the
    G and U that the forward call returned. The weights have no gradient. torch casts what a
    torch.autograd.Function returns to its input's type: for a float16 X the caller scales the
    loss, or keeps what is trained in bfloat16 or float32 and casts it before the call."""
    if dH.dim() != 2:
        raise ValueError("dH must be [M, N]")
    M, N = dH.shape
    _columns(N, 64)
    mat = K * (N // 32) * BLOCK_BYTES
    a = _act(act)
    i = dH.get_device()
    pd = _ptr(dH, "dH", torch.bfloat16, M * N, i)
    pG = _ptr(G, "G", torch.float16, M * N, i)
    pU = _ptr(U, "U", torch.float16, M * N, i)
    pg = _ptr(Wg, "Wg", torch.uint8, mat, i)
    pu = _ptr(Wu, "Wu", torch.uint8, mat, i)
    if dX is None:
        dX = dH.new_empty((M, K), dtype=torch.bfloat16)
    px = _ptr(dX, "dX", torch.bfloat16, M * K, i)
    _run(_lib.q4_0_glu_backward, q4_0_glu_backward_workspace_bytes(M, N, K), ws, i, pd, pG, pU, pg,
         pu, px, M, N, K, a)
    return dX


def q4_0_gemm_backward(dY: torch.Tensor, B: torch.Tensor, K: int, dX: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of Y = X . deq(B) with respect to X: dX [M, K] bf16 from dY [M, N] bf16."""
    if dY.dim() != 2:
        raise ValueError("dY must be [M, N]")
    M, N = dY.shape
    _columns(N, 64)
    i = dY.get_device()
    pd = _ptr(dY, "dY", torch.bfloat16, M * N, i)
    pb = _ptr(B, "B", torch.uint8, K * (N // 32) * BLOCK_BYTES, i)
    if dX is None:
        dX = dY.new_empty((M, K), dtype=torch.bfloat16)
    px = _ptr(dX, "dX", torch.bfloat16, M * K, i)
    _run(_lib.q4_0_gemm_backward, q4_0_gemm_backward_workspace_bytes(M, N, K), ws, i, pd, pb, px,
         M, N, K)
    return dX


def _lora(f, need, x, B, N, A, Bl, ids, scale, y, ws, dtype, block, names):
    if x.dim() != 2 or A.dim() != 3:
        raise ValueError(f"{names[0]} must be [M, K] and A [L, R, K]")
    M, K = x.shape
    L, R, _ = A.shape
    _columns(N, block)
    i = x.get_device()
    px = _ptr(x, names[0], dtype, M * K, i)
    pb = _ptr(B, "B", torch.uint8, K * (N // 32) * BLOCK_BYTES, i)
    pA = _ptr(A, "A", torch.float16, L * R * K, i)
    pB = _ptr(Bl, "Bl", torch.float16, L * N * R, i)
    pi = _ptr(ids, "ids", torch.int32, M, i)
    ps = _ptr(scale, "scale", torch.float32, L, i)
    if y is None:
        y = x.new_empty((M, N), dtype=dtype)
    py = _ptr(y, names[1], dtype, M * N, i)
    _run(f, need(M, N, K, R), ws, i, px, pb, pA, pB, pi, ps, py, M, N, K, R, L)
    return y


def q4_0_gemv_lora(x: torch.Tensor, B: torch.Tensor, N: int, A: torch.Tensor, Bl: torch.Tensor,
                   ids: torch.Tensor, scale: torch.Tensor, y: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[m] = x[m] . deq(B) + scale[i] * (x[m] . A[i]^T) . Bl[i]^T with i = ids[m]: one of L
    adapters (A [L, R, K], Bl [L, N, R], fp16) for each row, none where ids[m] is outside
    [0, L). x and y fp32, M <= 8."""
    return _lora(_lib.q4_0_gemv_lora, q4_0_gemv_lora_workspace_bytes, x, B, N, A, Bl, ids, scale,
                 y, ws, torch.float32, 32, ("x", "y"))


def q4_0_gemm_lora(X: torch.Tensor, B: torch.Tensor, N: int, A: torch.Tensor, Bl: torch.Tensor,
                   ids: torch.Tensor, scale: torch.Tensor, Y: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """q4_0_gemv_lora for any number of rows, X and Y fp16; K and N multiples of 64."""
    return _lora(_lib.q4_0_gemm_lora, q4_0_gemm_lora_workspace_bytes, X, B, N, A, Bl, ids, scale,
                 Y, ws, torch.float16, 64, ("X", "Y"))
