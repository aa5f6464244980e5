"""Thin Python binding of ``libmok.so`` (see ``include/mok.h``): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module only checks tensor
dtypes / devices / contiguity, passes ``data_ptr()``s and the current CUDA stream, and turns
status codes into exceptions.  PyTorch provides device memory and streams.

Importing this module loads the library and raises ``ImportError`` when it is missing; the norm,
dropout and feed-forward calls go through a compiled module beside it and raise ``ImportError``
without it.  There is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import sys
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmok.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libmok.so not found at {LIB_PATH}; build it with __graft_entry__.build() "
                      "(nvcc, sm_103a). There is no CPU fallback.")
_lib = ctypes.CDLL(LIB_PATH)


class _MissingBinding:
    """In place of the compiled binding of the norm, dropout and feed-forward calls where it cannot be loaded: the routed
    layer does without it, those calls raise."""

    def __init__(self, why: Exception):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs _mok_bind.so beside libmok.so; build it with __graft_entry__.build()") from self._why


try:
    from . import _mok_bind as _bind  # built beside libmok.so, which it calls
    _here = f"torch {torch.__version__}, python {sys.version_info.major}.{sys.version_info.minor}"
    _for = getattr(_bind, "built_for", "another torch or Python")
    if _for != _here:  # what it has inlined of torch may not match
        raise ImportError(f"_mok_bind.so is built for {_for}, this is {_here}")
except ImportError as e:
    _bind = _MissingBinding(e)

MOK_OK = 0
MOK_ERR_INVALID_ARG = 1
MOK_ERR_UNSUPPORTED = 2
MOK_ERR_WORKSPACE_TOO_SMALL = 3
MOK_ERR_CUDA = 4
MOK_ERR_BAD_EXPERT_ID = 5
MOK_ERR_CAPACITY = 6
MOK_ERR_TIMEOUT = 7
MOK_BF16 = 0
MOK_MXFP8 = 1


class MokError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = _lib.mok_status_string(code).decode()
        super().__init__(f"{where}: {msg} (status {code})")


class mok_config(ctypes.Structure):
    _fields_ = [("minibatch_rows", ctypes.c_int32), ("macrobatch_rows", ctypes.c_int32),
                ("num_ctas", ctypes.c_int32), ("precision", ctypes.c_int32), ("debug_flags", ctypes.c_uint32)]


class mok_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32)]


_P = ctypes.c_void_p


class mok_schedule(ctypes.Structure):
    _fields_ = [("shape", mok_shape), ("config", mok_config), ("rpad_max", ctypes.c_int64),
                ("tiles_max", ctypes.c_int64), ("mblocks_max", ctypes.c_int64), ("counts", _P), ("offsets", _P),
                ("poff", _P), ("perm", _P), ("inv", _P), ("tiles", _P), ("mblocks", _P), ("meta", _P),
                ("row_weight", _P), ("row_token", _P), ("status", _P), ("topk_weights", _P), ("ws", _P),
                ("ws_bytes", ctypes.c_size_t)]


MX_KEYS = ("q_gate", "s_gate", "q_up", "s_up", "q_down", "s_down",
           "qt_gate", "st_gate", "qt_up", "st_up", "qt_down", "st_down")


class mok_weights(ctypes.Structure):
    _fields_ = [("w_gate", _P), ("w_up", _P), ("w_down", _P)] + [(k, _P) for k in MX_KEYS]


class mok_grads(ctypes.Structure):
    _fields_ = [("dx", _P), ("dw_gate", _P), ("dw_up", _P), ("dw_down", _P), ("d_topk_weights", _P)]


_lib.mok_version.restype = ctypes.c_char_p
_lib.mok_version.argtypes = []
_lib.mok_status_string.restype = ctypes.c_char_p
_lib.mok_status_string.argtypes = [ctypes.c_int]
_lib.mok_workspace_bytes.restype = ctypes.c_size_t
_lib.mok_workspace_bytes.argtypes = [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape)]
_lib.mok_fwd_ctx_bytes.restype = ctypes.c_size_t
_lib.mok_fwd_ctx_bytes.argtypes = [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape)]
_lib.mok_mxfp8_quantize.restype = ctypes.c_int
_lib.mok_mxfp8_quantize.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P]
_lib.mok_build_schedule.restype = ctypes.c_int
_lib.mok_build_schedule.argtypes = [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, _P, _P,
                                    ctypes.c_size_t, ctypes.POINTER(mok_schedule), _P]
_lib.mok_forward.restype = ctypes.c_int
_lib.mok_forward.argtypes = [ctypes.POINTER(mok_schedule), _P, ctypes.POINTER(mok_weights), _P, _P,
                             ctypes.c_size_t, _P]
_lib.mok_backward.restype = ctypes.c_int
_lib.mok_backward.argtypes = [ctypes.POINTER(mok_schedule), _P, _P, ctypes.POINTER(mok_weights),
                              ctypes.POINTER(mok_grads), _P]


class mok_trace(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)), ("kinds", ctypes.POINTER(ctypes.c_int32)),
                ("capacity", ctypes.c_int32), ("count", ctypes.c_int32)]


_lib.mok_set_trace.restype = ctypes.c_int
_lib.mok_set_trace.argtypes = [ctypes.POINTER(mok_trace)]
_lib.mok_kernel_name.restype = ctypes.c_char_p
_lib.mok_kernel_name.argtypes = [ctypes.c_int32]
_lib.mok_read_device_status.restype = ctypes.c_int
_lib.mok_read_device_status.argtypes = [ctypes.POINTER(mok_schedule), ctypes.POINTER(ctypes.c_uint32), _P]
_lib.mok_selftest_wait_timeout.restype = ctypes.c_int
_lib.mok_selftest_wait_timeout.argtypes = [_P, _P]

class mok_mx_operands(ctypes.Structure):
    _fields_ = [(k, _P) for k in ("xq", "xs", "aq", "as_", "dyq", "dys", "dgq", "dgs", "xr", "xrs", "dyr", "dyrs",
                                  "dgr", "dgrs", "sar", "sars")] + \
        [("rows", ctypes.c_int64), ("rcap", ctypes.c_int64), ("xr_groups", ctypes.c_int32),
         ("sar_groups", ctypes.c_int32)]


_lib.mok_mx_operands_of.restype = ctypes.c_int
_lib.mok_mx_operands_of.argtypes = [ctypes.POINTER(mok_schedule), _P, ctypes.POINTER(mok_mx_operands)]

EXPORTED = ("mok_version", "mok_status_string", "mok_workspace_bytes", "mok_fwd_ctx_bytes", "mok_mxfp8_quantize",
            "mok_build_schedule", "mok_forward", "mok_backward", "mok_read_device_status", "mok_set_trace",
            "mok_kernel_name", "mok_build_schedule_noalloc", "mok_mx_operands_of", "mok_router_workspace_bytes",
            "mok_router_forward", "mok_router_backward", "mok_selftest_wait_timeout", "mok_ep_build_schedule",
            "mok_ep_forward", "mok_ep_backward", "mok_ep_combine", "mok_dropout_forward", "mok_dropout_backward",
            "mok_rmsnorm_forward", "mok_rmsnorm_workspace_bytes", "mok_rmsnorm_backward", "mok_ffn_ctx_bytes",
            "mok_ffn_forward", "mok_ffn_workspace_bytes", "mok_ffn_backward")
_lib.mok_router_workspace_bytes.restype = ctypes.c_size_t
_lib.mok_router_workspace_bytes.argtypes = [ctypes.POINTER(mok_shape)]
_lib.mok_router_forward.restype = ctypes.c_int
_lib.mok_router_forward.argtypes = [ctypes.POINTER(mok_shape), _P, _P, _P, _P, _P, _P, _P]
_lib.mok_router_backward.restype = ctypes.c_int
_lib.mok_router_backward.argtypes = [ctypes.POINTER(mok_schedule), _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                     _P, ctypes.c_size_t, _P]
_lib.mok_build_schedule_noalloc.restype = ctypes.c_int
_lib.mok_build_schedule_noalloc.argtypes = [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, _P,
                                            ctypes.POINTER(mok_schedule), _P]


# ---- expert parallelism ----
MOK_EP_MAX_RANKS = 8


class mok_ep_group(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("tokens_per_rank", ctypes.c_int64)]


_PT = ctypes.POINTER(_P)
_lib.mok_ep_build_schedule.restype = ctypes.c_int
_lib.mok_ep_build_schedule.argtypes = [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape),
                                       ctypes.POINTER(mok_ep_group), _PT, _PT, _P, ctypes.c_size_t,
                                       ctypes.POINTER(mok_schedule), _P]
_lib.mok_ep_forward.restype = ctypes.c_int
_lib.mok_ep_forward.argtypes = [ctypes.POINTER(mok_schedule), ctypes.POINTER(mok_ep_group), _PT,
                                ctypes.POINTER(mok_weights), _PT, _P, ctypes.c_size_t, _P]
_lib.mok_ep_backward.restype = ctypes.c_int
_lib.mok_ep_backward.argtypes = [ctypes.POINTER(mok_schedule), ctypes.POINTER(mok_ep_group), _P, _PT,
                                 ctypes.POINTER(mok_weights), _P, _P, _P, _PT, _PT, _P]
_lib.mok_ep_combine.restype = ctypes.c_int
_lib.mok_ep_combine.argtypes = [ctypes.POINTER(mok_shape), ctypes.POINTER(mok_ep_group), _P, _P, _P, _P, _P]


def _check(rc: int, where: str):
    if rc != MOK_OK:
        raise MokError(rc, where)


# the handle of a device's current stream without building a Stream object (0.1 against 2.9 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_stream(stream, x):
    """Refuses a torch stream of another device than tensor x's (a bare handle does not say which it is of)."""
    if isinstance(stream, torch.cuda.Stream) and isinstance(x, torch.Tensor) and x.is_cuda and stream.device != x.device:
        raise ValueError(f"the stream must be on {x.device}, as the tensors are, got {stream.device}")


def _on_stream(stream, x=None):
    """Makes `stream` (torch.cuda.Stream, or a handle on x's device; None: that device's current one) current: what a call
    allocates then belongs to the stream that it runs on, so that neither a workspace that it drops nor an output's
    earlier owner can still be in use there.  Without x the device is the current one."""
    device = x.device if isinstance(x, torch.Tensor) and x.is_cuda else None
    if stream is None:
        return torch.cuda.device(device)
    _check_stream(stream, x)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)  # 0: the default stream, of which ExternalStream makes a new stream of torch's pool
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def mok_version() -> str:
    return _lib.mok_version().decode()


MOK_FLAG_STATIC_TILES = 1  # static round-robin GEMM tile scheduling instead of cluster launch control


def make_config(minibatch_rows=512, macrobatch_rows=2048, num_ctas=0, precision=MOK_BF16, flags=0) -> mok_config:
    return mok_config(minibatch_rows, macrobatch_rows, num_ctas, precision, flags)


def make_shape(T, H, I, E, K) -> mok_shape:
    return mok_shape(T, H, I, E, K)


def mok_workspace_bytes(cfg: mok_config, shape: mok_shape) -> int:
    n = _lib.mok_workspace_bytes(ctypes.byref(cfg), ctypes.byref(shape))
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_workspace_bytes")
    return n


def mok_fwd_ctx_bytes(cfg: mok_config, shape: mok_shape) -> int:
    n = _lib.mok_fwd_ctx_bytes(ctypes.byref(cfg), ctypes.byref(shape))
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_fwd_ctx_bytes")
    return n


def mok_mxfp8_quantize(x: torch.Tensor, out_q: torch.Tensor | None = None, out_s: torch.Tensor | None = None,
                       stream=None):
    """MXFP8 of a 2-D bf16 tensor: (E4M3 bytes [rows, cols] uint8, E8M0 scales [rows, cols/32] uint8)."""
    if stream is not None:
        with _on_stream(stream):
            return mok_mxfp8_quantize(x, out_q, out_s)
    rows, cols = x.shape
    if out_q is None:
        out_q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if out_s is None:
        out_s = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    _check(_lib.mok_mxfp8_quantize(_ptr(x, torch.bfloat16, "x"), rows, cols, _ptr(out_q, torch.uint8, "out_q"),
                                   _ptr(out_s, torch.uint8, "out_s"), _stream(None)), "mok_mxfp8_quantize")
    return out_q, out_s


@dataclass
class Schedule:
    """A built schedule plus the tensors it refers to (kept alive here)."""
    c: mok_schedule
    ws: torch.Tensor
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor

    def _view(self, field, n, dtype=torch.int32):
        """Device tensor view of one schedule table (for tests and inspection)."""
        ptr = getattr(self.c, field)
        base = self.ws.data_ptr()
        off = ptr - base
        esz = torch.tensor([], dtype=dtype).element_size()
        assert off % esz == 0 and off >= 0
        return self.ws.view(torch.uint8)[off:off + n * esz].view(dtype)

    def tables(self) -> dict:
        E = self.c.shape.E
        R = self.c.shape.T * self.c.shape.K
        return dict(counts=self._view("counts", E), offsets=self._view("offsets", E + 1),
                    poff=self._view("poff", E + 1), perm=self._view("perm", self.c.rpad_max),
                    inv=self._view("inv", R), tiles=self._view("tiles", 4 * self.c.tiles_max).view(-1, 4),
                    mblocks=self._view("mblocks", 4 * self.c.mblocks_max).view(-1, 4),
                    meta=self._view("meta", 16), row_weight=self._view("row_weight", self.c.rpad_max, torch.float32),
                    row_token=self._view("row_token", self.c.rpad_max))


    def mx_operands(self, fwd_ctx: torch.Tensor) -> dict:
        """Device views of the MXFP8 operand copies (mok_mx_operands_of): E4M3 codes ([rows, n]
        quantised along each row, transposed [n, rcap] quantised along the rows) and their
        atom-tiled E8M0 scale arrays (flat uint8), plus the layout numbers rows, rcap, xr_groups,
        sar_groups."""
        m = mok_mx_operands()
        _check(_lib.mok_mx_operands_of(ctypes.byref(self.c), _ptr(fwd_ctx, None, "fwd_ctx"), ctypes.byref(m)),
               "mok_mx_operands_of")
        H, I, rows, rcap = self.c.shape.H, self.c.shape.I, m.rows, m.rcap
        rt = (rows + 127) // 128

        def v(ptr, n):
            for buf in (self.ws, fwd_ctx):
                base = buf.data_ptr()
                if base <= ptr < base + buf.numel() * buf.element_size():
                    return buf.view(torch.uint8)[ptr - base:ptr - base + n]
            raise ValueError("pointer outside the workspace and the context")
        return dict(xq=v(m.xq, rows * H).view(rows, H), xs=v(m.xs, rt * 128 * (H // 32)),
                    aq=v(m.aq, rows * I).view(rows, I), as_=v(m.as_, rt * 128 * (I // 32)),
                    dyq=v(m.dyq, rows * H).view(rows, H), dys=v(m.dys, rt * 128 * (H // 32)),
                    dgq=v(m.dgq, rows * 2 * I).view(rows, 2 * I), dgs=v(m.dgs, rt * 128 * (2 * I // 32)),
                    xr=v(m.xr, H * rcap).view(H, rcap), xrs=v(m.xrs, H * rcap // 32),
                    dyr=v(m.dyr, H * rcap).view(H, rcap), dyrs=v(m.dyrs, H * rcap // 32),
                    dgr=v(m.dgr, 2 * I * rcap).view(2 * I, rcap), dgrs=v(m.dgrs, 2 * I * rcap // 32),
                    sar=v(m.sar, I * rcap).view(I, rcap), sars=v(m.sars, I * rcap // 32),
                    rows=rows, rcap=rcap, xr_groups=m.xr_groups, sar_groups=m.sar_groups)


def alloc_workspace(cfg: mok_config, shape: mok_shape, device="cuda") -> torch.Tensor:
    return torch.empty(mok_workspace_bytes(cfg, shape), dtype=torch.uint8, device=device)


def alloc_fwd_ctx(cfg: mok_config, shape: mok_shape, device="cuda") -> torch.Tensor:
    return torch.empty(mok_fwd_ctx_bytes(cfg, shape), dtype=torch.uint8, device=device)


def mok_build_schedule(cfg: mok_config, shape: mok_shape, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                       ws: torch.Tensor, stream=None) -> Schedule:
    s = mok_schedule()
    _check(_lib.mok_build_schedule(ctypes.byref(cfg), ctypes.byref(shape), _ptr(topk_ids, torch.int32, "topk_ids"),
                                   _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(ws, None, "ws"),
                                   ws.numel() * ws.element_size(), ctypes.byref(s), _stream(stream)),
           "mok_build_schedule")
    return Schedule(s, ws, topk_ids, topk_weights)


def weights_struct(Wg=None, Wu=None, Wd=None, mx: dict | None = None) -> mok_weights:
    """bf16 weights for BF16 mode; ``mx`` = the pre-quantised copies (``quantize_weights``) for
    MXFP8 mode.  The struct holds raw pointers: keep the tensors alive while it is used."""
    w = mok_weights()
    w.w_gate = _ptr(Wg, torch.bfloat16, "w_gate")
    w.w_up = _ptr(Wu, torch.bfloat16, "w_up")
    w.w_down = _ptr(Wd, torch.bfloat16, "w_down")
    if mx:
        for k in MX_KEYS:
            setattr(w, k, _ptr(mx.get(k), torch.uint8, k))
    return w


def quantize_weights(Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, stream=None) -> dict:
    """The MXFP8 weight copies of mok_weights, made with mok_mxfp8_quantize on the device: forward
    copies along each GEMM's K and backward copies of the transposes."""
    if stream is not None:  # the transposed copies below are made on it as well
        with _on_stream(stream):
            return quantize_weights(Wg, Wu, Wd)
    E, I, H = Wg.shape
    out = {}
    out["q_gate"], out["s_gate"] = mok_mxfp8_quantize(Wg.reshape(E * I, H))
    out["q_up"], out["s_up"] = mok_mxfp8_quantize(Wu.reshape(E * I, H))
    out["q_down"], out["s_down"] = mok_mxfp8_quantize(Wd.reshape(E * H, I))
    out["qt_gate"], out["st_gate"] = mok_mxfp8_quantize(Wg.transpose(1, 2).contiguous().reshape(E * H, I))
    out["qt_up"], out["st_up"] = mok_mxfp8_quantize(Wu.transpose(1, 2).contiguous().reshape(E * H, I))
    out["qt_down"], out["st_down"] = mok_mxfp8_quantize(Wd.transpose(1, 2).contiguous().reshape(E * I, H))
    return out


def mok_forward(sched: Schedule, x: torch.Tensor, weights: mok_weights, out: torch.Tensor, fwd_ctx: torch.Tensor,
                stream=None) -> torch.Tensor:
    _check(_lib.mok_forward(ctypes.byref(sched.c), _ptr(x, torch.bfloat16, "x"), ctypes.byref(weights),
                            _ptr(out, torch.bfloat16, "out"), _ptr(fwd_ctx, None, "fwd_ctx"),
                            fwd_ctx.numel() * fwd_ctx.element_size(), _stream(stream)), "mok_forward")
    return out


@dataclass
class Grads:
    dx: torch.Tensor
    dw_gate: torch.Tensor
    dw_up: torch.Tensor
    dw_down: torch.Tensor
    d_topk_weights: torch.Tensor

    @staticmethod
    def empty(T, H, I, E, K, device="cuda") -> "Grads":
        return Grads(torch.empty((T, H), dtype=torch.bfloat16, device=device),
                     torch.empty((E, I, H), dtype=torch.float32, device=device),
                     torch.empty((E, I, H), dtype=torch.float32, device=device),
                     torch.empty((E, H, I), dtype=torch.float32, device=device),
                     torch.empty((T, K), dtype=torch.float32, device=device))

    def struct(self) -> mok_grads:
        g = mok_grads()
        g.dx = _ptr(self.dx, torch.bfloat16, "dx")
        g.dw_gate = _ptr(self.dw_gate, torch.float32, "dw_gate")
        g.dw_up = _ptr(self.dw_up, torch.float32, "dw_up")
        g.dw_down = _ptr(self.dw_down, torch.float32, "dw_down")
        g.d_topk_weights = _ptr(self.d_topk_weights, torch.float32, "d_topk_weights")
        return g


def mok_backward(sched: Schedule, fwd_ctx: torch.Tensor, dy: torch.Tensor, weights: mok_weights, grads: Grads,
                 stream=None) -> Grads:
    gs = grads.struct()
    _check(_lib.mok_backward(ctypes.byref(sched.c), _ptr(fwd_ctx, None, "fwd_ctx"), _ptr(dy, torch.bfloat16, "dy"),
                             ctypes.byref(weights), ctypes.byref(gs), _stream(stream)), "mok_backward")
    return grads


def make_ep_group(world: int, rank: int, tokens_per_rank: int) -> mok_ep_group:
    return mok_ep_group(world, rank, tokens_per_rank)


def _table(tensors, dtype, name):
    """Host array of per-rank device pointers (one per rank of the group)."""
    if len(tensors) > MOK_EP_MAX_RANKS:
        raise ValueError(f"at most {MOK_EP_MAX_RANKS} ranks")
    arr = (_P * MOK_EP_MAX_RANKS)()
    for r, t in enumerate(tensors):
        arr[r] = _ptr(t, dtype, f"{name}[{r}]")
    return arr


def mok_ep_build_schedule(cfg: mok_config, shape: mok_shape, ep: mok_ep_group, topk_ids: list, topk_weights: list,
                          ws: torch.Tensor, stream=None) -> Schedule:
    """This rank's schedule over the group's slots, from every rank's routing (lists of tensors)."""
    s = mok_schedule()
    ids_t, w_t = _table(topk_ids, torch.int32, "topk_ids"), _table(topk_weights, torch.float32, "topk_weights")
    _check(_lib.mok_ep_build_schedule(ctypes.byref(cfg), ctypes.byref(shape), ctypes.byref(ep), ids_t, w_t,
                                      _ptr(ws, None, "ws"), ws.numel() * ws.element_size(), ctypes.byref(s),
                                      _stream(stream)), "mok_ep_build_schedule")
    return Schedule(s, ws, topk_ids[ep.rank], topk_weights[ep.rank])


def mok_ep_forward(sched: Schedule, ep: mok_ep_group, x: list, weights: mok_weights, y_recv: list,
                   fwd_ctx: torch.Tensor, stream=None) -> None:
    _check(_lib.mok_ep_forward(ctypes.byref(sched.c), ctypes.byref(ep), _table(x, torch.bfloat16, "x"),
                               ctypes.byref(weights), _table(y_recv, torch.bfloat16, "y_recv"),
                               _ptr(fwd_ctx, None, "fwd_ctx"), fwd_ctx.numel() * fwd_ctx.element_size(),
                               _stream(stream)), "mok_ep_forward")


def mok_ep_backward(sched: Schedule, ep: mok_ep_group, fwd_ctx: torch.Tensor, dy: list, weights: mok_weights,
                    dw_gate: torch.Tensor, dw_up: torch.Tensor, dw_down: torch.Tensor, dx_recv: list,
                    d_topk_weights: list, stream=None) -> None:
    _check(_lib.mok_ep_backward(ctypes.byref(sched.c), ctypes.byref(ep), _ptr(fwd_ctx, None, "fwd_ctx"),
                                _table(dy, torch.bfloat16, "dy"), ctypes.byref(weights),
                                _ptr(dw_gate, torch.float32, "dw_gate"), _ptr(dw_up, torch.float32, "dw_up"),
                                _ptr(dw_down, torch.float32, "dw_down"), _table(dx_recv, torch.bfloat16, "dx_recv"),
                                _table(d_topk_weights, torch.float32, "d_topk_weights"), _stream(stream)),
           "mok_ep_backward")


def mok_ep_combine(shape: mok_shape, ep: mok_ep_group, topk_ids: torch.Tensor, topk_weights: torch.Tensor | None,
                   recv: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    _check(_lib.mok_ep_combine(ctypes.byref(shape), ctypes.byref(ep), _ptr(topk_ids, torch.int32, "topk_ids"),
                               _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(recv, torch.bfloat16, "recv"),
                               _ptr(out, torch.bfloat16, "out"), _stream(stream)), "mok_ep_combine")
    return out


def mok_read_device_status(sched: Schedule, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib.mok_read_device_status(ctypes.byref(sched.c), ctypes.byref(v), _stream(stream)),
           "mok_read_device_status")
    return v.value


def mok_selftest_wait_timeout(status: torch.Tensor, stream=None) -> None:
    """status: one int32 (bit pattern of a uint32) on the device; the timeout bit is OR-ed in."""
    if status.dtype != torch.int32 or status.numel() != 1 or not status.is_cuda:
        raise ValueError("status must be one int32 on the GPU")
    _check(_lib.mok_selftest_wait_timeout(ctypes.c_void_p(status.data_ptr()), _stream(stream)),
           "mok_selftest_wait_timeout")


# ---------------------------------------------------------------------------------------------
# router step (before the layer)
# ---------------------------------------------------------------------------------------------
def mok_router_workspace_bytes(shape: mok_shape) -> int:
    n = _lib.mok_router_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_router_workspace_bytes")
    return n


def mok_router_forward(shape: mok_shape, x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor | None,
                       logits: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, stream=None):
    _check(_lib.mok_router_forward(ctypes.byref(shape), _ptr(x, torch.bfloat16, "x"),
                                   _ptr(w_router, torch.bfloat16, "w_router"), _ptr(bias, torch.float32, "bias"),
                                   _ptr(logits, torch.float32, "logits"), _ptr(topk_ids, torch.int32, "topk_ids"),
                                   _ptr(topk_weights, torch.float32, "topk_weights"), _stream(stream)),
           "mok_router_forward")


def mok_router_backward(sched: Schedule, x: torch.Tensor, w_router: torch.Tensor, topk_ids: torch.Tensor,
                        topk_weights: torch.Tensor, d_topk_weights: torch.Tensor, dw_router: torch.Tensor,
                        d_bias: torch.Tensor | None, dx: torch.Tensor, accumulate_dx: bool, ws: torch.Tensor,
                        stream=None):
    _check(_lib.mok_router_backward(ctypes.byref(sched.c), _ptr(x, torch.bfloat16, "x"),
                                    _ptr(w_router, torch.bfloat16, "w_router"), _ptr(topk_ids, torch.int32, "ids"),
                                    _ptr(topk_weights, torch.float32, "topk_weights"),
                                    _ptr(d_topk_weights, torch.float32, "d_topk_weights"),
                                    _ptr(dw_router, torch.float32, "dw_router"), _ptr(d_bias, torch.float32, "d_bias"),
                                    _ptr(dx, torch.bfloat16, "dx"), 1 if accumulate_dx else 0, _ptr(ws, None, "ws"),
                                    ws.numel() * ws.element_size(), _stream(stream)), "mok_router_backward")


def router_forward(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor | None, K: int, stream=None):
    """Allocating form: returns (logits [T,E] fp32, topk_ids [T,K] int32, topk_weights [T,K] fp32)."""
    if stream is not None:
        with _on_stream(stream):
            return router_forward(x, w_router, bias, K)
    T, H = x.shape
    E = w_router.shape[1]
    shape = make_shape(T, H, 128, E, K)
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    ids = torch.empty((T, K), dtype=torch.int32, device=x.device)
    wts = torch.empty((T, K), dtype=torch.float32, device=x.device)
    mok_router_forward(shape, x, w_router, bias, logits, ids, wts)
    return logits, ids, wts


def router_backward(sched: Schedule, x: torch.Tensor, w_router: torch.Tensor, topk_ids: torch.Tensor,
                    topk_weights: torch.Tensor, d_topk_weights: torch.Tensor, with_bias: bool = False,
                    dx: torch.Tensor | None = None, stream=None):
    """Allocating form: returns (dw_router [H,E] fp32, d_bias [E] fp32 or None, dx [T,H] bf16).  A
    given dx receives the router's share added in place."""
    if stream is not None:
        with _on_stream(stream):
            return router_backward(sched, x, w_router, topk_ids, topk_weights, d_topk_weights, with_bias, dx)
    H, E = w_router.shape
    dw = torch.empty((H, E), dtype=torch.float32, device=x.device)
    db = torch.empty((E,), dtype=torch.float32, device=x.device) if with_bias else None
    acc = dx is not None
    if dx is None:
        dx = torch.empty_like(x)
    ws = torch.empty(mok_router_workspace_bytes(sched.c.shape), dtype=torch.uint8, device=x.device)
    mok_router_backward(sched, x, w_router, topk_ids, topk_weights, d_topk_weights, dw, db, dx, acc, ws)
    return dw, db, dx


class Layer:
    """Convenience owner of the workspace and forward context of one (shape, config) pair."""

    def __init__(self, T, H, I, E, K, cfg: mok_config | None = None, device="cuda"):
        self.shape = make_shape(T, H, I, E, K)
        self.cfg = cfg or make_config()
        self.ws = alloc_workspace(self.cfg, self.shape, device)
        self.ctx = alloc_fwd_ctx(self.cfg, self.shape, device)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.grads = Grads.empty(T, H, I, E, K, device)
        self.sched = None

    def schedule(self, topk_ids, topk_weights, stream=None) -> Schedule:
        self.sched = mok_build_schedule(self.cfg, self.shape, topk_ids, topk_weights, self.ws, stream)
        return self.sched

    def forward(self, x, weights: mok_weights, stream=None):
        return mok_forward(self.sched, x, weights, self.out, self.ctx, stream)

    def backward(self, dy, weights: mok_weights, stream=None) -> Grads:
        return mok_backward(self.sched, self.ctx, dy, weights, self.grads, stream)


# ---------------------------------------------------------------------------------------------
# dense operators around the layer: dropout, norm of the residual stream, gated feed-forward block
# ---------------------------------------------------------------------------------------------
MOK_DT_BF16 = 0
MOK_DT_FP32 = 1
MOK_ACT_SILU = 0
MOK_ACT_GELU = 1
_ACTS = {"silu": MOK_ACT_SILU, "gelu": MOK_ACT_GELU}
_STREAM_TYPES = {torch.bfloat16: MOK_DT_BF16, torch.float32: MOK_DT_FP32}


class mok_dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("rng", _P)]


class _placed_dropout(ctypes.Structure):  # with the index of the device that holds the state, for the compiled binding
    _fields_ = [("d", mok_dropout), ("device", ctypes.c_int32)]


class mok_norm_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("stream_type", ctypes.c_int32), ("eps", ctypes.c_float)]


class mok_ffn_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("act", ctypes.c_int32)]


class mok_ffn_grads(ctypes.Structure):
    _fields_ = [("dx", _P), ("dw_gate", _P), ("dw_up", _P), ("dw_down", _P), ("dw_type", ctypes.c_int32),
                ("dx_add", _P)]


_DROP, _NORM, _FFN = ctypes.POINTER(mok_dropout), ctypes.POINTER(mok_norm_shape), ctypes.POINTER(mok_ffn_shape)
_lib.mok_dropout_forward.restype = ctypes.c_int
_lib.mok_dropout_forward.argtypes = [ctypes.c_int64, ctypes.c_int32, _DROP, _P, _P, _P, _P]
_lib.mok_dropout_backward.restype = ctypes.c_int
_lib.mok_dropout_backward.argtypes = [ctypes.c_int64, ctypes.c_int32, _DROP, _P, _P, _P]
_lib.mok_rmsnorm_forward.restype = ctypes.c_int
_lib.mok_rmsnorm_forward.argtypes = [_NORM, _P, _P, _DROP, _P, _P, _P, _P, _P, _P, _P]
_lib.mok_rmsnorm_workspace_bytes.restype = ctypes.c_size_t
_lib.mok_rmsnorm_workspace_bytes.argtypes = [_NORM]
_lib.mok_rmsnorm_backward.restype = ctypes.c_int
_lib.mok_rmsnorm_backward.argtypes = [_NORM, _P, _P, _P, _P, _P, _DROP, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.mok_ffn_ctx_bytes.restype = ctypes.c_size_t
_lib.mok_ffn_ctx_bytes.argtypes = [_FFN, ctypes.c_int32]
_lib.mok_ffn_forward.restype = ctypes.c_int
_lib.mok_ffn_forward.argtypes = [_FFN, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, ctypes.c_int32, _P, _P]
_lib.mok_ffn_workspace_bytes.restype = ctypes.c_size_t
_lib.mok_ffn_workspace_bytes.argtypes = [_FFN]
_lib.mok_ffn_backward.restype = ctypes.c_int
_lib.mok_ffn_backward.argtypes = [_FFN, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, ctypes.POINTER(mok_ffn_grads), _P,
                                  ctypes.c_size_t, _P, _P]


def _arg(t: torch.Tensor | None, shape, dtype, name: str):
    """data_ptr of a contiguous CUDA tensor of that shape and dtype (None passes as NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _ptr(t, dtype, name)


class Dropout:
    """Dropout probability and generator state: rng, int64 [2] on the device, the bit patterns of
    {seed, offset}, read by the kernels when they run.  Each call that draws masks uses them all
    from the same state: advance the offset (``rng[1] += 1``) between calls."""

    def __init__(self, p: float, rng: torch.Tensor):
        self.rng = rng  # kept alive with the pointer
        ptr = _arg(rng, (2,), torch.int64, "rng")
        self._placed = _placed_dropout(mok_dropout(p, ptr), rng.device.index)
        self.c = self._placed.d
        self.ref = ctypes.byref(self.c)
        self.addr = ctypes.addressof(self._placed)

    def __reduce__(self):  # a copy has addresses of its own
        return Dropout, (self.c.p, self.rng)


def _refused(result, where: str, *args):
    """Raises for what a compiled call returned instead of its tensors: the library's status, or None for a tensor
    that is not what or where it has to be.  args: (tensor, shape, dtype, name) in the order of the call's checks, the
    first one's device being the call's."""
    if result is not None:
        raise MokError(result, where)
    for t, shape, dtype, name in args:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
        _arg(t, t.shape if shape is None else shape, dtype, name)
        if t.device != args[0][0].device:
            raise ValueError(f"{name} must be on {args[0][0].device}, as {args[0][3]} is, got {t.device}")
    raise ValueError(f"{where}: unsupported arguments")


def _rng_of(dropout):
    """The generator's state of an optional Dropout, as arguments of _refused."""
    return () if dropout is None else ((dropout.rng, (2,), torch.int64, "dropout.rng"),)


def _stream_type(t: torch.Tensor, name: str) -> int:
    st = _STREAM_TYPES.get(t.dtype)
    if st is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return st


def dropout_forward(x: torch.Tensor, dropout: Dropout, residual: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual + dropout(x): x bf16, residual bf16 or fp32 of x's shape; out of the residual's type
    (bf16 without one).  The number of values is a multiple of 8."""
    if stream is not None:
        with _on_stream(stream, x):
            return dropout_forward(x, dropout, residual, out)
    r = _bind.dropout_forward(x, dropout.addr, residual, out)
    if type(r) is not tuple:
        like = x if residual is None else residual
        _stream_type(like, "residual")
        _refused(r, "mok_dropout_forward", (x, None, torch.bfloat16, "x"), (like, x.shape, None, "residual"),
                 *(() if out is None else ((out, x.shape, like.dtype, "out"),)), *_rng_of(dropout))
    return r[0]


def dropout_backward(dout: torch.Tensor, dropout: Dropout, dx: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """The branch's gradient (bf16) for dout of the stream's type, under the forward's masks."""
    if stream is not None:
        with _on_stream(stream, dout):
            return dropout_backward(dout, dropout, dx)
    r = _bind.dropout_backward(dout, dropout.addr, dx)
    if type(r) is not tuple:
        _stream_type(dout, "dout")
        _refused(r, "mok_dropout_backward", (dout, None, None, "dout"),
                 *(() if dx is None else ((dx, dout.shape, torch.bfloat16, "dx"),)), *_rng_of(dropout))
    return r[0]


@dataclass
class NormOut:
    h: torch.Tensor               # the residual stream after the addition
    y: torch.Tensor | None        # normalised rows, bf16
    q: torch.Tensor | None        # the same in MXFP8: E4M3 codes (uint8) ...
    s: torch.Tensor | None        # ... and E8M0 scales (uint8) [T, H / 32]
    rstd: torch.Tensor            # 1 / rms of each row, fp32


def rmsnorm_forward(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                    dropout: Dropout | None = None, bf16: bool = True, mx: bool = False, stream=None) -> NormOut:
    """h = residual + dropout(x) and its root-mean-square norm times weight (mok_rmsnorm_forward):
    x [T, H] bf16, residual [T, H] bf16 or fp32 (the type of h), weight [H] bf16.  bf16 / mx choose the
    outputs.  Without residual and dropout h is x."""
    if stream is not None:
        with _on_stream(stream, x):
            return rmsnorm_forward(x, weight, eps, residual, dropout, bf16, mx)
    r = _bind.rmsnorm_forward(x, weight, eps, residual, None if dropout is None else dropout.addr, bf16, mx)
    if type(r) is not tuple:
        like = x if residual is None else residual
        _stream_type(like, "residual")
        T, H = x.shape
        _refused(r, "mok_rmsnorm_forward", (x, None, torch.bfloat16, "x"), (like, x.shape, None, "residual"),
                 (weight, (H,), torch.bfloat16, "weight"), *_rng_of(dropout))
    h, y, q, s, rstd = r
    return NormOut(x if h is None else h, y, q, s, rstd)


@dataclass
class NormGrads:
    dh: torch.Tensor         # of the residual, in the stream's type
    dx: torch.Tensor         # of the branch, bf16 (dh itself without dropout on a bf16 stream)
    dweight: torch.Tensor    # fp32 [H]


def mok_rmsnorm_workspace_bytes(shape: mok_norm_shape) -> int:
    n = _lib.mok_rmsnorm_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_rmsnorm_workspace_bytes")
    return n


def rmsnorm_backward(h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                     dres: torch.Tensor | None = None, dropout: Dropout | None = None, stream=None) -> NormGrads:
    """Gradients of rmsnorm_forward from dy [T, H] bf16 = dL/dy and dres = dL/dh from the stream's other
    uses (h's type, or None), under the forward's masks."""
    if stream is not None:
        with _on_stream(stream, h):
            return rmsnorm_backward(h, rstd, weight, dy, dres, dropout)
    r = _bind.rmsnorm_backward(h, rstd, weight, dy, dres, None if dropout is None else dropout.addr)
    if type(r) is not tuple:
        _stream_type(h, "h")
        T, H = h.shape
        _refused(r, "mok_rmsnorm_backward", (h, None, None, "h"), (rstd, (T,), torch.float32, "rstd"),
                 (weight, (H,), torch.bfloat16, "weight"), (dy, h.shape, torch.bfloat16, "dy"),
                 *(() if dres is None else ((dres, h.shape, h.dtype, "dres"),)), *_rng_of(dropout))
    dh, dx, dw = r
    return NormGrads(dh, dh if dx is None else dx, dw)


def mok_ffn_ctx_bytes(shape: mok_ffn_shape, save: bool) -> int:
    n = _lib.mok_ffn_ctx_bytes(ctypes.byref(shape), 1 if save else 0)
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_ffn_ctx_bytes")
    return n


def mok_ffn_workspace_bytes(shape: mok_ffn_shape) -> int:
    n = _lib.mok_ffn_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise MokError(MOK_ERR_INVALID_ARG, "mok_ffn_workspace_bytes")
    return n


@dataclass
class FFNGrads:
    dx: torch.Tensor
    dw_gate: torch.Tensor
    dw_up: torch.Tensor
    dw_down: torch.Tensor


class FFN:
    """Owner of the buffers of one dense gated feed-forward block (mok_ffn_forward / _backward):
    act(x Wg^T) * (x Wu^T) Wd^T + residual for exactly T tokens (another number is another plan; the C calls take any),
    w_gate, w_up [I, H] and w_down [H, I] bf16.  act: "silu" or "gelu" (tanh form).  train: the forward saves what the
    backward reads, 8 T I bytes beside the 2 T I of a forward alone (126 MB in all at T = 8192, I = 1536), and the plan has
    the backward's workspace, 4 T I bytes, and gradients.  dw_dtype: type of the weight gradients, torch.bfloat16 or
    torch.float32.  Outputs are the plan's own buffers, overwritten by the next call.  A copy (copy, deepcopy, pickle) is
    a new plan, whose buffers hold nothing yet."""

    def __init__(self, T: int, H: int, I: int, act: str = "silu", train: bool = True, dw_dtype=torch.bfloat16,
                 device="cuda"):
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
        if dw_dtype not in _STREAM_TYPES:
            raise ValueError(f"dw_dtype must be torch.bfloat16 or torch.float32, got {dw_dtype}")
        self.T, self.H, self.I, self.train = T, H, I, train
        self._made_of = (T, H, I, act, train, dw_dtype)
        self.shape = mok_ffn_shape(T, H, I, _ACTS[act])
        self.ctx = torch.empty(mok_ffn_ctx_bytes(self.shape, train), dtype=torch.uint8, device=device)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.status = torch.zeros((1,), dtype=torch.int32, device=device)
        self._device = self.out.device.index if self.out.is_cuda else -1
        self._fwd = (self._device, ctypes.addressof(self.shape), self.out.data_ptr(), self.ctx.data_ptr(), self.ctx.numel(),
                     1 if train else 0, self.status.data_ptr())
        if train:
            e = lambda *s: torch.empty(s, dtype=dw_dtype, device=device)  # noqa: E731
            self.grads = FFNGrads(torch.empty_like(self.out), e(I, H), e(I, H), e(H, I))
            self.ws = torch.empty(mok_ffn_workspace_bytes(self.shape), dtype=torch.uint8, device=device)
            g = self.grads
            self._grads = mok_ffn_grads(g.dx.data_ptr(), g.dw_gate.data_ptr(), g.dw_up.data_ptr(),
                                        g.dw_down.data_ptr(), _STREAM_TYPES[dw_dtype])
            self._bwd = (self._device, ctypes.addressof(self.shape), self.ctx.data_ptr(), self.ctx.numel(),
                         ctypes.addressof(self._grads), self.ws.data_ptr(), self.ws.numel(), self.status.data_ptr())

    def __reduce__(self):  # a copy has buffers, and addresses, of its own
        return FFN, (*self._made_of, self.out.device)

    def _in(self, x, w_gate, w_up, w_down):
        xs, ws, bf = (self.T, self.H), (self.I, self.H), torch.bfloat16
        return ((x, xs, bf, "x"), (w_gate, ws, bf, "w_gate"), (w_up, ws, bf, "w_up"),
                (w_down, (self.H, self.I), bf, "w_down"))

    def forward(self, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        _check_stream(stream, x)
        r = _bind.ffn_forward(*self._fwd, x, w_gate, w_up, w_down, residual, None if stream is None else _stream(stream))
        if type(r) is not tuple:
            _refused(r, "mok_ffn_forward", *self._in(x, w_gate, w_up, w_down),
                     *(() if residual is None else ((residual, (self.T, self.H), torch.bfloat16, "residual"),)),
                     (self.out, None, None, "the plan"))
        return self.out

    def backward(self, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                 dy: torch.Tensor, dx_add: torch.Tensor | None = None, stream=None) -> FFNGrads:
        """Gradients of the last forward; dx_add: x's gradient from its other uses, added to dx.  x and dy are not the
        plan's own dx (of a backward before); dx_add may be."""
        if not self.train:
            raise ValueError("backward needs a plan made with train=True")
        _check_stream(stream, x)
        r = _bind.ffn_backward(*self._bwd, x, w_gate, w_up, w_down, dy, dx_add, None if stream is None else _stream(stream))
        if type(r) is not tuple:
            like = (self.T, self.H), torch.bfloat16
            for t, name in ((x, "x"), (dy, "dy")):
                if r == MOK_ERR_INVALID_ARG and t.data_ptr() == self.grads.dx.data_ptr():
                    raise ValueError(f"{name} must not be the plan's dx, which is written while {name} is read")
            _refused(r, "mok_ffn_backward", *self._in(x, w_gate, w_up, w_down), (dy, *like, "dy"),
                     *(() if dx_add is None else ((dx_add, *like, "dx_add"),)), (self.out, None, None, "the plan"))
        return self.grads

    def device_status(self) -> int:
        """The block's device status word, bits (1 << status code), after all work on its device, on whatever stream;
        synchronises."""
        if self.status.is_cuda:
            torch.cuda.synchronize(self.status.device)
        return int(self.status.item())


def mok_kernel_name(kind: int) -> str:
    return _lib.mok_kernel_name(kind).decode()


def mok_set_trace(trace: "mok_trace | None"):
    _check(_lib.mok_set_trace(ctypes.byref(trace) if trace is not None else None), "mok_set_trace")


class Tracer:
    """Records a CUDA event pair around every kernel the library launches while active
    (``with Tracer(n) as tr: ...``), then reports per-launch device times in ms."""

    def __init__(self, capacity: int):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.events:
            e.record()  # creates the underlying cudaEvent_t
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * (2 * capacity))(*[e.cuda_event for e in self.events])
        self._kinds = (ctypes.c_int32 * capacity)()
        self.trace = mok_trace(self._handles, self._kinds, capacity, 0)

    def __enter__(self):
        self.trace.count = 0
        mok_set_trace(self.trace)
        return self

    def __exit__(self, *exc):
        mok_set_trace(None)
        return False

    def records(self):
        """[(kernel name, ms)] in launch order (synchronises)."""
        torch.cuda.synchronize()
        out = []
        for i in range(self.trace.count):
            out.append((mok_kernel_name(self._kinds[i]),
                        self.events[2 * i].elapsed_time(self.events[2 * i + 1])))
        return out
