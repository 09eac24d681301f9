"""Thin ctypes binding of libmoe.so (C ABI in include/moe.h).

Argument marshalling only: every step of the block runs in the library's HIP
kernels.  torch provides device memory (output tensors are allocated with
torch on the input's device) and the stream (torch's current stream, so
torch.cuda events and synchronisation see the library's work).  Nothing here
falls back to a CPU or torch implementation: if the library is not built, or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
ACT = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8}
MOE_LOGITS_GIVEN, MOE_IDENTITY_EXPERTS, MOE_KEEP_GATE_UP = 1, 2, 4

# every function the header declares, for the export check
EXPORTS = ["moe_version", "moe_status_string", "moe_workspace_bytes", "moe_packed_weight_bytes",
           "moe_pack_weights", "moe_route", "moe_dispatch", "moe_grouped_swiglu", "moe_combine",
           "moe_forward", "moe_forward_host_sync", "moe_set_profiling", "moe_kernel_times",
           "moe_set_gemm_grid_cap", "moe_backward_workspace_bytes", "moe_backward_weight_bytes",
           "moe_pack_weights_backward", "moe_backward", "moe_set_test_flags", "moe_route_noalloc",
           "moe_fused_status", "moe_norm", "moe_norm_backward_workspace_bytes", "moe_norm_backward",
           "moe_forward_quantized", "moe_balance_workspace_bytes", "moe_balance_loss",
           "moe_balance_loss_backward", "moe_router_backward_workspace_bytes", "moe_router_backward",
           "moe_backward_aux_workspace_bytes", "moe_backward_aux", "moe_decode_weight_bytes",
           "moe_decode_workspace_bytes", "moe_pack_weights_decode", "moe_decode_experts", "moe_decode"]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib().moe_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_hidden", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]

    @property
    def act(self) -> str:
        return {v: k for k, v in ACT.items()}[self.act_dtype]


def problem(T, d, E, k, H, act, logits_given=False, identity=False, keep_gate_up=False) -> Problem:
    flags = ((MOE_LOGITS_GIVEN if logits_given else 0) | (MOE_IDENTITY_EXPERTS if identity else 0)
             | (MOE_KEEP_GATE_UP if keep_gate_up else 0))
    return Problem(T, d, E, k, H, ACT[act], flags)


_LIB = None
_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_I32 = ctypes.c_int32


def lib():
    """Load libmoe.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "or python -m routing_dispatch_grouped_router_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        PP = ctypes.POINTER(Problem)
        L.moe_version.restype = ctypes.c_char_p
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [_I32]
        L.moe_workspace_bytes.argtypes = [PP, ctypes.POINTER(_SZ)]
        L.moe_packed_weight_bytes.argtypes = [PP, ctypes.POINTER(_SZ)]
        L.moe_pack_weights.argtypes = [PP, _P, _P, _P, _P, _P]
        L.moe_route.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_route_noalloc.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_dispatch.argtypes = [PP, _P, _P, _P, _P, _P]
        L.moe_grouped_swiglu.argtypes = [PP, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_combine.argtypes = [PP, _P, _P, _P, _P, _P]
        L.moe_forward.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward_host_sync.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]
        L.moe_set_profiling.argtypes = [_I32]
        L.moe_set_gemm_grid_cap.argtypes = [_I32]
        L.moe_set_test_flags.argtypes = [_I32]
        L.moe_fused_status.argtypes = [PP, _P, _SZ, _I32, ctypes.POINTER(_I32), _P]
        L.moe_backward_workspace_bytes.argtypes = [PP, ctypes.POINTER(_SZ)]
        L.moe_backward_weight_bytes.argtypes = [PP, ctypes.POINTER(_SZ)]
        L.moe_pack_weights_backward.argtypes = [PP, _P, _P, _P, _P, _P]
        L.moe_backward.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P, _P, _P, _P, _P,
                                   _P, _SZ, _P]
        for name in ("norm_backward_workspace", "balance_workspace", "router_backward_workspace",
                     "backward_aux_workspace", "decode_weight", "decode_workspace"):
            getattr(L, f"moe_{name}_bytes").argtypes = [PP, ctypes.POINTER(_SZ)]
        L.moe_norm.argtypes = [PP, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P]
        L.moe_norm_backward.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward_quantized.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_balance_loss.argtypes = [PP, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_balance_loss_backward.argtypes = [PP, _P, _P, _P, _P, _P, _P]
        L.moe_router_backward.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_backward_aux.argtypes = [*L.moe_backward.argtypes, _P, _P]
        L.moe_pack_weights_decode.argtypes = [PP, _P, _P, _P, _P, _P]
        L.moe_decode_experts.argtypes = [PP, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_decode.argtypes = [PP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float),
                                       _I32, ctypes.POINTER(_I32)]
        for name in EXPORTS:
            if name not in ("moe_version", "moe_status_string"):
                getattr(L, name).restype = _I32
        _LIB = L
    return _LIB


def _check(fn: str, status: int):
    if status != 0:
        raise MoeError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _own(t):
    """Address of a buffer that the caller's object allocated itself (or None)."""
    return None if t is None else t.data_ptr()


# The handle of a device's current stream without making a Stream object of it
# (0.1 instead of 2.9 us, of the 10 us that a small call took); not a documented
# function, so the documented way stands in where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, device=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    return torch.cuda.current_stream().cuda_stream


def _dev(t) -> torch.device:
    return t.device


def storage_dtype(act: str) -> torch.dtype:
    return torch.float32 if act == "f32" else torch.bfloat16


def _rows(p: Problem) -> tuple:
    """Shape and storage type of the problem's token rows [T, d]."""
    return (p.T, p.d_model), torch.float32 if p.act_dtype == MOE_F32 else torch.bfloat16


def out_dtype(act: str) -> torch.dtype:
    return torch.float32 if act == "f32" else torch.bfloat16


def _expect(t, shape, dtype, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def _bytes(fn: str, p: Problem) -> int:
    n = _SZ()
    _check(fn, getattr(lib(), fn)(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def _inputs(device, *tensors):
    """Addresses of a call's inputs: contiguous tensors (or None) on the current
    device, `device`, on whose given stream the kernels run."""
    ptrs = []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        if not t.is_cuda:
            raise ValueError("expected a device tensor")
        if t.get_device() != device:
            raise ValueError(f"a tensor is on {t.device}, expected cuda:{device}")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        ptrs.append(t.data_ptr())
    if torch.cuda.current_device() != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{torch.cuda.current_device()}")
    return ptrs


class _Operator:
    """An operator's problem (a copy: its buffers are of that size) and buffers.
    Another tensor may be put in a buffer's place (an output over an input, say),
    of the same shape and type; an optional one may be None."""

    def __init__(self, p: Problem, device):
        self.p = Problem.from_buffer_copy(p)
        self._p, self._device, self._specs = ctypes.byref(self.p), torch.device(device), {}
        self._index = -1 if self._device.type != "cuda" else (
            torch.cuda.current_device() if self._device.index is None else self._device.index)

    def _buffer(self, name, shape, dtype, wanted=True):
        self._specs[name] = shape, dtype
        self.__dict__[name] = torch.empty(shape, dtype=dtype, device=self._device) if wanted else None

    def __setattr__(self, name, value):
        if value is not None and name in self.__dict__.get("_specs", ()):
            _expect(value, *self._specs[name], name)
            if _ptr(value) is not None and value.get_device() != self._index:
                raise ValueError(f"{name} is on {value.device}, expected cuda:{self._index}")
        object.__setattr__(self, name, value)


# ----------------------------------------------------------------------------- host-only queries


def workspace_bytes(p: Problem) -> int:
    n = _SZ()
    _check("moe_workspace_bytes", lib().moe_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def packed_weight_bytes(p: Problem) -> int:
    n = _SZ()
    _check("moe_packed_weight_bytes", lib().moe_packed_weight_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def new_workspace(p: Problem, device) -> torch.Tensor:
    return torch.empty(workspace_bytes(p), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------------- entry points


def pack_weights(p: Problem, w_gate, w_up, w_down, stream=None) -> torch.Tensor:
    dt = storage_dtype(p.act)
    E, d, H = p.n_experts, p.d_model, p.d_hidden
    _expect(w_gate, (E, d, H), dt, "w_gate")
    _expect(w_up, (E, d, H), dt, "w_up")
    _expect(w_down, (E, H, d), dt, "w_down")
    packed = torch.empty(packed_weight_bytes(p), dtype=torch.uint8, device=w_gate.device)
    _check("moe_pack_weights", lib().moe_pack_weights(ctypes.byref(p), _ptr(w_gate), _ptr(w_up),
                                                      _ptr(w_down), _ptr(packed), _stream(stream)))
    return packed


def route(p: Problem, x=None, w_router=None, logits=None, ws=None, stream=None, stats=False) -> dict:
    """Returns dict(logits, idx, gate, counts, offsets, pos, row_token) as device tensors,
    plus router_stats [E + 2] (mean router probability per expert, balance scalar,
    worst-case imbalance) when stats=True."""
    T, E, k, d = p.T, p.n_experts, p.top_k, p.d_model
    dev = (logits if logits is not None else x).device
    if p.flags & MOE_LOGITS_GIVEN:
        _expect(logits, (T, E), torch.float32, "logits")
    else:
        _expect(x, (T, d), storage_dtype(p.act), "x")
        _expect(w_router, (d, E), storage_dtype(p.act), "w_router")
        logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    out = dict(logits=logits,
               idx=torch.empty((T, k), dtype=torch.int32, device=dev),
               gate=torch.empty((T, k), dtype=torch.float32, device=dev),
               counts=torch.empty((E,), dtype=torch.int32, device=dev),
               offsets=torch.empty((E + 1,), dtype=torch.int32, device=dev),
               pos=torch.empty((T, k), dtype=torch.int32, device=dev),
               row_token=torch.empty((T * k,), dtype=torch.int32, device=dev),
               router_stats=torch.empty((E + 2,), dtype=torch.float32, device=dev) if stats else None)
    ws = new_workspace(p, dev) if ws is None else ws
    _check("moe_route", lib().moe_route(
        ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(logits), _ptr(out["idx"]), _ptr(out["gate"]),
        _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["pos"]), _ptr(out["row_token"]),
        _ptr(out["router_stats"]), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def route_outputs(p: Problem, device, stats=False) -> dict:
    """Output tensors of route / route_noalloc for problem p (logits included)."""
    T, E, k = p.T, p.n_experts, p.top_k
    return dict(logits=torch.empty((T, E), dtype=torch.float32, device=device),
                idx=torch.empty((T, k), dtype=torch.int32, device=device),
                gate=torch.empty((T, k), dtype=torch.float32, device=device),
                counts=torch.empty((E,), dtype=torch.int32, device=device),
                offsets=torch.empty((E + 1,), dtype=torch.int32, device=device),
                pos=torch.empty((T, k), dtype=torch.int32, device=device),
                row_token=torch.empty((T * k,), dtype=torch.int32, device=device),
                router_stats=torch.empty((E + 2,), dtype=torch.float32, device=device) if stats else None)


def route_noalloc(p: Problem, out: dict, x=None, w_router=None, stream=None) -> dict:
    """moe_route_noalloc into the caller's tensors `out` (as route_outputs makes
    them; with MOE_LOGITS_GIVEN out["logits"] holds the input logits).  Neither
    this function nor the library allocates device memory."""
    T, E, k, d = p.T, p.n_experts, p.top_k, p.d_model
    _expect(out["logits"], (T, E), torch.float32, "logits")
    if not p.flags & MOE_LOGITS_GIVEN:
        _expect(x, (T, d), storage_dtype(p.act), "x")
        _expect(w_router, (d, E), storage_dtype(p.act), "w_router")
    for name, shape in (("idx", (T, k)), ("pos", (T, k)), ("counts", (E,)), ("offsets", (E + 1,)),
                        ("row_token", (T * k,))):
        _expect(out[name], shape, torch.int32, name)
    _expect(out["gate"], (T, k), torch.float32, "gate")
    if out.get("router_stats") is not None:
        _expect(out["router_stats"], (E + 2,), torch.float32, "router_stats")
    _check("moe_route_noalloc", lib().moe_route_noalloc(
        ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(out["logits"]), _ptr(out["idx"]), _ptr(out["gate"]),
        _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["pos"]), _ptr(out["row_token"]),
        _ptr(out.get("router_stats")), _stream(stream)))
    return out


def dispatch(p: Problem, x, pos, stream=None):
    """Returns (xe, xe_scale); xe_scale is None unless MXFP8, else uint8
    [d/128, R, 4]: the four E8M0 scales of each 128-wide slice of a row."""
    T, d, k = p.T, p.d_model, p.top_k
    R = T * k
    _expect(x, (T, d), storage_dtype(p.act), "x")
    _expect(pos, (T, k), torch.int32, "pos")
    if p.act == "mxfp8":
        xe = torch.empty((R, d), dtype=torch.uint8, device=x.device)
        xs = torch.empty((d // 128, R, 4), dtype=torch.uint8, device=x.device)   # slice-major scales
    else:
        xe = torch.empty((R, d), dtype=storage_dtype(p.act), device=x.device)
        xs = None
    _check("moe_dispatch", lib().moe_dispatch(ctypes.byref(p), _ptr(x), _ptr(pos), _ptr(xe), _ptr(xs),
                                              _stream(stream)))
    return xe, xs


def grouped_swiglu(p: Problem, xe, xe_scale, packed, offsets, ws=None, stream=None):
    R, d = p.T * p.top_k, p.d_model
    _expect(offsets, (p.n_experts + 1,), torch.int32, "offsets")
    ye = torch.empty((R, d), dtype=out_dtype(p.act), device=xe.device)
    ws = new_workspace(p, xe.device) if ws is None else ws
    _check("moe_grouped_swiglu", lib().moe_grouped_swiglu(
        ctypes.byref(p), _ptr(xe), _ptr(xe_scale), _ptr(packed), _ptr(offsets), _ptr(ye), _ptr(ws),
        ws.numel(), _stream(stream)))
    return ye


def combine(p: Problem, ye, gate, pos, stream=None):
    T, d, k = p.T, p.d_model, p.top_k
    _expect(ye, (T * k, d), out_dtype(p.act), "ye")
    _expect(gate, (T, k), torch.float32, "gate")
    _expect(pos, (T, k), torch.int32, "pos")
    y = torch.empty((T, d), dtype=out_dtype(p.act), device=ye.device)
    _check("moe_combine", lib().moe_combine(ctypes.byref(p), _ptr(ye), _ptr(gate), _ptr(pos), _ptr(y),
                                            _stream(stream)))
    return y


class Forward:
    """Preallocated state for repeated moe_forward calls (fixed buffer addresses)."""

    def __init__(self, p: Problem, device, debug_outputs: bool = True, host_sync: bool = False,
                 stats: bool = False):
        """host_sync: call moe_forward_host_sync (counts copied to a pinned host
        buffer and waited for before the grouped GEMMs) instead of moe_forward.
        stats: also compute the router statistics into self.router_stats [E + 2]."""
        self.p = p
        self.host_sync = host_sync
        self.host_counts = (torch.empty((p.n_experts,), dtype=torch.int32, pin_memory=True)
                            if host_sync else None)
        T, E, k, d = p.T, p.n_experts, p.top_k, p.d_model
        self.ws = new_workspace(p, device)
        self.y = torch.empty((T, d), dtype=out_dtype(p.act), device=device)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=device)
        self.debug = debug_outputs
        # whether the last call ran on code rows, which stay outside the workspace: what a Backward has to be given
        # (a replayed graph does not pass here: set it where the graph's forward was the other kind)
        self.quantized = False
        self.router_stats = (torch.empty((E + 2,), dtype=torch.float32, device=device) if stats else None)
        if debug_outputs:
            self.idx = torch.empty((T, k), dtype=torch.int32, device=device)
            self.gate = torch.empty((T, k), dtype=torch.float32, device=device)
            self.counts = torch.empty((E,), dtype=torch.int32, device=device)
            self.offsets = torch.empty((E + 1,), dtype=torch.int32, device=device)
            self.pos = torch.empty((T, k), dtype=torch.int32, device=device)
        else:
            self.idx = self.gate = self.counts = self.offsets = self.pos = None

    def __call__(self, x, packed=None, w_router=None, logits=None, stream=None, xq=None, xq_scale=None):
        """With xq [T, d] and xq_scale [T, d/32] (a Norm's q and q_scale) the block
        runs on these MXFP8 rows (moe_forward_quantized); x is then read by the
        learned router only, and may be None with given logits."""
        p = self.p
        if xq is not None:
            if self.host_sync:
                raise ValueError("quantised rows and host_sync do not go together")
            _expect(xq, (p.T, p.d_model), torch.uint8, "xq")
            _expect(xq_scale, (p.T, p.d_model // 32), torch.uint8, "xq_scale")
        if xq is None or x is not None or not p.flags & MOE_LOGITS_GIVEN:
            _expect(x, (p.T, p.d_model), storage_dtype(p.act), "x")
        if p.flags & MOE_LOGITS_GIVEN:
            _expect(logits, (p.T, p.n_experts), torch.float32, "logits")
            if logits.data_ptr() != self.logits.data_ptr():
                self.logits.copy_(logits)
        else:
            _expect(w_router, (p.d_model, p.n_experts), storage_dtype(p.act), "w_router")
        args = (ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(self.logits), _ptr(packed), _ptr(self.y),
                _ptr(self.idx), _ptr(self.gate), _ptr(self.counts), _ptr(self.offsets), _ptr(self.pos),
                _ptr(self.router_stats), _ptr(self.ws), self.ws.numel(), _stream(stream))
        if xq is not None:
            _check("moe_forward_quantized", lib().moe_forward_quantized(
                args[0], args[1], _ptr(xq), _ptr(xq_scale), *args[2:]))
        elif self.host_sync:
            _check("moe_forward_host_sync", lib().moe_forward_host_sync(
                *args, ctypes.c_void_p(self.host_counts.data_ptr())))
        else:
            _check("moe_forward", lib().moe_forward(*args))
        self.quantized = xq is not None
        return self.y


def forward(p: Problem, x, packed=None, w_router=None, logits=None, stream=None, host_sync=False,
            stats=False) -> dict:
    f = Forward(p, x.device, host_sync=host_sync, stats=stats)
    y = f(x, packed=packed, w_router=w_router, logits=logits, stream=stream)
    return dict(y=y, logits=f.logits, idx=f.idx, gate=f.gate, counts=f.counts, offsets=f.offsets,
                pos=f.pos, host_counts=f.host_counts, router_stats=f.router_stats)


def set_profiling(enable: bool):
    _check("moe_set_profiling", lib().moe_set_profiling(1 if enable else 0))


def backward_workspace_bytes(p: Problem) -> int:
    n = _SZ()
    _check("moe_backward_workspace_bytes", lib().moe_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def backward_weight_bytes(p: Problem) -> int:
    n = _SZ()
    _check("moe_backward_weight_bytes", lib().moe_backward_weight_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def pack_weights_backward(p: Problem, w_gate, w_up, w_down, stream=None) -> torch.Tensor:
    """The backward weight cache (moe_pack_weights_backward)."""
    dt = storage_dtype(p.act)
    E, d, H = p.n_experts, p.d_model, p.d_hidden
    _expect(w_gate, (E, d, H), dt, "w_gate")
    _expect(w_up, (E, d, H), dt, "w_up")
    _expect(w_down, (E, H, d), dt, "w_down")
    out = torch.empty(backward_weight_bytes(p), dtype=torch.uint8, device=w_gate.device)
    _check("moe_pack_weights_backward", lib().moe_pack_weights_backward(
        ctypes.byref(p), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(out), _stream(stream)))
    return out


class Backward:
    """Preallocated gradients and workspace for moe_backward of a Forward's last call
    (aux: for moe_backward_aux with another gradient for the logits)."""

    def __init__(self, p: Problem, device, aux: bool = False):
        self.p = p
        T, E, d, H = p.T, p.n_experts, p.d_model, p.d_hidden
        self.ws = torch.empty(_bytes("moe_backward_aux_workspace_bytes", p) if aux else backward_workspace_bytes(p),
                              dtype=torch.uint8, device=device)
        self.dx = torch.empty((T, d), dtype=out_dtype(p.act), device=device)
        self.dlogits = torch.empty((T, E), dtype=torch.float32, device=device)
        self.dw_gate = torch.empty((E, d, H), dtype=torch.float32, device=device)
        self.dw_up = torch.empty((E, d, H), dtype=torch.float32, device=device)
        self.dw_down = torch.empty((E, H, d), dtype=torch.float32, device=device)
        self.dw_router = (None if p.flags & MOE_LOGITS_GIVEN
                          else torch.empty((d, E), dtype=torch.float32, device=device))

    def __call__(self, fwd: "Forward", dy, packed, packed_bwd, x=None, w_router=None, stream=None,
                 dlogits_aux=None, xq=None):
        """dlogits_aux [T, E]: a gradient for the logits to be added (BalanceLoss.backward's);
        xq: the codes the forward was given, required if it was given any."""
        p = self.p
        dt = storage_dtype(p.act)
        if (xq is not None) != fwd.quantized:
            raise ValueError("xq: expected the codes that the forward ran on" if fwd.quantized else
                             "xq: not expected, the forward did not run on codes")
        if dlogits_aux is not None:
            _expect(dlogits_aux, (p.T, p.n_experts), torch.float32, "dlogits_aux")
        if xq is not None:
            _expect(xq, (p.T, p.d_model), torch.uint8, "xq")
        _expect(dy, (p.T, p.d_model), dt, "dy")
        if not p.flags & MOE_LOGITS_GIVEN:
            _expect(x, (p.T, p.d_model), dt, "x")
            _expect(w_router, (p.d_model, p.n_experts), dt, "w_router")
        elif x is not None:
            _expect(x, (p.T, p.d_model), dt, "x")
        args = (ctypes.byref(p), _ptr(dy), _ptr(x), _ptr(w_router), _ptr(packed), _ptr(packed_bwd),
                _ptr(fwd.idx), _ptr(fwd.gate), _ptr(fwd.offsets), _ptr(fwd.pos), _ptr(fwd.ws), fwd.ws.numel(),
                _ptr(self.dx), _ptr(self.dlogits), _ptr(self.dw_gate), _ptr(self.dw_up), _ptr(self.dw_down),
                _ptr(self.dw_router), _ptr(self.ws), self.ws.numel(), _stream(stream))
        if dlogits_aux is None and xq is None:
            _check("moe_backward", lib().moe_backward(*args))
        else:
            _check("moe_backward_aux", lib().moe_backward_aux(*args, _ptr(dlogits_aux), _ptr(xq)))
        return dict(dx=self.dx, dlogits=self.dlogits, dw_gate=self.dw_gate, dw_up=self.dw_up,
                    dw_down=self.dw_down, dw_router=self.dw_router)


class Norm(_Operator):
    """Preallocated outputs of moe_norm: y [T, d], rstd [T], with a residual its
    sum [T, d] (put None in its place where nothing reads it), for MXFP8 problems
    the rows' codes q [T, d] and scales q_scale [T, d/32] (uint8) unless quantized
    is False."""

    def __init__(self, p: Problem, device, eps: float = 1e-6, residual: bool = True, quantized: bool | None = None):
        super().__init__(p, device)
        self.eps, self.residual = float(eps), bool(residual)
        (T, d), dt = self._shape, self._dt = _rows(p)
        if quantized is None:
            quantized = p.act == "mxfp8"
        self._buffer("y", (T, d), dt)
        self._buffer("sum", (T, d), dt, residual)
        self._buffer("rstd", (T,), torch.float32)
        self._buffer("q", (T, d), torch.uint8, quantized)
        self._buffer("q_scale", (T, d // 32), torch.uint8, quantized)

    def __call__(self, x, weight, residual=None, stream=None):
        """y = norm(x + residual) weight; returns y."""
        shape, dt = self._shape, self._dt
        _expect(x, shape, dt, "x")
        _expect(weight, shape[1:], dt, "weight")
        if residual is None and self.sum is not None:
            raise ValueError("residual: expected")
        if residual is not None and self.sum is None and not self.residual:
            raise ValueError("residual: not expected")
        if residual is not None:
            _expect(residual, shape, dt, "residual")
        _check("moe_norm", lib().moe_norm(
            self._p, *_inputs(self._index, x, residual, weight), self.eps, _own(self.sum), _own(self.y),
            _own(self.q), _own(self.q_scale), _own(self.rstd), _stream(stream, self._index)))
        return self.y


class NormBackward(_Operator):
    """Preallocated gradients and workspace of moe_norm_backward."""

    def __init__(self, p: Problem, device):
        super().__init__(p, device)
        self._shape, self._dt = _rows(p)
        self._buffer("ws", (_bytes("moe_norm_backward_workspace_bytes", p),), torch.uint8)
        self._buffer("ds", self._shape, self._dt)
        self._buffer("dweight", (p.d_model,), torch.float32)

    def __call__(self, dy, s, weight, rstd, dsum=None, stream=None) -> dict:
        """dy: the gradient of y; s: the forward's sum (x without a residual); dsum: the
        gradient of that sum from elsewhere.  dict(ds, dweight)."""
        shape, dt = self._shape, self._dt
        _expect(dy, shape, dt, "dy")
        _expect(s, shape, dt, "s")
        _expect(weight, shape[1:], dt, "weight")
        _expect(rstd, shape[:1], torch.float32, "rstd")
        if dsum is not None:
            _expect(dsum, shape, dt, "dsum")
        _check("moe_norm_backward", lib().moe_norm_backward(
            self._p, *_inputs(self._index, dy, dsum, s, weight, rstd), _own(self.ds),
            _own(self.dweight), _own(self.ws), self.ws.numel(), _stream(stream, self._index)))
        return dict(ds=self.ds, dweight=self.dweight)


class BalanceLoss(_Operator):
    """Preallocated outputs and workspace of moe_balance_loss and its backward:
    loss [2] (balance, z), counts_live [E + 1] and its parts counts [E] and live [1]
    (tokens), dlogits [T, E]."""

    def __init__(self, p: Problem, device):
        super().__init__(p, device)
        self._shape, self._choices = (p.T, p.n_experts), (p.T, p.top_k)
        self._buffer("ws", (_bytes("moe_balance_workspace_bytes", p),), torch.uint8)
        self._buffer("loss", (2,), torch.float32)
        self._buffer("counts_live", (p.n_experts + 1,), torch.int32)
        self._parts()
        self._buffer("dlogits", self._shape, torch.float32)

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name == "counts_live":
            self._parts()

    def _parts(self):   # made when the buffer changes, not when they are asked for (1.5 us of a pass of 11)
        c = self.counts_live
        self._counts, self._live = (None, None) if c is None else (c[:-1], c[-1:])

    @property
    def counts(self):
        return self._counts

    @property
    def live(self):
        return self._live

    def _expect_logits(self, logits, mask):
        _expect(logits, self._shape, torch.float32, "logits")
        if mask is not None:
            _expect(mask, self._shape[:1], torch.uint8, "mask")

    def __call__(self, logits, idx, mask=None, stream=None):
        """loss [2] of the tokens whose mask (uint8 [T]; None: all) is not zero."""
        self._expect_logits(logits, mask)
        _expect(idx, self._choices, torch.int32, "idx")
        _check("moe_balance_loss", lib().moe_balance_loss(
            self._p, *_inputs(self._index, logits, idx, mask), _own(self.counts_live), _own(self.loss),
            _own(self.ws), self.ws.numel(), _stream(stream, self._index)))
        return self.loss

    def backward(self, logits, dloss, mask=None, stream=None):
        """dlogits for dloss [2], with the counts of the last call."""
        self._expect_logits(logits, mask)
        _expect(dloss, (2,), torch.float32, "dloss")
        logits, mask, dloss = _inputs(self._index, logits, mask, dloss)
        _check("moe_balance_loss_backward", lib().moe_balance_loss_backward(
            self._p, logits, mask, _own(self.counts_live), dloss, _own(self.dlogits),
            _stream(stream, self._index)))
        return self.dlogits


class RouterBackward(_Operator):
    """Preallocated gradients and workspace of moe_router_backward."""

    def __init__(self, p: Problem, device):
        super().__init__(p, device)
        self._shape, self._dt = _rows(p)
        self._logits, self._weight = (p.T, p.n_experts), (p.d_model, p.n_experts)
        self._buffer("ws", (_bytes("moe_router_backward_workspace_bytes", p),), torch.uint8)
        self._buffer("dx", self._shape, self._dt)
        self._buffer("dw_router", self._weight, torch.float32)

    def __call__(self, dlogits, x, w_router, dx_in=None, stream=None) -> dict:
        shape, dt = self._shape, self._dt
        _expect(dlogits, self._logits, torch.float32, "dlogits")
        _expect(x, shape, dt, "x")
        _expect(w_router, self._weight, dt, "w_router")
        if dx_in is not None:
            _expect(dx_in, shape, dt, "dx_in")
        _check("moe_router_backward", lib().moe_router_backward(
            self._p, *_inputs(self._index, dlogits, x, w_router, dx_in), _own(self.dx), _own(self.dw_router),
            _own(self.ws) if self.ws.numel() else None, self.ws.numel(), _stream(stream, self._index)))
        return dict(dx=self.dx, dw_router=self.dw_router)


MOE_DECODE_MAX_TOKENS = 256


def decode_weight_bytes(p: Problem) -> int:
    return _bytes("moe_decode_weight_bytes", p)


def pack_weights_decode(p: Problem, w_gate, w_up, w_down, stream=None) -> torch.Tensor:
    """The MXFP4 weights of moe_decode from bfloat16 ones."""
    E, d, H = p.n_experts, p.d_model, p.d_hidden
    _expect(w_gate, (E, d, H), torch.bfloat16, "w_gate")
    _expect(w_up, (E, d, H), torch.bfloat16, "w_up")
    _expect(w_down, (E, H, d), torch.bfloat16, "w_down")
    weights = _inputs(w_gate.get_device(), w_gate, w_up, w_down)
    packed = torch.empty(decode_weight_bytes(p), dtype=torch.uint8, device=w_gate.device)
    _check("moe_pack_weights_decode", lib().moe_pack_weights_decode(
        ctypes.byref(p), *weights, packed.data_ptr(), _stream(stream)))
    return packed


class Decode(_Operator):
    """Preallocated output and workspace of the block for a few tokens with 4-bit
    weights (moe_decode, moe_decode_experts): y [T, d], logits [T, E], idx and
    gate [T, k]."""

    def __init__(self, p: Problem, device):
        super().__init__(p, device)
        self._shape, self._choices = (p.T, p.d_model), (p.T, p.top_k)
        self.weight_bytes = decode_weight_bytes(p)
        self._buffer("ws", (_bytes("moe_decode_workspace_bytes", p),), torch.uint8)
        self._buffer("y", self._shape, torch.bfloat16)
        self._buffer("logits", (p.T, p.n_experts), torch.float32)
        self._buffer("idx", self._choices, torch.int32)
        self._buffer("gate", self._choices, torch.float32)

    def __call__(self, x, packed, w_router=None, logits=None, stream=None):
        """The block: router logits (or given ones), top-k and gates, experts; returns y."""
        p = self.p
        _expect(x, self._shape, torch.bfloat16, "x")
        _expect(packed, (self.weight_bytes,), torch.uint8, "packed")
        if p.flags & MOE_LOGITS_GIVEN:
            _expect(logits, (p.T, p.n_experts), torch.float32, "logits")
        else:
            _expect(w_router, (p.d_model, p.n_experts), torch.bfloat16, "w_router")
            logits = self.logits
        _check("moe_decode", lib().moe_decode(
            self._p, *_inputs(self._index, x, w_router, logits, packed), _own(self.y), _own(self.idx),
            _own(self.gate), _own(self.ws), self.ws.numel(), _stream(stream, self._index)))
        return self.y

    def experts(self, x, idx, gate, packed, stream=None):
        """The experts idx [T, k] (outside [0, E): unused) of each token, weighted by gate; returns y."""
        _expect(x, self._shape, torch.bfloat16, "x")
        _expect(idx, self._choices, torch.int32, "idx")
        _expect(gate, self._choices, torch.float32, "gate")
        _expect(packed, (self.weight_bytes,), torch.uint8, "packed")
        _check("moe_decode_experts", lib().moe_decode_experts(
            self._p, *_inputs(self._index, x, idx, gate, packed), _own(self.y), _own(self.ws),
            self.ws.numel(), _stream(stream, self._index)))
        return self.y


def set_gemm_grid_cap(cap: int):
    """Cap the grouped GEMMs' persistent grid at `cap` workgroups (multiple of 8, <= 256; 0 = no cap)."""
    _check("moe_set_gemm_grid_cap", lib().moe_set_gemm_grid_cap(int(cap)))


MOE_TEST_FFN_WAIT, MOE_TEST_FFN_GIVE_UP = 1, 2
MOE_STATUS_FORWARD, MOE_STATUS_BACKWARD = 0, 1


def set_test_flags(flags: int):
    """Test hooks of the fused bf16 grouped GEMMs (MOE_TEST_FFN_WAIT: every dependent tile waits
    for its rows before starting, the path taken when they are not yet done; MOE_TEST_FFN_GIVE_UP:
    every such wait ends at once as if its bound had been reached); 0 clears them."""
    _check("moe_set_test_flags", lib().moe_set_test_flags(int(flags)))


def fused_status(p: Problem, ws, which=MOE_STATUS_FORWARD, stream=None) -> int:
    """MOE_OK (0) or MOE_ERR_STATE (-6) from the error word of the last fused grouped-GEMM launch
    on workspace ws (synchronises on the stream)."""
    st = _I32()
    _check("moe_fused_status", lib().moe_fused_status(ctypes.byref(p), _ptr(ws), ws.numel(), int(which),
                                                      ctypes.byref(st), _stream(stream)))
    return st.value


def kernel_times() -> list[tuple[str, float]]:
    """(stage name, milliseconds) of the last profiled moe_forward (synchronises on it)."""
    names = (ctypes.c_char_p * 16)()
    ms = (ctypes.c_float * 16)()
    n = _I32()
    _check("moe_kernel_times", lib().moe_kernel_times(names, ms, 16, ctypes.byref(n)))
    return [(names[i].decode(), float(ms[i])) for i in range(n.value)]


def version() -> str:
    return lib().moe_version().decode()
