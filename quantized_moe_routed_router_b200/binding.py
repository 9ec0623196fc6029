"""ctypes binding of ``libts_moe.so`` (C ABI in ``include/ts_moe.h``).

Argument marshalling only: torch tensors are passed as device pointers plus
the current CUDA stream; every step of the routed half runs in the library's
kernels.  If the library is missing this module raises on import -- there is
no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional, Sequence

import numpy as np
import torch

from . import synth

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libts_moe.so")

TS_MOE_ABI_VERSION = 1
STATUS = {0: "OK", 1: "EINVAL", 2: "EUNSUPPORTED", 3: "ENOMEM", 4: "ECUDA", 5: "EDEVICE"}


class TsMoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class Config(C.Structure):
    _fields_ = [("abi_version", C.c_uint32), ("hidden", C.c_int32), ("moe_inter", C.c_int32),
                ("num_experts", C.c_int32), ("top_k", C.c_int32), ("num_layers", C.c_int32),
                ("max_tokens", C.c_int32), ("expert_fmt", C.c_int32), ("score", C.c_int32),
                ("bias_mode", C.c_int32), ("act", C.c_int32), ("act_alpha", C.c_float), ("act_limit", C.c_float),
                ("shared_inter", C.c_int32), ("device", C.c_int32), ("weights_mem", C.c_int32)]


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("router", "router_xscale", "router_bias", "per_expert_scale", "gate", "up",
                                           "down", "sh_gate", "sh_up", "sh_down")]


class Info(C.Structure):
    _fields_ = [("arena_bytes", C.c_uint64), ("workspace_bytes", C.c_uint64), ("expert_bytes", C.c_uint64),
                ("router_bytes", C.c_uint64), ("shared_bytes", C.c_uint64), ("num_ctas", C.c_int32),
                ("sm_count", C.c_int32), ("launch_tokens", C.c_int32)]


class RmsnormArgs(C.Structure):
    _fields_ = [("rows", C.c_int32), ("hidden", C.c_int32), ("resid_type", C.c_int32), ("delta_type", C.c_int32),
                ("gamma_type", C.c_int32), ("y_type", C.c_int32), ("eps", C.c_float),
                ("resid", C.c_void_p), ("ld_resid", C.c_int64), ("delta", C.c_void_p), ("ld_delta", C.c_int64),
                ("gamma", C.c_void_p), ("resid_out", C.c_void_p), ("ld_resid_out", C.c_int64),
                ("y", C.c_void_p), ("ld_y", C.c_int64), ("q", C.c_void_p), ("ld_q", C.c_int64),
                ("q_scale", C.c_void_p), ("qs_row", C.c_int64), ("qs_group", C.c_int64)]


class ActQuantArgs(C.Structure):
    _fields_ = [("rows", C.c_int32), ("inter", C.c_int32), ("act", C.c_int32), ("in_type", C.c_int32),
                ("act_alpha", C.c_float), ("act_limit", C.c_float),
                ("gate", C.c_void_p), ("ld_gate", C.c_int64), ("up", C.c_void_p), ("ld_up", C.c_int64),
                ("q", C.c_void_p), ("ld_q", C.c_int64), ("q_scale", C.c_void_p), ("qs_row", C.c_int64),
                ("qs_group", C.c_int64)]


class Fp8MatmulArgs(C.Structure):
    _fields_ = [("rows", C.c_int32), ("n", C.c_int32), ("k", C.c_int32), ("num_groups", C.c_int32),
                ("out_type", C.c_int32), ("reserved", C.c_int32),
                ("a", C.c_void_p), ("ld_a", C.c_int64), ("a_scale", C.c_void_p), ("as_row", C.c_int64),
                ("as_block", C.c_int64),
                ("b", C.c_void_p), ("ld_b", C.c_int64), ("b_group", C.c_int64), ("b_scale", C.c_void_p),
                ("bs_group", C.c_int64), ("bs_row", C.c_int64), ("bs_block", C.c_int64),
                ("offsets", C.c_void_p), ("add", C.c_void_p), ("ld_add", C.c_int64),
                ("out", C.c_void_p), ("ld_out", C.c_int64)]


class BalanceArgs(C.Structure):
    _fields_ = [("rows", C.c_int32), ("experts", C.c_int32), ("top_k", C.c_int32), ("score", C.c_int32),
                ("dtype", C.c_int32), ("coef", C.c_float),
                ("logits", C.c_void_p), ("ld_logits", C.c_int64), ("idx", C.c_void_p), ("ld_idx", C.c_int64),
                ("mask", C.c_void_p), ("dloss", C.c_void_p), ("loss", C.c_void_p), ("prob", C.c_void_p),
                ("counts", C.c_void_p), ("offsets", C.c_void_p), ("dlogits", C.c_void_p), ("ld_dlogits", C.c_int64),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_uint64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run quantized_moe_routed_router_b200.build.build()")
    lib = C.CDLL(LIB_PATH)
    vp, i32 = C.c_void_p, C.c_int
    lib.ts_moe_open.argtypes = [C.POINTER(Config), C.POINTER(LayerWeights), C.POINTER(vp)]
    lib.ts_moe_route.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp]
    lib.ts_moe_forward.argtypes = [vp, i32, vp, i32, vp, vp, vp]
    lib.ts_moe_device_status.argtypes = [vp, vp]
    lib.ts_moe_get_info.argtypes = [vp, C.POINTER(Info)]
    lib.ts_moe_set_timing_events.argtypes = [vp, vp]
    lib.ts_moe_last_error.argtypes = [vp]
    lib.ts_moe_last_error.restype = C.c_char_p
    lib.ts_moe_close.argtypes = [vp]
    lib.ts_moe_debug_range_start.argtypes = [C.c_uint64, i32, i32]
    lib.ts_moe_debug_range_start.restype = C.c_uint64
    lib.ts_moe_debug_owner_of.argtypes = [C.c_uint64, i32, C.c_uint64]
    lib.ts_moe_debug_partial_slot.argtypes = [C.c_uint64, i32, i32, C.c_uint64]
    lib.ts_moe_debug_group_size.argtypes = [i32]
    lib.ts_moe_debug_aligned_start.argtypes = [i32, i32, i32, i32]
    lib.ts_moe_debug_aligned_start.restype = C.c_uint64
    lib.ts_moe_debug_use_aligned.argtypes = [i32, i32]
    lib.ts_moe_debug_coresident.argtypes = [i32, i32, i32]
    lib.ts_moe_debug_layer_ctas.argtypes = [i32]
    lib.ts_moe_debug_validate.argtypes = [C.POINTER(Config), C.POINTER(LayerWeights)]
    lib.ts_moe_route_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp]
    lib.ts_moe_debug_skew_barrier.argtypes = [vp, vp]
    lib.ts_moe_rmsnorm.argtypes = [C.POINTER(RmsnormArgs), vp]
    lib.ts_moe_act_quant.argtypes = [C.POINTER(ActQuantArgs), vp]
    lib.ts_moe_fp8_matmul.argtypes = [C.POINTER(Fp8MatmulArgs), vp]
    lib.ts_moe_debug_fp8_matmul_plan.argtypes = [C.POINTER(Fp8MatmulArgs), i32, C.POINTER(C.c_int32)]
    lib.ts_moe_debug_fp8_matmul_plan.restype = None
    lib.ts_moe_debug_fp8_matmul_held.argtypes = [C.POINTER(Fp8MatmulArgs), i32, C.c_uint32, vp]
    lib.ts_moe_balance.argtypes = [C.POINTER(BalanceArgs), vp]
    lib.ts_moe_balance_workspace.argtypes = [C.c_int32, C.c_int32]
    lib.ts_moe_balance_workspace.restype = C.c_uint64
    for f in ("ts_moe_open", "ts_moe_route", "ts_moe_forward", "ts_moe_device_status", "ts_moe_get_info",
              "ts_moe_set_timing_events", "ts_moe_close", "ts_moe_debug_validate", "ts_moe_route_noalloc",
              "ts_moe_debug_skew_barrier", "ts_moe_rmsnorm", "ts_moe_act_quant", "ts_moe_fp8_matmul",
              "ts_moe_balance", "ts_moe_debug_fp8_matmul_held"):
        getattr(lib, f).restype = C.c_int
    return lib


lib = _load()


def make_config(shape: "synth.MoEShape", device: int = 0, weights_mem: int = 0) -> Config:
    return Config(TS_MOE_ABI_VERSION, shape.hidden, shape.moe_inter, shape.num_experts, shape.top_k, shape.num_layers,
                  shape.max_tokens, shape.expert_fmt, shape.score, shape.bias_mode, shape.act, shape.act_alpha,
                  shape.act_limit, shape.shared_inter, device, weights_mem)


def _ptr(a) -> Optional[int]:
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        return a.data_ptr()
    return a.ctypes.data


def layer_struct(L: "synth.LayerBlobs", keep: list) -> LayerWeights:
    """LayerWeights for one layer; host vectors are made contiguous and kept alive in `keep`."""
    def host(a, dt):
        if a is None:
            return None
        a = np.ascontiguousarray(a, dtype=dt)
        keep.append(a)
        return a.ctypes.data

    def blob(t):
        if t is None:
            return None
        t = t.contiguous()
        keep.append(t)
        return t.data_ptr()

    return LayerWeights(blob(L.router), host(L.xscale, np.uint16), host(L.bias, np.float32), host(L.pes, np.float32),
                        blob(L.gate), blob(L.up), blob(L.down), blob(L.sh_gate), blob(L.sh_up), blob(L.sh_down))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class MoE:
    """One ts_moe handle: all layers of `shape`, repacked on `device` at construction."""

    def __init__(self, shape: "synth.MoEShape", layers: Sequence["synth.LayerBlobs"], device: int = 0):
        assert len(layers) == shape.num_layers
        on_dev = layers[0].gate.is_cuda
        self.shape = shape
        self.cfg = make_config(shape, device, 1 if on_dev else 0)
        keep: list = []
        arr = (LayerWeights * shape.num_layers)(*[layer_struct(L, keep) for L in layers])
        h = C.c_void_p()
        st = lib.ts_moe_open(C.byref(self.cfg), arr, C.byref(h))
        if st != 0:
            raise TsMoeError(st, lib.ts_moe_last_error(None).decode())
        self.h = h

    def _check(self, st: int):
        if st != 0:
            raise TsMoeError(st, lib.ts_moe_last_error(self.h).decode())

    def route(self, layer: int, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor,
              logits: Optional[torch.Tensor] = None, stream=None):
        M = x.shape[0] if x is not None else 0
        self._check(lib.ts_moe_route(self.h, layer, _ptr(x), M, _ptr(idx), _ptr(w), _ptr(logits), _stream(stream)))

    def forward(self, layer: int, x: torch.Tensor, resid: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, stream=None, M: Optional[int] = None):
        if M is None:
            M = x.shape[0]
        self._check(lib.ts_moe_forward(self.h, layer, _ptr(x), M, _ptr(resid), _ptr(y), _stream(stream)))

    def forward_ptr(self, layer: int, x_ptr: int, M: int, resid_ptr: Optional[int], y_ptr: Optional[int],
                    stream: int):
        self._check(lib.ts_moe_forward(self.h, layer, x_ptr, M, resid_ptr, y_ptr, stream))

    def device_status(self, stream=None):
        self._check(lib.ts_moe_device_status(self.h, _stream(stream)))

    def info(self) -> Info:
        i = Info()
        self._check(lib.ts_moe_get_info(self.h, C.byref(i)))
        return i

    def set_timing_events(self, events: Optional[Sequence[torch.cuda.Event]]):
        if events is None:
            self._check(lib.ts_moe_set_timing_events(self.h, None))
            return
        self._evs = list(events)
        for e in self._evs:
            if not e.cuda_event:          # torch creates the CUDA event on first record
                e.record()
        arr = (C.c_void_p * 4)(*[e.cuda_event for e in self._evs])
        self._check(lib.ts_moe_set_timing_events(self.h, arr))

    def close(self):
        if getattr(self, "h", None):
            lib.ts_moe_close(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def route_noalloc(router: torch.Tensor, bias: Optional[torch.Tensor], pes: Optional[torch.Tensor], num_experts: int,
                  hidden: int, top_k: int, score: int, bias_mode: int, x: torch.Tensor, idx: torch.Tensor,
                  w: torch.Tensor, logits: Optional[torch.Tensor] = None, stream=None):
    """Router GEMV + top-k without a handle and without any device allocation
    (scratch lives in the library's static device array).  router: device Q8_0
    blob [E][H]; bias / pes: device float32 [E] or None; x: device bf16 [M][H]."""
    M = x.shape[0]
    st = lib.ts_moe_route_noalloc(_ptr(router), _ptr(bias), _ptr(pes), num_experts, hidden, top_k, score, bias_mode,
                                  _ptr(x), M, _ptr(idx), _ptr(w), _ptr(logits), _stream(stream))
    if st != 0:
        raise TsMoeError(st, lib.ts_moe_last_error(None).decode())


# ----------------------------------------------------------------------------- the operators next to the routed half

_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _refuse(msg: str):
    raise TsMoeError(1, msg)


def _check_op(st: int):
    if st != 0:
        raise TsMoeError(st, lib.ts_moe_last_error(None).decode())


def _rows(t: torch.Tensor, what: str, rows: int, cols: int, dev: int) -> int:
    """The row stride of a [rows][cols] tensor on device `dev` (-1: the CPU) with a contiguous last dimension."""
    if t.get_device() != dev:
        _refuse(f"{what} is on {t.device}, not on {_name(dev)}")
    if t.shape != (rows, cols):
        _refuse(f"{what} has shape {tuple(t.shape)}, not {(rows, cols)}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        _refuse(f"{what} needs a contiguous last dimension")
    return ld if rows > 1 else max(ld, cols)


def _dims(t: torch.Tensor, what: str, dims: str) -> tuple:
    """The sizes of a tensor of two dimensions."""
    try:
        rows, cols = t.shape
    except ValueError:
        _refuse(f"{what} must be [{dims}], not {list(t.shape)}")
    return rows, cols


def _name(dev: int) -> str:
    return "cpu" if dev < 0 else f"cuda:{dev}"


def _type(t: torch.Tensor, what: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        _refuse(f"{what} is {t.dtype}; bfloat16, float16 or float32 is needed")
    return dt


def _flat(t: torch.Tensor, what: str, n: int, dtype, dev: int) -> int:
    if t.get_device() != dev or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        _refuse(f"{what} must be a contiguous {dtype} tensor of {n} elements on {_name(dev)}")
    return t.data_ptr()


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _codes(t: torch.Tensor, what: str):
    if t.dtype not in _CODES:
        _refuse(f"{what} is {t.dtype}; float8_e4m3fn (or its bytes as uint8) is needed")


def _scales(t: torch.Tensor, what: str, shape: tuple, dev: int) -> tuple:
    if t.get_device() != dev or t.dtype != torch.float32 or t.shape != shape:
        _refuse(f"{what} must be a float32 tensor of shape {shape} on {_name(dev)}")
    return t.stride()


# The current stream's handle.  torch.cuda.current_stream(dev).cuda_stream builds an object for it, which takes 2 us; the
# direct call is torch's own but not public, so it may be missing.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Op:
    """An entry point whose argument struct is packed in one go: building the ctypes struct costs a decode step's call
    about a microsecond more."""

    def __init__(self, name: str, fmt: str, args: type):
        self.pack = struct.Struct(fmt).pack
        assert struct.calcsize(fmt) == C.sizeof(args)
        self.fn = lib[name]      # a function object of its own: the struct goes in as bytes
        self.fn.argtypes, self.fn.restype = [C.c_char_p, C.c_void_p], C.c_int

    def __call__(self, dev: int, stream, *fields):
        """Calls on the tensors' own device and, without a stream, on that device's current stream."""
        if dev < 0:
            _refuse("the tensors must be on a CUDA device")
        if stream is None:
            stream = _current_stream(dev)
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device.index != dev:
                _refuse(f"the stream belongs to {stream.device}, the tensors to {_name(dev)}")
            stream = stream.cuda_stream
        try:
            args = self.pack(*fields)
        except struct.error as e:
            _refuse(f"an argument does not fit its field: {e}")
        if torch.cuda.current_device() == dev:
            st = self.fn(args, stream)
        else:
            with torch.cuda.device(dev):
                st = self.fn(args, stream)
        if st != 0:
            _check_op(st)


_rmsnorm = _Op("ts_moe_rmsnorm", "@6ifPqPqPPqPqPqPqq", RmsnormArgs)
_act_quant = _Op("ts_moe_act_quant", "@4i2fPqPqPqPqq", ActQuantArgs)
_fp8_matmul = _Op("ts_moe_fp8_matmul", "@6iPqPqqPqqPqqqPPqPq", Fp8MatmulArgs)
_balance = _Op("ts_moe_balance", "@5ifPqPqPPPPPPPqPQ", BalanceArgs)


def rmsnorm(resid: torch.Tensor, gamma: Optional[torch.Tensor], eps: float, delta: Optional[torch.Tensor] = None,
            resid_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
            q: Optional[torch.Tensor] = None, q_scale: Optional[torch.Tensor] = None, stream=None):
    """ts_moe_rmsnorm: r = resid + delta (kept in resid_out, which may be resid),
    v = r / sqrt(mean(r^2) + eps) * gamma, written to y [M, H] and/or as 8-bit
    rows to q [M, H] with q_scale [M, ceil(H / 128)] (any strides)."""
    M, H = _dims(resid, "resid", "M, H")
    dev = resid.get_device()
    rt = _type(resid, "resid")
    ld = _rows(resid, "resid", M, H, dev)
    pd = ldd = td = pg = tg = po = ldo = py = ldy = ty = pq = ldq = ps = qr = qg = 0
    if delta is not None:
        pd, ldd, td = delta.data_ptr(), _rows(delta, "delta", M, H, dev), _type(delta, "delta")
    if gamma is not None:
        pg, tg = _flat(gamma, "gamma", H, gamma.dtype, dev), _type(gamma, "gamma")
    if resid_out is not None:
        if resid_out.dtype != resid.dtype:
            _refuse("resid_out must have resid's type")
        po, ldo = resid_out.data_ptr(), _rows(resid_out, "resid_out", M, H, dev)
    if y is not None:
        py, ldy, ty = y.data_ptr(), _rows(y, "y", M, H, dev), _type(y, "y")
    if q is not None:
        _codes(q, "q")
        pq, ldq = q.data_ptr(), _rows(q, "q", M, H, dev)
    if q_scale is not None:
        qr, qg = _scales(q_scale, "q_scale", (M, -(-H // 128)), dev)
        ps = q_scale.data_ptr()
    if M == 0:
        return
    _rmsnorm(dev, stream, M, H, rt, td, tg, ty, eps, resid.data_ptr(), ld, pd, ldd, pg, po, ldo, py, ldy, pq, ldq, ps, qr, qg)


def act_quant(gate: torch.Tensor, up: torch.Tensor, act: int, q: torch.Tensor, q_scale: torch.Tensor,
              act_alpha: float = 1.702, act_limit: float = 7.0, stream=None):
    """ts_moe_act_quant: the activation of gate and up ([M, I], e.g. two halves
    of one product) as 8-bit rows q [M, I] with q_scale [M, ceil(I / 128)]."""
    M, inter = _dims(gate, "gate", "M, I")
    dev = gate.get_device()
    if up.dtype != gate.dtype:
        _refuse("gate and up must have one type")
    _codes(q, "q")
    qs = _scales(q_scale, "q_scale", (M, -(-inter // 128)), dev)
    fields = (M, inter, act, _type(gate, "gate"), act_alpha, act_limit,
              gate.data_ptr(), _rows(gate, "gate", M, inter, dev), up.data_ptr(), _rows(up, "up", M, inter, dev),
              q.data_ptr(), _rows(q, "q", M, inter, dev), q_scale.data_ptr(), qs[0], qs[1])
    if M == 0:
        return
    _act_quant(dev, stream, *fields)


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, out: torch.Tensor,
               add: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None, stream=None):
    """ts_moe_fp8_matmul: out [M, N] = a [M, K] b^T with scales per row and 128
    columns (a_scale [M, ceil(K / 128)]) and per 128 x 128 block (b_scale
    [ceil(N / 128), ceil(K / 128)]), plus add [M, N] in out's type (out itself
    is allowed).  b is [N, K], or with offsets (int32 [G + 1] on the device)
    [G, N, K] with b_scale [G, ..., ...]: rows offsets[g] .. offsets[g + 1] - 1
    use b[g], other rows of out are left as they were."""
    M, K = _dims(a, "a", "M, K")
    N = _dims(out, "out", "M, N")[1]
    dev = a.get_device()
    kb = -(-K // 128)
    _codes(a, "a")
    _codes(b, "b")
    sa = _scales(a_scale, "a_scale", (M, kb), dev)
    if offsets is None:
        G, group, ldb, off = 1, 0, _rows(b, "b", N, K, dev), 0
        sb = (0, *_scales(b_scale, "b_scale", (-(-N // 128), kb), dev))
    else:
        if b.dim() != 3 or b.shape[0] < 1:
            _refuse("b must be [G, N, K] when offsets are given")
        G, group, ldb = b.shape[0], b.stride(0), _rows(b[0], "b[g]", N, K, dev)
        sb = _scales(b_scale, "b_scale", (G, -(-N // 128), kb), dev)
        off = _flat(offsets, "offsets", G + 1, torch.int32, dev)
    pa = lda = 0
    if add is not None:
        if add.dtype != out.dtype:
            _refuse("add must have out's type")
        pa, lda = add.data_ptr(), _rows(add, "add", M, N, dev)
    fields = (M, N, K, G, _type(out, "out"), 0, a.data_ptr(), _rows(a, "a", M, K, dev), a_scale.data_ptr(), *sa,
              b.data_ptr(), ldb, group, b_scale.data_ptr(), *sb, off, pa, lda, out.data_ptr(), _rows(out, "out", M, N, dev))
    if M == 0:
        return
    _fp8_matmul(dev, stream, *fields)


def balance(logits: torch.Tensor, idx: torch.Tensor, score: int, loss: torch.Tensor, counts: torch.Tensor,
            prob: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
            dlogits: Optional[torch.Tensor] = None, dloss: Optional[torch.Tensor] = None, coef: float = 1.0,
            offsets: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """ts_moe_balance: per-expert counts (int32 [E]) and their running sum
    (offsets, int32 [E + 1]), the mean probabilities prob (float32 [E]), the
    balance loss (float32, one element) and, with dlogits [M, E], its gradient
    times dloss (float32, one element; None = 1).  mask: bool or uint8 [M], rows
    that count.  Without a workspace one is taken from torch's allocator."""
    M, E = _dims(logits, "logits", "M, E")
    K = _dims(idx, "idx", "M, K")[1]
    dev = logits.get_device()
    if idx.dtype != torch.int32:
        _refuse(f"idx is {idx.dtype}; int32 is needed")
    pm = pd = pp = po = pg = ldg = 0
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            _refuse(f"mask is {mask.dtype}; bool or uint8 is needed")
        pm = _flat(mask, "mask", M, mask.dtype, dev)
    if dloss is not None:
        pd = _flat(dloss, "dloss", 1, torch.float32, dev)
    if prob is not None:
        pp = _flat(prob, "prob", E, torch.float32, dev)
    if offsets is not None:
        po = _flat(offsets, "offsets", E + 1, torch.int32, dev)
    if dlogits is not None:
        if dlogits.dtype != logits.dtype:
            _refuse("dlogits must have the type of logits")
        pg, ldg = dlogits.data_ptr(), _rows(dlogits, "dlogits", M, E, dev)
    fields = (M, E, K, score, _type(logits, "logits"), coef, logits.data_ptr(), _rows(logits, "logits", M, E, dev),
              idx.data_ptr(), _rows(idx, "idx", M, K, dev), pm, pd, _flat(loss, "loss", 1, torch.float32, dev), pp,
              _flat(counts, "counts", E, torch.int32, dev), po, pg, ldg)
    if workspace is None:
        if dev < 0:
            _refuse("the tensors must be on a CUDA device")
        need = lib.ts_moe_balance_workspace(M, E)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
        elif isinstance(stream, torch.cuda.Stream):
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
        else:
            _refuse("a raw stream handle needs a workspace of the caller's")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(f"workspace must be a contiguous tensor on {_name(dev)}")
    _balance(dev, stream, *fields, workspace.data_ptr(), workspace.numel() * workspace.element_size())


def validate(shape: "synth.MoEShape", layers: Sequence["synth.LayerBlobs"], **cfg_over) -> tuple:
    """Runs the library's host-side open-time validation only (no CUDA); returns (status, message)."""
    cfg = make_config(shape)
    for k, v in cfg_over.items():
        setattr(cfg, k, v)
    keep: list = []
    arr = (LayerWeights * max(1, len(layers)))(*[layer_struct(L, keep) for L in layers])
    st = lib.ts_moe_debug_validate(C.byref(cfg), arr)
    return st, lib.ts_moe_last_error(None).decode()
