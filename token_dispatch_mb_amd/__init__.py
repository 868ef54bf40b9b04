"""Python binding of libmoebal (include/moebal.h).

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every step of plan / dispatch / combine runs in the HIP
kernels of ``libmoebal.so``. There is no fallback: importing this package
fails if the library is not built.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoebal.so")

F32, BF16, FP8_E4M3, MX4 = 0, 1, 2, 3
DTYPES = {"f32": F32, "bf16": BF16, "fp8": FP8_E4M3, "mx4": MX4}
TORCH_DTYPES = {F32: torch.float32, BF16: torch.bfloat16, FP8_E4M3: torch.uint8}
ELT_BYTES = {F32: 4, BF16: 2, FP8_E4M3: 1}

OK, ERR_INVALID_ARG, ERR_WORKSPACE, ERR_HIP = 0, -1, -2, -3
ST_BAD_ID, ST_DUP_ID, ST_UNBALANCED, ST_CAPACITY = 1, 2, 4, 8
ST_FATAL = ST_BAD_ID | ST_DUP_ID | ST_CAPACITY

MAX_RANKS, MAX_EXPERTS, MAX_TOPK, MAX_SLOTS = 64, 1024, 32, 16

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; build it with `python -c 'import __graft_entry__ as g; g.build()'`"
    )
_lib = ctypes.CDLL(LIB_PATH)


class Dims(ctypes.Structure):
    """mb_dims."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_tokens", "top_k", "n_experts", "n_ranks", "slots_per_rank", "hidden", "cap",
        "dtype_in", "dtype_out")]

    @classmethod
    def make(cls, n_tokens, top_k, n_experts, n_ranks, slots_per_rank, hidden, cap=None,
             dtype_in="bf16", dtype_out="bf16") -> "Dims":
        if cap is None:
            cap = (n_tokens // n_ranks) * top_k if n_ranks else 0
        di = DTYPES[dtype_in] if isinstance(dtype_in, str) else dtype_in
        do = DTYPES[dtype_out] if isinstance(dtype_out, str) else dtype_out
        return cls(n_tokens, top_k, n_experts, n_ranks, slots_per_rank, hidden, max(cap, 1), di, do)

    @classmethod
    def for_workload(cls, wl, cap=None, n_tokens=None) -> "Dims":
        n = wl.n_tokens if n_tokens is None else n_tokens
        if cap is None and n_tokens is None:
            cap = wl.cap
        return cls.make(n, wl.top_k, wl.n_experts, wl.n_ranks, wl.slots_per_rank, wl.hidden,
                        cap=cap, dtype_in=wl.dtype_in, dtype_out=wl.dtype_out)

    @property
    def eh(self) -> int:
        return self.n_experts // self.n_ranks

    @property
    def n_slots(self) -> int:
        return self.eh + self.slots_per_rank

    @property
    def rows(self) -> int:
        return self.n_ranks * self.cap


_i32p = ctypes.POINTER(ctypes.c_int32)


class _PlanBufsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "counts", "load_pre", "load_post", "rep_expert", "slot_quota", "cu_seqlens", "pos",
        "row_src", "status")]


_vp = ctypes.c_void_p
_lib.mb_version.restype = ctypes.c_int
_lib.mb_strerror.argtypes = [ctypes.c_int]
_lib.mb_strerror.restype = ctypes.c_char_p
_lib.mb_plan_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
_lib.mb_plan_workspace_bytes.restype = ctypes.c_size_t
_lib.mb_plan.argtypes = [ctypes.POINTER(Dims), _vp, _vp, ctypes.c_size_t,
                         ctypes.POINTER(_PlanBufsC), _vp]
_lib.mb_plan.restype = ctypes.c_int
_lib.mb_plan_noalloc.argtypes = [ctypes.POINTER(Dims), _vp, ctypes.POINTER(_PlanBufsC), _vp]
_lib.mb_plan_noalloc.restype = ctypes.c_int
_lib.mb_plan_weighted.argtypes = [ctypes.POINTER(Dims), _vp, _i32p, _vp, ctypes.c_size_t,
                                  ctypes.POINTER(_PlanBufsC), _vp]
_lib.mb_plan_weighted.restype = ctypes.c_int


class DriftParams(ctypes.Structure):
    """mb_drift_params: replan when d > delta_num / delta_den, checked every
    check_every calls, reference of up to `window` calls; a kept placement
    replayed above cap or (tol_den > 0) above (1 + tol_num / tol_den) times a
    target replans in the same call. tol_num = tol_den = 0 (the default)
    guards cap only."""
    _fields_ = [(n, ctypes.c_int32) for n in ("delta_num", "delta_den", "window", "check_every",
                                             "tol_num", "tol_den")]


class _PlanOptionsC(ctypes.Structure):
    _fields_ = [("rank_speed", _i32p), ("drift", ctypes.POINTER(DriftParams)),
                ("drift_state", _vp), ("quota_repair", ctypes.c_int32)]


_lib.mb_plan_ex.argtypes = [ctypes.POINTER(Dims), _vp, ctypes.POINTER(_PlanOptionsC), _vp,
                            ctypes.c_size_t, ctypes.POINTER(_PlanBufsC), _vp]
_lib.mb_plan_ex.restype = ctypes.c_int
_lib.mb_drift_state_bytes.argtypes = [ctypes.POINTER(Dims)]
_lib.mb_drift_state_bytes.restype = ctypes.c_size_t
_lib.mb_plan_drift.argtypes = [ctypes.POINTER(Dims), _vp, _i32p, ctypes.POINTER(DriftParams), _vp,
                               _vp, ctypes.c_size_t, ctypes.POINTER(_PlanBufsC), _vp]
_lib.mb_plan_drift.restype = ctypes.c_int
_lib.mb_dispatch.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _vp, _vp, _vp,
                             _vp, _vp]
_lib.mb_dispatch.restype = ctypes.c_int
_lib.mb_combine.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _vp, _vp, _vp, _vp]
_lib.mb_combine.restype = ctypes.c_int
_lib.mb_combine_fp8.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _vp, _vp, _vp,
                                _vp, _vp]
_lib.mb_combine_fp8.restype = ctypes.c_int
_lib.mb_plan_status.argtypes = [ctypes.POINTER(_PlanBufsC), _vp, _i32p]
_lib.mb_plan_status.restype = ctypes.c_int

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
ACT_NONE, ACT_SWIGLU = 0, 1
ACTS = {"none": ACT_NONE, "swiglu": ACT_SWIGLU}
MAX_GROUPS, MAX_NORM_HIDDEN, MAX_LORA_RANK = 64, 16384, 256


class RouteParams(ctypes.Structure):
    """mb_route_params."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_tokens", "n_experts", "top_k", "dtype", "score", "n_groups", "top_groups", "group_top",
        "renorm")] + [("scale", ctypes.c_float)]

    @classmethod
    def make(cls, n_tokens, n_experts, top_k, dtype="f32", score="softmax", n_groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0) -> "RouteParams":
        return cls(n_tokens, n_experts, top_k, DTYPES[dtype] if isinstance(dtype, str) else dtype,
                   SCORES[score] if isinstance(score, str) else score, n_groups, top_groups,
                   group_top, int(bool(renorm)), scale)


_i32, _f32 = ctypes.c_int32, ctypes.c_float
_lib.mb_route.argtypes = [ctypes.POINTER(RouteParams), _vp, _vp, _vp, _vp, _vp]
_lib.mb_route.restype = ctypes.c_int
_lib.mb_rmsnorm_fp8.argtypes = [_i32, _i32, _i32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.mb_rmsnorm_fp8.restype = ctypes.c_int
_lib.mb_quantize_mx4.argtypes = [_i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mb_quantize_mx4.restype = ctypes.c_int
_lib.mb_dequantize_mx4.argtypes = [_i32, _i32, _i32, _vp, _vp, _vp, _vp]
_lib.mb_dequantize_mx4.restype = ctypes.c_int
_lib.mb_expert_mx4.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _i32, _i32, _vp,
                               _vp, _vp, _vp, _vp, _vp]
_lib.mb_expert_mx4.restype = ctypes.c_int


class LoraParams(ctypes.Structure):
    """mb_lora_params."""

    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_rows", "n_out", "k_in", "rank", "n_adapters", "dtype_out")]

    @classmethod
    def make(cls, n_rows, n_out, k_in, rank, n_adapters, dtype_out="bf16") -> "LoraParams":
        return cls(n_rows, n_out, k_in, rank, n_adapters,
                   DTYPES[dtype_out] if isinstance(dtype_out, str) else dtype_out)


_lib.mb_combine_grad.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _vp, _vp, _vp,
                                 _vp, _vp, _vp]
_lib.mb_combine_grad.restype = ctypes.c_int
_lib.mb_lora_workspace_bytes.argtypes = [ctypes.POINTER(LoraParams)]
_lib.mb_lora_workspace_bytes.restype = ctypes.c_size_t
_lib.mb_project_lora.argtypes = [ctypes.POINTER(LoraParams), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 ctypes.c_size_t, _vp, _vp]
_lib.mb_project_lora.restype = ctypes.c_int
_lib.mb_expert_bf16.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _i32, _i32, _i32,
                                _vp, _vp, _vp, _vp, _vp]
_lib.mb_expert_bf16.restype = ctypes.c_int
_lib.mb_expert_bf16_dgrad.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _i32, _i32,
                                      _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mb_expert_bf16_dgrad.restype = ctypes.c_int
_lib.mb_expert_bf16_wgrad.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_PlanBufsC), _i32, _i32,
                                      _i32, _i32, _vp, _vp, _vp, _vp]
_lib.mb_expert_bf16_wgrad.restype = ctypes.c_int

EXPORTS = ("mb_version", "mb_strerror", "mb_plan_workspace_bytes", "mb_plan",
           "mb_plan_noalloc", "mb_plan_weighted", "mb_drift_state_bytes", "mb_plan_drift", "mb_plan_ex",
           "mb_dispatch", "mb_combine", "mb_combine_fp8", "mb_plan_status", "mb_route",
           "mb_rmsnorm_fp8", "mb_quantize_mx4", "mb_dequantize_mx4", "mb_expert_mx4",
           "mb_expert_bf16", "mb_expert_bf16_dgrad", "mb_expert_bf16_wgrad", "mb_combine_grad",
           "mb_lora_workspace_bytes", "mb_project_lora")
ST_REPLANNED = 16
ST_GUARDED = 32
NOALLOC_WS_BYTES = 4 << 20
MAX_WINDOW = 4096
MAX_SPEED = 1 << 20


class MoebalError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")
        self.code = code


def version() -> int:
    return _lib.mb_version()


def strerror(code: int) -> str:
    return _lib.mb_strerror(code).decode()


def workspace_bytes(dims: Dims) -> int:
    return int(_lib.mb_plan_workspace_bytes(ctypes.byref(dims)))


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _check(t, name: str, dtype=None, numel: int | None = None, nbytes: int | None = None) -> None:
    """Refuse, before any C call, what the kernels cannot take: a tensor off
    the GPU (a host pointer would fault the device), a strided view, a wrong
    dtype or too few elements / bytes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (it is on {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (it is {t.dtype})")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, {numel} needed")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, {nbytes} needed")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _speeds(dims: "Dims", speeds):
    if len(speeds) < dims.n_ranks:
        raise ValueError(f"speeds lists {len(speeds)} ranks, {dims.n_ranks} needed")
    return (ctypes.c_int32 * dims.n_ranks)(*[int(v) for v in speeds[: dims.n_ranks]])


def _dims_key(dims: "Dims") -> tuple:
    return (dims.n_tokens, dims.top_k, dims.n_experts, dims.n_ranks, dims.slots_per_rank,
            dims.hidden, dims.cap, dims.dtype_in, dims.dtype_out)


# handle of a device's current stream, without a Stream object for it (1.5 us
# of a call); absent in builds of torch without GPU support
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, *tensors) -> ctypes.c_void_p:
    """The stream's HIP handle (torch's current stream by default), after
    checking that the given tensors live on the stream's GPU (a pointer into
    another GPU's memory would fault in the kernel)."""
    if stream is None:
        if _raw_stream is not None:
            at = torch.cuda.current_device()
            for t in tensors:
                if t is not None and t.get_device() != at:
                    raise ValueError(f"a tensor is on {t.device}, the stream on cuda:{at}")
            return ctypes.c_void_p(_raw_stream(at))
        stream = torch.cuda.current_stream()
    dev = stream.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"a tensor is on {t.device}, the stream on {dev}")
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class PlanBuffers:
    """Caller-owned device outputs of mb_plan (torch int32 tensors)."""

    counts: torch.Tensor
    load_pre: torch.Tensor
    load_post: torch.Tensor
    rep_expert: torch.Tensor
    slot_quota: torch.Tensor
    cu_seqlens: torch.Tensor
    pos: torch.Tensor
    row_src: torch.Tensor
    status: torch.Tensor
    _key: tuple | None = field(default=None, init=False, repr=False, compare=False)
    _c: _PlanBufsC | None = field(default=None, init=False, repr=False, compare=False)

    @classmethod
    def allocate(cls, dims: Dims, device) -> "PlanBuffers":
        P, E, R, N, K = dims.n_ranks, dims.n_experts, dims.slots_per_rank, dims.n_tokens, dims.top_k
        ns = dims.n_slots
        z = lambda *s: torch.empty(s, dtype=torch.int32, device=device)  # noqa: E731
        return cls(counts=z(P, E), load_pre=z(P), load_post=z(P), rep_expert=z(P, max(R, 1)),
                   slot_quota=z(P, ns), cu_seqlens=z(P, ns + 1), pos=z(N, K),
                   row_src=z(dims.rows), status=z(4))

    def check(self, dims: Dims) -> None:
        """Every buffer an int32 GPU tensor with room for its output."""
        P, E, R, N, K, ns = (dims.n_ranks, dims.n_experts, dims.slots_per_rank, dims.n_tokens,
                             dims.top_k, dims.n_slots)
        need = {"counts": P * E, "load_pre": P, "load_post": P, "rep_expert": P * R,
                "slot_quota": P * ns, "cu_seqlens": P * (ns + 1), "pos": N * K,
                "row_src": dims.rows, "status": 4}
        for name, n in need.items():
            _check(getattr(self, name), name, torch.int32, numel=n)
            if getattr(self, name).device != self.status.device:
                raise ValueError(f"{name} is on another GPU than status")

    def c_struct(self, dims: Dims | None = None) -> _PlanBufsC:
        """The mb_plan_bufs of these tensors; with `dims`, checked against
        them first (once per set of pointers and sizes)."""
        ts = (self.counts, self.load_pre, self.load_post, self.rep_expert, self.slot_quota,
              self.cu_seqlens, self.pos, self.row_src, self.status)
        ptrs = tuple([t.data_ptr() for t in ts])
        if dims is None:
            return self._c if self._key is not None and self._key[0] == ptrs else _PlanBufsC(*ptrs)
        # the key holds the sizes too: a smaller tensor at the same address
        # is checked again
        key = (ptrs, _dims_key(dims), tuple([t.numel() for t in ts]),
               tuple([t.is_contiguous() for t in ts]))
        if key != self._key:
            self.check(dims)
            self._c, self._key = _PlanBufsC(*ptrs), key
        return self._c


def alloc_workspace(dims: Dims, device) -> torch.Tensor:
    n = workspace_bytes(dims)
    if n == 0:
        raise MoebalError("mb_plan_workspace_bytes", ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def plan(dims: Dims, ids: torch.Tensor, ws: torch.Tensor, bufs: PlanBuffers, stream=None,
         speeds=None, drift=None, repair: bool = False) -> None:
    """mb_plan: enqueue the plan of one MoE layer call on `stream`; with
    ``speeds`` (P host ints), mb_plan_weighted; with ``drift`` =
    (DriftParams, state tensor), mb_plan_drift; with ``repair``, mb_plan_ex
    (any of the three options)."""
    _check(ids, "ids", torch.int32, numel=dims.n_tokens * dims.top_k)
    _check(ws, "ws")
    cb = bufs.c_struct(dims)
    sp = None if speeds is None else _speeds(dims, speeds)
    if drift is not None:
        prm, state = drift
        _check(state, "drift state", nbytes=int(_lib.mb_drift_state_bytes(ctypes.byref(dims))))
    st = _stream(stream, ids, ws, bufs.status, drift[1] if drift is not None else None)
    if repair:
        opt = _PlanOptionsC(ctypes.cast(sp, _i32p) if sp is not None else None,
                            ctypes.pointer(drift[0]) if drift else None,
                            _ptr(drift[1]) if drift else None, 1)
        rc = _lib.mb_plan_ex(ctypes.byref(dims), _ptr(ids), ctypes.byref(opt), _ptr(ws),
                             _nbytes(ws), ctypes.byref(cb), st)
        if rc != OK:
            raise MoebalError("mb_plan_ex", rc)
        return
    if drift is not None:
        rc = _lib.mb_plan_drift(ctypes.byref(dims), _ptr(ids), sp, ctypes.byref(prm), _ptr(state),
                                _ptr(ws), _nbytes(ws), ctypes.byref(cb), st)
        if rc != OK:
            raise MoebalError("mb_plan_drift", rc)
        return
    if sp is None:
        rc = _lib.mb_plan(ctypes.byref(dims), _ptr(ids), _ptr(ws), _nbytes(ws), ctypes.byref(cb), st)
        if rc != OK:
            raise MoebalError("mb_plan", rc)
        return
    rc = _lib.mb_plan_weighted(ctypes.byref(dims), _ptr(ids), sp, _ptr(ws), _nbytes(ws),
                               ctypes.byref(cb), st)
    if rc != OK:
        raise MoebalError("mb_plan_weighted", rc)


def plan_noalloc(dims: Dims, ids: torch.Tensor, bufs: PlanBuffers, stream=None) -> None:
    """mb_plan_noalloc: mb_plan with the library's own per-GPU workspace (no
    workspace argument; calls on one GPU must not overlap in time)."""
    _check(ids, "ids", torch.int32, numel=dims.n_tokens * dims.top_k)
    cb = bufs.c_struct(dims)
    rc = _lib.mb_plan_noalloc(ctypes.byref(dims), _ptr(ids), ctypes.byref(cb),
                              _stream(stream, ids, bufs.status))
    if rc != OK:
        raise MoebalError("mb_plan_noalloc", rc)


def dispatch(dims: Dims, bufs: PlanBuffers, x: torch.Tensor, buf: torch.Tensor,
             x_scale: torch.Tensor | None = None, buf_scale: torch.Tensor | None = None,
             stream=None) -> None:
    """mb_dispatch: buf[pos[t][k]] = x[t] (and the scale rows: fp32
    [N, H/128] for fp8, uint8 [N, H/32] for 4-bit rows)."""
    row = dims.hidden // 2 if dims.dtype_in == MX4 else dims.hidden * ELT_BYTES.get(dims.dtype_in, 0)
    _check(x, "x", nbytes=dims.n_tokens * row)
    _check(buf, "buf", nbytes=dims.rows * row)
    if dims.dtype_in == FP8_E4M3:
        _check(x_scale, "x_scale", torch.float32, numel=dims.n_tokens * (dims.hidden // 128))
        _check(buf_scale, "buf_scale", torch.float32, numel=dims.rows * (dims.hidden // 128))
    elif dims.dtype_in == MX4:
        _check(x_scale, "x_scale", torch.uint8, numel=dims.n_tokens * (dims.hidden // 32))
        _check(buf_scale, "buf_scale", torch.uint8, numel=dims.rows * (dims.hidden // 32))
    rc = _lib.mb_dispatch(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), _ptr(x),
                          _ptr(x_scale), _ptr(buf), _ptr(buf_scale),
                          _stream(stream, x, buf, x_scale, buf_scale, bufs.status))
    if rc != OK:
        raise MoebalError("mb_dispatch", rc)


def combine(dims: Dims, bufs: PlanBuffers, y_exp: torch.Tensor, w: torch.Tensor, y: torch.Tensor,
            stream=None) -> None:
    """mb_combine: y[t] = sum_k w[t][k] * y_exp[pos[t][k]] (fp32 accumulation)."""
    row = dims.hidden * ELT_BYTES.get(dims.dtype_out, 0)
    _check(y_exp, "y_exp", nbytes=dims.rows * row)
    _check(w, "w", torch.float32, numel=dims.n_tokens * dims.top_k)
    _check(y, "y", nbytes=dims.n_tokens * row)
    rc = _lib.mb_combine(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), _ptr(y_exp), _ptr(w),
                         _ptr(y), _stream(stream, y_exp, w, y, bufs.status))
    if rc != OK:
        raise MoebalError("mb_combine", rc)


def alloc_drift_state(dims: Dims, device) -> torch.Tensor:
    """A zero-filled (fresh) drift state buffer for one layer."""
    n = _lib.mb_drift_state_bytes(ctypes.byref(dims))
    if n == 0:
        raise MoebalError("mb_drift_state_bytes", ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def drift_header(state: torch.Tensor) -> dict:
    """The mb_drift_header fields of a state buffer (copies to the host)."""
    import numpy as np

    b = state[:64].cpu().numpy().tobytes()
    i32 = np.frombuffer(b[:16], np.int32)
    i64 = np.frombuffer(b[16:32], np.int64)
    return {"have_plan": int(i32[0]), "countdown": int(i32[1]), "nwin": int(i32[2]),
            "n_moves": int(i32[3]), "calls": int(i64[0]), "replans": int(i64[1]),
            "last_d": float(np.frombuffer(b[32:40], np.float64)[0]),
            "guarded": int(np.frombuffer(b[40:48], np.int64)[0])}


def combine_fp8(dims: Dims, bufs: PlanBuffers, y_exp: torch.Tensor, y_scale: torch.Tensor,
                w: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """mb_combine_fp8: y[t] = sum_k w[t][k] * dequant(y_exp[pos[t][k]]) from
    fp8 e4m3 rows (uint8 [rows, H]) and fp32 scales [rows, H/128]."""
    _check(y_exp, "y_exp", torch.uint8, numel=dims.rows * dims.hidden)
    _check(y_scale, "y_scale", torch.float32, numel=dims.rows * (dims.hidden // 128))
    _check(w, "w", torch.float32, numel=dims.n_tokens * dims.top_k)
    _check(y, "y", nbytes=dims.n_tokens * dims.hidden * ELT_BYTES.get(dims.dtype_out, 0))
    rc = _lib.mb_combine_fp8(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), _ptr(y_exp),
                             _ptr(y_scale), _ptr(w), _ptr(y),
                             _stream(stream, y_exp, y_scale, w, y, bufs.status))
    if rc != OK:
        raise MoebalError("mb_combine_fp8", rc)


def route(prm: RouteParams, logits: torch.Tensor, ids: torch.Tensor, w: torch.Tensor,
          bias: torch.Tensor | None = None, stream=None) -> None:
    """mb_route: router logits [N, E] to expert ids (int32) and gate weights
    (fp32) [N, K], the inputs of ``plan`` and ``combine``."""
    n = prm.n_tokens
    _check(logits, "logits", _row_dtype(prm.dtype), numel=n * prm.n_experts)
    _check(ids, "ids", torch.int32, numel=n * prm.top_k)
    _check(w, "w", torch.float32, numel=n * prm.top_k)
    if bias is not None:
        _check(bias, "bias", torch.float32, numel=prm.n_experts)
    rc = _lib.mb_route(ctypes.byref(prm), _ptr(logits), _ptr(bias), _ptr(ids), _ptr(w),
                       _stream(stream, logits, bias, ids, w))
    if rc != OK:
        _refused("mb_route", rc, (logits, n * prm.n_experts * logits.element_size(), False),
                 (bias, 4 * prm.n_experts, False), (ids, 4 * n * prm.top_k, True),
                 (w, 4 * n * prm.top_k, True))


def _row_dtype(code: int) -> torch.dtype:
    if code not in (F32, BF16):
        raise ValueError(f"rows must be f32 or bf16 (dtype code {code})")
    return TORCH_DTYPES[code]


def _rows(t, name: str) -> tuple[int, int, int]:
    """(rows, row length, dtype code) of a 2-D f32 or bf16 GPU tensor."""
    _check(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions (it has {t.dim()})")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16 (it is {t.dtype})")
    return t.shape[0], t.shape[1], F32 if t.dtype == torch.float32 else BF16


def _distinct(spans: list) -> None:
    """Refuse outputs that overlap each other or an input: `spans` lists
    (first byte, past the last, is it written)."""
    spans.sort()
    end, written = 0, False
    for lo, hi, out in spans:
        if lo < end and hi > lo and (written or out):
            raise ValueError("outputs must not overlap each other or the inputs (but "
                             "rmsnorm_fp8's residual_out may be its x or residual)")
        if hi > end:
            end, written = hi, out
        else:
            written |= out


def _refused(fn: str, rc: int, *spans) -> None:
    """Raise for a call the library refused: as a ValueError where it is for
    outputs that overlap. `spans`: (tensor or None, bytes, is it written)."""
    if rc == ERR_INVALID_ARG:
        _distinct([(t.data_ptr(), t.data_ptr() + n, out) for t, n, out in spans
                   if t is not None and n > 0])
    raise MoebalError(fn, rc)


def rmsnorm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float, q: torch.Tensor,
                q_scale: torch.Tensor, residual: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None) -> None:
    """mb_rmsnorm_fp8: root-mean-square norm of x [N, H] (plus ``residual``)
    to fp8 rows q (uint8 [N, H]) with fp32 scales [N, H/128], the rows
    ``dispatch`` takes; optionally the sum x + residual (``residual_out``,
    which may be x or residual themselves) and the normed rows ``y``."""
    n, h, code = _rows(x, "x")
    dtype, m = x.dtype, n * h
    _check(weight, "weight", dtype, numel=h)
    _check(q, "q", torch.uint8, numel=m)
    _check(q_scale, "q_scale", torch.float32, numel=n * (h // 128))
    ptr = x.data_ptr()
    size = m * ELT_BYTES[code]
    spans = [(ptr, ptr + size, False)]
    p_r = p_o = p_y = None
    if residual is not None:
        _check(residual, "residual", dtype, numel=m)
        p_r = residual.data_ptr()
        spans.append((p_r, p_r + size, False))
    if residual_out is not None:
        _check(residual_out, "residual_out", dtype, numel=m)
        p_o = residual_out.data_ptr()
        if p_o == ptr or p_o == p_r:  # in place: that input is written
            spans = [(lo, hi, lo == p_o) for lo, hi, _ in spans if lo != p_o or ptr != p_r]
            if ptr == p_r:  # x and residual are one tensor
                spans.append((ptr, ptr + size, True))
        else:
            spans.append((p_o, p_o + size, True))
    if y is not None:
        _check(y, "y", dtype, numel=m)
        p_y = y.data_ptr()
        spans.append((p_y, p_y + size, True))
    p_w, p_q, p_s = weight.data_ptr(), q.data_ptr(), q_scale.data_ptr()
    spans += [(p_w, p_w + size // n if n else p_w, False), (p_q, p_q + m, True),
              (p_s, p_s + m // 32, True)]
    _distinct(spans)
    rc = _lib.mb_rmsnorm_fp8(n, h, code, eps, ptr, p_r, p_w, p_o, p_y, p_q, p_s,
                             _stream(stream, x, residual, weight, residual_out, y, q, q_scale))
    if rc != OK:
        raise MoebalError("mb_rmsnorm_fp8", rc)


def quantize_mx4(x: torch.Tensor, q: torch.Tensor, q_scale: torch.Tensor, act: str = "none",
                 row_src: torch.Tensor | None = None, stream=None) -> None:
    """mb_quantize_mx4: rows x [M, H] to packed e2m1 codes (uint8 [M, H/2])
    and e8m0 scale bytes [M, H/32]; with act="swiglu" x rows are [gate | up]
    of 2H. Rows with a negative ``row_src`` entry are skipped."""
    m, h, code = _rows(x, "x")
    a = ACTS[act]
    if a == ACT_SWIGLU:
        if h % 2:
            raise ValueError(f"swiglu rows must have an even length (it is {h})")
        h //= 2
    _check(q, "q", torch.uint8, numel=m * (h // 2))
    _check(q_scale, "q_scale", torch.uint8, numel=m * (h // 32))
    if row_src is not None:
        _check(row_src, "row_src", torch.int32, numel=m)
    rc = _lib.mb_quantize_mx4(m, h, code, a, _ptr(x), _ptr(row_src), _ptr(q), _ptr(q_scale),
                              _stream(stream, x, row_src, q, q_scale))
    if rc != OK:
        _refused("mb_quantize_mx4", rc, (x, x.numel() * x.element_size(), False),
                 (row_src, 4 * m, False), (q, m * (h // 2), True), (q_scale, m * (h // 32), True))


def dequantize_mx4(q: torch.Tensor, q_scale: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """mb_dequantize_mx4: packed 4-bit rows back to rows x [M, H]."""
    m, h, code = _rows(x, "x")
    _check(q, "q", torch.uint8, numel=m * (h // 2))
    _check(q_scale, "q_scale", torch.uint8, numel=m * (h // 32))
    rc = _lib.mb_dequantize_mx4(m, h, code, _ptr(q), _ptr(q_scale), _ptr(x),
                                _stream(stream, q, q_scale, x))
    if rc != OK:
        _refused("mb_dequantize_mx4", rc, (q, m * (h // 2), False),
                 (q_scale, m * (h // 32), False), (x, x.numel() * x.element_size(), True))


def expert_mx4(dims: Dims, bufs: PlanBuffers, n_out: int, k_in: int, a: torch.Tensor,
               a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, y: torch.Tensor,
               stream=None) -> None:
    """mb_expert_mx4: y[p] = a[p] @ w[expert of p's slot].T over the plan's
    rows, from packed 4-bit rows a [P*cap, k_in/2] and weights
    [E, n_out, k_in/2] with their scale bytes (one per 32)."""
    _check(a, "a", torch.uint8, numel=dims.rows * (k_in // 2))
    _check(a_scale, "a_scale", torch.uint8, numel=dims.rows * (k_in // 32))
    _check(w, "w", torch.uint8, numel=dims.n_experts * n_out * (k_in // 2))
    _check(w_scale, "w_scale", torch.uint8, numel=dims.n_experts * n_out * (k_in // 32))
    _check(y, "y", TORCH_DTYPES.get(dims.dtype_out), numel=dims.rows * n_out)
    rc = _lib.mb_expert_mx4(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), n_out, k_in,
                            _ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(y),
                            _stream(stream, a, a_scale, w, w_scale, y, bufs.status))
    if rc != OK:
        rows, wide = dims.rows, dims.n_experts * n_out
        _refused("mb_expert_mx4", rc, (a, rows * (k_in // 2), False),
                 (a_scale, rows * (k_in // 32), False), (w, wide * (k_in // 2), False),
                 (w_scale, wide * (k_in // 32), False), (y, rows * n_out * y.element_size(), True),
                 *((t, t.numel() * 4, False) for t in (bufs.cu_seqlens, bufs.rep_expert,
                                                       bufs.status)))


def _plan_spans(bufs: PlanBuffers) -> tuple:
    """The plan's arrays that the experts' products read, for `_refused`."""
    return tuple((t, t.numel() * 4, False) for t in (bufs.cu_seqlens, bufs.rep_expert, bufs.status))


def expert_bf16(dims: Dims, bufs: PlanBuffers, n_out: int, k_in: int, a: torch.Tensor,
                w: torch.Tensor, y: torch.Tensor, act: str = "none",
                pre: torch.Tensor | None = None, stream=None) -> None:
    """mb_expert_bf16: y[p] = a[p] @ w[expert of p's slot].T over the plan's
    rows, from bf16 rows a [P*cap, k_in] and weights [E, n_out, k_in]. With
    act="swiglu" the weights are [E, 2 n_out, k_in] (gate rows, then up), y is
    silu(gate) * up in bf16, and ``pre`` [P*cap, 2 n_out] keeps gate and up
    for ``expert_bf16_dgrad``."""
    rows, gated = dims.rows, ACTS[act] == ACT_SWIGLU
    wide = dims.n_experts * n_out * (2 if gated else 1)
    _check(a, "a", torch.bfloat16, numel=rows * k_in)
    _check(w, "w", torch.bfloat16, numel=wide * k_in)
    _check(y, "y", torch.bfloat16 if gated else TORCH_DTYPES.get(dims.dtype_out), numel=rows * n_out)
    if pre is not None:
        _check(pre, "pre", torch.bfloat16, numel=rows * 2 * n_out)
    rc = _lib.mb_expert_bf16(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), ACTS[act], n_out,
                             k_in, _ptr(a), _ptr(w), _ptr(y), _ptr(pre),
                             _stream(stream, a, w, y, pre, bufs.status))
    if rc != OK:
        _refused("mb_expert_bf16", rc, (a, rows * k_in * 2, False), (w, wide * k_in * 2, False),
                 (y, rows * n_out * y.element_size(), True), (pre, rows * n_out * 4, True),
                 *_plan_spans(bufs))


def expert_bf16_dgrad(dims: Dims, bufs: PlanBuffers, n_out: int, k_in: int, dy: torch.Tensor,
                      w: torch.Tensor, da: torch.Tensor, act: str = "none",
                      pre: torch.Tensor | None = None, stream=None) -> None:
    """mb_expert_bf16_dgrad: the gradient of a product's rows, da[p] = dy[p] @
    w[expert], from dy [P*cap, n_out] and the weights [E, n_out, k_in]. With
    act="swiglu" the rows were silu(gate) * up of ``pre`` [P*cap, 2 k_in], and
    da is the gradient of those, in bf16."""
    rows, gated = dims.rows, ACTS[act] == ACT_SWIGLU
    wide = k_in * (2 if gated else 1)
    _check(dy, "dy", torch.bfloat16, numel=rows * n_out)
    _check(w, "w", torch.bfloat16, numel=dims.n_experts * n_out * k_in)
    _check(da, "da", torch.bfloat16 if gated else TORCH_DTYPES.get(dims.dtype_out),
           numel=rows * wide)
    if pre is not None:
        _check(pre, "pre", torch.bfloat16, numel=rows * 2 * k_in)
    rc = _lib.mb_expert_bf16_dgrad(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), ACTS[act],
                                   n_out, k_in, _ptr(dy), _ptr(w), _ptr(pre), _ptr(da),
                                   _stream(stream, dy, w, da, pre, bufs.status))
    if rc != OK:
        _refused("mb_expert_bf16_dgrad", rc, (dy, rows * n_out * 2, False),
                 (w, dims.n_experts * n_out * k_in * 2, False),
                 (da, rows * wide * da.element_size(), True), (pre, rows * k_in * 4, False),
                 *_plan_spans(bufs))


def expert_bf16_wgrad(dims: Dims, bufs: PlanBuffers, n_out: int, k_in: int, dy: torch.Tensor,
                      a: torch.Tensor, dw: torch.Tensor, accumulate: bool = False,
                      stream=None) -> None:
    """mb_expert_bf16_wgrad: the gradient of a product's weights, dw[e] =
    dy.T @ a over the rows of every slot that holds e, into dw [E, n_out, k_in]
    (float32 or bfloat16); added to what dw holds with ``accumulate``."""
    rows = dims.rows
    _check(dy, "dy", torch.bfloat16, numel=rows * n_out)
    _check(a, "a", torch.bfloat16, numel=rows * k_in)
    _check(dw, "dw", numel=dims.n_experts * n_out * k_in)
    if dw.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dw must be torch.float32 or torch.bfloat16 (it is {dw.dtype})")
    rc = _lib.mb_expert_bf16_wgrad(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), n_out, k_in,
                                   F32 if dw.dtype == torch.float32 else BF16, int(bool(accumulate)),
                                   _ptr(dy), _ptr(a), _ptr(dw),
                                   _stream(stream, dy, a, dw, bufs.status))
    if rc != OK:
        _refused("mb_expert_bf16_wgrad", rc, (dy, rows * n_out * 2, False),
                 (a, rows * k_in * 2, False),
                 (dw, dims.n_experts * n_out * k_in * dw.element_size(), True), *_plan_spans(bufs))


def combine_grad(dims: Dims, bufs: PlanBuffers, dy: torch.Tensor, y_exp: torch.Tensor | None,
                 w: torch.Tensor | None, dy_exp: torch.Tensor | None,
                 dw: torch.Tensor | None = None, stream=None) -> None:
    """mb_combine_grad: the gradients of ``combine``, dy_exp[pos[t][k]] =
    w[t][k] * dy[t] and dw[t][k] = dy[t] . y_exp[pos[t][k]]. Either output may
    be None; y_exp is needed for dw only, w for dy_exp only."""
    row, pairs = dims.hidden * ELT_BYTES.get(dims.dtype_out, 0), dims.n_tokens * dims.top_k
    _check(dy, "dy", TORCH_DTYPES.get(dims.dtype_out), nbytes=dims.n_tokens * row)
    if dw is not None:
        _check(y_exp, "y_exp", dy.dtype, nbytes=dims.rows * row)
        _check(dw, "dw", torch.float32, numel=pairs)
    if dy_exp is not None:
        _check(w, "w", torch.float32, numel=pairs)
        _check(dy_exp, "dy_exp", dy.dtype, nbytes=dims.rows * row)
    for name, t in (("y_exp", y_exp), ("w", w)):
        if t is not None:
            _check(t, name)
    rc = _lib.mb_combine_grad(ctypes.byref(dims), ctypes.byref(bufs.c_struct(dims)), _ptr(dy),
                              _ptr(y_exp), _ptr(w), _ptr(dy_exp), _ptr(dw),
                              _stream(stream, dy, y_exp, w, dy_exp, dw, bufs.status))
    if rc != OK:
        _refused("mb_combine_grad", rc, (dy, dims.n_tokens * row, False),
                 (y_exp if dw is not None else None, dims.rows * row, False),
                 (w if dy_exp is not None else None, 4 * pairs, False),
                 (dy_exp, dims.rows * row, True), (dw, 4 * pairs, True),
                 (bufs.pos, 4 * pairs, False), (bufs.status, 16, False))


def lora_workspace_bytes(prm: LoraParams) -> int:
    return int(_lib.mb_lora_workspace_bytes(ctypes.byref(prm)))


def alloc_lora_workspace(prm: LoraParams, device) -> torch.Tensor:
    n = lora_workspace_bytes(prm)
    if n == 0:
        raise MoebalError("mb_lora_workspace_bytes", ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def project_lora(prm: LoraParams, x: torch.Tensor, w: torch.Tensor, lora_a: torch.Tensor,
                 lora_b: torch.Tensor, scale: torch.Tensor, adapter: torch.Tensor,
                 ws: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """mb_project_lora: y[t] = x[t] @ w.T, plus scale[a] * (x[t] @ lora_a[a].T)
    @ lora_b[a].T where a = adapter[t] is in [0, L); x [T, k_in], w [n_out,
    k_in], lora_a [L, rank, k_in], lora_b [L, n_out, rank] in bf16, scale [L]
    fp32, adapter [T] int32, ws from ``alloc_lora_workspace``."""
    t, n, k, low = prm.n_rows, prm.n_out, prm.k_in, prm.n_adapters * prm.rank
    _check(x, "x", torch.bfloat16, numel=t * k)
    _check(w, "w", torch.bfloat16, numel=n * k)
    _check(lora_a, "lora_a", torch.bfloat16, numel=low * k)
    _check(lora_b, "lora_b", torch.bfloat16, numel=low * n)
    _check(scale, "scale", torch.float32, numel=prm.n_adapters)
    _check(adapter, "adapter", torch.int32, numel=t)
    _check(ws, "ws")
    _check(y, "y", TORCH_DTYPES.get(prm.dtype_out), numel=t * n)
    rc = _lib.mb_project_lora(ctypes.byref(prm), _ptr(x), _ptr(w), _ptr(lora_a), _ptr(lora_b),
                              _ptr(scale), _ptr(adapter), _ptr(ws), _nbytes(ws), _ptr(y),
                              _stream(stream, x, w, lora_a, lora_b, scale, adapter, ws, y))
    if rc != OK:
        _refused("mb_project_lora", rc, (x, t * k * 2, False), (w, n * k * 2, False),
                 (lora_a, low * k * 2, False), (lora_b, low * n * 2, False),
                 (scale, 4 * prm.n_adapters, False), (adapter, 4 * t, False),
                 (ws, lora_workspace_bytes(prm), True), (y, t * n * y.element_size(), True))


def plan_status(bufs: PlanBuffers, stream=None):
    """mb_plan_status: [flags, T, max load, moves] on the host (synchronises)."""
    import numpy as np

    _check(bufs.status, "status", torch.int32, numel=4)
    out = (ctypes.c_int32 * 4)()
    rc = _lib.mb_plan_status(ctypes.byref(bufs.c_struct()), _stream(stream, bufs.status), out)
    if rc != OK:
        raise MoebalError("mb_plan_status", rc)
    return np.array(list(out), dtype=np.int32)


def raw_call(fn: str, *args) -> int:
    """Call an exported mb_* function with raw ctypes arguments (for tests of
    the argument checks)."""
    return getattr(_lib, fn)(*args)
