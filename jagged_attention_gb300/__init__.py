"""Python binding of libjfa (jagged FlashAttention for GB300, sm_103a).

Argument marshalling only: every step of the forward and backward runs in the
CUDA kernels of ``libjfa.so`` behind the C ABI in ``include/jfa.h``.  torch is
used for device memory and streams.  There is no fallback: if the library
is missing or the device is not an sm_103 GPU, calls raise.

    plan = Plan(kv_offsets, q_offsets=None, H=4, Lq=256, D=128)   # broadcast-Q
    out, lse = fwd(plan, q, k, v, scale)
    dq, dk, dv = bwd(plan, q, k, v, out, dout, lse, scale)

Positions (before the forward, and back after the backward):

    rotary = Rotary(*rotary_pairs(128, sections=(16, 24, 24)), D=128)
    q, k = rotate(rotary, positions, q, k)              # positions int32 [rows, axes]
    dq, dk = rotate(rotary, positions, dq, dk, inverse=True)

Serving from a paged cache, one step:

    lens, n_free, slots, positions, offsets = paged_tables(pager, lens, delta, table, free, n_free, rows=n)
    q = paged_append(pager, k, v, slots, k_pages, v_pages, rotary=rotary, positions=positions, q=q)
    out, lse = paged_decode(pager, q, k_pages, v_pages, table, lens, scale)

The same from a cache of 8 or 4 bits, and its rows read back for the forward of prompts:

    pager = Pager(..., bits=4)
    k_pages, v_pages, k_scales, v_scales = pager.pages()
    held = dict(k_scales=k_scales, v_scales=v_scales)
    q = paged_append(pager, k, v, slots, k_pages, v_pages, **held, rotary=rotary, positions=positions, q=q)
    k, v = paged_gather(pager, k_pages, v_pages, table, offsets, rows=n, **held)
    out, lse = paged_decode(pager, q, k_pages, v_pages, table, lens, scale, **held)
"""
from __future__ import annotations

import ctypes
import struct
import threading
from pathlib import Path

import numpy as np
import torch

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libjfa.so"
HEADER = PKG.parent / "include" / "jfa.h"

JFA_OK = 0
STATUS_NAMES = {
    0: "JFA_OK", 1: "JFA_ERR_INVALID_ARG", 2: "JFA_ERR_UNSUPPORTED", 3: "JFA_ERR_BAD_OFFSETS",
    4: "JFA_ERR_ALIGNMENT", 5: "JFA_ERR_WORKSPACE", 6: "JFA_ERR_CUDA", 7: "JFA_ERR_DEVICE_TIMEOUT",
    8: "JFA_ERR_PAGES",
}
BLOCK_M = BLOCK_N = 128
PLAN_PACK_SHORT = 1  # JFA_PLAN_PACK_SHORT
PLAN_DYNAMIC = 2  # JFA_PLAN_DYNAMIC
PLAN_DELTA_PREPASS = 4  # JFA_PLAN_DELTA_PREPASS
PLAN_DELTA_IN_TILES = 8  # JFA_PLAN_DELTA_IN_TILES
PLAN_NO_PACK = 32  # JFA_PLAN_NO_PACK
PLAN_FWD_PAIRS = 64  # JFA_PLAN_FWD_PAIRS
PLAN_STATIC = 128  # JFA_PLAN_STATIC
PLAN_FWD_TWO = 256  # JFA_PLAN_FWD_TWO
PLAN_FWD_ONE = 512  # JFA_PLAN_FWD_ONE
ROTARY_INTERLEAVED = 1  # JFA_ROTARY_INTERLEAVED
ROTATE_INVERSE = 1  # JFA_ROTATE_INVERSE
ROTATE_X_FP32 = 2  # JFA_ROTATE_X_FP32
ROTATE_Y_FP32 = 4  # JFA_ROTATE_Y_FP32
PAGER_8BIT = 1  # JFA_PAGER_8BIT
PAGER_4BIT = 2  # JFA_PAGER_4BIT
PAGER_NO_PAGES = 1  # JFA_PAGER_NO_PAGES
PAGER_BAD_LENGTH = 2  # JFA_PAGER_BAD_LENGTH
PAGER_BAD_PAGE = 4  # JFA_PAGER_BAD_PAGE


class JfaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where} failed: {STATUS_NAMES.get(code, code)}")


_lib = None
_lib_lock = threading.Lock()
_vp = ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int32)
_ip = ctypes.POINTER(ctypes.c_int)
_f64p = ctypes.POINTER(ctypes.c_double)
_u64p = ctypes.POINTER(ctypes.c_uint64)


class _Pages(ctypes.Structure):
    """jfa_pages"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page", ctypes.c_int64),
                ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class _Scales(ctypes.Structure):
    """jfa_scales"""
    _fields_ = _Pages._fields_


_packed = struct.Struct("@5q").pack  # either, in a quarter of the time: ctypes takes bytes for a pointer



def build(force: bool = False) -> Path:
    """Compile libjfa.so in-tree (nvcc, sm_103a)."""
    from . import buildlib
    return buildlib.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            if not LIB_PATH.exists():
                raise RuntimeError(f"{LIB_PATH} is missing: build it with jagged_attention_gb300.build()")
            L = ctypes.CDLL(str(LIB_PATH))
            L.jfa_plan_create.argtypes = [_i32p, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, _vp, ctypes.POINTER(_vp)]
            L.jfa_plan_destroy.argtypes = [_vp]
            L.jfa_plan_tiles.argtypes = [_vp, ctypes.c_int, _i32p, _i32p, _ip, _ip]
            L.jfa_build_tiles.argtypes = [_i32p, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_uint, _i32p, _i32p,
                                          _ip, _ip]
            L.jfa_plan_create_ex.argtypes = [_i32p, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_uint, _vp,
                                             ctypes.POINTER(_vp)]
            L.jfa_fwd.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp]
            L.jfa_bwd_workspace_bytes.argtypes = [_vp]
            L.jfa_bwd_workspace_bytes.restype = ctypes.c_size_t
            L.jfa_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp,
                                  _vp, ctypes.c_size_t, _vp]
            L.jfa_bwd_preprocess.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
            L.jfa_bwd_main.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp,
                                       _vp, ctypes.c_size_t, _vp]
            L.jfa_delta_in_tiles.argtypes = [_i32p, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_uint, _ip]
            _ci = ctypes.c_int
            L.jfa_fwd_simple.argtypes = [_vp, _vp, _vp, _i32p, _i32p, _ci, _ci, _ci, _ci, ctypes.c_float,
                                         _vp, _vp, _vp]
            L.jfa_bwd_simple.argtypes = [_vp, _vp, _vp, _i32p, _i32p, _ci, _ci, _ci, _ci, ctypes.c_float,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp]
            L.jfa_simple_device_status.argtypes = [_vp, _ip]
            L.jfa_simple_release.argtypes = []
            L.jfa_plan_device_status.argtypes = [_vp, _vp, _ip]
            L.jfa_plan_selftest.argtypes = [_vp, ctypes.c_int, ctypes.c_uint]
            L.jfa_plan_forward_pairs.argtypes = [_vp, _ip]
            L.jfa_plan_claims.argtypes = [_vp, _ip, _ip]
            L.jfa_plan_forward_form.argtypes = [_vp, _ip]
            _cl, _cu = ctypes.c_int64, ctypes.c_uint
            L.jfa_rotary_turns.argtypes = [_f64p, _ci, _u64p]
            L.jfa_rotary_create.argtypes = [_f64p, _i32p, _ci, _ci, _cu, ctypes.POINTER(_vp)]
            L.jfa_rotary_destroy.argtypes = [_vp]
            L.jfa_rotate.argtypes = [_vp, _vp, _cl, _cl, _cl, _cu, _vp, _cl, _vp, _cl, _ci, _vp, _cl, _vp,
                                     _cl, _ci, _vp]
            L.jfa_pager_block_bytes.argtypes = [_ci, _ci, _ci]
            L.jfa_pager_block_bytes.restype = ctypes.c_size_t
            L.jfa_pager_block_bytes_ex.argtypes = [_ci, _ci, _ci, _cu]
            L.jfa_pager_block_bytes_ex.restype = ctypes.c_size_t
            L.jfa_pager_create.argtypes = [_ci, _ci, _cl, _ci, _ci, _ci, _ci, _vp, ctypes.c_size_t, _vp,
                                           ctypes.POINTER(_vp)]
            L.jfa_pager_destroy.argtypes = [_vp]
            L.jfa_pager_status.argtypes = [_vp, _vp, _ip]
            L.jfa_paged_tables.argtypes = [_vp, _ci, _vp, _vp, _vp, _vp, _cl, _vp, _vp, _vp, _cl, _vp, _vp,
                                           _vp, _vp]
            L.jfa_paged_append.argtypes = [_vp, _cl, _vp, _cl, _vp, _cl, _vp, _vp, _vp, _vp, _cl, _cl, _vp,
                                           _cl, _vp, _cl, _vp]
            L.jfa_paged_decode.argtypes = [_vp, _ci, _vp, _cl, _vp, _vp, _cl, _vp, ctypes.c_float, _vp, _vp,
                                           _vp]
            L.jfa_pager_create_ex.argtypes = [_ci, _ci, _cl, _ci, _ci, _ci, _ci, _cu, _vp, ctypes.c_size_t, _vp,
                                              ctypes.POINTER(_vp)]
            L.jfa_paged_append_ex.argtypes = [_vp, _cl, _vp, _cl, _vp, _cl, _vp, _vp, _vp, _vp, _vp, _cl, _cl, _vp,
                                              _cl, _vp, _cl, _vp]
            L.jfa_paged_gather.argtypes = [_vp, _ci, _vp, _vp, _vp, _cl, _vp, _vp, _cl, _vp, _cl, _vp, _cl, _vp]
            L.jfa_paged_decode_ex.argtypes = [_vp, _ci, _vp, _cl, _vp, _vp, _vp, _cl, _vp, ctypes.c_float, _vp,
                                              _vp, _vp]
            L.jfa_status_string.argtypes = [ctypes.c_int]
            L.jfa_status_string.restype = ctypes.c_char_p
            for name in ("jfa_plan_create", "jfa_plan_create_ex", "jfa_plan_destroy", "jfa_plan_tiles", "jfa_build_tiles",
                         "jfa_fwd", "jfa_bwd", "jfa_bwd_preprocess", "jfa_bwd_main",
                         "jfa_plan_device_status", "jfa_delta_in_tiles", "jfa_fwd_simple",
                         "jfa_bwd_simple", "jfa_simple_device_status", "jfa_simple_release",
                         "jfa_plan_selftest", "jfa_plan_forward_pairs", "jfa_plan_claims",
                         "jfa_plan_forward_form", "jfa_rotary_turns", "jfa_rotary_create",
                         "jfa_rotary_destroy", "jfa_rotate", "jfa_pager_create", "jfa_pager_destroy",
                         "jfa_pager_status", "jfa_paged_tables", "jfa_paged_append", "jfa_paged_decode",
                         "jfa_pager_create_ex", "jfa_paged_append_ex", "jfa_paged_gather",
                         "jfa_paged_decode_ex"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def selftest_mma_cycles(form: int, count: int = 4096, group: int = 0, stream=None) -> tuple[float, float]:
    """(cycles per product to completion, cycles per product spent issuing) of
    one form (jfa_selftest_mma_cycles): 0 M128 N128, 1 M128 N256, 2 M128 N128
    with A in TMEM, 3 M128 N64, 4 form 0 with B MN-major, 5 form 0 with A and
    B MN-major, 6 form 2 with B MN-major; count a multiple of 8; group > 0
    waits for each group of that many products before issuing the next."""
    L = lib()
    fn = L.jfa_selftest_mma_cycles
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_ulonglong),
                   ctypes.POINTER(ctypes.c_ulonglong), _vp]
    fn.restype = ctypes.c_int
    c, ci = ctypes.c_ulonglong(), ctypes.c_ulonglong()
    _check(fn(form, count, group, ctypes.byref(c), ctypes.byref(ci), _stream(stream)),
           "jfa_selftest_mma_cycles")
    return c.value / count, ci.value / count


def selftest_wait_timeout(limit_us: int = 20000, stream=None) -> tuple[int, int]:
    """Run the library's bounded-wait self-test (jfa_selftest_wait_timeout):
    returns (status code, measured wait in ns).  JFA_ERR_DEVICE_TIMEOUT (7) is
    the expected status."""
    L = lib()
    fn = L.jfa_selftest_wait_timeout
    fn.argtypes = [ctypes.c_uint, ctypes.POINTER(ctypes.c_ulonglong), _vp]
    fn.restype = ctypes.c_int
    waited = ctypes.c_ulonglong()
    rc = fn(int(limit_us), ctypes.byref(waited), None if not torch.cuda.is_available() else _stream(stream))
    return rc, waited.value


def _check(rc: int, where: str):
    if rc != JFA_OK:
        raise JfaError(rc, where)


def _offsets(a) -> np.ndarray | None:
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _i32ptr(a: np.ndarray | None):
    return None if a is None else a.ctypes.data_as(_i32p)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def build_tiles(kv_offsets, q_offsets=None, *, H: int, Lq: int = 0, num_ctas: int, direction: int,
                flags: int = 0):
    """Host-only schedule (no GPU): tiles int32 [T, 4] and cta_ptr int32 [P + 1]."""
    kv = _offsets(kv_offsets)
    qo = _offsets(q_offsets)
    B = kv.size - 1
    T, P = ctypes.c_int(), ctypes.c_int()
    L = lib()
    _check(L.jfa_build_tiles(_i32ptr(kv), _i32ptr(qo), B, H, Lq, num_ctas, direction, flags, None,
                             None, ctypes.byref(T), ctypes.byref(P)), "jfa_build_tiles")
    tiles = np.zeros((T.value, 4), dtype=np.int32)
    ptr = np.zeros(P.value + 1, dtype=np.int32)
    _check(L.jfa_build_tiles(_i32ptr(kv), _i32ptr(qo), B, H, Lq, num_ctas, direction, flags,
                             tiles.ctypes.data_as(_i32p), ptr.ctypes.data_as(_i32p),
                             ctypes.byref(T), ctypes.byref(P)), "jfa_build_tiles")
    return tiles, ptr


def delta_in_tiles(kv_offsets, q_offsets=None, *, Lq: int = 0, flags: int = 0) -> bool:
    """Host-only (no GPU): whether a plan with these offsets and flags has its
    backward tiles form Delta (then the backward does not read ``out``)."""
    kv = _offsets(kv_offsets)
    qo = _offsets(q_offsets)
    res = ctypes.c_int()
    _check(lib().jfa_delta_in_tiles(_i32ptr(kv), _i32ptr(qo), kv.size - 1, Lq, flags,
                                    ctypes.byref(res)), "jfa_delta_in_tiles")
    return bool(res.value)


def plan_choices(kv_offsets, q_offsets=None, *, H: int, D: int, Lq: int = 0, num_ctas: int,
                 flags: int = 0) -> dict:
    """Host-only (no GPU): the schedule choices a plan with these arguments makes
    on a device of ``num_ctas`` SMs (jfa_plan_choices): ``forward_form`` (0 one
    query tile per CTA, 1 CTA pairs, 2 two query tiles per CTA), whether the
    forward / backward claim their tiles at run time, and whether short
    sequences are packed."""
    kv = _offsets(kv_offsets)
    qo = _offsets(q_offsets)
    fn = lib().jfa_plan_choices
    fn.argtypes = [_i32p, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                   ctypes.c_uint, _ip, _ip, _ip, _ip]
    fn.restype = ctypes.c_int
    form, fc, bc, pk = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(fn(_i32ptr(kv), _i32ptr(qo), kv.size - 1, H, Lq, D, num_ctas, flags, ctypes.byref(form),
              ctypes.byref(fc), ctypes.byref(bc), ctypes.byref(pk)), "jfa_plan_choices")
    return {"forward_form": form.value, "claims": (bool(fc.value), bool(bc.value)), "packed": bool(pk.value)}


class Plan:
    """A jfa_plan_t: offsets and tile schedules resident on the current device,
    which must be current again whenever the plan is used."""

    def __init__(self, kv_offsets, q_offsets=None, *, H: int, D: int, Lq: int = 0,
                 num_ctas: int = 0, flags: int = 0, stream=None):
        self.kv_offsets = _offsets(kv_offsets)
        self.q_offsets = _offsets(q_offsets)
        self.B = self.kv_offsets.size - 1
        self.H, self.D = H, D
        self.broadcast = q_offsets is None
        self.Lq = Lq if self.broadcast else 0
        self.n_kv = int(self.kv_offsets[-1])
        self.n_q = self.Lq if self.broadcast else int(self.q_offsets[-1])
        self.n_o = self.B * self.Lq if self.broadcast else self.n_q
        h = _vp()
        self.flags = flags
        _check(lib().jfa_plan_create_ex(_i32ptr(self.kv_offsets), _i32ptr(self.q_offsets), self.B,
                                        H, self.Lq, D, num_ctas, flags, _stream(stream),
                                        ctypes.byref(h)),
               "jfa_plan_create_ex")
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan already destroyed")
        return self._h

    def tiles(self, direction: int):
        T, P = ctypes.c_int(), ctypes.c_int()
        L = lib()
        _check(L.jfa_plan_tiles(self.handle, direction, None, None, ctypes.byref(T), ctypes.byref(P)),
               "jfa_plan_tiles")
        tiles = np.zeros((T.value, 4), dtype=np.int32)
        ptr = np.zeros(P.value + 1, dtype=np.int32)
        _check(L.jfa_plan_tiles(self.handle, direction, tiles.ctypes.data_as(_i32p),
                                ptr.ctypes.data_as(_i32p), ctypes.byref(T), ctypes.byref(P)),
               "jfa_plan_tiles")
        return tiles, ptr

    def claims(self) -> tuple:
        """(forward, backward): whether each pass claims its tiles at run time."""
        f, b = ctypes.c_int(), ctypes.c_int()
        _check(lib().jfa_plan_claims(self.handle, ctypes.byref(f), ctypes.byref(b)), "jfa_plan_claims")
        return bool(f.value), bool(b.value)

    def forward_form(self) -> int:
        """0: one query tile per CTA, 1: CTA pairs, 2: two query tiles per CTA."""
        v = ctypes.c_int()
        _check(lib().jfa_plan_forward_form(self.handle, ctypes.byref(v)), "jfa_plan_forward_form")
        return v.value

    def forward_pairs(self) -> bool:
        """Whether the plan's forward runs as CTA pairs over pair tiles."""
        v = ctypes.c_int()
        _check(lib().jfa_plan_forward_pairs(self.handle, ctypes.byref(v)), "jfa_plan_forward_pairs")
        return bool(v.value)

    def workspace_bytes(self) -> int:
        return int(lib().jfa_bwd_workspace_bytes(self.handle))

    def device_status(self, stream=None) -> int:
        """Raise JfaError if a kernel recorded a timed-out wait; returns the raw word."""
        raw = ctypes.c_int()
        _check(lib().jfa_plan_device_status(self.handle, _stream(stream), ctypes.byref(raw)),
               "jfa_plan_device_status")
        return raw.value

    def selftest(self, skip: int, limit_us: int = 0):
        """Failure-path test only (jfa_plan_selftest): shorten every device wait of
        this plan's later launches to limit_us and withhold one arrival (skip 1:
        forward, 2: backward; 0: none)."""
        _check(lib().jfa_plan_selftest(self.handle, skip, limit_us), "jfa_plan_selftest")

    def close(self):
        if self._h is not None:
            _check(lib().jfa_plan_destroy(self._h), "jfa_plan_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _dev(t: torch.Tensor, name: str, dtype) -> int:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def fwd(plan: Plan, q, k, v, scale: float, out=None, lse=None, stream=None):
    """O (bf16 [n_o, H, D]) and LSE (fp32 [H, n_o]) through jfa_fwd."""
    dev = k.device if k.numel() else q.device
    if out is None:
        out = torch.empty((plan.n_o, plan.H, plan.D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((plan.H, plan.n_o), dtype=torch.float32, device=dev)
    _check(lib().jfa_fwd(plan.handle, _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                         _dev(v, "v", torch.bfloat16), float(scale), _dev(out, "out", torch.bfloat16),
                         _dev(lse, "lse", torch.float32), _stream(stream)), "jfa_fwd")
    return out, lse


def bwd(plan: Plan, q, k, v, out, dout, lse, scale: float, dq=None, dk=None, dv=None,
        workspace=None, stream=None):
    """dQ (fp32, shape of q), dK and dV (bf16) through jfa_bwd."""
    if dq is None:
        dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    ws_bytes = plan.workspace_bytes()
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=k.device)
    _check(lib().jfa_bwd(plan.handle, _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                         _dev(v, "v", torch.bfloat16), _dev(out, "out", torch.bfloat16),
                         _dev(dout, "dout", torch.bfloat16), _dev(lse, "lse", torch.float32),
                         float(scale), _dev(dq, "dq", torch.float32), _dev(dk, "dk", torch.bfloat16),
                         _dev(dv, "dv", torch.bfloat16), workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), _stream(stream)), "jfa_bwd")
    return dq, dk, dv


def _simple_sizes(q, k, kv_offsets, q_offsets):
    kv = _offsets(kv_offsets)
    qo = _offsets(q_offsets)
    B = kv.size - 1
    H, D = int(k.shape[1]), int(k.shape[2])
    Lq = int(q.shape[0]) if qo is None else 0
    n_o = B * Lq if qo is None else int(qo[-1])
    return kv, qo, B, H, Lq, D, n_o


def fwd_simple(q, k, v, kv_offsets, q_offsets=None, *, scale: float, out=None, lse=None,
               stream=None):
    """O and LSE through jfa_fwd_simple: no plan object (the library caches one per
    distinct offsets).  q_offsets None: broadcast mode, q holds the Lq shared rows."""
    kv, qo, B, H, Lq, D, n_o = _simple_sizes(q, k, kv_offsets, q_offsets)
    if out is None:
        out = torch.empty((n_o, H, D), dtype=torch.bfloat16, device=k.device)
    if lse is None:
        lse = torch.empty((H, n_o), dtype=torch.float32, device=k.device)
    _check(lib().jfa_fwd_simple(_dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                                _dev(v, "v", torch.bfloat16), _i32ptr(kv), _i32ptr(qo), B, H, Lq, D,
                                float(scale), _dev(out, "out", torch.bfloat16),
                                _dev(lse, "lse", torch.float32), _stream(stream)), "jfa_fwd_simple")
    return out, lse


def bwd_simple(q, k, v, out, dout, lse, kv_offsets, q_offsets=None, *, scale: float, dq=None,
               dk=None, dv=None, stream=None):
    """dQ (fp32), dK, dV through jfa_bwd_simple (cached plan and workspace)."""
    kv, qo, B, H, Lq, D, _ = _simple_sizes(q, k, kv_offsets, q_offsets)
    if dq is None:
        dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    _check(lib().jfa_bwd_simple(_dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                                _dev(v, "v", torch.bfloat16), _i32ptr(kv), _i32ptr(qo), B, H, Lq, D,
                                float(scale), _dev(out, "out", torch.bfloat16),
                                _dev(dout, "dout", torch.bfloat16), _dev(lse, "lse", torch.float32),
                                _dev(dq, "dq", torch.float32), _dev(dk, "dk", torch.bfloat16),
                                _dev(dv, "dv", torch.bfloat16), _stream(stream)), "jfa_bwd_simple")
    return dq, dk, dv


def simple_device_status(stream=None) -> int:
    """jfa_simple_device_status: status code (JFA_OK or JFA_ERR_DEVICE_TIMEOUT)."""
    raw = ctypes.c_int()
    return int(lib().jfa_simple_device_status(_stream(stream), ctypes.byref(raw)))


def simple_release():
    """Release the plans and workspaces the plan-free calls cached."""
    _check(lib().jfa_simple_release(), "jfa_simple_release")


def header_functions() -> list[str]:
    """Names of the functions include/jfa.h declares."""
    import re
    text = HEADER.read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(jfa_[a-z_0-9]+)\s*\(", text)))


def bwd_preprocess(plan: Plan, out, dout, dq, dk, dv, workspace, stream=None):
    """Delta into ``workspace`` (unless the plan's main pass forms it), dq cleared,
    dK/dV of query-less sequences zeroed."""
    _check(lib().jfa_bwd_preprocess(plan.handle, _dev(out, "out", torch.bfloat16),
                                    _dev(dout, "dout", torch.bfloat16), _dev(dq, "dq", torch.float32),
                                    _dev(dk, "dk", torch.bfloat16), _dev(dv, "dv", torch.bfloat16),
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "jfa_bwd_preprocess")


def bwd_main(plan: Plan, q, k, v, dout, lse, scale: float, dq, dk, dv, workspace, stream=None):
    """The key/value-stationary backward pass (after bwd_preprocess on the same stream)."""
    _check(lib().jfa_bwd_main(plan.handle, _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                              _dev(v, "v", torch.bfloat16), _dev(dout, "dout", torch.bfloat16),
                              _dev(lse, "lse", torch.float32), float(scale),
                              _dev(dq, "dq", torch.float32), _dev(dk, "dk", torch.bfloat16),
                              _dev(dv, "dv", torch.bfloat16), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "jfa_bwd_main")


def rotary_pairs(rotary_dim: int, sections=None, base: float = 10000.0):
    """(inv_freq, axis) of the usual rotary positions: base^(-2i / rotary_dim) for
    pair i, the pairs dealt to the axes in runs of ``sections`` (None: one axis)."""
    half = rotary_dim // 2
    sections = (half,) if sections is None else tuple(sections)
    if rotary_dim % 2 or sum(sections) != half:
        raise ValueError(f"sections {sections} must add up to {rotary_dim}/2 pairs")
    inv_freq = float(base) ** (-2.0 * np.arange(half) / rotary_dim)
    return inv_freq, np.repeat(np.arange(len(sections), dtype=np.int32), sections)


def _pair_arrays(inv_freq, axis=None):
    f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64)).reshape(-1)
    a = np.zeros(f.size, np.int32) if axis is None else np.ascontiguousarray(np.asarray(axis, np.int32)).reshape(-1)
    if a.size != f.size:
        raise ValueError(f"{a.size} axes for {f.size} frequencies")
    return f, a


def rotary_turns(inv_freq) -> np.ndarray:
    """Host-only (no GPU): the 64-bit turn fractions a Rotary holds (jfa_rotary_turns)."""
    f, _ = _pair_arrays(inv_freq)
    out = np.zeros(f.size, dtype=np.uint64)
    _check(lib().jfa_rotary_turns(f.ctypes.data_as(_f64p), f.size, out.ctypes.data_as(_u64p)),
           "jfa_rotary_turns")
    return out


class Rotary:
    """A jfa_rotary_t: inverse frequencies and axes of the pairs of a head of D
    values (see rotary_pairs).  Holds no device memory."""

    def __init__(self, inv_freq, axis=None, *, D: int, interleaved: bool = False):
        self._h = None
        f, a = _pair_arrays(inv_freq, axis)
        self.D, self.pairs, self.interleaved = D, f.size, interleaved
        self.axes = int(a.max()) + 1 if a.size else 1
        h = _vp()
        _check(lib().jfa_rotary_create(f.ctypes.data_as(_f64p), _i32ptr(a), f.size, D,
                                       ROTARY_INTERLEAVED if interleaved else 0, ctypes.byref(h)),
               "jfa_rotary_create")
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("rotary already destroyed")
        return self._h

    def close(self):
        if self._h is not None:
            _check(lib().jfa_rotary_destroy(self._h), "jfa_rotary_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _refuse(name: str, t, dtype, device: int, shape):
    """Raises what is wrong with a tensor, in the order type, device, shape."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise TypeError(f"{name} must be on cuda:{device}, got {t.device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, innermost dimensions contiguous, got {tuple(t.shape)} "
                     f"with strides {t.stride()}")


def _rows(name: str, t: torch.Tensor, shape, dtype, device: int) -> tuple[int, int]:
    """(address, elements from row to row) of a tensor [rows, heads, D] whose heads are contiguous."""
    if t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _refuse(name, t, dtype, device, shape)
    row, head, one = t.stride()
    rows, heads, D = shape
    if one != 1 or head != D and heads > 1:
        if t.numel():
            _refuse(name, t, dtype, device, shape)
    return t.data_ptr(), row if rows > 1 else heads * D


def _ints(name: str, t: torch.Tensor, n: int, device: int) -> int:
    """Address of a contiguous int32 tensor of n values."""
    if t.dtype != torch.int32 or t.get_device() != device or t.shape != (n,) or n > 1 and t.stride(0) != 1:
        _refuse(name, t, torch.int32, device, (n,))
    return t.data_ptr()


def _table(t: torch.Tensor, pager, B: int, device: int) -> tuple[int, int]:
    """(address, entries from row to row) of a block table [B, max_pages]."""
    width = pager.max_pages
    if t.dtype != torch.int32 or t.get_device() != device or t.shape != (B, width):
        _refuse("table", t, torch.int32, device, (B, width))
    row, one = t.stride()
    if one != 1 and width > 1:
        _refuse("table", t, torch.int32, device, (B, width))
    return t.data_ptr(), row if B > 1 else width


def _positions(positions: torch.Tensor, rotary: Rotary, rows: int, device: int) -> tuple[int, int, int]:
    """(address, row distance, axis distance): int32 [rows, axes], or [rows] for one position on every axis."""
    if positions.dtype != torch.int32 or positions.get_device() != device:
        _refuse("positions", positions, torch.int32, device, (rows, rotary.axes))
    shape, stride = positions.shape, positions.stride()
    if len(shape) == 1 and shape[0] == rows:
        return positions.data_ptr(), stride[0], 0
    if len(shape) != 2 or shape[0] != rows or shape[1] < rotary.axes:
        raise ValueError(f"positions must be [{rows}] or [{rows}, {rotary.axes}], got {tuple(shape)}")
    return positions.data_ptr(), stride[0], stride[1]


def _on(stream):
    """The context in which `stream` (a torch stream or a cudaStream_t) is current:
    outputs made there belong to it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _raw_stream(device: int) -> int:
    """The current stream's handle, as torch.cuda.current_stream(device).cuda_stream, in a tenth of the time."""
    return torch._C._cuda_getCurrentRawStream(device)


def rotate(rotary: Rotary, positions, q, k=None, *, inverse: bool = False, q_out=None, k_out=None,
           stream=None):
    """q (and k) [rows, heads, D], bf16 or fp32, rotated by their positions through
    jfa_rotate; ``inverse`` rotates back, which takes dq and dk (of the rotated
    q and k) to the gradients of the unrotated ones.  Rows may lie apart (slices
    of a fused projection).  q_out / k_out may be q / k.  Returns q_out, or
    (q_out, k_out) with k."""
    if stream is not None:
        with _on(stream):
            return rotate(rotary, positions, q, k, inverse=inverse, q_out=q_out, k_out=k_out)
    dev = q.get_device()
    if dev < 0:
        raise TypeError(f"q must be a CUDA tensor, got {q.device}")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"q on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    if q.dim() != 3 or k is not None and k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, D]")
    rows, hq, _ = q.shape
    flags = ROTATE_INVERSE if inverse else 0
    if q.dtype == torch.float32:
        flags |= ROTATE_X_FP32
    elif q.dtype != torch.bfloat16:
        raise TypeError(f"q must be {torch.bfloat16} or {torch.float32}, got {q.dtype}")
    shape = (rows, hq, rotary.D)
    if q_out is None:
        q_out = torch.empty(shape, dtype=q.dtype, device=q.device)
    args = (*_rows("q", q, shape, q.dtype, dev), *_rows("q_out", q_out, shape, q.dtype, dev), hq)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        args += (None, 0, None, 0, 0)
    else:
        hk = k.shape[1]
        if k.dtype == torch.float32:
            flags |= ROTATE_Y_FP32
        elif k.dtype != torch.bfloat16:
            raise TypeError(f"k must be {torch.bfloat16} or {torch.float32}, got {k.dtype}")
        shape = (rows, hk, rotary.D)
        if k_out is None:
            k_out = torch.empty(shape, dtype=k.dtype, device=k.device)
        args += (*_rows("k", k, shape, k.dtype, dev), *_rows("k_out", k_out, shape, k.dtype, dev), hk)
    rc = (_lib or lib()).jfa_rotate(rotary.handle, *_positions(positions, rotary, rows, dev), rows, flags, *args,
                                    _raw_stream(dev))
    if rc:
        _check(rc, "jfa_rotate")
    return q_out if k is None else (q_out, k_out)


class Pager:
    """A jfa_pager_t: the geometry of a paged key/value cache, with its status word
    and workspace in ``block``, which is cleared before the pager is there (created
    within a capture: by the graph, on the capturing stream).  One pager for each
    stream that decodes at the same time: its launches must be stream-ordered.  It may
    be dropped while eager calls run, on whatever streams: the block's memory is not
    given away before they are done (a stream that is not torch's own has to live as
    long).  Keep it as long as graphs that captured its calls.

    ``bits`` 8 or 4: pages hold uint8 codes [num_pages, page_size, Hkv, D * bits / 8],
    and uint8 scales [num_pages, page_size, Hkv, n] go with them, n = 1 or D / 16 (see
    jfa_pager_create_ex; ``pages()`` makes them)."""

    def __init__(self, *, max_seqs: int, max_pages: int, num_pages: int, page_size: int, H: int, Hkv: int,
                 D: int, bits: int = 16):
        self._h = None
        if bits not in (16, 8, 4):
            raise ValueError(f"bits must be 16, 8 or 4, got {bits}")
        self.bits, self.scale_bytes = bits, 1 if bits == 8 else D // 16
        shape = (num_pages, page_size, Hkv)
        self._pages_shape = (*shape, D if bits == 16 else D * bits // 8)
        self._pages_dtype = torch.bfloat16 if bits == 16 else torch.uint8
        self._scales_shape = (*shape, self.scale_bytes)
        self.max_seqs, self.max_pages, self.num_pages, self.page_size = max_seqs, max_pages, num_pages, page_size
        self.H, self.Hkv, self.D = H, Hkv, D
        self.device = torch.device("cuda", torch.cuda.current_device())
        self.index = self.device.index
        flags = {16: 0, 8: PAGER_8BIT, 4: PAGER_4BIT}[bits]
        n = lib().jfa_pager_block_bytes_ex(H, Hkv, D, flags)
        self.block = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
        stream = torch.cuda.current_stream()
        self._streams = {stream.cuda_stream}  # those that the block's memory is kept for
        h = _vp()
        _check(lib().jfa_pager_create_ex(max_seqs, max_pages, num_pages, page_size, H, Hkv, D, flags,
                                         self.block.data_ptr(), n, stream.cuda_stream, ctypes.byref(h)),
               "jfa_pager_create_ex")
        self._h = h
        if not torch.cuda.is_current_stream_capturing():
            stream.synchronize()  # cleared for calls on any stream

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("pager already destroyed")
        return self._h

    def pages(self):
        """A cache for this pager, all zeros: (k_pages, v_pages, k_scales, v_scales), scales
        None with 16 bits.  The scales of a head's rows lie one behind the other."""
        k, v = (torch.zeros(self._pages_shape, dtype=self._pages_dtype, device=self.device) for _ in range(2))
        if self.bits == 16:
            return k, v, None, None
        pages, rows, heads, n = self._scales_shape
        k_scales, v_scales = (torch.zeros((pages, heads, rows, n), dtype=torch.uint8, device=self.device).transpose(1, 2)
                              for _ in range(2))
        return k, v, k_scales, v_scales

    def _launch_stream(self) -> int:
        """The handle of the current stream, which a call is about to use.  The block
        belongs to the stream of its creation: of another the allocator is told, once
        (a captured call's work is no eager work)."""
        s = _raw_stream(self.index)
        if s not in self._streams and not torch.cuda.is_current_stream_capturing():
            self.block.record_stream(torch.cuda.current_stream(self.index))
            self._streams.add(s)
        return s

    def status(self, stream=None) -> int:
        """The status bits (PAGER_*) set since the last call, which it clears."""
        if stream is not None:
            with _on(stream):
                return self.status()
        raw = ctypes.c_int()
        rc = lib().jfa_pager_status(self.handle, self._launch_stream(), ctypes.byref(raw))
        if rc != 8:  # JFA_ERR_PAGES: the bits say what
            _check(rc, "jfa_pager_status")
        return raw.value

    def close(self):
        if self._h is not None:
            _check(lib().jfa_pager_destroy(self._h), "jfa_pager_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _pages(pager: Pager, k_pages, v_pages) -> bytes:
    """jfa_pages."""
    return _packed(*_pair("pages", k_pages, v_pages, pager._pages_shape, pager._pages_dtype, pager.index))


def _pair(what: str, k, v, shape, dtype, dev: int) -> tuple:
    """(address of k, of v, distances of pages, rows and heads) of two tensors alike.  The
    stride of a dimension of one says nothing: 0."""
    st, sv = k.stride(), v.stride()
    pages, rows, heads, n = shape
    if k.dtype != dtype or k.get_device() != dev or k.shape != shape or st[3] != 1 and n > 1:
        _refuse("k_" + what, k, dtype, dev, shape)
    if v.dtype != dtype or v.get_device() != dev or v.shape != shape or sv[3] != 1 and n > 1:
        _refuse("v_" + what, v, dtype, dev, shape)
    page, row, head = st[0] if pages > 1 else 0, st[1] if rows > 1 else 0, st[2] if heads > 1 else 0
    if st != sv and (page, row, head) != (sv[0] if pages > 1 else 0, sv[1] if rows > 1 else 0, sv[2] if heads > 1 else 0):
        raise ValueError(f"k_{what} and v_{what} must have the same strides, got {st} and {sv}")
    return k.data_ptr(), v.data_ptr(), page, row, head


def _scales(pager: Pager, k_scales, v_scales):
    """jfa_scales, None with 16 bits."""
    if pager.bits == 16:
        if k_scales is None and v_scales is None:
            return None
    elif k_scales is not None and v_scales is not None:
        return _packed(*_pair("scales", k_scales, v_scales, pager._scales_shape, torch.uint8, pager.index))
    raise ValueError(f"a cache of {pager.bits} bits {'has no' if pager.bits == 16 else 'needs'} k_scales and v_scales")


def paged_tables(pager: Pager, lens, delta, table, free_list, n_free, *, rows: int, lens_out=None,
                 n_free_out=None, slots=None, positions=None, row_offsets=None, stream=None):
    """Lengths, block table, free list, slots and positions of a step through
    jfa_paged_tables: request b of at least one goes from lens[b] to lens[b] + delta[b] rows.
    table [B, max_pages] and free_list [num_pages] are updated in place; lens and
    n_free too where lens_out and n_free_out are given as them.  Returns
    (lens_out, n_free_out, slots, positions, row_offsets)."""
    if stream is not None:
        with _on(stream):
            return paged_tables(pager, lens, delta, table, free_list, n_free, rows=rows, lens_out=lens_out,
                                n_free_out=n_free_out, slots=slots, positions=positions, row_offsets=row_offsets)
    dev = pager.index
    B = lens.shape[0]
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if n_free_out is None:
        n_free_out = torch.empty_like(n_free)
    if slots is None:
        slots = torch.empty(rows, dtype=torch.int32, device=pager.device)
    if positions is None:
        positions = torch.empty_like(slots)
    if row_offsets is None:
        row_offsets = torch.empty(B + 1, dtype=torch.int32, device=pager.device)
    rc = (_lib or lib()).jfa_paged_tables(
        pager.handle, B, _ints("lens", lens, B, dev), _ints("delta", delta, B, dev),
        _ints("lens_out", lens_out, B, dev), *_table(table, pager, B, dev),
        _ints("free_list", free_list, pager.num_pages, dev), _ints("n_free", n_free, 1, dev),
        _ints("n_free_out", n_free_out, 1, dev), rows, _ints("slots", slots, rows, dev),
        _ints("positions", positions, rows, dev), _ints("row_offsets", row_offsets, B + 1, dev),
        pager._launch_stream())
    if rc:
        _check(rc, "jfa_paged_tables")
    return lens_out, n_free_out, slots, positions, row_offsets


def paged_append(pager: Pager, k, v, slots, k_pages, v_pages, *, k_scales=None, v_scales=None,
                 rotary: Rotary | None = None, positions=None, q=None, q_out=None, stream=None):
    """New rows k, v [rows, Hkv, D] into the pages at their slots through
    jfa_paged_append_ex, quantised into a cache of 8 or 4 bits; with ``rotary``, k and q
    [rows, H, D] rotated by ``positions`` on the way.  Returns q_out (which may be q),
    None without q."""
    if stream is not None:
        with _on(stream):
            return paged_append(pager, k, v, slots, k_pages, v_pages, k_scales=k_scales, v_scales=v_scales,
                                rotary=rotary, positions=positions, q=q, q_out=q_out)
    dev = pager.index
    rows = k.shape[0]
    shape = (rows, pager.Hkv, pager.D)
    rot, pos, q_args = None, (None, 0, 0), (None, 0, None, 0)
    if rotary is not None:
        if positions is None:
            raise ValueError("rotary without positions")
        rot, pos = rotary.handle, _positions(positions, rotary, rows, dev)
    elif positions is not None or q is not None:
        raise ValueError("positions and q go with rotary")
    if q is not None:
        q_shape = (rows, pager.H, pager.D)
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=torch.bfloat16, device=pager.device)
            to_q = q_out.data_ptr(), pager.H * pager.D
        else:
            to_q = _rows("q_out", q_out, q_shape, torch.bfloat16, dev)
        q_args = (*_rows("q", q, q_shape, torch.bfloat16, dev), *to_q)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = (_lib or lib()).jfa_paged_append_ex(
        pager.handle, rows, *_rows("k", k, shape, torch.bfloat16, dev), *_rows("v", v, shape, torch.bfloat16, dev),
        _ints("slots", slots, rows, dev), _pages(pager, k_pages, v_pages),
        _scales(pager, k_scales, v_scales), rot, *pos, *q_args, pager._launch_stream())
    if rc:
        _check(rc, "jfa_paged_append_ex")
    return q_out


def paged_gather(pager: Pager, k_pages, v_pages, table, offsets, *, rows: int, starts=None, k_scales=None,
                 v_scales=None, k_out=None, v_out=None, stream=None):
    """Cached rows read back into packed bf16 rows k_out, v_out [rows, Hkv, D] through
    jfa_paged_gather: packed row r with offsets[b] <= r < offsets[b + 1] is cached row
    starts[b] + r - offsets[b] of request b (starts None: 0).  Rows behind offsets[B] stay
    as they were.  offsets [B + 1], starts [B], table [B, max_pages], B at least 1.  Returns
    (k_out, v_out), which fwd takes as k and v where Hkv is its H; with grouped heads q
    [n, H, D] goes there as q.view(n, Hkv, H // Hkv, D).transpose(1, 2).reshape(-1, Hkv, D),
    its offsets times H // Hkv.  fwd is not causal: each of a prompt's rows would attend to
    all rows gathered of its request, those behind it too, which is not what a causal model
    wants of them (its newest row is paged_decode's)."""""
    if stream is not None:
        with _on(stream):
            return paged_gather(pager, k_pages, v_pages, table, offsets, rows=rows, starts=starts, k_scales=k_scales,
                                v_scales=v_scales, k_out=k_out, v_out=v_out)
    dev, B = pager.index, offsets.shape[0] - 1
    shape = (rows, pager.Hkv, pager.D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=pager.device)
        to_k = k_out.data_ptr(), pager.Hkv * pager.D
    else:
        to_k = _rows("k_out", k_out, shape, torch.bfloat16, dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=pager.device)
        to_v = v_out.data_ptr(), pager.Hkv * pager.D
    else:
        to_v = _rows("v_out", v_out, shape, torch.bfloat16, dev)
    rc = (_lib or lib()).jfa_paged_gather(
        pager.handle, B, _pages(pager, k_pages, v_pages), _scales(pager, k_scales, v_scales),
        *_table(table, pager, B, dev), None if starts is None else _ints("starts", starts, B, dev),
        _ints("offsets", offsets, B + 1, dev), rows, *to_k, *to_v, pager._launch_stream())
    if rc:
        _check(rc, "jfa_paged_gather")
    return k_out, v_out


def paged_decode(pager: Pager, q, k_pages, v_pages, table, lens, scale: float, *, k_scales=None, v_scales=None,
                 out=None, lse=None, stream=None):
    """O (bf16 [B, H, D]) and LSE (fp32 [H, B]) of one new token per request over
    its cached rows, through jfa_paged_decode_ex.  q [B, H, D], B at least 1; rows may lie apart.
    out may not be q."""
    if stream is not None:
        with _on(stream):
            return paged_decode(pager, q, k_pages, v_pages, table, lens, scale, k_scales=k_scales, v_scales=v_scales,
                                out=out, lse=lse)
    dev, H, D = pager.index, pager.H, pager.D
    B = q.shape[0]
    shape = (B, H, D)
    q_at = _rows("q", q, shape, torch.bfloat16, dev)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=pager.device)
    if lse is None:
        lse = torch.empty((H, B), dtype=torch.float32, device=pager.device)
    elif lse.dtype != torch.float32 or lse.get_device() != dev or lse.shape != (H, B) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous float32 [{H}, {B}] on {pager.device}")
    out_at, out_row = _rows("out", out, shape, torch.bfloat16, dev)
    if out_row != H * D:
        raise ValueError("out must be contiguous")
    rc = (_lib or lib()).jfa_paged_decode_ex(
        pager.handle, B, *q_at, _pages(pager, k_pages, v_pages), _scales(pager, k_scales, v_scales),
        *_table(table, pager, B, dev), _ints("lens", lens, B, dev), float(scale), out_at, lse.data_ptr(),
        pager._launch_stream())
    if rc:
        _check(rc, "jfa_paged_decode_ex")
    return out, lse
