"""Python binding of libgdnspec (include/gdn_spec.h): argument marshalling only.

Every step of the path runs in the library's CUDA kernels.  PyTorch supplies
device memory and streams; tensors are passed as raw device pointers.  If the
library has not been built, the first call raises with the build command; there
is no fallback of any kind.

Names follow the C ABI: ``verify``, ``commit``, ``fold``, ``reset``,
``read_status`` wrap ``gdn_spec_verify`` ... ``gdn_spec_read_status``.
``SpecLayer`` and ``SpecCursors`` allocate the per-layer state and the shared
cursors with torch and produce the C descriptors.

The softmax-attention layers of a hybrid model: ``KvCache`` is the paged cache of
all of them, ``kv_*`` its pages, ``RopePlan`` / ``rope`` / ``rope_append`` the
rotary positions and ``tree_attn`` the attention of a drafted window.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

GATE_SCALAR, GATE_PER_KEY = 0, 1
DTYPE_BF16, DTYPE_FP32 = 0, 1
ST_ACCEPT_RANGE, ST_SLOT_OOR, ST_RING_OVERFLOW, ST_CURSOR_CORRUPT, ST_TIMEOUT = 1, 2, 4, 8, 16
ST_UNFOLDED = 32
ST_NO_PAGES, ST_PAGE_OOR, ST_SLOT_BUSY = 64, 128, 256
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = 0, 1, 2, 3, 4
TREE_MAX = 64                     # drafted tokens of a window (bits of a tree mask)

_IO_TORCH = {DTYPE_BF16: torch.bfloat16, DTYPE_FP32: torch.float32}
_NAME_TO_DTYPE = {"bf16": DTYPE_BF16, "fp32": DTYPE_FP32}


class GdnSpecError(RuntimeError):
    pass


class LayerDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("HV", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("T", ctypes.c_int32), ("L", ctypes.c_int32),
                ("num_slots", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("checkpoint", ctypes.c_void_p),
                ("rawv", ctypes.c_void_p), ("rawk", ctypes.c_void_p),
                ("ring_g", ctypes.c_void_p), ("ring_beta", ctypes.c_void_p)]


class CursorDesc(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("write_pos", ctypes.c_void_p),
                ("cache_base", ctypes.c_void_p), ("is_flush", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("HKV", ctypes.c_int32), ("P", ctypes.c_int32), ("D", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("num_slots", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_void_p),
                ("length", ctypes.c_void_p), ("ref", ctypes.c_void_p),
                ("free_bits", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class RopeScalingDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("factor", ctypes.c_double), ("original", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class RopePlanDesc(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int32), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("freq", ctypes.c_uint64 * 128)]


_lib = None
EXPORTS = ("gdn_spec_verify", "gdn_spec_verify_d", "gdn_spec_commit", "gdn_spec_fold",
           "gdn_spec_reset", "gdn_spec_prefill",
           "gdn_spec_snapshot_verify", "gdn_spec_snapshot_commit",
           "gdn_spec_read_status", "gdn_spec_strerror", "gdn_spec_abi_version",
           "gdn_spec_verify_path", "gdn_spec_prefill_path", "gdn_spec_set_wait_limit",
           "gdn_spec_kv_init", "gdn_spec_kv_reserve", "gdn_spec_kv_fork", "gdn_spec_kv_commit",
           "gdn_spec_kv_free", "gdn_spec_kv_read_status", "gdn_spec_rope_init",
           "gdn_spec_rope_init_freqs", "gdn_spec_rope", "gdn_spec_rope_append",
           "gdn_spec_tree_attn", "gdn_spec_tree_attn_workspace", "gdn_spec_tree_attn_path")


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libgdnspec.so (built in-tree).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise GdnSpecError(
            f"libgdnspec.so not found at {path}; build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P, I32 = ctypes.c_void_p, ctypes.c_int32
    LP, CP = ctypes.POINTER(LayerDesc), ctypes.POINTER(CursorDesc)
    lib.gdn_spec_verify.argtypes = [LP, CP, P, I32, P, P, P, P, P, P, P, P, P]
    lib.gdn_spec_verify_d.argtypes = [LP, P, CP, P, I32, P, P, P, P, P, P, P, P, P]
    lib.gdn_spec_commit.argtypes = [CP, I32, I32, P, I32, P, P]
    lib.gdn_spec_fold.argtypes = [LP, I32, CP, P, I32, P]
    lib.gdn_spec_reset.argtypes = [CP, P, I32, P]
    lib.gdn_spec_prefill.argtypes = [LP, CP, P, I32, I32, P, P, P, P, P, P, P, P, I32, P]
    lib.gdn_spec_snapshot_verify.argtypes = [LP, CP, P, I32, P, P, P, P, P, P, P, P, P, P]
    lib.gdn_spec_snapshot_commit.argtypes = [LP, CP, P, I32, P, P, P]
    lib.gdn_spec_read_status.argtypes = [CP, ctypes.POINTER(ctypes.c_uint32), I32, P]
    for name in ("gdn_spec_verify", "gdn_spec_verify_d", "gdn_spec_commit", "gdn_spec_fold",
                 "gdn_spec_reset",
                 "gdn_spec_prefill", "gdn_spec_snapshot_verify", "gdn_spec_snapshot_commit",
                 "gdn_spec_read_status"):
        getattr(lib, name).restype = ctypes.c_int
    lib.gdn_spec_strerror.argtypes = [ctypes.c_int]
    lib.gdn_spec_strerror.restype = ctypes.c_char_p
    lib.gdn_spec_abi_version.argtypes = []
    lib.gdn_spec_abi_version.restype = ctypes.c_int
    lib.gdn_spec_verify_path.argtypes = [LP]
    lib.gdn_spec_verify_path.restype = ctypes.c_char_p
    lib.gdn_spec_prefill_path.argtypes = [LP]
    lib.gdn_spec_prefill_path.restype = ctypes.c_char_p
    lib.gdn_spec_set_wait_limit.argtypes = [ctypes.c_uint32]
    lib.gdn_spec_set_wait_limit.restype = ctypes.c_uint32
    KP, RP, I64, F64 = (ctypes.POINTER(KvCacheDesc), ctypes.POINTER(RopePlanDesc), ctypes.c_int64,
                        ctypes.c_double)
    lib.gdn_spec_kv_init.argtypes = [KP, P]
    lib.gdn_spec_kv_reserve.argtypes = [KP, P, I32, I32, P, P, P]
    lib.gdn_spec_kv_fork.argtypes = [KP, P, P, I32, P, P]
    lib.gdn_spec_kv_commit.argtypes = [KP, P, I32, I32, P, P, P]
    lib.gdn_spec_kv_free.argtypes = [KP, P, I32, P]
    lib.gdn_spec_kv_read_status.argtypes = [KP, ctypes.POINTER(ctypes.c_uint32), I32, P]
    lib.gdn_spec_rope_init.argtypes = [RP, I32, I32, I32, F64, ctypes.POINTER(RopeScalingDesc)]
    lib.gdn_spec_rope_init_freqs.argtypes = [RP, I32, I32, I32, ctypes.POINTER(F64), F64]
    lib.gdn_spec_rope.argtypes = [RP, I32, I32, I32, P, P, I64, P, I64, I32, P]
    lib.gdn_spec_rope_append.argtypes = [RP, KP, I32, P, I32, I32, P, P, I32, P, I64, P, I64, P, I64, P, P]
    lib.gdn_spec_tree_attn.argtypes = [KP, I32, P, I32, I32, I32, P, P, P, ctypes.c_float, P, P, P, I64, P]
    lib.gdn_spec_tree_attn_workspace.argtypes = [KP, I32, I32, I32]
    lib.gdn_spec_tree_attn_workspace.restype = I64
    lib.gdn_spec_tree_attn_path.argtypes = [KP, I32, I32]
    lib.gdn_spec_tree_attn_path.restype = ctypes.c_char_p
    for name in ("gdn_spec_kv_init", "gdn_spec_kv_reserve", "gdn_spec_kv_fork", "gdn_spec_kv_commit",
                 "gdn_spec_kv_free", "gdn_spec_kv_read_status", "gdn_spec_rope_init",
                 "gdn_spec_rope_init_freqs", "gdn_spec_rope", "gdn_spec_rope_append",
                 "gdn_spec_tree_attn"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise GdnSpecError(f"{what}: {load().gdn_spec_strerror(rc).decode()} (code {rc})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (some 4 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and torch.cuda.is_initialized():
        return _raw_stream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _scratch(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory for one call on ``stream``, from that stream's pool: when it is dropped with the kernels
    still queued, the allocator hands it out again to work behind them on the same stream only."""
    if stream is None or stream.cuda_stream == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """A result that a call on ``stream`` writes and the caller gets: from that stream's pool, so that
    nothing queued before on the current stream still uses the memory, and noted as used on the
    current stream too, where the caller may read it (after a wait) and drop it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    out = _scratch(shape, dtype, device, stream)
    if stream.cuda_stream != _stream(None):
        out.record_stream(torch.cuda.current_stream())
    return out


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise GdnSpecError(f"{name}: want contiguous CUDA {dtype} {tuple(shape)}, got "
                           f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} "
                           f"device={t.device}")


class SpecCursors:
    """Per-slot cursors (shared by all layers) and the device status word."""

    def __init__(self, num_slots: int, device="cuda"):
        self.num_slots = num_slots
        z = lambda: torch.zeros(num_slots, dtype=torch.int32, device=device)  # noqa: E731
        self.write_pos, self.cache_base, self.is_flush = z(), z(), z()
        self.status = torch.zeros(4, dtype=torch.int32, device=device)  # word 0 is used

    def desc(self) -> CursorDesc:
        return CursorDesc(self.num_slots, self.write_pos.data_ptr(), self.cache_base.data_ptr(),
                          self.is_flush.data_ptr(), self.status.data_ptr())


class SpecLayer:
    """One GDN layer's dimensions and per-slot state (checkpoint + raw ring)."""

    def __init__(self, H: int, HV: int, K: int, V: int, T: int, L: int, num_slots: int,
                 per_key_gate: bool = False, io_dtype: str = "bf16", scale: float = 1.0,
                 l2_eps: float = 1e-6, device="cuda"):
        self.H, self.HV, self.K, self.V, self.T, self.L = H, HV, K, V, T, L
        self.num_slots = num_slots
        self.per_key_gate = per_key_gate
        self.io_code = _NAME_TO_DTYPE[io_dtype]
        self.io_torch = _IO_TORCH[self.io_code]
        self.scale, self.l2_eps = scale, l2_eps
        f32 = torch.float32
        self.checkpoint = torch.zeros(num_slots, HV, V, K, dtype=f32, device=device)
        self.rawv = torch.zeros(num_slots, HV, L, V, dtype=self.io_torch, device=device)
        self.rawk = torch.zeros(num_slots, H, L, K, dtype=self.io_torch, device=device)
        gshape = (num_slots, HV, L, K) if per_key_gate else (num_slots, HV, L)
        self.ring_g = torch.zeros(gshape, dtype=f32, device=device)
        self.ring_beta = torch.zeros(num_slots, HV, L, dtype=f32, device=device)

    def desc(self) -> LayerDesc:
        return LayerDesc(self.H, self.HV, self.K, self.V, self.T, self.L, self.num_slots,
                         GATE_PER_KEY if self.per_key_gate else GATE_SCALAR, self.io_code,
                         self.scale, self.l2_eps, self.checkpoint.data_ptr(),
                         self.rawv.data_ptr(), self.rawk.data_ptr(), self.ring_g.data_ptr(),
                         self.ring_beta.data_ptr())

    def new_dring(self) -> torch.Tensor:
        """A zeroed d ring for gdn_spec_verify_d: fp32 [num_slots, HV, L, V]."""
        return torch.zeros(self.num_slots, self.HV, self.L, self.V, dtype=torch.float32,
                           device=self.checkpoint.device)

    def window_shapes(self, B: int) -> dict:
        T, H, HV, K, V = self.T, self.H, self.HV, self.K, self.V
        return {"q": (B, T, H, K), "k": (B, T, H, K), "v": (B, T, HV, V),
                "a": (B, T, HV, K) if self.per_key_gate else (B, T, HV), "b": (B, T, HV),
                "A_log": (HV,), "dt_bias": (HV, K) if self.per_key_gate else (HV,),
                "out": (B, T, HV, V)}


def verify_path(layer: SpecLayer) -> str:
    r = load().gdn_spec_verify_path(ctypes.byref(layer.desc()))
    if r is None:
        raise GdnSpecError("invalid layer descriptor")
    return r.decode()


def prefill_path(layer: SpecLayer) -> str:
    r = load().gdn_spec_prefill_path(ctypes.byref(layer.desc()))
    if r is None:
        raise GdnSpecError("invalid layer descriptor")
    return r.decode()


def verify(layer: SpecLayer, cursors: SpecCursors, slot_idx: torch.Tensor, q, k, v, a, b,
           A_log, dt_bias, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gdn_spec_verify: outputs of the draft window [B, T, HV, V]; writes the ring."""
    B = slot_idx.shape[0]
    shp = layer.window_shapes(B)
    io = layer.io_torch
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need(t, name, io, shp[name])
    _need(A_log, "A_log", torch.float32, shp["A_log"])
    _need(dt_bias, "dt_bias", torch.float32, shp["dt_bias"])
    if out is None:
        out = _result(shp["out"], io, q.device, stream)
    _need(out, "out", io, shp["out"])
    rc = load().gdn_spec_verify(ctypes.byref(layer.desc()), ctypes.byref(cursors.desc()),
                                _ptr(slot_idx), B, _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                _ptr(A_log), _ptr(dt_bias), _ptr(out), _stream(stream))
    _check(rc, "gdn_spec_verify")
    return out


def verify_d(layer: SpecLayer, dring: torch.Tensor, cursors: SpecCursors, slot_idx: torch.Tensor,
             q, k, v, a, b, A_log, dt_bias, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """gdn_spec_verify_d (comparison variant): outputs of the draft window
    [B, T, HV, V] from a ring that also caches each token's corrected delta;
    writes the window's raw records into the ring and its d into ``dring``
    (fp32 [num_slots, HV, L, V], see ``SpecLayer.new_dring``)."""
    B = slot_idx.shape[0]
    shp = layer.window_shapes(B)
    io = layer.io_torch
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need(t, name, io, shp[name])
    _need(A_log, "A_log", torch.float32, shp["A_log"])
    _need(dt_bias, "dt_bias", torch.float32, shp["dt_bias"])
    _need(dring, "dring", torch.float32, (layer.num_slots, layer.HV, layer.L, layer.V))
    if out is None:
        out = _result(shp["out"], io, q.device, stream)
    _need(out, "out", io, shp["out"])
    rc = load().gdn_spec_verify_d(ctypes.byref(layer.desc()), _ptr(dring), ctypes.byref(cursors.desc()),
                                  _ptr(slot_idx), B, _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                  _ptr(A_log), _ptr(dt_bias), _ptr(out), _stream(stream))
    _check(rc, "gdn_spec_verify_d")
    return out


def commit(cursors: SpecCursors, T: int, L: int, slot_idx: torch.Tensor,
           accept_len: torch.Tensor, stream=None) -> None:
    B = slot_idx.shape[0]
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    _need(accept_len, "accept_len", torch.int32, (B,))
    rc = load().gdn_spec_commit(ctypes.byref(cursors.desc()), T, L, _ptr(slot_idx), B,
                                _ptr(accept_len), _stream(stream))
    _check(rc, "gdn_spec_commit")


def fold(layers, cursors: SpecCursors, slot_idx: torch.Tensor, stream=None) -> None:
    if isinstance(layers, SpecLayer):
        layers = [layers]
    B = slot_idx.shape[0]
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    arr = (LayerDesc * len(layers))(*[ly.desc() for ly in layers])
    rc = load().gdn_spec_fold(arr, len(layers), ctypes.byref(cursors.desc()), _ptr(slot_idx), B,
                              _stream(stream))
    _check(rc, "gdn_spec_fold")


def prefill(layer: SpecLayer, cursors: SpecCursors, slot_idx: torch.Tensor, q, k, v, a, b,
            A_log, dt_bias, out: torch.Tensor | None = None, from_zero: bool = True,
            stream=None) -> torch.Tensor:
    """gdn_spec_prefill: outputs of the N prompt tokens [B, N, HV, V]; the final
    states become the slots' checkpoints and the slots' cursors are reset."""
    B = slot_idx.shape[0]
    N = q.shape[1]
    T, H, HV, K, V = N, layer.H, layer.HV, layer.K, layer.V
    io = layer.io_torch
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    shp = {"q": (B, T, H, K), "k": (B, T, H, K), "v": (B, T, HV, V),
           "a": (B, T, HV, K) if layer.per_key_gate else (B, T, HV), "b": (B, T, HV)}
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need(t, name, io, shp[name])
    _need(A_log, "A_log", torch.float32, (HV,))
    _need(dt_bias, "dt_bias", torch.float32, (HV, K) if layer.per_key_gate else (HV,))
    if out is None:
        out = _result((B, N, HV, V), io, q.device, stream)
    _need(out, "out", io, (B, N, HV, V))
    rc = load().gdn_spec_prefill(ctypes.byref(layer.desc()), ctypes.byref(cursors.desc()),
                                 _ptr(slot_idx), B, N, _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                 _ptr(A_log), _ptr(dt_bias), _ptr(out), int(bool(from_zero)),
                                 _stream(stream))
    _check(rc, "gdn_spec_prefill")
    return out


def snapshot_verify(layer: SpecLayer, cursors: SpecCursors, slot_idx: torch.Tensor, q, k, v, a, b,
                    A_log, dt_bias, out: torch.Tensor | None = None,
                    snap: torch.Tensor | None = None, stream=None):
    """Comparison variant (per-draft snapshots): returns (out [B, T, HV, V],
    snap fp32 [B, T, HV, V, K]); the checkpoint is only read."""
    B = slot_idx.shape[0]
    shp = layer.window_shapes(B)
    io = layer.io_torch
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need(t, name, io, shp[name])
    _need(A_log, "A_log", torch.float32, shp["A_log"])
    _need(dt_bias, "dt_bias", torch.float32, shp["dt_bias"])
    if out is None:
        out = _result(shp["out"], io, q.device, stream)
    _need(out, "out", io, shp["out"])
    sshape = (B, layer.T, layer.HV, layer.V, layer.K)
    if snap is None:
        snap = _result(sshape, torch.float32, q.device, stream)
    _need(snap, "snap", torch.float32, sshape)
    rc = load().gdn_spec_snapshot_verify(ctypes.byref(layer.desc()), ctypes.byref(cursors.desc()),
                                         _ptr(slot_idx), B, _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                         _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(out), _ptr(snap),
                                         _stream(stream))
    _check(rc, "gdn_spec_snapshot_verify")
    return out, snap


def snapshot_commit(layer: SpecLayer, cursors: SpecCursors, slot_idx: torch.Tensor,
                    accept_len: torch.Tensor, snap: torch.Tensor, stream=None) -> None:
    """Comparison variant: checkpoint[slot] = snap[b, accept_len - 1]."""
    B = slot_idx.shape[0]
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(snap, "snap", torch.float32, (B, layer.T, layer.HV, layer.V, layer.K))
    rc = load().gdn_spec_snapshot_commit(ctypes.byref(layer.desc()), ctypes.byref(cursors.desc()),
                                         _ptr(slot_idx), B, _ptr(accept_len), _ptr(snap),
                                         _stream(stream))
    _check(rc, "gdn_spec_snapshot_commit")


def reset(cursors: SpecCursors, slot_idx: torch.Tensor, stream=None) -> None:
    B = slot_idx.shape[0]
    _need(slot_idx, "slot_idx", torch.int32, (B,))
    rc = load().gdn_spec_reset(ctypes.byref(cursors.desc()), _ptr(slot_idx), B, _stream(stream))
    _check(rc, "gdn_spec_reset")


def read_status(cursors: SpecCursors, clear: bool = True, stream=None) -> int:
    v = ctypes.c_uint32(0)
    rc = load().gdn_spec_read_status(ctypes.byref(cursors.desc()), ctypes.byref(v), int(clear),
                                     _stream(stream))
    _check(rc, "gdn_spec_read_status")
    return int(v.value)


WAIT_LIMIT_DEFAULT = 0xFFFFFFFF


def set_wait_limit(polls: int) -> int:
    """gdn_spec_set_wait_limit (diagnostic): polls after which the first wait on
    each data copy gives up; WAIT_LIMIT_DEFAULT restores the default.  Returns
    the previous limit."""
    return int(load().gdn_spec_set_wait_limit(ctypes.c_uint32(polls & 0xFFFFFFFF)))


# ------------------------------------------------ softmax-attention layers

class KvCache:
    """The paged key/value cache of all softmax-attention layers: ``k`` and ``v``
    [n_layers, num_pages, HKV, P, D], the slots' page tables and lengths, the pages'
    holders.  A new cache is empty (keys and values uninitialised); ``tensors`` gives
    some or all of its tensors instead (as they are, nothing is reset).  A tensor may be
    replaced by another of its shape (``cache.length = x``: the calls from then on use x); the
    dimensions are fixed."""

    _DIMS = ("n_layers", "num_pages", "HKV", "P", "D", "num_slots", "max_pages", "io_code", "io_torch")

    def __init__(self, n_layers: int, num_pages: int, HKV: int, P: int, D: int, num_slots: int,
                 max_pages: int, io_dtype: str = "bf16", device="cuda", tensors: dict | None = None):
        self.n_layers, self.num_pages, self.HKV, self.P, self.D = n_layers, num_pages, HKV, P, D
        self.num_slots, self.max_pages = num_slots, max_pages
        self.io_code = _NAME_TO_DTYPE[io_dtype]
        self.io_torch = _IO_TORCH[self.io_code]
        t = dict(tensors or {})
        shape, i32 = (n_layers, num_pages, HKV, P, D), torch.int32
        new = {"k": lambda: torch.empty(shape, dtype=self.io_torch, device=device),
               "v": lambda: torch.empty(shape, dtype=self.io_torch, device=device),
               "page_table": lambda: torch.full((num_slots, max_pages), -1, dtype=i32, device=device),
               "n_pages": lambda: torch.zeros(num_slots, dtype=i32, device=device),
               "length": lambda: torch.zeros(num_slots, dtype=i32, device=device),
               "ref": lambda: torch.zeros(num_pages, dtype=i32, device=device),
               "free_bits": lambda: self._all_free(num_pages, device),
               "status": lambda: torch.zeros(4, dtype=i32, device=device)}
        for name, make in new.items():
            x = t.pop(name, None)
            if x is None:
                x = make()
            else:
                self._need_tensor(name, x)
            setattr(self, name, x)
        if t:
            raise GdnSpecError(f"unknown cache tensors: {sorted(t)}")
        self._tensors = tuple(new)
        self._desc = KvCacheDesc(n_layers, num_pages, HKV, P, D, self.io_code, num_slots, max_pages,
                                 *(getattr(self, n).data_ptr() for n in new))
        self._ref = ctypes.byref(self._desc)

    def _need_tensor(self, name: str, x: torch.Tensor) -> None:
        pool = (self.n_layers, self.num_pages, self.HKV, self.P, self.D)
        want = {"k": pool, "v": pool, "page_table": (self.num_slots, self.max_pages),
                "n_pages": (self.num_slots,), "length": (self.num_slots,), "ref": (self.num_pages,),
                "free_bits": ((self.num_pages + 31) // 32,), "status": x.shape}
        if name == "status" and x.numel() < 1:
            raise GdnSpecError("status: want one word at least")
        _need(x, name, self.io_torch if name in ("k", "v") else torch.int32, want[name])

    def __setattr__(self, name: str, value) -> None:
        # The calls pass the descriptor's addresses, so they follow a tensor that is replaced.
        if "_desc" in self.__dict__:
            if name in self._DIMS:
                raise GdnSpecError(f"{name}: a cache's dimensions are fixed")
            if name in self._tensors:
                self._need_tensor(name, value)
                setattr(self._desc, name, value.data_ptr())
        object.__setattr__(self, name, value)

    @staticmethod
    def _all_free(num_pages: int, device) -> torch.Tensor:
        bits = torch.full(((num_pages + 31) // 32,), -1, dtype=torch.int32, device=device)
        if num_pages % 32:
            bits[-1] = (1 << num_pages % 32) - 1
        return bits

    def desc(self) -> KvCacheDesc:
        return self._desc


def kv_init(cache: KvCache, stream=None) -> None:
    """gdn_spec_kv_init: every slot empty, every page free."""
    _check(load().gdn_spec_kv_init(cache._ref, _stream(stream)), "gdn_spec_kv_init")


def _done(done: torch.Tensor | None, like: torch.Tensor, stream) -> torch.Tensor:
    if done is None:
        return _result(like.shape, torch.int32, like.device, stream)
    _need(done, "done", torch.int32, like.shape)
    return done


def _rows(t: torch.Tensor, name: str) -> int:
    shape = t.shape
    if len(shape) != 1:
        raise GdnSpecError(f"{name}: want one dimension, got {tuple(shape)}")
    _need(t, name, torch.int32, shape)
    return shape[0]


def kv_reserve(cache: KvCache, slot_idx: torch.Tensor, T: int, n_tokens: torch.Tensor | None = None,
               done: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gdn_spec_kv_reserve: pages for T (or n_tokens[b] <= T) more tokens of every row's
    slot.  Returns int32 [B]: 1 where the row is served."""
    B = _rows(slot_idx, "slot_idx")
    done = _done(done, slot_idx, stream)
    if n_tokens is not None:
        _need(n_tokens, "n_tokens", torch.int32, (B,))
    rc = load().gdn_spec_kv_reserve(cache._ref, _ptr(slot_idx), B, T, _ptr(n_tokens), _ptr(done),
                                    _stream(stream))
    _check(rc, "gdn_spec_kv_reserve")
    return done


def kv_fork(cache: KvCache, src_idx: torch.Tensor, dst_idx: torch.Tensor,
            done: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gdn_spec_kv_fork: slots dst_idx become copies of slots src_idx, full pages
    shared.  Returns int32 [B]: 1 where the row is served."""
    B = _rows(src_idx, "src_idx")
    _need(dst_idx, "dst_idx", torch.int32, (B,))
    done = _done(done, src_idx, stream)
    rc = load().gdn_spec_kv_fork(cache._ref, _ptr(src_idx), _ptr(dst_idx), B, _ptr(done),
                                 _stream(stream))
    _check(rc, "gdn_spec_kv_fork")
    return done


def kv_commit(cache: KvCache, slot_idx: torch.Tensor, accept_len: torch.Tensor, T: int,
              path: torch.Tensor | None = None, stream=None) -> None:
    """gdn_spec_kv_commit: the accepted drafts (nodes path[b, :accept_len[b]], or the first
    accept_len[b]) become the slots' next committed tokens, in every layer."""
    B = _rows(slot_idx, "slot_idx")
    _need(accept_len, "accept_len", torch.int32, (B,))
    if path is not None:
        _need(path, "path", torch.int32, (B, T))
    rc = load().gdn_spec_kv_commit(cache._ref, _ptr(slot_idx), B, T, _ptr(path), _ptr(accept_len),
                                   _stream(stream))
    _check(rc, "gdn_spec_kv_commit")


def kv_free(cache: KvCache, slot_idx: torch.Tensor, stream=None) -> None:
    """gdn_spec_kv_free: the slots become empty, pages that nobody holds free."""
    B = _rows(slot_idx, "slot_idx")
    _check(load().gdn_spec_kv_free(cache._ref, _ptr(slot_idx), B, _stream(stream)),
           "gdn_spec_kv_free")


def kv_read_status(cache: KvCache, clear: bool = True, stream=None) -> int:
    v = ctypes.c_uint32(0)
    rc = load().gdn_spec_kv_read_status(cache._ref, ctypes.byref(v), int(clear), _stream(stream))
    _check(rc, "gdn_spec_kv_read_status")
    return int(v.value)


_ROPE_LAYOUT = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
_ROPE_KIND = {"none": ROPE_NONE, "linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN,
              "bands": ROPE_BANDS}


class RopePlan:
    """gdn_spec_rope_init: the rotary positions of heads of D dims, the first ``rot`` of
    them turned, frequencies base^(-2i/rot) scaled for long contexts by ``scaling``
    ("none", "linear", "ntk", "yarn" with fast and slow, "bands" with low and high), or
    given as ``freqs`` (radians a position, rot / 2 of them; then ``mscale`` is the
    factor on cos and sin)."""

    def __init__(self, D: int, rot: int | None = None, layout: str = "half", base: float = 1.0e4,
                 scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                 fast: float = 32.0, slow: float = 1.0, low: float = 1.0, high: float = 4.0,
                 freqs=None, mscale: float = 1.0):
        rot = D if rot is None else rot
        if layout not in _ROPE_LAYOUT or scaling not in _ROPE_KIND:
            raise GdnSpecError(f"rotary layout {layout!r} or scaling {scaling!r} is not known")
        self._desc = RopePlanDesc()
        self._ref = ctypes.byref(self._desc)
        if freqs is not None:
            f = [float(x) for x in freqs]
            if len(f) != rot // 2:
                raise GdnSpecError(f"freqs: want {rot // 2} values, got {len(f)}")
            arr = (ctypes.c_double * max(len(f), 1))(*f)
            rc = load().gdn_spec_rope_init_freqs(self._ref, D, rot, _ROPE_LAYOUT[layout], arr, mscale)
            _check(rc, "gdn_spec_rope_init_freqs")
            return
        yarn = scaling == "yarn"
        sc = RopeScalingDesc(_ROPE_KIND[scaling], 0, factor, original, fast if yarn else low,
                             slow if yarn else high)
        rc = load().gdn_spec_rope_init(self._ref, D, rot, _ROPE_LAYOUT[layout], base,
                                       ctypes.byref(sc))
        _check(rc, "gdn_spec_rope_init")

    # What the calls are checked against is what the kernels get.
    D = property(lambda self: self._desc.D)
    rot = property(lambda self: self._desc.rot)

    def desc(self) -> RopePlanDesc:
        return self._desc


def _token_stride(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Elements between tokens of [..tokens.., heads, D] whose heads are dense and whose
    tokens are evenly spaced."""
    st, nd = t.stride(), len(shape)
    ok = t.dtype == dtype and t.shape == shape and t.is_cuda
    if ok and nd == 4 and st[3] == 1 and st[2] == shape[3] and shape[0] > 1:   # the usual case at once
        if shape[1] == 1:
            return st[0]
        if st[0] == st[1] * shape[1]:
            return st[1]
    ok = ok and (shape[-1] == 1 or st[-1] == 1) and (shape[-2] == 1 or st[-2] == shape[-1])
    step, span = None, 1
    for i in range(nd - 3, -1, -1):
        if shape[i] != 1 and ok:
            if step is None:
                ok = st[i] % span == 0
                step = st[i] // span
            else:
                ok = st[i] == step * span
        span *= shape[i]
    if not ok:
        raise GdnSpecError(f"{name}: want CUDA {dtype} {tuple(shape)} with dense heads and evenly spaced "
                           f"tokens, got {t.dtype} {tuple(t.shape)} strides={tuple(st)} device={t.device}")
    return shape[-1] * shape[-2] if step is None else step


def rope(plan: RopePlan, pos: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
         transpose: bool = False, stream=None) -> torch.Tensor:
    """gdn_spec_rope: x [N, heads, D] (tokens may be strided) turned to positions pos
    [N]; transpose gives the gradient of x from that of the result.  out may be x."""
    N, heads, D = x.shape if x.dim() == 3 else (0, 0, 0)
    if x.dim() != 3 or x.dtype not in (torch.bfloat16, torch.float32) or D != plan.D:
        raise GdnSpecError(f"x: want bf16 or fp32 [N, heads, {plan.D}], got {x.dtype} {tuple(x.shape)}")
    _need(pos, "pos", torch.int32, (N,))
    xs = _token_stride(x, "x", x.dtype, (N, heads, D))
    if out is None:
        out, os_ = _result((N, heads, D), x.dtype, x.device, stream), heads * D
    else:
        os_ = _token_stride(out, "out", x.dtype, (N, heads, D))
    code = DTYPE_BF16 if x.dtype == torch.bfloat16 else DTYPE_FP32
    rc = load().gdn_spec_rope(plan._ref, N, heads, code, _ptr(pos), _ptr(x), xs, _ptr(out), os_,
                              int(bool(transpose)), _stream(stream))
    _check(rc, "gdn_spec_rope")
    return out


def rope_append(plan: RopePlan, cache: KvCache, layer: int, slot_idx: torch.Tensor, q, k, v,
                pos: torch.Tensor | None = None, n_tokens: torch.Tensor | None = None,
                q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gdn_spec_rope_append: rotated q [B, T, HQ, D]; rotated k and v [B, T, HKV, D] go
    behind the slots' committed tokens in ``layer`` of the cache.  q, k, v may be
    slices of one projection's output."""
    B = _rows(slot_idx, "slot_idx")
    if q.dim() != 4:
        raise GdnSpecError(f"q: want [B, T, heads, D], got {tuple(q.shape)}")
    _, T, HQ, _ = q.shape
    io, kv_shape = cache.io_torch, (B, T, cache.HKV, cache.D)
    qs = _token_stride(q, "q", io, (B, T, HQ, cache.D))
    ks = _token_stride(k, "k", io, kv_shape)
    vs = _token_stride(v, "v", io, kv_shape)
    if pos is not None:
        _need(pos, "pos", torch.int32, (B, T))
    if n_tokens is not None:
        _need(n_tokens, "n_tokens", torch.int32, (B,))
    if q_out is None:
        q_out = _result((B, T, HQ, cache.D), io, q.device, stream)
    else:
        _need(q_out, "q_out", io, (B, T, HQ, cache.D))
    rc = load().gdn_spec_rope_append(plan._ref, cache._ref, layer, _ptr(slot_idx), B, T,
                                     _ptr(n_tokens), _ptr(pos), HQ, _ptr(q), qs, _ptr(k), ks,
                                     _ptr(v), vs, _ptr(q_out), _stream(stream))
    _check(rc, "gdn_spec_rope_append")
    return q_out


def tree_attn_path(cache: KvCache, T: int, HQ: int) -> str:
    r = load().gdn_spec_tree_attn_path(cache._ref, T, HQ)
    if r is None:
        raise GdnSpecError("invalid cache descriptor, window or head count")
    return r.decode()


def tree_attn_workspace(cache: KvCache, B: int, T: int, HQ: int) -> int:
    """gdn_spec_tree_attn_workspace: bytes that a call of this size needs on the current device."""
    n = load().gdn_spec_tree_attn_workspace(cache._ref, B, T, HQ)
    if n < 0:
        _check(n, "gdn_spec_tree_attn_workspace")
    return n


def tree_attn(cache: KvCache, layer: int, slot_idx: torch.Tensor, q: torch.Tensor,
              tree_mask: torch.Tensor | None = None, tree_len: torch.Tensor | None = None,
              scale: float | None = None, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """gdn_spec_tree_attn: attention [B, T, HQ, D] of a window of drafted tokens over
    ``layer`` of the cache.  tree_mask int64 [B, T]: bit n of a node's word lets it
    attend to node n (None: a chain); tree_len int32 [B]: the rows' nodes (None: T);
    scale: D^-0.5 by default; lse fp32 [B, T, HQ]: written when given; workspace: uint8,
    at least ``tree_attn_workspace`` bytes (None: allocated for the call on its stream)."""
    B = _rows(slot_idx, "slot_idx")
    if q.dim() != 4:
        raise GdnSpecError(f"q: want [B, T, HQ, D], got {tuple(q.shape)}")
    _, T, HQ, _ = q.shape
    _need(q, "q", cache.io_torch, (B, T, HQ, cache.D))
    if tree_mask is not None:
        _need(tree_mask, "tree_mask", torch.int64, (B, T))
    if tree_len is not None:
        _need(tree_len, "tree_len", torch.int32, (B,))
    if out is None:
        out = _result(q.shape, q.dtype, q.device, stream)
    else:
        _need(out, "out", cache.io_torch, (B, T, HQ, cache.D))
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, T, HQ))
    if workspace is None:
        workspace = _scratch(max(16, tree_attn_workspace(cache, B, T, HQ)), torch.uint8, q.device, stream)
    else:
        _need(workspace, "workspace", torch.uint8, (workspace.numel(),))
    rc = load().gdn_spec_tree_attn(cache._ref, layer, _ptr(slot_idx), B, T, HQ, _ptr(q),
                                   _ptr(tree_mask), _ptr(tree_len),
                                   cache.D ** -0.5 if scale is None else scale, _ptr(out), _ptr(lse),
                                   _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "gdn_spec_tree_attn")
    return out
