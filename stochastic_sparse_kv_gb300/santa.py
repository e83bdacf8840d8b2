"""ctypes binding to libsanta.so (the C ABI in include/santa.h).

Argument marshalling only: every step of the decode step runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  If the library has not been built
or cannot be loaded, every call raises -- there is no CPU path.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsanta.so")

OK = 0
DENSE, STRATIFIED, SYSTEMATIC, IID = 0, 1, 2, 3
MODES = {"dense": DENSE, "stratified": STRATIFIED, "systematic": SYSTEMATIC, "iid": IID}
GROUP_DEDUP = 0x100  # or-ed into a sampling mode: V rows loaded once per KV-head group
OUT_BF16 = 0x200     # or-ed into any mode: out is bf16 (the fp32 result rounded once)
BERNOULLI_QK = 0x400  # or-ed into any mode: score with each head's ternary query draw
TWO_PASS = 0x800      # or-ed into a sampling mode: never the single-pass cluster kernel
CLEAR_REST = 1 << 30  # or-ed into T: rows of the result that no live token writes become zeros
DEV_BAD_SEQLEN, DEV_TIMEOUT, DEV_BAD_POSITION, DEV_BAD_PAGE = 1, 2, 4, 8
ROPE_LAYOUTS = {"halves": 0, "pairs": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

# every symbol include/santa.h declares
EXPORTS = ("santa_workspace_size", "santa_workspace_init", "santa_decode", "santa_sample_points",
           "santa_device_status", "santa_status_string", "santa_version", "santa_decode_static",
           "santa_set_wait_limit", "santa_ternary_query", "santa_call_info", "santa_timeline_buffer",
           "santa_kv4_append", "santa_kv4_read", "santa_decode_kv4", "santa_decode_window",
           "santa_window_workspace_size", "santa_rope_turns", "santa_rope", "santa_paged_append",
           "santa_attend_workspace_size", "santa_attend_paged")
ERR_UNSUPPORTED = -4
ERR_DEVICE = -6
ERR_SCRATCH = -7
STATIC_SCRATCH_BYTES = (16 << 20) + 65536


class SantaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("n_max", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Kv4(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3)]


class _Rotation(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amplitude", ctypes.c_float)]


class _RopeSpec(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("scaling", ctypes.c_int32), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("original", ctypes.c_int32)]


class _Paged(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None
_lib_path = None


def load(path: str | None = None):
    """Load libsanta.so (raises if it is missing: build it with __graft_entry__.build()).
    The SANTA_LIBRARY environment variable, if set, names another build to load; so does
    `path`, on the first call of a process (one build per process)."""
    global _lib, _lib_path
    with _lock:
        if _lib is not None:
            if path is not None and os.path.realpath(path) != _lib_path:
                raise RuntimeError(f"{_lib_path} is loaded already; one libsanta build per process")
            return _lib
        p = path or os.environ.get("SANTA_LIBRARY", LIB_PATH)
        if not os.path.exists(p):
            raise RuntimeError(f"libsanta.so not found at {p}; build it first (python -c "
                               "'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
        lib.santa_workspace_size.argtypes = [ctypes.POINTER(Shape), i32, i32, ctypes.POINTER(sz)]
        lib.santa_workspace_size.restype = ctypes.c_int
        lib.santa_workspace_init.argtypes = [vp, sz, vp]
        lib.santa_workspace_init.restype = ctypes.c_int
        lib.santa_decode.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, vp, i32, i32, u64, vp, vp, vp, sz, vp]
        lib.santa_decode.restype = ctypes.c_int
        lib.santa_sample_points.argtypes = [i32, i32, i32, i32, u64, vp, vp]
        lib.santa_sample_points.restype = ctypes.c_int
        lib.santa_device_status.argtypes = [vp, ctypes.POINTER(i32), vp]
        lib.santa_device_status.restype = ctypes.c_int
        lib.santa_status_string.argtypes = [ctypes.c_int]
        lib.santa_status_string.restype = ctypes.c_char_p
        lib.santa_decode_static.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, vp, i32, i32, u64, vp, vp, vp]
        lib.santa_decode_static.restype = ctypes.c_int
        lib.santa_ternary_query.argtypes = [i32, i32, i32, vp, u64, vp, vp]
        lib.santa_ternary_query.restype = ctypes.c_int
        lib.santa_call_info.argtypes = [ctypes.POINTER(Shape), i32, i32, ctypes.POINTER(i32)]
        lib.santa_call_info.restype = ctypes.c_int
        lib.santa_timeline_buffer.argtypes = [vp, sz]
        lib.santa_timeline_buffer.restype = ctypes.c_int
        lib.santa_set_wait_limit.argtypes = [u64]
        lib.santa_set_wait_limit.restype = ctypes.c_int
        shp, kvp, rwp = ctypes.POINTER(Shape), ctypes.POINTER(_Kv4), ctypes.POINTER(_Rows)
        for f in (lib.santa_kv4_append, lib.santa_kv4_read):
            f.argtypes = [shp, kvp, rwp, i32, vp, vp, vp, vp]
            f.restype = ctypes.c_int
        lib.santa_decode_kv4.argtypes = [shp, vp, kvp, vp, i32, i32, i32, vp, vp, sz, vp]
        lib.santa_decode_kv4.restype = ctypes.c_int
        lib.santa_decode_window.argtypes = [shp, vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]
        lib.santa_decode_window.restype = ctypes.c_int
        lib.santa_window_workspace_size.argtypes = [shp, ctypes.POINTER(sz)]
        lib.santa_window_workspace_size.restype = ctypes.c_int
        i64p, rtp, pgp = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(_Rotation), ctypes.POINTER(_Paged)
        lib.santa_rope_turns.argtypes = [ctypes.POINTER(_RopeSpec), i32, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_float)]
        lib.santa_rope.argtypes = [i32, i32, i32, i32, vp, i64p, vp, i64p, rtp, vp, vp, vp, vp]
        lib.santa_paged_append.argtypes = [shp, pgp, rwp, i32, vp, vp, rtp, vp, i64p, vp, i64p, vp, vp]
        lib.santa_attend_workspace_size.argtypes = [shp, i32, ctypes.POINTER(sz)]
        lib.santa_attend_paged.argtypes = [shp, vp, i64p, pgp, i32, vp, vp, i32, i32, vp, vp, sz, vp]
        for f in (lib.santa_rope_turns, lib.santa_rope, lib.santa_paged_append, lib.santa_attend_workspace_size,
                  lib.santa_attend_paged):
            f.restype = ctypes.c_int
        lib.santa_version.argtypes = []
        lib.santa_version.restype = ctypes.c_int
        _lib, _lib_path = lib, os.path.realpath(p)
        return lib


def status_string(status: int) -> str:
    return load().santa_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise SantaError(rc, what)


def _mode(mode) -> int:
    return MODES[mode] if isinstance(mode, str) else int(mode)


def make_shape(B, H_q, H_kv, d, n_max, scale: float = 0.0) -> Shape:
    return Shape(int(B), int(H_q), int(H_kv), int(d), int(n_max), float(scale))


def workspace_size(shape: Shape, S: int, mode) -> int:
    n = ctypes.c_size_t(0)
    _check(load().santa_workspace_size(ctypes.byref(shape), int(S), _mode(mode), ctypes.byref(n)),
           "santa_workspace_size")
    return int(n.value)


def _stream_ptr(stream) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def new_workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """A zero-initialised workspace (torch allocation, 256-byte aligned), for calls on `stream`."""
    if stream is not None:
        with _current(stream, device):
            return new_workspace(nbytes, device)
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    _check(load().santa_workspace_init(ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                       ctypes.c_void_p(_stream_ptr(None))), "santa_workspace_init")
    return ws


def _current(stream, device):
    """A context in which `stream` is the current one.  What a call on an explicit stream
    allocates is allocated in it: torch hands a block's memory on in the order of the stream that
    the block was allocated on, and a capture is the stream's that is captured."""
    dev = torch.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, dev)
    if dev.index is not None and stream.device != dev:
        raise ValueError(f"the stream is not one of {dev}")
    return torch.cuda.stream(stream)


_ws_cache: dict = {}     # (kind of call, device, stream) -> workspace
_ws_captured: dict = {}  # address -> workspace whose address a captured decode() holds: never freed


def _own_workspace(kind: str, nbytes: int, dev, raw) -> torch.Tensor:
    """The workspace of a call on the current stream (handle `raw`) that was given none: one for each
    kind of call, device and stream, allocated on that stream, so that a smaller one is not
    reused before the calls on it have ended.  Inside a capture it is one of the graph's own,
    cleared in the graph (two graphs that share one could not be replayed at the same time);
    decode() takes the stream's own there if a call before the capture has made it."""
    ws = _ws_cache.get((kind, dev, raw))
    if ws is not None and ws.numel() < nbytes:
        ws = None
    if torch.cuda.is_current_stream_capturing():
        if ws is None or kind != "decode":
            return new_workspace(nbytes, dev)
        _ws_captured[ws.data_ptr()] = ws
    elif ws is None:
        ws = _ws_cache[(kind, dev, raw)] = new_workspace(nbytes, dev)
    return ws


def _cached_workspace(nbytes: int, device, stream) -> torch.Tensor:
    """The workspace of decode()."""
    if stream is not None:
        with _current(stream, device):
            return _cached_workspace(nbytes, device, None)
    return _own_workspace("decode", nbytes, torch.device(device), _stream_ptr(None))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seq_lens: torch.Tensor,
           S: int, mode="systematic", seed: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
           idx_out: torch.Tensor | None = None, want_idx: bool = True, workspace: torch.Tensor | None = None,
           stream=None, group_dedup: bool = False, out_dtype: torch.dtype = torch.float32,
           bernoulli: bool = False, two_pass: bool = False):
    """One SANTA (or dense) decode step on the GPU.  q [B,H_q,d], k/v [B,H_kv,n_max,d] bf16,
    seq_lens [B] int32, all on one CUDA device.  Returns (out [B,H_q,d], idx int32
    [B,H_q,S] or None).  out is fp32, or bf16 (SANTA_OUT_BF16) when `out` is a bf16 tensor
    or out_dtype is torch.bfloat16.  group_dedup: load each sampled V row once per group of
    query heads sharing a KV head (SANTA_GROUP_DEDUP).  bernoulli: score with each head's
    ternary query draw (SANTA_BERNOULLI_QK).  two_pass: the score and value stages as two
    launches even where the single-pass cluster kernel applies (SANTA_TWO_PASS)."""
    m = _mode(mode)
    B, H_q, d = q.shape
    _, H_kv, n_max, d2 = k_cache.shape
    for t, name in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise ValueError("seq_lens must be an int32 CUDA tensor")
    if v_cache.shape != k_cache.shape or d2 != d:
        raise ValueError("k_cache/v_cache/q shapes disagree")
    shape = make_shape(B, H_q, H_kv, d, n_max, scale)
    dev = q.device
    if stream is not None:
        caller = torch.cuda.current_stream(dev)
        with _current(stream, dev):
            got = decode(q, k_cache, v_cache, seq_lens, S, m, seed, scale, out, idx_out, want_idx, workspace, None,
                         group_dedup, out_dtype, bernoulli, two_pass)
        for t, given in zip(got, (out, idx_out)):
            if t is not None and given is None:  # the caller may use it on its own stream
                t.record_stream(caller)
        return got
    if out is None:
        out = torch.empty(B, H_q, d, dtype=out_dtype, device=dev)
    if out.dtype not in (torch.float32, torch.bfloat16) or not out.is_contiguous() or out.shape != (B, H_q, d):
        raise ValueError("out must be a contiguous fp32 or bf16 [B, H_q, d] tensor")
    if m != DENSE and want_idx and idx_out is None:
        idx_out = torch.empty(B, H_q, S, dtype=torch.int32, device=dev)
    nbytes = workspace_size(shape, S if m != DENSE else 1, m)
    ws = workspace if workspace is not None else _cached_workspace(nbytes, dev, None)
    mf = m | (GROUP_DEDUP if (group_dedup and m != DENSE) else 0) | (OUT_BF16 if out.dtype == torch.bfloat16 else 0) \
        | (BERNOULLI_QK if bernoulli else 0) | (TWO_PASS if (two_pass and m != DENSE) else 0)
    rc = load().santa_decode(ctypes.byref(shape), ctypes.c_void_p(q.data_ptr()),
                             ctypes.c_void_p(k_cache.data_ptr()), ctypes.c_void_p(v_cache.data_ptr()),
                             ctypes.c_void_p(seq_lens.data_ptr()), int(S), mf, ctypes.c_uint64(seed),
                             ctypes.c_void_p(out.data_ptr()),
                             ctypes.c_void_p(idx_out.data_ptr() if (idx_out is not None and m != DENSE) else 0),
                             ctypes.c_void_p(ws.data_ptr()), ws.numel(), ctypes.c_void_p(_stream_ptr(None)))
    _check(rc, "santa_decode")
    return out, (idx_out if m != DENSE else None)


class DecodePlan:
    """santa_decode with every argument but the seed marshalled once: the checks of
    decode(), the shape, the workspace and the ctypes arguments are built in the
    constructor, and each call is one foreign call.  For decode loops where the tensors
    stay put (the call reads whatever the tensors hold at that time)."""

    def __init__(self, q, k_cache, v_cache, seq_lens, S: int, mode="systematic", scale: float = 0.0,
                 out: torch.Tensor | None = None, idx_out: torch.Tensor | None = None, want_idx: bool = True,
                 workspace: torch.Tensor | None = None, stream=None, group_dedup: bool = False,
                 out_dtype: torch.dtype = torch.float32, bernoulli: bool = False, two_pass: bool = False):
        m = _mode(mode)
        # one checked call through decode() fixes every buffer (and runs the step once)
        self.out, self.idx_out = decode(q, k_cache, v_cache, seq_lens, S, m, 0, scale, out, idx_out, want_idx,
                                        workspace, stream, group_dedup, out_dtype, bernoulli, two_pass)
        B, H_q, d = q.shape
        _, H_kv, n_max, _ = k_cache.shape
        self._shape = make_shape(B, H_q, H_kv, d, n_max, scale)
        nbytes = workspace_size(self._shape, S if m != DENSE else 1, m)
        ws = workspace if workspace is not None else _cached_workspace(nbytes, q.device, stream)
        # the buffers (and the stream object, if one was given) stay alive with the plan
        self._keep = (q, k_cache, v_cache, seq_lens, ws, stream)
        flags = m | (GROUP_DEDUP if (group_dedup and m != DENSE) else 0) | \
            (OUT_BF16 if self.out.dtype == torch.bfloat16 else 0) | (BERNOULLI_QK if bernoulli else 0) | \
            (TWO_PASS if (two_pass and m != DENSE) else 0)
        vp = ctypes.c_void_p
        self._fn = load().santa_decode
        self._pre = (ctypes.byref(self._shape), vp(q.data_ptr()), vp(k_cache.data_ptr()), vp(v_cache.data_ptr()),
                     vp(seq_lens.data_ptr()), int(S), flags)
        self._post = (vp(self.out.data_ptr()),
                      vp(self.idx_out.data_ptr() if (self.idx_out is not None and m != DENSE) else 0),
                      vp(ws.data_ptr()), ws.numel(), vp(_stream_ptr(stream)))

    def __call__(self, seed: int):
        rc = self._fn(*self._pre, ctypes.c_uint64(seed), *self._post)
        if rc != 0:
            _check(rc, "santa_decode")
        return self.out, self.idx_out


def call_info(shape: Shape, S: int, mode, group_dedup: bool = False, bernoulli: bool = False,
              two_pass: bool = False) -> int:
    """santa_call_info: the kernel launches one decode call with this shape, S and mode
    enqueues on the current device (1: the single-pass cluster kernel)."""
    m = _mode(mode) | (GROUP_DEDUP if group_dedup else 0) | (BERNOULLI_QK if bernoulli else 0) | \
        (TWO_PASS if two_pass else 0)
    n = ctypes.c_int32(0)
    _check(load().santa_call_info(ctypes.byref(shape), int(S), m, ctypes.byref(n)), "santa_call_info")
    return int(n.value)


def set_wait_limit(limit_ns: int) -> None:
    """santa_set_wait_limit: how long a kernel's pipeline waits may last before it gives
    up with SANTA_DEV_TIMEOUT (0: the default of 2 s).  A diagnostic knob."""
    _check(load().santa_set_wait_limit(ctypes.c_uint64(int(limit_ns))), "santa_set_wait_limit")


def sample_points(B: int, H_q: int, S: int, mode, seed: int, device="cuda", stream=None) -> torch.Tensor:
    if stream is not None:
        caller = torch.cuda.current_stream(device)
        with _current(stream, device):
            t = sample_points(B, H_q, S, mode, seed, device)
        t.record_stream(caller)
        return t
    t = torch.empty(B, H_q, S, dtype=torch.float64, device=device)
    _check(load().santa_sample_points(int(B), int(H_q), int(S), _mode(mode), ctypes.c_uint64(seed),
                                      ctypes.c_void_p(t.data_ptr()), ctypes.c_void_p(_stream_ptr(None))),
           "santa_sample_points")
    return t


def ternary_query(q: torch.Tensor, seed: int, stream=None) -> torch.Tensor:
    """santa_ternary_query: each head's Bernoulli qK^T draw (bf16 [B,H_q,d])."""
    if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be a contiguous bf16 CUDA tensor [B, H_q, d]")
    if stream is not None:
        caller = torch.cuda.current_stream(q.device)
        with _current(stream, q.device):
            out = ternary_query(q, seed)
        out.record_stream(caller)
        return out
    B, H_q, d = q.shape
    out = torch.empty_like(q)
    _check(load().santa_ternary_query(int(B), int(H_q), int(d), ctypes.c_void_p(q.data_ptr()), ctypes.c_uint64(seed),
                                      ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(_stream_ptr(None))),
           "santa_ternary_query")
    return out


def device_status(workspace: torch.Tensor | None, stream=None) -> int:
    """santa_device_status: the device error word of `workspace` (None: the static scratch
    of santa_decode_static on the current device), read and cleared."""
    code = ctypes.c_int32(0)
    rc = load().santa_device_status(ctypes.c_void_p(workspace.data_ptr() if workspace is not None else 0),
                                    ctypes.byref(code), ctypes.c_void_p(_stream_ptr(stream)))
    if rc not in (OK, ERR_DEVICE):
        _check(rc, "santa_device_status")
    return int(code.value)


# ------------------------------------------------------------------ 4-bit KV cache, windowed attention

class KV4Cache(NamedTuple):
    """A 4-bit KV cache: uint8 codes [B, H_kv, n_max, d/2] and scales [B, H_kv, n_max, d/16]
    for K and V, contiguous on one CUDA device (the format is described in santa.h)."""
    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor


def new_kv4_cache(B: int, H_kv: int, n_max: int, d: int, device="cuda") -> KV4Cache:
    """An empty cache (all values zero) of capacity n_max rounded up to a multiple of 16."""
    n = -(-int(n_max) // 16) * 16
    return KV4Cache(*(torch.zeros(B, H_kv, n, w, dtype=torch.uint8, device=device) for w in (d // 2, d // 16) * 2))


def _cuda_bf16(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def _int_vector(t: torch.Tensor, name: str, B: int, dev):
    if t.dtype != torch.int32 or t.device != dev or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [B] on the inputs' device")


def _kv4_dims(cache: KV4Cache):
    """(B, H_kv, n_max, d, device) of a checked cache."""
    k, ks, v, vs = cache
    shape, dev = k.shape, k.device
    if len(shape) != 4 or not k.is_cuda:
        raise ValueError("a 4-bit cache holds CUDA tensors of four dimensions")
    B, H_kv, n_max, half = shape
    if v.shape != shape or ks.shape != vs.shape or ks.shape != (B, H_kv, n_max, half // 8):
        raise ValueError("4-bit cache shapes disagree: codes [B, H_kv, n_max, d/2], scales [B, H_kv, n_max, d/16]")
    for t in cache:
        if t.dtype != torch.uint8 or t.device != dev or not t.is_contiguous():
            raise ValueError("a 4-bit cache holds contiguous uint8 tensors on one CUDA device")
    return B, H_kv, n_max, half * 2, dev


def _kv4_arg(cache: KV4Cache):
    k, ks, v, vs = cache
    return ctypes.byref(_Kv4(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr()))


class _on_device:
    """The library launches on the current device: make it the tensors' own for the call."""
    __slots__ = ("dev", "ctx")

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        self.ctx = None
        if self.dev.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(self.dev)
            self.ctx.__enter__()

    def __exit__(self, *e):
        if self.ctx is not None:
            self.ctx.__exit__(*e)


_shapes: dict = {}


def _shape_of(key):
    """(the shape as a C argument, the workspace bytes of a windowed call), kept per shape."""
    got = _shapes.get(key)
    if got is None:
        shape, n = make_shape(*key), ctypes.c_size_t(0)
        _check(load().santa_window_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "santa_window_workspace_size")
        if len(_shapes) >= 1024:
            _shapes.clear()
        got = _shapes[key] = (ctypes.byref(shape), int(n.value))
    return got


def _raw_stream(stream, dev) -> int:
    """The CUDA handle of `stream`, or of the current one on `dev` (looked up without making a
    torch.cuda.Stream, which would be a tenth of a small call)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)


def _move_rows(fn, what: str, cache, k, v, pos, counts, workspace, stream):
    B, H_kv, n_max, d, dev = _kv4_dims(cache)
    for t, name in ((k, "K rows"), (v, "V rows")):
        if t.dtype != torch.bfloat16 or t.device != dev or t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{name} must be a bf16 tensor [B, T, H_kv, d] on the cache's device, contiguous in d")
        if t.shape != (B, k.shape[1], H_kv, d):
            raise ValueError(f"{name} [B, T, H_kv, d] and the cache's shape disagree")
    _int_vector(pos, "pos", B, dev)
    if counts is not None:
        _int_vector(counts, "counts", B, dev)
    rows = _Rows(k.data_ptr(), v.data_ptr(), k.stride()[:3], v.stride()[:3])
    shape, _ = _shape_of((B, H_kv, H_kv, d, n_max))
    with _on_device(dev):
        rc = fn(shape, _kv4_arg(cache), ctypes.byref(rows), k.shape[1], pos.data_ptr(),
                counts.data_ptr() if counts is not None else None,
                workspace.data_ptr() if workspace is not None else None, _raw_stream(stream, dev))
    if rc:
        _check(rc, what)


def kv4_append(cache: KV4Cache, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor,
               counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> None:
    """Quantise new rows [B, T, H_kv, d] (bf16, any strides that are multiples of 8) into the
    cache at rows pos[b] .. pos[b] + T - 1, or only the first counts[b] of them (int32 [B]).
    Batch rows that would leave the cache are skipped; give a `workspace` to have that
    reported by device_status (DEV_BAD_POSITION)."""
    if k_new.dim() == 4 and k_new.shape[1] == 0:
        return
    _move_rows(load().santa_kv4_append, "santa_kv4_append", cache, k_new, v_new, pos, counts, workspace, stream)


def kv4_read(cache: KV4Cache, pos: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
             counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Rows pos[b] + t of the cache into k_out, v_out [B, T, H_kv, d] (bf16, strided as for
    kv4_append) for t < counts[b] (default T); other rows stay as they were.  Exact.  For a
    bf16 cache [B, H_kv, n, d] pass its transpose(1, 2).  Returns (k_out, v_out)."""
    if k_out.dim() != 4 or k_out.shape[1] != 0:
        if k_out.is_cuda and k_out.data_ptr() == v_out.data_ptr():
            raise ValueError("k_out and v_out are the same rows")
        _move_rows(load().santa_kv4_read, "santa_kv4_read", cache, k_out, v_out, pos, counts, workspace, stream)
    return k_out, v_out


def _window_call(q, dims, cache_args, fn, what, seq_lens, window, sinks, scale, out, out_dtype, workspace, stream):
    B, H_kv, n_max, d, dev = dims
    qs = q.shape
    if len(qs) != 3 or qs[0] != B or qs[2] != d or q.device != dev:
        raise ValueError("q [B, H_q, d] and the cache's shape or device disagree")
    _int_vector(seq_lens, "seq_lens", B, dev)
    if not (-1 << 31 <= window < 1 << 31 and -1 << 31 <= sinks < 1 << 31):
        raise ValueError("window and sinks are 32-bit numbers")
    if stream is not None:
        caller = torch.cuda.current_stream(dev)
        with _current(stream, dev):
            got = _window_call(q, dims, cache_args, fn, what, seq_lens, window, sinks, scale, out, out_dtype, workspace, None)
        if out is None:  # the caller may use it on its own stream
            got.record_stream(caller)
        return got
    shape, nbytes = _shape_of((B, qs[1], H_kv, d, n_max, scale))
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
        out = torch.empty(qs, dtype=out_dtype, device=dev)
    elif out.dtype not in (torch.float32, torch.bfloat16) or not out.is_contiguous() or out.shape != qs or out.device != dev:
        raise ValueError("out must be a contiguous fp32 or bf16 [B, H_q, d] tensor on q's device")
    with _on_device(dev):
        raw = _raw_stream(None, dev)
        ws = workspace if workspace is not None else _own_workspace("window", nbytes, dev, raw)
        rc = fn(shape, q.data_ptr(), *cache_args, seq_lens.data_ptr(), window, sinks,
                OUT_BF16 if out.dtype == torch.bfloat16 else 0, out.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc, what)
    return out


def decode_window(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seq_lens: torch.Tensor, window: int,
                  sinks: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None, stream=None):
    """One step of exact attention over the last `window` keys of each sequence and its first
    `sinks` (window = 0: every key).  q [B, H_q, d], k/v [B, H_kv, n_max, d] bf16, seq_lens
    [B] int32, all on one CUDA device.  Returns out [B, H_q, d], fp32 or bf16.  On an explicit `stream`,
    the call and all that it allocates are that stream's: order its inputs and its result with
    the current stream as for any work on another one."""
    for t, name in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda_bf16(t, name)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.device != k_cache.device:
        raise ValueError("k_cache and v_cache [B, H_kv, n_max, d] disagree")
    return _window_call(q, (*k_cache.shape, k_cache.device), (k_cache.data_ptr(), v_cache.data_ptr()),
                        load().santa_decode_window, "santa_decode_window", seq_lens, window, sinks, scale, out, out_dtype,
                        workspace, stream)


def decode_kv4(q: torch.Tensor, cache: KV4Cache, seq_lens: torch.Tensor, window: int = 0, sinks: int = 0,
               scale: float = 0.0, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
               workspace: torch.Tensor | None = None, stream=None):
    """One step of exact attention over a 4-bit cache: every key, or with window > 0 the last
    `window` keys and the first `sinks`.  Arguments and result as for decode_window."""
    _cuda_bf16(q, "q")
    return _window_call(q, _kv4_dims(cache), (_kv4_arg(cache),), load().santa_decode_kv4, "santa_decode_kv4", seq_lens,
                        window, sinks, scale, out, out_dtype, workspace, stream)


# ------------------------------------------------------------------ rotary positions, paged cache

class RopeTable(NamedTuple):
    """Rotary frequencies: turns int64 [rot/2] on the device (the bits of unsigned numbers, turns a
    position in units of 2^-64), the number of features they rotate, how those pair up ("halves":
    (i, i + rot/2); "pairs": (2i, 2i + 1)), and a factor of the rotated features."""
    turns: torch.Tensor
    rot: int
    layout: str = "halves"
    amplitude: float = 1.0


def rope_table(rot: int, base: float = 10000.0, layout: str = "halves", scaling: str = "none", factor: float = 1.0,
               low: float = 1.0, high: float = 4.0, original: int = 8192, device="cuda") -> RopeTable:
    """Frequencies base^(-2i/rot), scaled for long contexts: "linear", "base", "bands" or "ramp"
    (santa_rope_spec in santa.h has the formulas; `low` and `high` are turns over the `original`
    context).  rot: a multiple of 16 up to the head dimension."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"layout is one of {list(ROPE_LAYOUTS)}, scaling one of {list(ROPE_SCALINGS)}")
    if not (-1 << 31 <= original < 1 << 31 and -1 << 31 <= rot < 1 << 31):
        raise ValueError("rot and original are 32-bit numbers")
    spec = _RopeSpec(base, ROPE_SCALINGS[scaling], factor, low, high, original)
    turns, amplitude = (ctypes.c_uint64 * max(min(int(rot), 65536) // 2, 1))(), ctypes.c_float(0)
    _check(load().santa_rope_turns(ctypes.byref(spec), int(rot), turns, ctypes.byref(amplitude)), "santa_rope_turns")
    bits = torch.tensor([x - (1 << 64) if x >> 63 else x for x in turns], dtype=torch.int64)
    return RopeTable(bits.to(device), int(rot), layout, float(amplitude.value))


class PagedCache(NamedTuple):
    """A bf16 cache in pages: k and v [n_pages, H_kv, page, d], table int32 [B, columns]; key j of
    sequence b is row j % page of page table[b, j // page].  Contiguous, on one CUDA device."""
    k: torch.Tensor
    v: torch.Tensor
    table: torch.Tensor


def new_paged_cache(n_pages: int, H_kv: int, page: int, d: int, B: int, columns: int, device="cuda") -> PagedCache:
    """An empty pool and a table whose entries name no page yet (-1)."""
    k, v = (torch.zeros(n_pages, H_kv, page, d, dtype=torch.bfloat16, device=device) for _ in range(2))
    return PagedCache(k, v, torch.full((B, columns), -1, dtype=torch.int32, device=device))


def _rotation_arg(table: RopeTable, dev):
    t = table.turns
    if t.dtype != torch.int64 or t.device != dev or t.shape != (table.rot // 2,) or not t.is_contiguous():
        raise ValueError("a rope table holds contiguous int64 turns [rot/2] on the inputs' device")
    if table.layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout is one of {list(ROPE_LAYOUTS)}")
    return ctypes.byref(_Rotation(t.data_ptr(), table.rot, ROPE_LAYOUTS[table.layout], table.amplitude))


_strides = ctypes.c_int64 * 3
_stride_args: dict = {}   # strides of a [B, T, H, d] tensor -> those of (batch, token, head) as a C argument
_append_shapes: dict = {}


def _kept(cache: dict, key, make):
    """cache[key], made on first use; these are C arguments of plain numbers."""
    got = cache.get(key)
    if got is None:
        if len(cache) >= 1024:
            cache.clear()
        got = cache[key] = make(key)
    return got


def _checked_shape(key):
    """make_shape of sizes that C's 32 bits hold."""
    if max(key[:5]) >= 1 << 31:
        raise SantaError(ERR_UNSUPPORTED, f"sizes {key[:5]}")
    return make_shape(*key)


def _check_tokens(T: int):
    """T is a number of tokens below CLEAR_REST, which goes into the same C argument."""
    if T >= CLEAR_REST:
        raise SantaError(ERR_UNSUPPORTED, f"{T} tokens")


def _workspace_ptr(workspace: torch.Tensor | None, dev):
    """The address of a workspace that was given, which the kernels write to."""
    if workspace is None:
        return None
    if workspace.device != dev:
        raise ValueError("the workspace is not on the inputs' device")
    return workspace.data_ptr()


def _row_tensor(t: torch.Tensor, name: str, shape, dev):
    st = t.stride()
    if t.dtype is not torch.bfloat16 or t.device != dev or len(st) != 4 or st[3] != 1:
        raise ValueError(f"{name} must be a bf16 tensor [B, T, H, d] on the inputs' device, contiguous in d")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return t.data_ptr(), _kept(_stride_args, st, lambda x: _strides(*x[:3]))


def _on_stream(stream, dev, call, made):
    """call() with `stream` current; what it returns is the caller's to use on its own one (`made`)."""
    caller = torch.cuda.current_stream(dev)
    with _current(stream, dev):
        got = call()
    if made and got is not None:
        got.record_stream(caller)
    return got


def _out_rows(x: torch.Tensor) -> torch.Tensor:
    """Rows for a result; the call gets CLEAR_REST, so that those that no live token writes are zeros."""
    return torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)


def rope(x: torch.Tensor, table: RopeTable, pos: torch.Tensor, counts: torch.Tensor | None = None,
         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows x [B, T, H, d] (bf16, any strides that are multiples of 8) rotated to the positions
    pos[b] + t (int32 [B]), for t < counts[b] (default T).  Into `out` (x itself: in place), whose
    other rows stay as they were; without it into new rows, the others zero.  Batch rows with a position or
    a count out of range are skipped (in new rows: zeros); give a `workspace` to have that reported by
    device_status (DEV_BAD_POSITION)."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dev = x.device
    if stream is not None:
        return _on_stream(stream, dev, lambda: rope(x, table, pos, counts, out, workspace), out is None)
    x_ptr, x_st = _row_tensor(x, "x", None, dev)
    B, T, H, d = x.shape
    _check_tokens(T)
    if B | H >= 1 << 31:
        raise SantaError(ERR_UNSUPPORTED, f"{B} batch rows, {H} heads")
    _int_vector(pos, "pos", B, dev)
    if counts is not None:
        _int_vector(counts, "counts", B, dev)
    rotation = _rotation_arg(table, dev)
    if out is None:
        out, clear = _out_rows(x), CLEAR_REST
    else:
        clear = 0
    o_ptr, o_st = _row_tensor(out, "out", x.shape, dev)
    if T == 0:
        return out
    with _on_device(dev):
        rc = (_lib or load()).santa_rope(B, T | clear, H, d, x_ptr, x_st, o_ptr, o_st, rotation, pos.data_ptr(),
                               counts.data_ptr() if counts is not None else None,
                               _workspace_ptr(workspace, dev), _raw_stream(None, dev))
    if rc:
        _check(rc, "santa_rope")
    return out


def _paged_dims(cache: PagedCache):
    """(B, H_kv, n_max, d, page, device) of a checked cache."""
    k, v, table = cache
    dev, size, columns = k.device, k.shape, table.shape
    if len(size) != 4 or v.shape != size or not k.is_cuda:
        raise ValueError("a paged cache holds CUDA tensors k and v [n_pages, H_kv, page, d]")
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or v.device != dev or not k.is_contiguous() or \
            not v.is_contiguous():
        raise ValueError("a paged cache holds contiguous bf16 tensors on one CUDA device")
    if table.dtype is not torch.int32 or table.device != dev or len(columns) != 2 or not table.is_contiguous():
        raise ValueError("a paged cache's table is a contiguous int32 tensor [B, columns] on its device")
    _, H_kv, page, d = size
    return columns[0], H_kv, columns[1] * page, d, page, dev


def _paged_arg(cache: PagedCache):
    k, v, table = cache
    return ctypes.byref(_Paged(k.data_ptr(), v.data_ptr(), table.data_ptr(), k.shape[0], k.shape[2]))


def paged_append(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor,
                 counts: torch.Tensor | None = None, rope: RopeTable | None = None, q: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Write new rows [B, T, H_kv, d] (bf16, any strides that are multiples of 8) to positions
    pos[b] + t of a paged cache, for t < counts[b] (default T), K rotated by `rope` if one is given.
    With it, the same tokens' queries q [B, T, H_q, d] can be rotated in the same launch: into
    q_out (q itself: in place) or into new rows, which are returned (as for rope).  Batch rows that would
    leave the table, and tokens without a page, are not written; give a `workspace` to have that reported
    by device_status (DEV_BAD_POSITION, DEV_BAD_PAGE)."""
    B, H_kv, n_max, d, _, dev = _paged_dims(cache)
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    if q is not None and rope is None:
        raise ValueError("q is rotated: give a rope table")
    if stream is not None:
        return _on_stream(stream, dev, lambda: paged_append(cache, k_new, v_new, pos, counts, rope, q, q_out, workspace),
                          q_out is None)
    T = k_new.shape[1] if k_new.dim() == 4 else -1
    _check_tokens(T)
    k_ptr, k_st = _row_tensor(k_new, "K rows", (B, T, H_kv, d), dev)
    v_ptr, v_st = _row_tensor(v_new, "V rows", (B, T, H_kv, d), dev)
    _int_vector(pos, "pos", B, dev)
    if counts is not None:
        _int_vector(counts, "counts", B, dev)
    H_q, q_arg, clear = H_kv, (None,) * 4, 0
    if q is not None:
        H_q = q.shape[2] if q.dim() == 4 else 0
        q_args = _row_tensor(q, "q", (B, T, H_q, d), dev)
        if q_out is None:
            q_out, clear = _out_rows(q), CLEAR_REST
        q_arg = (*q_args, *_row_tensor(q_out, "q_out", q.shape, dev))
    rotation = _rotation_arg(rope, dev) if rope is not None else None
    if T == 0:
        return q_out
    shape = _kept(_append_shapes, (B, H_q, H_kv, d, n_max), lambda x: ctypes.byref(_checked_shape(x)))
    with _on_device(dev):
        rc = (_lib or load()).santa_paged_append(shape, _paged_arg(cache), ctypes.byref(_Rows(k_ptr, v_ptr, k_st, v_st)),
                                       T | clear, pos.data_ptr(), counts.data_ptr() if counts is not None else None, rotation, *q_arg,
                                       _workspace_ptr(workspace, dev), _raw_stream(None, dev))
    if rc:
        _check(rc, "santa_paged_append")
    return q_out


_attend_shapes: dict = {}


def _attend_shape_of(key):
    """(the shape as a C argument, the workspace bytes of attend_paged), kept per shape and T."""
    shape, n = _checked_shape(key[:-1]), ctypes.c_size_t(0)
    _check_tokens(key[-1])
    _check(load().santa_attend_workspace_size(ctypes.byref(shape), key[-1], ctypes.byref(n)), "santa_attend_workspace_size")
    return ctypes.byref(shape), int(n.value)


def attend_paged(q: torch.Tensor, cache: PagedCache, pos: torch.Tensor, counts: torch.Tensor | None = None, window: int = 0,
                 sinks: int = 0, scale: float = 0.0, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Causal attention of T new tokens a sequence (1: a decode step) over a paged cache that holds
    their K and V already.  q [B, T, H_q, d] (bf16, any strides that are multiples of 8); token t < counts[b]
    (default T) sits at pos[b] + t (int32 [B]) and sees the keys up to its own, with window > 0 the
    last `window` of them and the first `sinks`.  Returns bf16 [B, T, H_q, d]: `out`, whose other rows
    stay as they were, or new rows, the others zero.  Batch rows with a position or a count out of range are
    skipped (in new rows: zeros), and a key without a page counts as zeros; give a `workspace` to have that
    reported by device_status (DEV_BAD_POSITION, DEV_BAD_PAGE).  On an explicit `stream`, the call and all that it
    allocates are that stream's: order its inputs and its result with the current stream as for any
    work on another one."""
    B, H_kv, n_max, d, _, dev = _paged_dims(cache)
    if not (-1 << 31 <= window < 1 << 31 and -1 << 31 <= sinks < 1 << 31):
        raise ValueError("window and sinks are 32-bit numbers")
    if stream is not None:
        return _on_stream(stream, dev, lambda: attend_paged(q, cache, pos, counts, window, sinks, scale, out, workspace),
                          out is None)
    q_ptr, q_st = _row_tensor(q, "q", None, dev)
    size = q.shape
    if size[0] != B or size[3] != d:
        raise ValueError("q [B, T, H_q, d] and the cache's shape disagree")
    _int_vector(pos, "pos", B, dev)
    if counts is not None:
        _int_vector(counts, "counts", B, dev)
    T = size[1]
    shape, nbytes = _kept(_attend_shapes, (B, size[2], H_kv, d, n_max, scale, T), _attend_shape_of)
    clear = 0
    if out is None:
        out, clear = _out_rows(q), CLEAR_REST
    elif out.dtype is not torch.bfloat16 or not out.is_contiguous() or out.shape != size or out.device != dev:
        raise ValueError("out must be a contiguous bf16 tensor [B, T, H_q, d] on q's device")
    if T == 0:
        return out
    _workspace_ptr(workspace, dev)
    with _on_device(dev):
        raw = _raw_stream(None, dev)
        ws = workspace if workspace is not None else _own_workspace("attend", nbytes, dev, raw)
        rc = (_lib or load()).santa_attend_paged(shape, q_ptr, q_st, _paged_arg(cache), T | clear, pos.data_ptr(),
                                       counts.data_ptr() if counts is not None else None, window, sinks, out.data_ptr(),
                                       ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc, "santa_attend_paged")
    return out
