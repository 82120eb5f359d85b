"""ctypes binding of libdspark's C ABI (include/dspark.h), same names, argument marshalling only.

Every function takes CUDA torch tensors (torch supplies device memory and streams, nothing
else), checks dtype / device / contiguity / size on the host, passes raw pointers and the
current CUDA stream, and raises DSparkError when the library returns an error code. All the
work of the hot path runs in the library's kernels; if the library is not built, the first
call raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

STATIC, COMPACT, CAP_ACCEPT = 0, 1, 2
MODES = {"static": STATIC, "compact": COMPACT, "cap_accept": CAP_ACCEPT}
BF16, F32 = 0, 1

STATUS_TIER_OVERFLOW = 0x01
STATUS_PACK_CAPACITY = 0x02
STATUS_BAD_WINDOW = 0x04
STATUS_OUT_OVERFLOW = 0x08
STATUS_BAD_COST = 0x10
STATUS_BAD_ROWS = 0x20
STATUS_BAD_TOKEN = 0x40
STATUS_BAD_LENGTH = 0x80
STATUS_STALL = 0x100
STATUS_BAD_PAGE = 0x200
STATUS_BAD_VALUE = 0x400
STATUS_NO_TOKEN = 0x800

ROPE_PLAIN, ROPE_LINEAR, ROPE_BY_PARTS = 0, 1, 2
ROPE_SCALINGS = {"none": ROPE_PLAIN, "linear": ROPE_LINEAR, "by_parts": ROPE_BY_PARTS}

STREAM_AUTO, STREAM_REGISTER, STREAM_BULK = 0, 1, 2

MAX_GAMMA = 32
MAX_CANDIDATES = 16384
MAX_BATCH = 8192
MAX_HISTORY = 524000
MAX_BIAS = 2047

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdspark.so")
_LOCK = threading.Lock()
_LIB = None

_p = ctypes.c_void_p
_i = ctypes.c_int
_u64 = ctypes.c_uint64
_i64 = ctypes.c_int64
_d = ctypes.c_double


class DSparkError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


class _Cost(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_double), ("alpha", ctypes.c_void_p), ("alpha_len", ctypes.c_int32),
                ("theta", ctypes.c_void_p), ("theta_len", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("heads", ctypes.c_int32), ("page", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("width", ctypes.c_int32)]


class _Adjustments(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("history_cap", ctypes.c_int32),
                ("bias_cap", ctypes.c_int32), ("repetition", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_len", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_row", ctypes.c_void_p), ("mask_stride", ctypes.c_int64),
                ("mask_rows", ctypes.c_int32)]


SYMBOLS = {
    "dspark_schedule": ([_p, _i, _i, ctypes.POINTER(_Cost), _p, _p, _p, _p], _i),
    "dspark_pack": ([_p, _p, _i, _i, _p, _i, _p, _p, _p, _p, _i, _p, _p, _p], _i),
    "dspark_verify": ([_i, _i, _p, _i, _p, _i, _i, _p, _p, _p, _i, _i, ctypes.c_float, _u64, _u64,
                       _p, _p, _p, _p, _p, ctypes.c_size_t, _p, _p], _i),
    "dspark_verify_workspace_bytes": ([_i, _i, _i, _i], ctypes.c_size_t),
    "dspark_scatter": ([_p, _p, _i, _i, _p, _p, _i, _p, _p], _i),
    "dspark_schedule_pack": ([_p, _i, _i, ctypes.POINTER(_Cost), _p, _p, _i, _p, _p, _p, _p, _p,
                              _p, _i, _p, _p, _p], _i),
    "dspark_verify_scatter": ([_i, _i, _p, _i, _p, _i, _i, _p, _p, _p, _i, _i, ctypes.c_float,
                               _u64, _u64, _p, _p, _p, _p, _p, ctypes.c_size_t, _p, _p, _i, _p,
                               _p], _i),
    "dspark_verify_noalloc": ([_i, _i, _p, _i, _p, _i, _i, _p, _p, _p, _i, _i, ctypes.c_float,
                               _u64, _u64, _p, _p, _p, _p, _p, _p], _i),
    "dspark_observe": ([_p, _p, _p, _i, _i, _i, _p, _p, _p, _p], _i),
    "dspark_rope_turns": ([_i, _d, _i, _d, _d, _d, _d, _p], _i),
    "dspark_rotate": ([_p, _i64, _p, _i64, _i, _i, _i, _i, _p, ctypes.POINTER(_Rope), _i, _p], _i),
    "dspark_append": ([ctypes.POINTER(_Cache), ctypes.POINTER(_Rope), _p, _i64, _p, _i64, _p, _i64,
                       _p, _i64, _i, _i, _i, _p, _p, _p, _i, _p, _p], _i),
    "dspark_attend": ([ctypes.POINTER(_Cache), _p, _i64, _p, _i64, _i, _i, _i, _p, _p, _i,
                       ctypes.c_float, _i, _p, _p, ctypes.c_size_t, _p, _p], _i),
    "dspark_attend_workspace_bytes": ([_i, _i], ctypes.c_size_t),
    "dspark_attend_sinks": ([ctypes.POINTER(_Cache), _p, _i64, _p, _i64, _i, _i, _i, _p, _p, _i,
                             ctypes.c_float, _i, _i, _p, _p, ctypes.c_size_t, _p, _p], _i),
    "dspark_attend_shared": ([ctypes.POINTER(_Cache), _p, _i64, _p, _i64, _i, _i, _i, _p, _p, _i,
                              _p, _p, _i, ctypes.c_float, _p, _p, ctypes.c_size_t, _p, _p], _i),
    "dspark_attend_shared_workspace_bytes": ([_i, _i, _i, _i, _i], ctypes.c_size_t),
    "dspark_adjust": ([_p, _i64, _p, _i64, _i, _i, _i, _p, _p, _i, _i,
                       ctypes.POINTER(_Adjustments), _p, _p], _i),
    "dspark_graph_begin": ([_p], _i),
    "dspark_graph_end": ([_p, ctypes.POINTER(_p)], _i),
    "dspark_graph_launch": ([_p, _p], _i),
    "dspark_graph_destroy": ([_p], _i),
    "dspark_set_stream_kernel": ([_i], _i),
    "dspark_set_stream_events": ([_p, _p], _i),
    "dspark_last_error": ([], ctypes.c_char_p),
    "dspark_version": ([], _i),
}


def lib():
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _LIB
    with _LOCK:
        if _LIB is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is not built: run speculative_decoding_ragged_gb300.build.build()")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SYMBOLS.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _LIB = handle
    return _LIB


def last_error() -> str:
    return lib().dspark_last_error().decode()


def _check(fn: str, rc: int):
    if rc != 0:
        raise DSparkError(fn, rc, last_error())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, numel=None, min_numel=None,
         required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} must have at least {min_numel} elements, got {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


class Prepared:
    """One checked, marshalled call: calling it re-issues the same C call (same pointers,
    sizes and stream) with no Python-side checks, for tight step loops."""

    __slots__ = ("name", "fn", "args")

    def __init__(self, name, args):
        self.name = name
        self.fn = getattr(lib(), name)
        self.args = args

    def __call__(self):
        rc = self.fn(*self.args)
        if rc != 0:
            raise DSparkError(self.name, rc, last_error())


def _call(name: str, args, prepare: bool):
    if prepare:
        return Prepared(name, args)
    _check(name, getattr(lib(), name)(*args))
    return None


def set_stream_kernel(which: int) -> None:
    """Which kernel streams the logits inside verify (STREAM_AUTO, STREAM_REGISTER,
    STREAM_BULK); results are bit-identical, only speed differs."""
    _check("dspark_set_stream_kernel", lib().dspark_set_stream_kernel(int(which)))


def set_stream_events(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]):
    """Record `start` / `stop` around the logit-streaming kernel of every later verify call
    (None, None: off). The events must have been recorded once (torch creates them lazily)."""
    def handle(ev):
        if ev is None:
            return None
        h = int(ev.cuda_event)
        if h == 0:
            raise ValueError("record the event once before handing it to the library")
        return ctypes.c_void_p(h)
    _check("dspark_set_stream_events", lib().dspark_set_stream_events(handle(start), handle(stop)))


class StepGraph:
    """Library calls captured once as a CUDA graph through the C ABI (dspark_graph_begin /
    dspark_graph_end) and replayed with one cudaGraphLaunch (dspark_graph_launch).

        s = torch.cuda.Stream()              # capture needs a stream other than the default
        with torch.cuda.stream(s):
            calls = [...]                    # prepared while s is current: bound to s
            g = StepGraph(s)
            for c in calls: c()
            g.end()
        g.launch()                           # replays on torch's current stream
    """

    def __init__(self, stream):
        self._stream = _stream(stream)
        self._h = ctypes.c_void_p()
        _check("dspark_graph_begin", lib().dspark_graph_begin(self._stream))

    def end(self):
        _check("dspark_graph_end", lib().dspark_graph_end(self._stream, ctypes.byref(self._h)))
        return self

    def prepare_launch(self, stream=None) -> "Prepared":
        """The replay as a prepared call bound to `stream` (torch's current by default)."""
        return Prepared("dspark_graph_launch", (self._h, _stream(stream)))

    def launch(self, stream=None):
        _check("dspark_graph_launch", lib().dspark_graph_launch(self._h, _stream(stream)))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _LIB is not None:
            _LIB.dspark_graph_destroy(h)
            self._h = ctypes.c_void_p()


def version() -> int:
    return lib().dspark_version()


class CostTable:
    """T(bs, K) = bias + alpha[bs] + theta[bs + K]; alpha and theta are float64 CUDA tensors."""

    def __init__(self, bias: float, alpha: torch.Tensor, theta: torch.Tensor):
        self.bias = float(bias)
        self.alpha = alpha
        self.theta = theta
        self._c = _Cost(self.bias, _ptr(alpha, "alpha", torch.float64), alpha.numel(),
                        _ptr(theta, "theta", torch.float64), theta.numel())

    @property
    def c(self):
        return self._c


def dspark_schedule(conf: torch.Tensor, cost: CostTable, windows: torch.Tensor,
                    k_star: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None,
                    prepare: bool = False):
    B = windows.numel()
    L = conf.shape[-1] if conf.dim() == 2 else 0
    gamma = L + 1
    args = (_ptr(conf, "conf", torch.float32, numel=B * L, required=L > 0 and B > 0), B, gamma,
            ctypes.byref(cost.c), _ptr(windows, "windows", torch.int32),
            _ptr(k_star, "k_star", torch.int32, min_numel=1),
            _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_schedule", args, prepare)


def dspark_pack(windows: torch.Tensor, block_tokens: torch.Tensor, tiers: torch.Tensor,
                cu_seqlens: torch.Tensor, packed_ids: torch.Tensor, meta: torch.Tensor,
                row_req: Optional[torch.Tensor] = None, row_pos: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    B, gamma = block_tokens.shape
    cap = packed_ids.numel()
    args = (
        _ptr(windows, "windows", torch.int32, numel=B, required=B > 0),
        _ptr(block_tokens, "block_tokens", torch.int32, required=B > 0), B, gamma,
        _ptr(tiers, "tiers", torch.int32), tiers.numel(),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=B + 1),
        _ptr(packed_ids, "packed_ids", torch.int32, required=cap > 0),
        _ptr(row_req, "row_req", torch.int32, min_numel=cap, required=False),
        _ptr(row_pos, "row_pos", torch.int32, min_numel=cap, required=False), cap,
        _ptr(meta, "meta", torch.int32, min_numel=2),
        _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_pack", args, prepare)


def dspark_schedule_pack(conf: torch.Tensor, cost: CostTable, block_tokens: torch.Tensor,
                         tiers: torch.Tensor, windows: torch.Tensor, k_star: torch.Tensor,
                         cu_seqlens: torch.Tensor, packed_ids: torch.Tensor, meta: torch.Tensor,
                         row_req: Optional[torch.Tensor] = None,
                         row_pos: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None,
                         prepare: bool = False):
    """dspark_schedule then dspark_pack of the windows it writes, in one kernel."""
    B, gamma = block_tokens.shape
    L = gamma - 1
    if conf.dim() == 2 and tuple(conf.shape) != (B, L):
        raise ValueError(f"conf must be [{B}, {L}]")
    cap = packed_ids.numel()
    args = (
        _ptr(conf, "conf", torch.float32, numel=B * L, required=L > 0 and B > 0), B, gamma,
        ctypes.byref(cost.c), _ptr(block_tokens, "block_tokens", torch.int32, required=B > 0),
        _ptr(tiers, "tiers", torch.int32), tiers.numel(),
        _ptr(windows, "windows", torch.int32, numel=B),
        _ptr(k_star, "k_star", torch.int32, min_numel=1),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=B + 1),
        _ptr(packed_ids, "packed_ids", torch.int32, required=cap > 0),
        _ptr(row_req, "row_req", torch.int32, min_numel=cap, required=False),
        _ptr(row_pos, "row_pos", torch.int32, min_numel=cap, required=False), cap,
        _ptr(meta, "meta", torch.int32, min_numel=2),
        _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_schedule_pack", args, prepare)


def dspark_verify_workspace_bytes(B: int, gamma: int, V: int, stochastic: bool) -> int:
    return int(lib().dspark_verify_workspace_bytes(B, gamma, V, int(bool(stochastic))))


def _dtype_code(t: torch.Tensor, name: str = "logits") -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _verify_args(mode, target, block_tokens, accept_len, committed, workspace, stochastic,
                 draft, cu_seqlens, windows, ceiling_len, row_prob, temperature, seed, step):
    mode = MODES[mode] if isinstance(mode, str) else int(mode)
    B, gamma = block_tokens.shape
    rows, V = target.shape
    dt = _dtype_code(target)
    if draft is not None:
        if draft.dtype != target.dtype or draft.shape[-1] != V:
            raise ValueError("draft logits must match the target's dtype and vocabulary")
        if draft.numel() != B * (gamma - 1) * V:
            raise ValueError(f"draft logits must hold B*(gamma-1) = {B * (gamma - 1)} rows")
    return (
        mode, int(bool(stochastic)), _ptr(target, "target"), rows,
        _ptr(draft, "draft", required=False), dt, V,
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=B + 1, required=False),
        _ptr(windows, "windows", torch.int32, min_numel=B, required=False),
        _ptr(block_tokens, "block_tokens", torch.int32), B, gamma, float(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _ptr(accept_len, "accept_len", torch.int32, min_numel=B),
        _ptr(committed, "committed", torch.int32, min_numel=B * gamma),
        _ptr(ceiling_len, "ceiling_len", torch.int32, min_numel=B, required=False),
        _ptr(row_prob, "row_prob", torch.float32, min_numel=2 * rows, required=False),
        _ptr(workspace, "workspace", required=False),
        workspace.numel() * workspace.element_size() if workspace is not None else 0)


def dspark_verify(mode, target: torch.Tensor, block_tokens: torch.Tensor,
                  accept_len: torch.Tensor, committed: torch.Tensor, workspace: torch.Tensor, *,
                  stochastic: bool = False, draft: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None,
                  windows: Optional[torch.Tensor] = None,
                  ceiling_len: Optional[torch.Tensor] = None,
                  row_prob: Optional[torch.Tensor] = None, temperature: float = 1.0,
                  seed: int = 0, step: int = 0, status: Optional[torch.Tensor] = None,
                  stream=None, prepare: bool = False):
    args = _verify_args(mode, target, block_tokens, accept_len, committed, workspace,
                        stochastic, draft, cu_seqlens, windows, ceiling_len, row_prob,
                        temperature, seed, step)
    args += (_ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_verify", args, prepare)


def dspark_verify_scatter(mode, target: torch.Tensor, block_tokens: torch.Tensor,
                          accept_len: torch.Tensor, committed: torch.Tensor,
                          workspace: torch.Tensor, out_tokens: torch.Tensor,
                          out_len: torch.Tensor, *, stochastic: bool = False,
                          draft: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None,
                          windows: Optional[torch.Tensor] = None,
                          ceiling_len: Optional[torch.Tensor] = None,
                          row_prob: Optional[torch.Tensor] = None, temperature: float = 1.0,
                          seed: int = 0, step: int = 0, status: Optional[torch.Tensor] = None,
                          stream=None, prepare: bool = False):
    """dspark_verify then dspark_scatter of its committed tokens, without the scatter launch."""
    B = block_tokens.shape[0]
    cap = out_tokens.shape[1] if out_tokens.dim() == 2 else 0
    args = _verify_args(mode, target, block_tokens, accept_len, committed, workspace,
                        stochastic, draft, cu_seqlens, windows, ceiling_len, row_prob,
                        temperature, seed, step)
    args += (_ptr(out_tokens, "out_tokens", torch.int32, min_numel=B * cap, required=B * cap > 0),
             _ptr(out_len, "out_len", torch.int32, min_numel=B, required=B > 0), cap,
             _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_verify_scatter", args, prepare)


def dspark_scatter(committed: torch.Tensor, accept_len: torch.Tensor, out_tokens: torch.Tensor,
                   out_len: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None,
                   prepare: bool = False):
    B, gamma = committed.shape
    cap = out_tokens.shape[1] if out_tokens.dim() == 2 else 0
    args = (
        _ptr(committed, "committed", torch.int32, required=B > 0),
        _ptr(accept_len, "accept_len", torch.int32, min_numel=B, required=B > 0), B, gamma,
        _ptr(out_tokens, "out_tokens", torch.int32, min_numel=B * cap, required=B * cap > 0),
        _ptr(out_len, "out_len", torch.int32, min_numel=B, required=B > 0), cap,
        _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_scatter", args, prepare)


def dspark_observe(conf: torch.Tensor, accept_len: torch.Tensor, ceiling_len: torch.Tensor,
                   hist: torch.Tensor, util: torch.Tensor, status: Optional[torch.Tensor] = None,
                   stream=None, prepare: bool = False):
    """Accumulate calibration counters (hist: int64 [n_bins, 3]) and utilisation counters
    (util: int64 [2]) on the device; see ece() and utilisation() for the derived metrics."""
    B = accept_len.numel()
    L = conf.shape[-1] if conf.dim() == 2 else 0
    n_bins = hist.numel() // 3
    if hist.numel() != 3 * n_bins or n_bins < 1:
        raise ValueError("hist must hold 3 counters per bin")
    args = (_ptr(conf, "conf", torch.float32, numel=B * L, required=B > 0 and L > 0),
            _ptr(accept_len, "accept_len", torch.int32, required=B > 0),
            _ptr(ceiling_len, "ceiling_len", torch.int32, numel=B, required=B > 0), B, L + 1,
            n_bins, _ptr(hist, "hist", torch.int64), _ptr(util, "util", torch.int64, numel=2),
            _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_observe", args, prepare)


def ece(hist) -> float:
    """Expected calibration error from dspark_observe's counters (n_bins x 3, host array)."""
    import numpy as np
    h = np.asarray(hist, dtype=np.float64).reshape(-1, 3)
    n = h[:, 0]
    N = n.sum()
    if N == 0:
        return 0.0
    nz = n > 0
    conf = h[nz, 1] / 4294967296.0 / n[nz]
    acc = h[nz, 2] / n[nz]
    return float((n[nz] / N * np.abs(acc - conf)).sum())


def utilisation(util) -> float:
    """Committed tokens over the acceptance ceiling, from dspark_observe's counters."""
    c, ceil = int(util[0]), int(util[1])
    return c / ceil if ceil else 0.0


# ---- the target forward's ragged operators: rotary positions, paged cache, attention -------
def rope_turns(rot: int, base: float = 10000.0, scaling="none", factor: float = 1.0,
               trained: float = 1.0, slow: float = 1.0, fast: float = 32.0):
    """dspark_rope_turns: the frequencies of rot / 2 pairs as 64-bit fractions of a turn per
    position, a host array (numpy uint64) to copy to the device once (Rope does)."""
    import numpy as np
    code = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    out = np.zeros(max(int(rot) // 2, 1), np.uint64)
    _check("dspark_rope_turns",
           lib().dspark_rope_turns(int(rot), float(base), code, float(factor), float(trained),
                                   float(slow), float(fast), out.ctypes.data))
    return out[:int(rot) // 2]


class Rope:
    """A rotation of the first 2 * len(turns) elements of every head: `turns` is an int64 (or
    uint64) CUDA tensor of dspark_rope_turns' values, `mscale` the factor on cos and sin."""

    def __init__(self, turns: torch.Tensor, mscale: float = 1.0, interleaved: bool = False):
        if turns.dtype not in (torch.int64, torch.uint64):
            raise ValueError(f"turns must be int64 or uint64, got {turns.dtype}")
        self.turns = turns
        self.mscale = float(mscale)
        self.interleaved = bool(interleaved)
        self._c = _Rope(_ptr(turns, "turns"), 2 * turns.numel(), int(interleaved), self.mscale)

    @classmethod
    def make(cls, rot: int, base: float = 10000.0, *, scaling="none", factor: float = 1.0,
             trained: float = 1.0, slow: float = 1.0, fast: float = 32.0, mscale=None,
             interleaved: bool = False, device="cuda"):
        """The rope of these frequencies; mscale None: 0.1 ln(factor) + 1 by parts, else 1."""
        import math
        import numpy as np
        turns = rope_turns(rot, base, scaling, factor, trained, slow, fast)
        if mscale is None:
            by_parts = scaling in ("by_parts", ROPE_BY_PARTS)
            mscale = 0.1 * math.log(factor) + 1.0 if by_parts else 1.0
        return cls(torch.as_tensor(turns.view(np.int64)).to(device), mscale, interleaved)

    @property
    def c(self):
        return self._c


class PagedCache:
    """An 8-bit paged key/value cache (dspark_cache) over the caller's tensors: k and v
    [n_pages, heads, page, dim] float8_e4m3fn (or uint8 codes), k_scale and v_scale
    [n_pages, heads] float32, table [B, width] int32."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, table: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must both be [n_pages, heads, page, dim]")
        for name, t in (("k", k), ("v", v)):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise ValueError(f"{name} must be float8_e4m3fn or uint8, got {t.dtype}")
        if table.dim() != 2:
            raise ValueError("table must be [B, width]")
        n, heads, page, dim = k.shape
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.n_pages, self.heads, self.page, self.dim = n, heads, page, dim
        self.B, self.width = table.shape
        scales = dict(dtype=torch.float32, numel=n * heads)
        self._c = _Cache(_ptr(k, "k"), _ptr(v, "v"), _ptr(k_scale, "k_scale", **scales),
                         _ptr(v_scale, "v_scale", **scales), _ptr(table, "table", torch.int32),
                         n, heads, page, dim, self.width)

    @classmethod
    def empty(cls, n_pages: int, heads: int, page: int, dim: int, table: torch.Tensor):
        """A zeroed cache of n_pages pages on the table's device."""
        dev = table.device
        pages = [torch.zeros(n_pages, heads, page, dim, dtype=torch.uint8, device=dev)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones(n_pages, heads, dtype=torch.float32, device=dev) for _ in range(2)]
        return cls(*pages, *scales, table)

    @property
    def c(self):
        return self._c


def _heads(t: torch.Tensor, name: str, dtype=None, rows=None, heads=None, dim=None):
    """(pointer, row stride) of rows of heads: [rows, heads, dim], the heads of a row dense, rows
    at any stride (a slice of a projection's output)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, dim]")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    r, h, d = t.shape
    if (rows is not None and r != rows) or (heads is not None and h != heads) or \
            (dim is not None and d != dim):
        raise ValueError(f"{name} must be [{rows}, {heads}, {dim}], got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a row must be dense")
    if r > 1 and s0 < h * d:
        raise ValueError(f"{name}: rows overlap")
    return ctypes.c_void_p(t.data_ptr()), s0 if r > 1 else h * d


def dspark_rotate(x: torch.Tensor, y: torch.Tensor, positions: torch.Tensor, rope: Rope, *,
                  inverse: bool = False, stream=None, prepare: bool = False):
    """y = x rotated by each row's position; inverse: rotated back, which is the gradient."""
    xp, xs = _heads(x, "x")
    rows, heads, dim = x.shape
    yp, ys = _heads(y, "y", x.dtype, rows, heads, dim)
    args = (xp, xs, yp, ys, _dtype_code(x, "x"), rows, heads, dim,
            _ptr(positions, "positions", torch.int32, numel=rows, required=rows > 0),
            ctypes.byref(rope.c), int(bool(inverse)), _stream(stream))
    return _call("dspark_rotate", args, prepare)


def dspark_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, row_req: torch.Tensor,
                  row_pos: torch.Tensor, lengths: torch.Tensor, *, rope: Optional[Rope] = None,
                  q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    """The packed rows' keys (rotated) and values into the cache; q, if given, rotated to q_out."""
    kp, ks = _heads(k, "k", None, None, cache.heads, cache.dim)
    rows = k.shape[0]
    vp, vs = _heads(v, "v", k.dtype, rows, cache.heads, cache.dim)
    if (q is None) != (q_out is None):
        raise ValueError("give both q and q_out or neither")
    qp, qs, op, os_, hq = None, 0, None, 0, 0
    if q is not None:
        qp, qs = _heads(q, "q", k.dtype, rows, None, cache.dim)
        hq = q.shape[1]
        op, os_ = _heads(q_out, "q_out", k.dtype, rows, hq, cache.dim)
    args = (ctypes.byref(cache.c), ctypes.byref(rope.c) if rope is not None else None,
            kp, ks, vp, vs, qp, qs, op, os_, hq, _dtype_code(k, "k"), rows,
            _ptr(row_req, "row_req", torch.int32, min_numel=rows, required=rows > 0),
            _ptr(row_pos, "row_pos", torch.int32, min_numel=rows, required=rows > 0),
            _ptr(lengths, "lengths", torch.int32, numel=cache.B), cache.B,
            _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    return _call("dspark_append", args, prepare)


def dspark_attend_workspace_bytes(heads: int, dim: int) -> int:
    return int(lib().dspark_attend_workspace_bytes(int(heads), int(dim)))


def _attend_args(cache, q, out, cu_seqlens, lengths, scale):
    qp, qs = _heads(q, "q", None, None, None, cache.dim)
    rows, hq, dim = q.shape
    op, os_ = _heads(out, "out", q.dtype, rows, hq, dim)
    if lengths.numel() != cache.B:
        raise ValueError(f"lengths must have {cache.B} elements, got {lengths.numel()}")
    return ((ctypes.byref(cache.c), qp, qs, op, os_, hq, _dtype_code(q, "q"), rows,
             _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=cache.B + 1),
             _ptr(lengths, "lengths", torch.int32), cache.B),
            float(dim) ** -0.5 if scale is None else float(scale))


def _attend_tail(q, lse, workspace, status, stream):
    return (_ptr(lse, "lse", torch.float32, min_numel=q.shape[0] * q.shape[1], required=False),
            _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))


def dspark_attend(cache: PagedCache, q: torch.Tensor, out: torch.Tensor, cu_seqlens: torch.Tensor,
                  lengths: torch.Tensor, workspace: torch.Tensor, *,
                  scale: Optional[float] = None, window: int = 0,
                  lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None, prepare: bool = False):
    """Attention of the packed rows over the cache; scale None: 1 / sqrt(dim); window 0: every
    token up to the row's own."""
    args, scale = _attend_args(cache, q, out, cu_seqlens, lengths, scale)
    args += (scale, int(window)) + _attend_tail(q, lse, workspace, status, stream)
    return _call("dspark_attend", args, prepare)


def dspark_attend_sinks(cache: PagedCache, q: torch.Tensor, out: torch.Tensor,
                        cu_seqlens: torch.Tensor, lengths: torch.Tensor, workspace: torch.Tensor, *,
                        window: int, sinks: int, scale: Optional[float] = None,
                        lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream=None, prepare: bool = False):
    """dspark_attend over the last `window` tokens and the first `sinks` tokens of each request."""
    args, scale = _attend_args(cache, q, out, cu_seqlens, lengths, scale)
    args += (scale, int(window), int(sinks)) + _attend_tail(q, lse, workspace, status, stream)
    return _call("dspark_attend_sinks", args, prepare)


def dspark_attend_shared_workspace_bytes(rows: int, q_heads: int, heads: int, dim: int, B: int) -> int:
    return int(lib().dspark_attend_shared_workspace_bytes(int(rows), int(q_heads), int(heads), int(dim), int(B)))


def dspark_attend_shared(cache: PagedCache, q: torch.Tensor, out: torch.Tensor,
                         cu_seqlens: torch.Tensor, lengths: torch.Tensor, group_cu: torch.Tensor,
                         prefix: torch.Tensor, workspace: torch.Tensor, *,
                         scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    """dspark_attend where the first prefix[g] tokens of the requests group_cu[g] .. group_cu[g + 1] - 1
    are the same tokens in the same pages: read once for the group."""
    args, scale = _attend_args(cache, q, out, cu_seqlens, lengths, scale)
    groups = prefix.numel()
    args += (_ptr(group_cu, "group_cu", torch.int32, min_numel=groups + 1, required=groups > 0),
             _ptr(prefix, "prefix", torch.int32), groups, scale)
    args += _attend_tail(q, lse, workspace, status, stream)
    return _call("dspark_attend_shared", args, prepare)


# ---- the logits between the target forward and verify ---------------------------------------
class Adjustments:
    """What dspark_adjust applies to a step's logits (dspark_adjustments), over the caller's CUDA
    tensors; what is None is left out. For B requests: history [B, cap] int32 with history_len and
    prompt_len [B] int32; repetition, presence, frequency [B] float32; bias_tokens [B, n] int32,
    bias_values [B, n] float32, bias_len [B] int32; mask [mask rows, >= V / 32 words] int32 (or
    uint32), its rows dense, and mask_row, int32, the mask row of each logits row (-1: none)."""

    def __init__(self, *, history=None, history_len=None, prompt_len=None, repetition=None,
                 presence=None, frequency=None, bias_tokens=None, bias_values=None, bias_len=None,
                 mask=None, mask_row=None):
        self.history, self.history_len, self.prompt_len = history, history_len, prompt_len
        self.repetition, self.presence, self.frequency = repetition, presence, frequency
        self.bias_tokens, self.bias_values, self.bias_len = bias_tokens, bias_values, bias_len
        self.mask, self.mask_row = mask, mask_row
        self.B = None                        # requests, by the first array given

        def rows(name, t, dtype, dims, like=None):
            if t is None:
                return None
            if t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
            if self.B is None:
                self.B = t.shape[0]
            if t.shape[0] != self.B:
                raise ValueError(f"{name} must be for {self.B} requests, got {t.shape[0]}")
            if like is not None and t.shape != like.shape:
                raise ValueError(f"{name} must be {tuple(like.shape)}, got {tuple(t.shape)}")
            return _ptr(t, name, dtype)

        if (history is None) != (history_len is None) or (history is None and prompt_len is not None):
            raise ValueError("history and history_len go together, prompt_len with them")
        if not (bias_tokens is None) == (bias_values is None) == (bias_len is None):
            raise ValueError("bias_tokens, bias_values and bias_len go together")
        if mask is None and mask_row is not None:
            raise ValueError("mask_row needs a mask")
        c = _Adjustments()
        c.history = rows("history", history, torch.int32, 2)
        c.history_len = rows("history_len", history_len, torch.int32, 1)
        c.prompt_len = rows("prompt_len", prompt_len, torch.int32, 1)
        c.history_cap = 0 if history is None else history.shape[1]
        c.repetition = rows("repetition", repetition, torch.float32, 1)
        c.presence = rows("presence", presence, torch.float32, 1)
        c.frequency = rows("frequency", frequency, torch.float32, 1)
        c.bias_tokens = rows("bias_tokens", bias_tokens, torch.int32, 2)
        c.bias_values = rows("bias_values", bias_values, torch.float32, 2, bias_tokens)
        c.bias_len = rows("bias_len", bias_len, torch.int32, 1)
        c.bias_cap = 0 if bias_tokens is None else bias_tokens.shape[1]
        if mask is not None:
            if mask.dim() != 2 or mask.dtype not in (torch.int32, torch.uint32):
                raise ValueError("mask must be [mask rows, words] int32 or uint32")
            if not mask.is_cuda:
                raise ValueError("mask must be a CUDA tensor")
            if mask.shape[1] > 1 and mask.stride(1) != 1:
                raise ValueError("mask: the words of a row must be dense")
            c.mask = ctypes.c_void_p(mask.data_ptr())
            c.mask_rows = mask.shape[0]
            c.mask_stride = mask.stride(0) if mask.shape[0] > 1 else mask.shape[1]
            c.mask_row = _ptr(mask_row, "mask_row", torch.int32, required=False)
        self._c = c

    @property
    def c(self):
        return self._c


def _rows_of(t: torch.Tensor, name: str):
    """(pointer, row stride) of [rows, V], a row's elements dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, V]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be dense")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap")
    return ctypes.c_void_p(t.data_ptr()), t.stride(0) if t.shape[0] > 1 else t.shape[1]


def dspark_adjust(logits: torch.Tensor, out: torch.Tensor, block_tokens: torch.Tensor,
                  how: Adjustments, *, cu_seqlens: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    """out = the rows' logits with penalties, biases and masks applied (out may be logits);
    cu_seqlens None: row b * gamma + i is request b's, as in the static verify mode."""
    xp, xs = _rows_of(logits, "logits")
    yp, ys = _rows_of(out, "out")
    if out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must have the shape and type of logits")
    rows, V = logits.shape
    B, gamma = block_tokens.shape
    if how.B is not None and how.B != B:
        raise ValueError(f"the adjustments are for {how.B} requests, the block tokens for {B}")
    if how.mask is not None and how.mask.shape[1] * 32 < V:
        raise ValueError(f"a mask row must have {-(-V // 32)} words, got {how.mask.shape[1]}")
    if how.mask_row is not None and how.mask_row.numel() < rows:
        raise ValueError(f"mask_row must have {rows} elements, got {how.mask_row.numel()}")
    args = (xp, xs, yp, ys, _dtype_code(logits), rows, V,
            _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=B + 1, required=False),
            _ptr(block_tokens, "block_tokens", torch.int32, required=B > 0), B, gamma,
            ctypes.byref(how.c), _ptr(status, "status", torch.int32, min_numel=1, required=False),
            _stream(stream))
    return _call("dspark_adjust", args, prepare)


NOALLOC_SCRATCH_BYTES = 4 << 20


def dspark_verify_noalloc(mode, target: torch.Tensor, block_tokens: torch.Tensor,
                          accept_len: torch.Tensor, committed: torch.Tensor, *,
                          stochastic: bool = False, draft: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None,
                          windows: Optional[torch.Tensor] = None,
                          ceiling_len: Optional[torch.Tensor] = None,
                          row_prob: Optional[torch.Tensor] = None, temperature: float = 1.0,
                          seed: int = 0, step: int = 0, status: Optional[torch.Tensor] = None,
                          stream=None):
    """dspark_verify without a workspace argument, for callers that cannot provide scratch
    memory: the library keeps a static 4 MiB device array per GPU and uses that instead.
    Calls that overlap on the GPU share the array; keep them ordered on one stream."""
    mode = MODES[mode] if isinstance(mode, str) else int(mode)
    B, gamma = block_tokens.shape
    rows, V = target.shape
    dt = _dtype_code(target)
    if draft is not None:
        if draft.dtype != target.dtype or draft.shape[-1] != V:
            raise ValueError("draft logits must match the target's dtype and vocabulary")
        if draft.numel() != B * (gamma - 1) * V:
            raise ValueError(f"draft logits must hold B*(gamma-1) = {B * (gamma - 1)} rows")
    rc = lib().dspark_verify_noalloc(
        mode, int(bool(stochastic)), _ptr(target, "target"), rows,
        _ptr(draft, "draft", required=False), dt, V,
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, min_numel=B + 1, required=False),
        _ptr(windows, "windows", torch.int32, min_numel=B, required=False),
        _ptr(block_tokens, "block_tokens", torch.int32), B, gamma, float(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _ptr(accept_len, "accept_len", torch.int32, min_numel=B),
        _ptr(committed, "committed", torch.int32, min_numel=B * gamma),
        _ptr(ceiling_len, "ceiling_len", torch.int32, min_numel=B, required=False),
        _ptr(row_prob, "row_prob", torch.float32, min_numel=2 * rows, required=False),
        _ptr(status, "status", torch.int32, min_numel=1, required=False), _stream(stream))
    _check("dspark_verify_noalloc", rc)
