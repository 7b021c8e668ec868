"""Python binding of libmoe, the sm_100a routed-expert MoE layer library.

Argument marshalling only: every function below checks that its torch tensors
have the dtype and shape the C ABI expects, passes their device pointers and
the current CUDA stream to the function of the same name in libmoe.so
(include/moe.h), and raises ``MoeError`` on a non-zero status.  Every step of
the layer runs in the library's kernels; there is no fallback: if libmoe.so
is missing or fails to load, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_LIBRARY=bounds loads the bounds-checked build (every index the kernels
# read from data range-checked into the status word), for tests
LIB_PATH = os.path.join(_PKG, "libmoe_bounds.so" if os.environ.get("MOE_LIBRARY") == "bounds" else "libmoe.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "moe.h")

MOE_OK, MOE_EINVAL, MOE_EALIGN, MOE_ENOSPACE, MOE_ECUDA, MOE_ETIMEOUT, MOE_EDEVICE = 0, -1, -2, -3, -4, -5, -6
MOE_IO_X_HOST, MOE_IO_OUT_HOST = 1, 2  # moe_layer_opts.io_host bits
MOE_F32, MOE_BF16, MOE_I8 = 0, 1, 2
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_GROUP_TOP2, MOE_GROUP_MAX = 0, 1
MOE_PATH_AUTO, MOE_PATH_MULTI, MOE_PATH_DECODE, MOE_PATH_TC = 0, 1, 2, 3


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status}: {detail}")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("f", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("has_shared", ctypes.c_int32), ("wbits", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("tc_min_tokens", ctypes.c_int32), ("topp", ctypes.c_float)]

    @property
    def blob_bytes(self) -> int:
        return 3 * self.d * self.f * self.wbits // 8

    @property
    def n_blobs(self) -> int:
        return self.n_experts + self.has_shared

    @property
    def scale_rows(self) -> int:
        return 2 * self.f + self.d


class MoeLayerOpts(ctypes.Structure):
    _fields_ = [("events", ctypes.c_void_p * 4), ("path", ctypes.c_int32), ("n_launches", ctypes.c_int32),
                ("trace", ctypes.c_void_p), ("path_ran", ctypes.c_int32),
                ("wait_limit_us", ctypes.c_int32), ("test_skip_h", ctypes.c_int32), ("io_host", ctypes.c_int32)]


class MoePool(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("s", ctypes.c_void_p), ("slot_of", ctypes.c_void_p),
                ("n_slots", ctypes.c_int32)]
    _tensors = ()  # make_pool's


class MoeCache(ctypes.Structure):
    _fields_ = [("host_w", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("slot_of", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("n_slots", ctypes.c_int32)]


class MoeCacheStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int64), ("misses", ctypes.c_int64), ("bytes", ctypes.c_int64)]


class MoeGateRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_value", ctypes.c_int32), ("raw_weights", ctypes.c_int32)]


class MoeAdapters(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("r_max", ctypes.c_int32), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("scale", ctypes.c_void_p)]
    _device = None  # make_adapters': the tables' device


def config(d: int, f: int, n_experts: int, top_k: int, has_shared: int = 1, wbits: int = 4,
           routed_scale: float = 2.5, tc_min_tokens: int = 0, topp: float = 0.0) -> MoeConfig:
    return MoeConfig(d, f, n_experts, top_k, has_shared, wbits, routed_scale, tc_min_tokens, topp)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python expert_ffn_router_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    C = ctypes.POINTER(MoeConfig)
    PL, R, I64 = ctypes.POINTER(MoePool), ctypes.POINTER(MoeGateRule), ctypes.c_int64
    sig = {
        "moe_workspace_bytes": (SZ, [C, I32]),
        "moe_workspace_init": (I32, [P, SZ, P]),
        "moe_quantize": (I32, [C, P, I32, I32, P, P, P]),
        "moe_route": (I32, [C, P, I32, I32, P, P, P, P, P, SZ, P]),
        "moe_route_static": (I32, [C, P, I32, I32, P, P, P, P, P]),
        "moe_expert_ffn": (I32, [C, PL, I32, P, P, I32, P, P, P, P, P, P, SZ, P]),
        "moe_expert_down": (I32, [C, PL, I32, P, P, I32, P, P, P, SZ, P]),
        "moe_layer": (I32, [C, PL, P, P, P, I32, I32, P, I32, P, P, P, SZ, P]),
        "moe_layer_ex": (I32, [C, PL, P, P, P, I32, I32, P, I32, P, P, P, SZ, P, ctypes.POINTER(MoeLayerOpts)]),
        "moe_gate": (I32, [C, R, P, I32, I64, I32, P, P, P, P]),
        "moe_route_gated": (I32, [C, R, P, I32, I32, P, P, P, P, P, SZ, P]),
        "moe_layer_routed": (I32, [C, PL, P, P, P, I32, I32, P, I32, P, SZ, P]),
        "moe_adapter_plan_bytes": (SZ, [I32, I32]),
        "moe_adapter_plan": (I32, [I32, P, I32, P, SZ, P]),
        "moe_adapter": (I32, [ctypes.POINTER(MoeAdapters), P, SZ, P, I32, P, I64, I32, P, I64, P, I64, P]),
        "moe_rmsnorm": (I32, [P, I32, I32, I32, F, P, P, P]),
        "moe_poll_status": (I32, [P, ctypes.POINTER(I32), P]),
        "moe_cache_state_bytes": (SZ, [C, I32]),
        "moe_cache_init": (I32, [C, ctypes.POINTER(MoeCache), P]),
        "moe_cache_fetch": (I32, [C, ctypes.POINTER(MoeCache), P, I32, P, ctypes.POINTER(MoeCacheStats)]),
        "moe_status_string": (ctypes.c_char_p, [I32]),
        "moe_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def declared_symbols() -> list:
    """Names of the entry points include/moe.h declares."""
    with open(HEADER) as fh:
        return re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", fh.read())


def _check(st: int, where: str):
    if st != MOE_OK:
        raise MoeError(st, where, lib.moe_last_error().decode())


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor], dtype=None, numel: Optional[int] = None, name: str = "",
         host: bool = False) -> Optional[int]:
    if t is None:
        return None
    if host:
        if t.is_cuda or not t.is_pinned():
            raise ValueError(f"{name}: expected a pinned host tensor")
    elif not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _xdtype(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return MOE_F32
    if x.dtype == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")


def make_pool(w: torch.Tensor, s: torch.Tensor, slot_of: Optional[torch.Tensor] = None,
              n_slots: int = 0) -> MoePool:
    """The C struct over device tensors; it keeps references to them, so their
    memory stays allocated for as long as the struct is in use.  With
    ``slot_of`` (an HBM expert cache's slot table) ``w`` holds ``n_slots``
    blobs."""
    pool = MoePool(_ptr(w, torch.uint8, name="pool.w"), _ptr(s, torch.float32, name="pool.s"),
                   _ptr(slot_of, torch.int32, name="pool.slot_of"), n_slots if slot_of is not None else 0)
    pool._tensors = (w, s, slot_of)
    return pool


class ExpertCache:
    """An HBM expert cache over one layer's pool in pinned host memory
    (moe_cache_init / moe_cache_fetch): ``n_slots`` device blobs, the slot
    table and the host book-keeping, all owned here.  ``pool`` is the
    moe_pool over the slots to pass to moe_layer after ``fetch``."""

    def __init__(self, cfg: MoeConfig, host_w: torch.Tensor, scales: torch.Tensor, n_slots: int, device="cuda",
                 stream=None):
        if host_w.is_cuda or not host_w.is_pinned():
            raise ValueError("host_w: expected a pinned host tensor")
        self.cfg = cfg
        B = cfg.blob_bytes
        self.host_w = host_w
        self.slots = torch.empty(n_slots * B, dtype=torch.uint8, device=device)
        self.slot_of = torch.empty(cfg.n_experts + cfg.has_shared, dtype=torch.int32, device=device)
        nb = lib.moe_cache_state_bytes(ctypes.byref(cfg), n_slots)
        if nb == 0:
            raise MoeError(MOE_EINVAL, "moe_cache_state_bytes", lib.moe_last_error().decode())
        self.state = (ctypes.c_uint64 * ((nb + 7) // 8))()
        self.c = MoeCache(host_w.data_ptr(), self.slots.data_ptr(), self.slot_of.data_ptr(),
                          ctypes.addressof(self.state), n_slots)
        self.pool = make_pool(self.slots, scales, self.slot_of, n_slots)
        _check(lib.moe_cache_init(ctypes.byref(cfg), ctypes.byref(self.c), _stream(stream)), "moe_cache_init")

    def fetch(self, idx_host: torch.Tensor, stream=None) -> MoeCacheStats:
        """Makes the experts of ``idx_host`` (int32 [T][top_k] on the host)
        resident; returns this call's hits, misses and copied bytes."""
        idx_host = idx_host.contiguous()
        if idx_host.is_cuda or idx_host.dtype != torch.int32:
            raise ValueError("idx_host: expected an int32 host tensor")
        st = MoeCacheStats()
        _check(lib.moe_cache_fetch(ctypes.byref(self.cfg), ctypes.byref(self.c), idx_host.data_ptr(),
                                   idx_host.shape[0], _stream(stream), ctypes.byref(st)), "moe_cache_fetch")
        return st


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def moe_workspace_bytes(cfg: MoeConfig, max_tokens: int) -> int:
    n = lib.moe_workspace_bytes(ctypes.byref(cfg), max_tokens)
    if n == 0:
        raise MoeError(MOE_EINVAL, "moe_workspace_bytes", lib.moe_last_error().decode())
    return n


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib.moe_workspace_init(_ptr(ws, torch.uint8, name="ws"), ws.numel(), _stream(stream)),
           "moe_workspace_init")


def workspace(cfg: MoeConfig, max_tokens: int, device="cuda") -> torch.Tensor:
    """Allocate (through torch) and initialise a workspace for up to max_tokens."""
    ws = torch.empty(moe_workspace_bytes(cfg, max_tokens), dtype=torch.uint8, device=device)
    moe_workspace_init(ws)
    return ws


def moe_quantize(cfg: MoeConfig, x: torch.Tensor, xq: torch.Tensor, sx: torch.Tensor, stream=None):
    T = x.shape[0]
    _check(lib.moe_quantize(ctypes.byref(cfg), _ptr(x, name="x"), _xdtype(x), T,
                            _ptr(xq, torch.int8, T * cfg.d, "xq"), _ptr(sx, torch.float32, T, "sx"),
                            _stream(stream)), "moe_quantize")


def moe_route(cfg: MoeConfig, x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor,
              topk_idx: torch.Tensor, topk_w: torch.Tensor, ws: torch.Tensor, stream=None):
    T = x.shape[0]
    _check(lib.moe_route(ctypes.byref(cfg), _ptr(x, name="x"), _xdtype(x), T,
                         _ptr(w_router, torch.float32, cfg.n_experts * cfg.d, "w_router"),
                         _ptr(bias, torch.float32, cfg.n_experts, "bias"),
                         _ptr(topk_idx, torch.int32, T * cfg.top_k, "topk_idx"),
                         _ptr(topk_w, torch.float32, T * cfg.top_k, "topk_w"),
                         _ptr(ws, torch.uint8, name="ws"), ws.numel(), _stream(stream)), "moe_route")


def moe_route_static(cfg: MoeConfig, x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor,
                     topk_idx: torch.Tensor, topk_w: torch.Tensor, stream=None):
    """moe_route without a workspace, for callers that cannot allocate device
    memory on their call path; its scratch is a fixed array inside libmoe.so.
    Up to 8 tokens per call; calls that overlap on the GPU race."""
    T = x.shape[0]
    _check(lib.moe_route_static(ctypes.byref(cfg), _ptr(x, name="x"), _xdtype(x), T,
                                _ptr(w_router, torch.float32, cfg.n_experts * cfg.d, "w_router"),
                                _ptr(bias, torch.float32, cfg.n_experts, "bias"),
                                _ptr(topk_idx, torch.int32, T * cfg.top_k, "topk_idx"),
                                _ptr(topk_w, torch.float32, T * cfg.top_k, "topk_w"), _stream(stream)),
           "moe_route_static")


def moe_expert_ffn(cfg: MoeConfig, pool: MoePool, expert: int, xq: torch.Tensor, sx: torch.Tensor,
                   y: torch.Tensor, ws: torch.Tensor, dbg_acc_gu=None, dbg_hq=None, dbg_sh=None,
                   dbg_acc_d=None, stream=None):
    T = xq.shape[0]
    _check(lib.moe_expert_ffn(ctypes.byref(cfg), ctypes.byref(pool), expert,
                              _ptr(xq, torch.int8, T * cfg.d, "xq"), _ptr(sx, torch.float32, T, "sx"), T,
                              _ptr(y, torch.float32, T * cfg.d, "y"),
                              _ptr(dbg_acc_gu, torch.int32, T * 2 * cfg.f, "dbg_acc_gu"),
                              _ptr(dbg_hq, torch.int8, T * cfg.f, "dbg_hq"),
                              _ptr(dbg_sh, torch.float32, T, "dbg_sh"),
                              _ptr(dbg_acc_d, torch.int32, T * cfg.d, "dbg_acc_d"),
                              _ptr(ws, torch.uint8, name="ws"), ws.numel(), _stream(stream)), "moe_expert_ffn")


def moe_expert_down(cfg: MoeConfig, pool: MoePool, expert: int, hq: torch.Tensor, sh: torch.Tensor,
                    y: torch.Tensor, ws: torch.Tensor, dbg_acc_d=None, stream=None):
    T = hq.shape[0]
    _check(lib.moe_expert_down(ctypes.byref(cfg), ctypes.byref(pool), expert,
                               _ptr(hq, torch.int8, T * cfg.f, "hq"), _ptr(sh, torch.float32, T, "sh"), T,
                               _ptr(y, torch.float32, T * cfg.d, "y"),
                               _ptr(dbg_acc_d, torch.int32, T * cfg.d, "dbg_acc_d"),
                               _ptr(ws, torch.uint8, name="ws"), ws.numel(), _stream(stream)), "moe_expert_down")


def moe_layer(cfg: MoeConfig, pool: MoePool, w_router: torch.Tensor, bias: torch.Tensor, x: torch.Tensor,
              out: torch.Tensor, ws: torch.Tensor, accumulate: bool = False, topk_idx_out=None,
              topk_w_out=None, stream=None, opts: Optional[MoeLayerOpts] = None):
    """moe_layer, or moe_layer_ex when ``opts`` is given."""
    T = x.shape[0]
    io = opts.io_host if opts is not None else 0
    args = (ctypes.byref(cfg), ctypes.byref(pool),
            _ptr(w_router, torch.float32, cfg.n_experts * cfg.d, "w_router"),
            _ptr(bias, torch.float32, cfg.n_experts, "bias"), _ptr(x, name="x", host=bool(io & MOE_IO_X_HOST)),
            _xdtype(x), T,
            _ptr(out, torch.float32, T * cfg.d, "out", host=bool(io & MOE_IO_OUT_HOST)), 1 if accumulate else 0,
            _ptr(topk_idx_out, torch.int32, T * cfg.top_k, "topk_idx_out"),
            _ptr(topk_w_out, torch.float32, T * cfg.top_k, "topk_w_out"),
            _ptr(ws, torch.uint8, name="ws"), ws.numel(), _stream(stream))
    if opts is None:
        _check(lib.moe_layer(*args), "moe_layer")
    else:
        _check(lib.moe_layer_ex(*args, ctypes.byref(opts)), "moe_layer_ex")


def gate_rule(score: str = "sigmoid", n_groups: int = 0, topk_groups: int = 0, group_value: str = "top2",
              renorm: bool = True) -> MoeGateRule:
    """A selection rule: ``score`` "sigmoid" or "softmax"; with ``n_groups`` > 1
    a row selects from its ``topk_groups`` best groups, a group's value the sum
    of its two largest ("top2") or its largest ("max"); ``renorm`` divides the
    weights by their sum."""
    return MoeGateRule({"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}[score], n_groups, topk_groups,
                       {"top2": MOE_GROUP_TOP2, "max": MOE_GROUP_MAX}[group_value], 0 if renorm else 1)


def _here(t: torch.Tensor, name: str) -> int:
    """The current device, which ``t`` must be on."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device, cuda:{dev}, got {t.device}")
    return dev


def _arg(t: torch.Tensor, dev: int, dtype, numel: int, name: str) -> int:
    """_ptr for a tensor on the current device (its checks in one expression:
    a call of the small operators is shorter than their host time)."""
    if t.get_device() != dev or t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        _ptr(t, dtype, numel, name)
        raise ValueError(f"{name}: expected a tensor on the current device, cuda:{dev}, got {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, dev: int, d: int, name: str, dtype=None):
    """Pointer and row stride of a [T][d] matrix whose rows may lie apart."""
    if t.get_device() != dev:
        _here(t, name)
    if t.dim() != 2 or t.shape[1] != d:
        raise ValueError(f"{name}: expected [T][{d}], got {list(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    ld, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{name}: expected rows of neighbouring elements")
    return t.data_ptr(), ld if t.shape[0] > 1 else d  # one row's distance to the next says nothing


def _stream_on(stream: Optional[torch.cuda.Stream], dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.int8: MOE_I8}


def moe_gate(cfg: MoeConfig, rule: MoeGateRule, logits: torch.Tensor, bias: Optional[torch.Tensor],
             topk_idx: torch.Tensor, topk_w: torch.Tensor, stream=None):
    """Selects experts from logits [T][E] (float32 or bfloat16; rows may be a
    slice of a wider matrix): indices (-1: no expert) and weights."""
    dev = _here(logits, "logits")
    p, ld = _rows(logits, dev, cfg.n_experts, "logits")
    T, k = logits.shape[0], cfg.top_k
    st = lib.moe_gate(ctypes.byref(cfg), ctypes.byref(rule), p, _xdtype(logits), ld, T,
                      None if bias is None else _arg(bias, dev, torch.float32, cfg.n_experts, "bias"),
                      _arg(topk_idx, dev, torch.int32, T * k, "topk_idx"),
                      _arg(topk_w, dev, torch.float32, T * k, "topk_w"), _stream_on(stream, dev))
    if st != MOE_OK:
        _check(st, "moe_gate")


def moe_route_gated(cfg: MoeConfig, rule: MoeGateRule, x: torch.Tensor, w_router: torch.Tensor,
                    bias: Optional[torch.Tensor], topk_idx: torch.Tensor, topk_w: torch.Tensor, ws: torch.Tensor,
                    stream=None):
    """moe_route with the selection of moe_gate."""
    dev = _here(x, "x")
    T, n = x.shape[0], ws.numel()
    _check(lib.moe_route_gated(ctypes.byref(cfg), ctypes.byref(rule), _ptr(x, None, T * cfg.d, "x"), _xdtype(x), T,
                               _arg(w_router, dev, torch.float32, cfg.n_experts * cfg.d, "w_router"),
                               None if bias is None else _arg(bias, dev, torch.float32, cfg.n_experts, "bias"),
                               _arg(topk_idx, dev, torch.int32, T * cfg.top_k, "topk_idx"),
                               _arg(topk_w, dev, torch.float32, T * cfg.top_k, "topk_w"),
                               _arg(ws, dev, torch.uint8, n, "ws"), n, _stream(stream)), "moe_route_gated")


def moe_layer_routed(cfg: MoeConfig, pool: MoePool, topk_idx: torch.Tensor, topk_w: torch.Tensor, x: torch.Tensor,
                     out: torch.Tensor, ws: torch.Tensor, accumulate: bool = False, stream=None):
    """moe_layer for a routing the caller has."""
    dev = _here(x, "x")
    T, n = x.shape[0], ws.numel()
    for t, name in zip(pool._tensors, ("pool.w", "pool.s", "pool.slot_of")):
        if t is not None:
            _here(t, name)
    _check(lib.moe_layer_routed(ctypes.byref(cfg), ctypes.byref(pool),
                                _arg(topk_idx, dev, torch.int32, T * cfg.top_k, "topk_idx"),
                                _arg(topk_w, dev, torch.float32, T * cfg.top_k, "topk_w"),
                                _ptr(x, None, T * cfg.d, "x"), _xdtype(x), T,
                                _arg(out, dev, torch.float32, T * cfg.d, "out"), 1 if accumulate else 0,
                                _arg(ws, dev, torch.uint8, n, "ws"), n, _stream(stream)), "moe_layer_routed")


def make_adapters(a: torch.Tensor, b: torch.Tensor, rank: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None) -> MoeAdapters:
    """The C struct over ``a`` [n][r_max][d_in] and ``b`` [n][d_out][r_max]
    (bfloat16), ``rank`` [n] (int32) and ``scale`` [n] (float32), all on one
    device; it keeps references to them."""
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
        raise ValueError(f"adapters: expected a [n][r][d_in] and b [n][d_out][r], got {list(a.shape)}, {list(b.shape)}")
    n, r, d_in = a.shape
    ad = MoeAdapters(n, r, d_in, b.shape[1], _ptr(a, torch.bfloat16, name="adapters.a"),
                     _ptr(b, torch.bfloat16, name="adapters.b"), _ptr(rank, torch.int32, n, "adapters.rank"),
                     _ptr(scale, torch.float32, n, "adapters.scale"))
    ad._tensors = (a, b, rank, scale)
    ad._device = a.get_device()
    for t, name in ((b, "b"), (rank, "rank"), (scale, "scale")):
        if t is not None and t.get_device() != ad._device:
            raise ValueError(f"adapters.{name}: expected a tensor on the device of adapters.a, {a.device}, got {t.device}")
    return ad


def moe_adapter_plan_bytes(n_adapters: int, max_tokens: int) -> int:
    n = lib.moe_adapter_plan_bytes(n_adapters, max_tokens)
    if n == 0:
        raise MoeError(MOE_EINVAL, "moe_adapter_plan_bytes", lib.moe_last_error().decode())
    return n


def moe_adapter_plan(n_adapters: int, adapter_of: torch.Tensor, plan: torch.Tensor, stream=None):
    """The plan of a batch whose row t has the adapter ``adapter_of[t]`` (int32,
    -1: none), into ``plan``."""
    dev, T, n = _here(adapter_of, "adapter_of"), adapter_of.numel(), plan.numel()
    _check(lib.moe_adapter_plan(n_adapters, _arg(adapter_of, dev, torch.int32, T, "adapter_of"), T,
                                _arg(plan, dev, torch.uint8, n, "plan"), n, _stream(stream)),
           "moe_adapter_plan")


def adapter_plan(n_adapters: int, adapter_of: torch.Tensor, stream=None) -> torch.Tensor:
    """Allocate (through torch) and make the plan of a batch.  It is the current
    stream's memory: another ``stream`` that fills it waits for the current one
    first, and calls that read it on a third wait for ``stream``."""
    plan = torch.empty(moe_adapter_plan_bytes(n_adapters, adapter_of.numel()), dtype=torch.uint8,
                       device=adapter_of.device)
    if stream is not None and stream != torch.cuda.current_stream():
        stream.wait_stream(torch.cuda.current_stream())  # the memory may be a plan's that is still read there
        plan.record_stream(stream)
    moe_adapter_plan(n_adapters, adapter_of, plan, stream)
    return plan


def moe_adapter(ad: MoeAdapters, plan: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                base: Optional[torch.Tensor] = None, sx: Optional[torch.Tensor] = None, stream=None):
    """y = base + the rows' adapters of x (float32, bfloat16, or int8 codes
    with ``sx``); ``base`` may be ``y``; rows may lie apart."""
    dev = _here(x, "x")
    if ad._device != dev and ad._device is not None:
        raise ValueError(f"adapters: expected tables on the current device, cuda:{dev}, got cuda:{ad._device}")
    T = x.shape[0]
    xp, ldx = _rows(x, dev, ad.d_in, "x")
    yp, ldy = _rows(y, dev, ad.d_out, "y", torch.float32)
    bp, ldb = _rows(base, dev, ad.d_out, "base", torch.float32) if base is not None else (None, 0)
    if y.shape[0] != T or (base is not None and base.shape[0] != T):
        raise ValueError(f"x, y and base: expected {T} rows each")
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be float32, bfloat16 or int8, got {x.dtype}")
    n = plan.numel()
    st = lib.moe_adapter(ctypes.byref(ad), _arg(plan, dev, torch.uint8, n, "plan"), n, xp, _DTYPES[x.dtype],
                         None if sx is None else _arg(sx, dev, torch.float32, T, "sx"), ldx, T, bp, ldb, yp, ldy,
                         _stream_on(stream, dev))
    if st != MOE_OK:
        _check(st, "moe_adapter")


def moe_rmsnorm(x: torch.Tensor, x_in: torch.Tensor, eps: float = 1e-6, x_copy=None, stream=None):
    T, d = x.shape
    _check(lib.moe_rmsnorm(_ptr(x, name="x"), _xdtype(x), T, d, eps, _ptr(x_in, torch.float32, T * d, "x_in"),
                           _ptr(x_copy, torch.float32, T * d, "x_copy"), _stream(stream)), "moe_rmsnorm")


def moe_poll_status(ws: torch.Tensor, stream=None) -> int:
    info = ctypes.c_int32(0)
    st = lib.moe_poll_status(_ptr(ws, torch.uint8, name="ws"), ctypes.byref(info), _stream(stream))
    return st


__all__ = [n for n in dir() if n.startswith("moe_")] + ["MoeConfig", "MoePool", "MoeLayerOpts", "MoeGateRule",
                                                         "MoeAdapters", "MoeError", "config", "make_pool",
                                                         "gate_rule", "make_adapters", "adapter_plan", "workspace",
                                                         "lib"]
