"""Python binding of libpkv, the paged-KV decode step for GB300 (sm_103a).

The functions here have the names of the C ABI in ``include/pkv.h`` and do
argument marshalling only: they check dtypes, devices and contiguity of torch
tensors and pass their data pointers (and the current CUDA stream) to the
library.  Every step of the computation runs in the library's CUDA kernels;
there is no fallback.  If ``libpkv.so`` has not been built, importing the
binding's functions raises.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK, PKV_EINVAL, PKV_ERANGE, PKV_ENOMEM, PKV_ECUDA, PKV_EWORKSPACE, PKV_EDEVICE, PKV_ENOTIMPL = \
    0, -1, -2, -3, -4, -5, -6, -7
PKV_DEVERR_POSITION, PKV_DEVERR_PAGE, PKV_DEVERR_ROW, PKV_DEVERR_SLOT, PKV_DEVERR_TIMEOUT = 1, 2, 4, 8, 16

# Every symbol include/pkv.h declares.
ABI_SYMBOLS = ("pkv_config_default", "pkv_strerror", "pkv_pool_alloc", "pkv_pool_wrap", "pkv_pool_free",
               "pkv_pool_kv", "pkv_workspace_bytes", "pkv_decode", "pkv_step", "pkv_prefill", "pkv_check_errors",
               "pkv_set_ctas", "pkv_set_wait_limit", "pkv_timer_enable", "pkv_timer_read", "pkv_decode_static",
               "pkv_linear_workspace_bytes", "pkv_linear", "pkv_qkv_proj", "pkv_qkv_proj_append",
               "pkv_decode_appended", "pkv_output_gate", "pkv_q4_pool_bytes", "pkv_q4_pool_alloc", "pkv_q4_pool_wrap",
               "pkv_q4_pool_data", "pkv_q4_append", "pkv_q4_read", "pkv_q4_decode", "pkv_norm_rope",
               "pkv_rope_frequencies", "pkv_pool_set_rope")

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}                  # PKV_ROPE_HALF, PKV_ROPE_INTERLEAVED
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}  # PKV_ROPE_NONE ...

# Size of the scratch array pkv_decode_static uses in place of a workspace.
PKV_STATIC_SCRATCH_BYTES = 32 << 20


class PkvConfig(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_seq", ctypes.c_int),
                ("rope_theta", ctypes.c_double), ("eps", ctypes.c_double), ("rotary_dim", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class PkvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {pkv_strerror(code)} ({code})")
        self.code = code


_lib = None
_fast = None   # the module _pkv_torch (csrc/pkv_torch.cpp), if it was built for this torch
_BF16, _I32 = torch.bfloat16, torch.int32


def _raw_stream(device: int) -> int:
    """Handle of the device's current stream, without making a torch stream of it."""
    return torch._C._cuda_getCurrentRawStream(device)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libpkv.so (built by ``__graft_entry__.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libpkv.so not found at {path}: build it first (python -c 'import __graft_entry__ as g; "
                           f"g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(PkvConfig)
    sig = {
        "pkv_config_default": ([cfgp], i32),
        "pkv_strerror": ([i32], ctypes.c_char_p),
        "pkv_pool_alloc": ([cfgp, i32, vp, ctypes.POINTER(vp)], i32),
        "pkv_pool_wrap": ([cfgp, i32, vp, vp, vp, ctypes.POINTER(vp)], i32),
        "pkv_pool_free": ([vp], i32),
        "pkv_pool_kv": ([vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(i64)], i32),
        "pkv_workspace_bytes": ([vp, i32, i32, i32, ctypes.POINTER(sz)], i32),
        "pkv_decode": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp], i32),
        "pkv_step": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp], i32),
        "pkv_prefill": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp], i32),
        "pkv_check_errors": ([vp, vp, ctypes.POINTER(ctypes.c_uint32)], i32),
        "pkv_set_ctas": ([vp, i32], i32),
        "pkv_set_wait_limit": ([vp, i64], i32),
        "pkv_timer_enable": ([vp, i32], i32),
        "pkv_timer_read": ([vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)], i32),
        "pkv_decode_static": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp], i32),
        "pkv_linear_workspace_bytes": ([vp, i32, i32, i32, ctypes.POINTER(sz)], i32),
        "pkv_linear": ([vp, vp, vp, vp, i32, i32, i32, vp, sz, vp], i32),
        "pkv_qkv_proj": ([vp, vp, vp, i32, i32, vp, vp, vp, vp], i32),
        "pkv_qkv_proj_append": ([vp, vp, vp, i32, i32, vp, vp, vp, vp, i32, vp, vp], i32),
        "pkv_decode_appended": ([vp, vp, vp, vp, i32, i32, vp, vp, sz, vp], i32),
        "pkv_output_gate": ([vp, vp, vp, i32, vp], i32),
        "pkv_q4_pool_bytes": ([cfgp, i32, ctypes.POINTER(sz)], i32),
        "pkv_q4_pool_alloc": ([cfgp, i32, ctypes.c_float, ctypes.c_float, vp, ctypes.POINTER(vp)], i32),
        "pkv_q4_pool_wrap": ([cfgp, i32, vp, ctypes.c_float, ctypes.c_float, vp, ctypes.POINTER(vp)], i32),
        "pkv_q4_pool_data": ([vp, ctypes.POINTER(vp), ctypes.POINTER(sz)], i32),
        "pkv_q4_append": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp], i32),
        "pkv_q4_read": ([vp, vp, vp, vp, i32, i32, i32, vp, vp, i64, i64, vp], i32),
        "pkv_q4_decode": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp], i32),
        "pkv_norm_rope": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i64, vp, vp, i64, i64, vp], i32),
        "pkv_rope_frequencies": ([cfgp, i32, ctypes.c_double, i32, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_double)], i32),
        "pkv_pool_set_rope": ([vp, ctypes.POINTER(ctypes.c_double), ctypes.c_double, vp], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    _load_fast(lib)
    return lib


def _load_fast(lib) -> None:
    """The calls of a few microseconds go through a CPython module where it was built: 0.5 us of checks in place of 4."""
    global _fast
    try:
        from . import _pkv_torch as fast
    except ImportError:
        return
    if fast.torch_version == torch.__version__:
        fast.bind(*(ctypes.cast(getattr(lib, "pkv_" + name), ctypes.c_void_p).value
                    for name in ("q4_decode", "q4_append", "q4_read", "norm_rope")))
        _fast = fast


def _check(rc: int, what: str):
    if rc != PKV_OK:
        raise PkvError(rc, what)


def _stream(stream) -> int:
    """The stream's handle; None: the current device's current stream (asked for without making a torch stream)."""
    if stream is None:
        return _raw_stream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _capturing(stream) -> bool:
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


def _on(stream):
    """Allocations inside are ordered on `stream` (a torch stream or a handle; None: the current stream)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _dev(t: torch.Tensor | None, dtype: torch.dtype, what: str, allow_none: bool = False) -> int | None:
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{what} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    raise ValueError(f"{what} must be contiguous")


# ------------------------------------------------------------------ C ABI, one function each

def pkv_strerror(code: int) -> str:
    return load_library().pkv_strerror(int(code)).decode()


def pkv_config_default() -> PkvConfig:
    c = PkvConfig()
    _check(load_library().pkv_config_default(ctypes.byref(c)), "pkv_config_default")
    return c


def _cfg(cfg) -> PkvConfig:
    if cfg is None:
        return pkv_config_default()
    if isinstance(cfg, PkvConfig):
        return cfg
    c = pkv_config_default()
    for k, v in dict(cfg).items():
        setattr(c, k, v)
    return c


def pkv_pool_alloc(cfg, num_pages: int, stream=None) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check(load_library().pkv_pool_alloc(ctypes.byref(_cfg(cfg)), int(num_pages), _stream(stream),
                                         ctypes.byref(out)), "pkv_pool_alloc")
    return out


def pkv_pool_wrap(cfg, num_pages: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check(load_library().pkv_pool_wrap(ctypes.byref(_cfg(cfg)), int(num_pages), _dev(k, torch.bfloat16, "k"),
                                        _dev(v, torch.bfloat16, "v"), _stream(stream), ctypes.byref(out)),
           "pkv_pool_wrap")
    return out


def pkv_pool_free(pool) -> None:
    _check(load_library().pkv_pool_free(pool), "pkv_pool_free")


def pkv_pool_kv(pool):
    k, v, n = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_int64()
    _check(load_library().pkv_pool_kv(pool, ctypes.byref(k), ctypes.byref(v), ctypes.byref(n)), "pkv_pool_kv")
    return k.value, v.value, n.value


def pkv_workspace_bytes(pool, rows: int, pages: int, prefill_tokens: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(load_library().pkv_workspace_bytes(pool, int(rows), int(pages), int(prefill_tokens), ctypes.byref(n)),
           "pkv_workspace_bytes")
    return n.value


def _table(table, rows, pages):
    """(pointer, rows, pages) of a page table, or of the contiguous-row layout when ``table`` is None."""
    if table is None:
        if rows is None or pages is None:
            raise ValueError("without a table, rows and pages are required")
        return None, int(rows), int(pages)
    if table.dim() != 2:
        raise ValueError(f"table must be [rows][pages], got {tuple(table.shape)}")
    rows, pages = table.shape
    return _dev(table, torch.int32, "table"), rows, pages


def pkv_decode(pool, q, k, v, q_norm_w, k_norm_w, positions, table, out, workspace, stream=None,
               pages=None) -> None:
    """decode_paged; ``table=None`` with ``pages`` is decode_rows over contiguous rows."""
    tp, rows, pages = _table(table, positions.shape[0], pages)
    _check(load_library().pkv_decode(
        pool, _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), tp, rows, pages,
        _dev(out, torch.bfloat16, "out"), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "pkv_decode")


def pkv_decode_static(pool, q, k, v, q_norm_w, k_norm_w, positions, table, out, stream=None, pages=None) -> None:
    """pkv_decode without a workspace: the library's static scratch array is used instead."""
    tp, rows, pages = _table(table, positions.shape[0], pages)
    _check(load_library().pkv_decode_static(
        pool, _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), tp, rows, pages,
        _dev(out, torch.bfloat16, "out"), _stream(stream)), "pkv_decode_static")


def pkv_step(pool, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, step_positions, table, out, workspace,
             stream=None, pages=None) -> None:
    """step_paged; ``table=None`` with ``pages`` is step_packed over contiguous rows."""
    P = int(positions.shape[0])
    tp, rows, pages = _table(table, step_positions.shape[0], pages)
    _check(load_library().pkv_step(
        pool, _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), _dev(prow, torch.int32, "prow"),
        _dev(slots, torch.int32, "slots", allow_none=True), _dev(step_positions, torch.int32, "step_positions"),
        tp, P, rows, pages, _dev(out, torch.bfloat16, "out"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "pkv_step")


def pkv_prefill(pool, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, table, out, workspace, stream=None,
                rows=None, pages=None) -> None:
    """prefill_paged; ``table=None`` with ``rows`` and ``pages`` is prefill over contiguous rows."""
    P = int(positions.shape[0])
    tp, rows, pages = _table(table, rows, pages)
    _check(load_library().pkv_prefill(
        pool, _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), _dev(prow, torch.int32, "prow"),
        _dev(slots, torch.int32, "slots", allow_none=True), tp, P, rows, pages,
        _dev(out, torch.bfloat16, "out"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream)), "pkv_prefill")


def pkv_linear_workspace_bytes(pool, tokens: int, in_features: int, out_features: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().pkv_linear_workspace_bytes(pool, int(tokens), int(in_features), int(out_features),
                                                      ctypes.byref(n)), "pkv_linear_workspace_bytes")
    return n.value


def pkv_linear(pool, x, w, y, workspace=None, stream=None) -> None:
    """y = x w^T: x [tokens][in], w [out][in] (nn.Linear layout), y [tokens][out], all bf16."""
    if x.dim() != 2 or w.dim() != 2 or y.dim() != 2 or x.shape[1] != w.shape[1] or y.shape != (x.shape[0], w.shape[0]):
        raise ValueError(f"shapes x {tuple(x.shape)}, w {tuple(w.shape)}, y {tuple(y.shape)} do not match y = x w^T")
    ws = ctypes.c_void_p(None) if workspace is None else _dev(workspace, torch.uint8, "workspace")
    _check(load_library().pkv_linear(
        pool, _dev(x, torch.bfloat16, "x"), _dev(w, torch.bfloat16, "w"), _dev(y, torch.bfloat16, "y"),
        int(x.shape[0]), int(x.shape[1]), int(w.shape[0]), ws, 0 if workspace is None else workspace.numel(),
        _stream(stream)), "pkv_linear")


def pkv_qkv_proj(pool, x, w_qkv, q, k, v, stream=None) -> None:
    """q, k, v = x Wq^T, x Wk^T, x Wv^T with w_qkv = [Wq; Wk; Wv] stacked row-wise (one launch)."""
    tokens, hidden = int(x.shape[0]), int(x.shape[1])
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.shape[0] != tokens:
            raise ValueError(f"{name} has {t.shape[0]} tokens, x has {tokens}")
    if w_qkv.dim() != 2 or w_qkv.shape[1] != hidden or w_qkv.shape[0] != q[0].numel() + k[0].numel() + v[0].numel():
        raise ValueError(f"w_qkv {tuple(w_qkv.shape)} does not stack the q, k, v projections of x {tuple(x.shape)}")
    _check(load_library().pkv_qkv_proj(
        pool, _dev(x, torch.bfloat16, "x"), _dev(w_qkv, torch.bfloat16, "w_qkv"), tokens, hidden,
        _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), _stream(stream)),
        "pkv_qkv_proj")


def pkv_qkv_proj_append(pool, x, w_qkv, q_norm_w, k_norm_w, positions, table, q_hat, stream=None,
                        pages=None) -> None:
    """q/k/v projection of decode rows with QK-norm, RoPE and the k/v append in its epilogue;
    q_hat (fp32 [tokens][heads][head_dim]) receives the normed, roped q."""
    tokens, hidden = int(x.shape[0]), int(x.shape[1])
    tp, rows, pages = _table(table, positions.shape[0], pages)
    if rows != tokens or q_hat.shape[0] != tokens:
        raise ValueError(f"x has {tokens} tokens, positions/table {rows}, q_hat {q_hat.shape[0]}")
    _check(load_library().pkv_qkv_proj_append(
        pool, _dev(x, torch.bfloat16, "x"), _dev(w_qkv, torch.bfloat16, "w_qkv"), tokens, hidden,
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), tp, pages, _dev(q_hat, torch.float32, "q_hat"),
        _stream(stream)), "pkv_qkv_proj_append")


def pkv_decode_appended(pool, q_hat, positions, table, out, workspace, stream=None, pages=None) -> None:
    """decode_paged's attention after pkv_qkv_proj_append (q prepared, k/v already in the pool)."""
    tp, rows, pages = _table(table, positions.shape[0], pages)
    _check(load_library().pkv_decode_appended(
        pool, _dev(q_hat, torch.float32, "q_hat"), _dev(positions, torch.int32, "positions"), tp, rows, pages,
        _dev(out, torch.bfloat16, "out"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream)), "pkv_decode_appended")


def pkv_output_gate(pool, out, gate, stream=None) -> None:
    """out *= sigmoid(gate) in place (the gated-attention variant's output gate)."""
    if out.shape != gate.shape:
        raise ValueError(f"gate {tuple(gate.shape)} does not match out {tuple(out.shape)}")
    _check(load_library().pkv_output_gate(pool, _dev(out, torch.bfloat16, "out"), _dev(gate, torch.bfloat16, "gate"),
                                          int(out.shape[0]), _stream(stream)), "pkv_output_gate")


# ---- 4-bit pools

def pkv_q4_pool_bytes(cfg, num_pages: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().pkv_q4_pool_bytes(ctypes.byref(_cfg(cfg)), int(num_pages), ctypes.byref(n)),
           "pkv_q4_pool_bytes")
    return n.value


def pkv_q4_pool_alloc(cfg, num_pages: int, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check(load_library().pkv_q4_pool_alloc(ctypes.byref(_cfg(cfg)), int(num_pages), float(k_scale), float(v_scale),
                                            _stream(stream), ctypes.byref(out)), "pkv_q4_pool_alloc")
    return out


def pkv_q4_pool_wrap(cfg, num_pages: int, data: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0,
                     stream=None) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check(load_library().pkv_q4_pool_wrap(ctypes.byref(_cfg(cfg)), int(num_pages), _dev(data, torch.uint8, "data"),
                                           float(k_scale), float(v_scale), _stream(stream), ctypes.byref(out)),
           "pkv_q4_pool_wrap")
    return out


def pkv_q4_pool_data(pool):
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    _check(load_library().pkv_q4_pool_data(pool, ctypes.byref(p), ctypes.byref(n)), "pkv_q4_pool_data")
    return p.value, n.value


def _prow(prow, tokens):
    if prow is None:
        return None
    if prow.shape[0] != tokens:
        raise ValueError(f"prow has {prow.shape[0]} tokens, positions {tokens}")
    return _dev(prow, torch.int32, "prow")


def pkv_q4_append(pool, k, v, k_norm_w, positions, prow, table, stream=None, rows=None, pages=None) -> None:
    """Quantise k, v [tokens][kv_heads][head_dim] into the pool; ``prow=None``: token t is row t."""
    tokens = positions.shape[0]
    if k.shape != v.shape or k.shape[0] != tokens:
        raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)} and {tokens} positions do not match")
    tp, rows, pages = _table(table, rows, pages)
    _check(load_library().pkv_q4_append(
        pool, _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), _prow(prow, tokens), tp, tokens, rows, pages, _stream(stream)),
        "pkv_q4_append")


def pkv_q4_read(pool, positions, prow, table, k, v, stream=None, rows=None, pages=None) -> None:
    """Cached k and v of the tokens, into views [tokens][kv_heads][head_dim] whose heads are contiguous
    (a bf16 pool's K[:, s:s+n].transpose(0, 1) is one)."""
    tokens, strides = positions.shape[0], k.stride()
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or not k.is_cuda or not v.is_cuda:
        raise TypeError("k and v must be bf16 CUDA tensors")
    if len(strides) != 3 or strides[2] != 1 or v.stride() != strides or v.shape != k.shape or k.shape[0] != tokens:
        raise ValueError(f"k and v must be [{tokens}][kv_heads][head_dim] with contiguous heads, both alike")
    tp, rows, pages = _table(table, rows, pages)
    _check(load_library().pkv_q4_read(
        pool, _dev(positions, torch.int32, "positions"), _prow(prow, tokens), tp, tokens, rows, pages,
        k.data_ptr(), v.data_ptr(), strides[0], strides[1], _stream(stream)),
        "pkv_q4_read")


def pkv_q4_decode(pool, q, k, v, q_norm_w, k_norm_w, positions, table, out, workspace, stream=None,
                  pages=None) -> None:
    """decode_paged over a 4-bit pool; ``table=None`` with ``pages`` is the contiguous-row layout."""
    tp, rows, pages = _table(table, positions.shape[0], pages)
    if positions.shape[0] != rows:
        raise ValueError(f"table has {rows} rows, positions {positions.shape[0]}")
    _check(load_library().pkv_q4_decode(
        pool, _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
        _dev(q_norm_w, torch.bfloat16, "q_norm_w"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(positions, torch.int32, "positions"), tp, rows, pages, _dev(out, torch.bfloat16, "out"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "pkv_q4_decode")


# ---- norm + rotation

def pkv_norm_rope(pool, q, k, q_norm_w, k_norm_w, positions, q_out, k_out, layout="half", stream=None,
                  shape=None) -> None:
    """QK-norm and RoPE of q [tokens][heads][head_dim] and k [tokens][kv_heads][head_dim] (heads contiguous, any
    token stride) into q_out and k_out (both bf16 or both fp32).  q or k may be None; no weights: no norm.
    shape: the pool's (heads, kv_heads, head_dim), to be checked if given."""
    tokens = positions.shape[0]
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q and q_out, and k and k_out, are given together")
    if q is None and k is None:
        raise ValueError("q or k is required")
    kind = (k_out if q_out is None else q_out).dtype
    if kind is not _BF16 and kind is not torch.float32:
        raise TypeError(f"outputs must be bf16 or fp32, got {kind}")
    qp = qs = qo = qos = kp = ks = ko = kos = 0
    if q is not None:
        s = q.shape if shape is None else (tokens, shape[0], shape[2])
        qp, qs = _heads(q, _BF16, "q", tokens, s)
        qo, qos = _heads(q_out, kind, "q_out", tokens, s)
    if k is not None:
        s = k.shape if shape is None else (tokens, shape[1], shape[2])
        kp, ks = _heads(k, _BF16, "k", tokens, s)
        ko, kos = _heads(k_out, kind, "k_out", tokens, s)
    for w in (q_norm_w, k_norm_w):
        if w is not None and w.numel() != s[2]:
            raise ValueError(f"norm weights must be [{s[2]}], got {tuple(w.shape)}")
    rc = load_library().pkv_norm_rope(
        pool, qp, kp, None if q_norm_w is None else _dev(q_norm_w, _BF16, "q_norm_w"),
        None if k_norm_w is None else _dev(k_norm_w, _BF16, "k_norm_w"), _dev(positions, _I32, "positions"), tokens,
        ROPE_LAYOUTS[layout], kind is not _BF16, qs, ks, qo, ko, qos, kos, _stream(stream))
    if rc:
        raise PkvError(rc, "pkv_norm_rope")


def _heads(x, dtype, what, tokens, shape):
    """(pointer, token stride) of a tensor of that shape, [tokens][heads][head_dim], with contiguous heads."""
    if x.dtype is not dtype or not x.is_cuda:
        raise TypeError(f"{what} must be a {dtype} CUDA tensor, got {x.dtype}")
    if x.shape != shape or len(shape) != 3 or shape[0] != tokens:
        raise ValueError(f"{what} must be {list(shape)} for {tokens} positions, got {tuple(x.shape)}")
    token, head, dim = x.stride()
    if dim != 1 or (head != shape[2] and shape[1] > 1):
        raise ValueError(f"{what} must have contiguous heads, got strides {x.stride()}")
    return x.data_ptr(), token if tokens > 1 else shape[1] * shape[2]


def pkv_rope_frequencies(cfg, scaling="none", factor: float = 1.0, trained: int = 0):
    """(inverse frequencies of the rotated pairs, factor on cos and sin) of a scaled rotation."""
    c = _cfg(cfg)
    freq = (ctypes.c_double * max(1, (c.rotary_dim or c.head_dim) // 2))()
    m = ctypes.c_double()
    _check(load_library().pkv_rope_frequencies(ctypes.byref(c), ROPE_SCALINGS[scaling], float(factor), int(trained),
                                               freq, ctypes.byref(m)), "pkv_rope_frequencies")
    return list(freq), m.value


def pkv_pool_set_rope(pool, inv_freq, mscale: float = 1.0, stream=None) -> None:
    _check(load_library().pkv_pool_set_rope(pool, (ctypes.c_double * len(inv_freq))(*inv_freq), float(mscale),
                                            _stream(stream)), "pkv_pool_set_rope")


def pkv_check_errors(pool, stream=None) -> int:
    f = ctypes.c_uint32()
    _check(load_library().pkv_check_errors(pool, _stream(stream), ctypes.byref(f)), "pkv_check_errors")
    return f.value


def pkv_set_ctas(pool, ctas: int) -> None:
    _check(load_library().pkv_set_ctas(pool, int(ctas)), "pkv_set_ctas")


def pkv_set_wait_limit(pool, ns: int) -> None:
    _check(load_library().pkv_set_wait_limit(pool, int(ns)), "pkv_set_wait_limit")


def pkv_timer_enable(pool, enable) -> None:
    """enable: False/0 off, True/1 every timed launch, 2 the attention launches only."""
    _check(load_library().pkv_timer_enable(pool, int(enable)), "pkv_timer_enable")


def pkv_timer_read(pool):
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(load_library().pkv_timer_read(pool, ctypes.byref(ms), ctypes.byref(n)), "pkv_timer_read")
    return ms.value, n.value


# ------------------------------------------------------------------ convenience (marshalling only)

def _on_device(index: int, **tensors) -> None:
    """Refuses tensors of another device than the pool's: its kernels would read their pointers there."""
    for what, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.get_device() != index:
            raise ValueError(f"{what} lies on {t.device}, the pool on cuda:{index}")


class _Pool:
    """What pools of either format share: the workspace, norm + rotation, errors, closing."""

    handle = None
    _ws = None
    _shape = None   # (heads, kv_heads, head_dim)
    _spec = None    # (device index, heads, kv_heads, head_dim)
    _h = 0          # the handle's value

    def workspace(self, rows: int, pages: int, prefill_tokens: int = 0) -> torch.Tensor:
        n = pkv_workspace_bytes(self.handle, rows, pages, prefill_tokens)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        return self._ws

    def set_rope(self, inv_freq, mscale: float = 1.0, stream=None) -> None:
        """Other frequencies for this pool's rotation (see pkv_rope_frequencies)."""
        if len(inv_freq) != (self.cfg.rotary_dim or self.cfg.head_dim) // 2:
            raise ValueError(f"{len(inv_freq)} frequencies for a rotation of {self.cfg.rotary_dim} dims")
        pkv_pool_set_rope(self.handle, inv_freq, mscale, stream)

    def norm_rope(self, q, k, q_norm_w, k_norm_w, positions, layout="half", q_out=None, k_out=None,
                  dtype=torch.bfloat16, stream=None):
        """(q, k) normed over each head and rotated; fp32 q is what pkv_decode_appended takes."""
        if q is not None and q_out is None:
            with _on(stream):
                q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
        if k is not None and k_out is None:
            with _on(stream):
                k_out = torch.empty(k.shape, dtype=dtype, device=k.device)
        if _fast is not None and layout in ROPE_LAYOUTS:
            raw = _raw_stream(self._spec[0]) if stream is None else _stream(stream)
            rc = _fast.norm_rope(self._h, self._spec, q, k, q_norm_w, k_norm_w, positions, ROPE_LAYOUTS[layout],
                                 q_out, k_out, raw)
            if rc is not None:
                _check(rc, "pkv_norm_rope")
                return q_out, k_out
        _on_device(self._spec[0], q=q, k=k, q_norm_w=q_norm_w, k_norm_w=k_norm_w, positions=positions, q_out=q_out,
                   k_out=k_out)
        pkv_norm_rope(self.handle, q, k, q_norm_w, k_norm_w, positions, q_out, k_out, layout, stream, self._shape)
        return q_out, k_out

    def check_errors(self, stream=None) -> int:
        return pkv_check_errors(self.handle, stream)

    def close(self):
        if self.handle is not None and self.handle.value:
            pkv_pool_free(self.handle)
        self.handle, self._h = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedKVPool(_Pool):
    """A pool over caller-owned K/V torch tensors [kv_heads][num_pages*page_size][head_dim] (bf16).  Its calls share one
    workspace: on one stream and from one host thread at a time."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, cfg=None, stream=None):
        c = _cfg(cfg)
        if K.shape != V.shape or K.dim() != 3 or K.shape[0] != c.kv_heads or K.shape[2] != c.head_dim \
                or K.shape[1] % c.page_size:
            raise ValueError(f"K/V must be [kv_heads][num_pages*page_size][head_dim], got {tuple(K.shape)}")
        self.K, self.V, self.cfg = K, V, c
        self.num_pages = K.shape[1] // c.page_size
        self.device, self._shape = K.device, (c.heads, c.kv_heads, c.head_dim)
        self.handle = pkv_pool_wrap(c, self.num_pages, K, V, stream)
        self._h, self._spec = self.handle.value, (K.get_device(), *self._shape)
        self._lws = None

    def decode(self, q, k, v, q_norm_w, k_norm_w, positions, table, out=None, stream=None,
               pages=None) -> torch.Tensor:
        if out is None:
            out = torch.empty_like(q)
        pages = table.shape[1] if table is not None else pages
        ws = self.workspace(positions.shape[0], pages, 0)
        pkv_decode(self.handle, q, k, v, q_norm_w, k_norm_w, positions, table, out, ws, stream, pages=pages)
        return out

    def step(self, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, step_positions, table, out=None,
             stream=None, pages=None) -> torch.Tensor:
        if out is None:
            out = torch.empty_like(q)
        pages = table.shape[1] if table is not None else pages
        ws = self.workspace(step_positions.shape[0], pages, positions.shape[0])
        pkv_step(self.handle, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, step_positions, table, out, ws,
                 stream, pages=pages)
        return out

    def prefill(self, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, table, out=None, stream=None,
                rows=None, pages=None) -> torch.Tensor:
        if out is None:
            out = torch.empty_like(q)
        pages = table.shape[1] if table is not None else pages
        ws = self.workspace(0, pages, positions.shape[0])
        pkv_prefill(self.handle, q, k, v, q_norm_w, k_norm_w, positions, prow, slots, table, out, ws, stream,
                    rows=rows, pages=pages)
        return out

    def linear(self, x, w, y=None, stream=None) -> torch.Tensor:
        """y = x w^T on this pool's device (a projection before or after the attention)."""
        if y is None:
            y = torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device=x.device)
        n = pkv_linear_workspace_bytes(self.handle, x.shape[0], x.shape[1], w.shape[0])
        ws = None
        if n:
            if self._lws is None or self._lws.numel() < n:
                self._lws = torch.empty(n, dtype=torch.uint8, device=x.device)
            ws = self._lws
        pkv_linear(self.handle, x, w, y, ws, stream)
        return y

    def qkv_proj(self, x, w_qkv, q=None, k=None, v=None, stream=None):
        """q [tokens][heads][head_dim], k and v [tokens][kv_heads][head_dim] from x and the stacked weights."""
        c, n = self.cfg, x.shape[0]
        if q is None:
            q = torch.empty(n, c.heads, c.head_dim, dtype=torch.bfloat16, device=x.device)
        if k is None:
            k = torch.empty(n, c.kv_heads, c.head_dim, dtype=torch.bfloat16, device=x.device)
        if v is None:
            v = torch.empty(n, c.kv_heads, c.head_dim, dtype=torch.bfloat16, device=x.device)
        pkv_qkv_proj(self.handle, x, w_qkv, q, k, v, stream)
        return q, k, v

    def decode_layer_fused(self, x, w_qkv, q_norm_w, k_norm_w, positions, table, out=None, q_hat=None,
                           stream=None, pages=None) -> torch.Tensor:
        """The q/k/v projection with norm, RoPE and append fused in, then the attention."""
        c, n = self.cfg, x.shape[0]
        if q_hat is None:
            q_hat = torch.empty(n, c.heads, c.head_dim, dtype=torch.float32, device=x.device)
        if out is None:
            out = torch.empty(n, c.heads, c.head_dim, dtype=torch.bfloat16, device=x.device)
        pages = table.shape[1] if table is not None else pages
        pkv_qkv_proj_append(self.handle, x, w_qkv, q_norm_w, k_norm_w, positions, table, q_hat, stream, pages=pages)
        ws = self.workspace(n, pages, 0)
        pkv_decode_appended(self.handle, q_hat, positions, table, out, ws, stream, pages=pages)
        return out


class Q4KVPool(_Pool):
    """A 4-bit pool over a caller-owned uint8 tensor [num_pages][kv_heads][...] (pkv_q4_pool_bytes bytes; zeros are
    an empty pool, and ``Q4KVPool.empty`` makes one).  k_scale and v_scale are powers of two."""

    def __init__(self, data: torch.Tensor, cfg=None, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
        c = _cfg(cfg)
        per_page = pkv_q4_pool_bytes(c, 1)
        if data.dtype != torch.uint8 or data.numel() == 0 or data.numel() % per_page:
            raise ValueError(f"data must be uint8, a multiple of {per_page} bytes, got {data.dtype} x {data.numel()}")
        self.data, self.cfg, self.device, self._streams = data, c, data.device, {}
        self._shape = self._heads, self._kv_heads, self._dim = c.heads, c.kv_heads, c.head_dim
        self._lib, self._index, self._lock = load_library(), data.get_device(), threading.Lock()
        self.num_pages = data.numel() // per_page
        self.handle = pkv_q4_pool_wrap(c, self.num_pages, data, k_scale, v_scale, stream)
        self._h, self._spec = self.handle.value, (self._index, *self._shape)

    @classmethod
    def empty(cls, num_pages: int, cfg=None, k_scale: float = 1.0, v_scale: float = 1.0, device="cuda", stream=None):
        data = torch.zeros(pkv_q4_pool_bytes(cfg, num_pages), dtype=torch.uint8, device=device)
        return cls(data, cfg, k_scale, v_scale, stream)

    # A call whose arguments are as they should be goes through _fast, and a code that the library returns is raised.
    # What _fast returns None for, and every call where the module was not built, is checked here, and a wrong
    # argument raises.

    def append(self, k, v, k_norm_w, positions, prow, table, stream=None, rows=None, pages=None) -> None:
        """k normed and roped, then k and v quantised into their slots (prow None: token t is row t)."""
        raw = _raw_stream(self._index) if stream is None else _stream(stream)
        if _fast is not None:
            rc = _fast.append(self._h, self._spec, k, v, k_norm_w, positions, prow, table, rows, pages, raw)
            if rc is not None:
                return _check(rc, "pkv_q4_append")
        _on_device(self._index, k=k, v=v, k_norm_w=k_norm_w, positions=positions, prow=prow, table=table)
        n = positions.shape[0]
        shape = (n, self._kv_heads, self._dim)
        if k.shape != shape or v.shape != shape or k_norm_w.numel() != self._dim:
            raise ValueError(f"k and v must be {list(shape)} and k_norm_w [{self._dim}], got {tuple(k.shape)}, "
                             f"{tuple(v.shape)} and {tuple(k_norm_w.shape)}")
        tp, rows, pages = _table(table, rows, pages)
        rc = self._lib.pkv_q4_append(
            self.handle, _dev(k, _BF16, "k"), _dev(v, _BF16, "v"), _dev(k_norm_w, _BF16, "k_norm_w"),
            _dev(positions, _I32, "positions"), None if prow is None else _prow(prow, n), tp, n, rows, pages, raw)
        if rc:
            raise PkvError(rc, "pkv_q4_append")

    def read(self, positions, prow, table, k=None, v=None, stream=None, rows=None, pages=None):
        """(k, v) [tokens][kv_heads][head_dim] that the pool holds at the tokens' positions."""
        raw = _raw_stream(self._index) if stream is None else _stream(stream)
        n = positions.shape[0]
        shape = (n, self._kv_heads, self._dim)
        if k is None or v is None:
            with _on(stream):
                new = torch.empty(2, *shape, dtype=torch.bfloat16, device=self.device)
            k, v = new[0] if k is None else k, new[1] if v is None else v
        if _fast is not None:
            rc = _fast.read(self._h, self._spec, positions, prow, table, k, v, rows, pages, raw)
            if rc is not None:
                _check(rc, "pkv_q4_read")
                return k, v
        _on_device(self._index, positions=positions, prow=prow, table=table, k=k, v=v)
        strides = k.stride()
        if k.shape != shape or v.shape != shape or v.stride() != strides or strides[2] != 1:
            raise ValueError(f"k and v must be {list(shape)} with contiguous heads and the same strides, got "
                             f"{tuple(k.shape)} by {strides} and {tuple(v.shape)} by {v.stride()}")
        if k.dtype is not _BF16 or v.dtype is not _BF16 or not k.is_cuda or not v.is_cuda:
            raise TypeError("k and v must be bf16 CUDA tensors")
        tp, rows, pages = _table(table, rows, pages)
        rc = self._lib.pkv_q4_read(
            self.handle, _dev(positions, _I32, "positions"), None if prow is None else _prow(prow, n), tp, n, rows, pages,
            k.data_ptr(), v.data_ptr(), strides[0], strides[1], raw)
        if rc:
            raise PkvError(rc, "pkv_q4_read")
        return k, v

    def decode(self, q, k, v, q_norm_w, k_norm_w, positions, table, out=None, stream=None, pages=None) -> torch.Tensor:
        """One step of every row: append its k and v, attend over its cached positions.

        The workspace is the class's own: one kept per stream, and each captured call's in its graph, so that graphs
        and calls on other streams may run at the same time.  Host threads may share a stream: a call's launches go
        out together (the library runs without the interpreter's lock, and another thread's launches between them
        would find the same workspace)."""
        if out is None:
            with _on(stream):
                out = torch.empty_like(q)
        raw = _raw_stream(self._index) if stream is None else _stream(stream)
        with self._lock:
            self._decode(q, k, v, q_norm_w, k_norm_w, positions, table, out, stream, raw, pages)
        return out

    def _decode(self, q, k, v, q_norm_w, k_norm_w, positions, table, out, stream, raw, pages) -> None:
        ws = self._streams.get(raw)
        if ws is not None and raw != 0 and _capturing(stream):   # (the default stream is never captured)
            ws = None
        if ws is not None and _fast is not None:
            rc = _fast.decode(self._h, self._spec, q, k, v, q_norm_w, k_norm_w, positions, table, pages, out, ws[0], ws[1],
                              raw)
            if rc is not None and rc != PKV_EWORKSPACE:
                return _check(rc, "pkv_q4_decode")
        _on_device(self._index, q=q, k=k, v=v, q_norm_w=q_norm_w, k_norm_w=k_norm_w, positions=positions, table=table,
                   out=out)
        rows = positions.shape[0]
        qs, ks = (rows, self._heads, self._dim), (rows, self._kv_heads, self._dim)
        if q.shape != qs or out.shape != qs or k.shape != ks or v.shape != ks:
            raise ValueError(f"q and out must be {list(qs)}, k and v {list(ks)}, got {tuple(q.shape)}, "
                             f"{tuple(out.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
        if q_norm_w.numel() != self._dim or k_norm_w.numel() != self._dim:
            raise ValueError(f"q_norm_w and k_norm_w must be [{self._dim}]")
        tp, table_rows, pages = _table(table, rows, pages)
        if table_rows != rows:
            raise ValueError(f"table has {table_rows} rows, positions {rows}")
        args = (self.handle, _dev(q, _BF16, "q"), _dev(k, _BF16, "k"), _dev(v, _BF16, "v"),
                _dev(q_norm_w, _BF16, "q_norm_w"), _dev(k_norm_w, _BF16, "k_norm_w"), _dev(positions, _I32, "positions"),
                tp, rows, pages, _dev(out, _BF16, "out"))
        rc = PKV_EWORKSPACE
        if ws is not None:
            rc = self._lib.pkv_q4_decode(*args, ws[0], ws[1], raw)
        if rc == PKV_EWORKSPACE:   # a first call, more rows than any call on this stream so far, or a capture
            n = pkv_workspace_bytes(self.handle, rows, pages, 0)
            with _on(stream):
                buf = torch.empty(n, dtype=torch.uint8, device=self.device)
            if not _capturing(stream):
                self._streams[raw] = (buf.data_ptr(), n, buf)
            rc = self._lib.pkv_q4_decode(*args, buf.data_ptr(), n, raw)
        if rc:
            raise PkvError(rc, "pkv_q4_decode")
