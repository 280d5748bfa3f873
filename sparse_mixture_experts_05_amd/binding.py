"""ctypes binding of libmoe.so: argument marshalling only.

Tensors are PyTorch device tensors (memory and streams only); every
computation happens in the library's HIP kernels, enqueued on the current
stream. Missing library or non-GPU tensors raise: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
          -3: "MOE_ERR_WORKSPACE", -4: "MOE_ERR_HIP", -5: "MOE_ERR_SCRATCH"}

_vp, _i, _sz, _d = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
_f = ctypes.c_float

SIGNATURES = {
    "moe_route": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "moe_dispatch_workspace_bytes": (_sz, [_i, _i, _i]),
    "moe_dispatch": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_dispatch_capped": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _sz, _vp]),
    "moe_expert_ffn_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "moe_expert_ffn": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp,
                            _vp, _vp, _sz, _vp]),
    "moe_expert_ffn_gather": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i,
                                   _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "moe_expert_ffn_gather_timed": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                                         _i, _i, _i, _vp, _vp, _vp, _sz, _vp, _vp]),
    "moe_combine": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "moe_load_stats": (_i, [_vp, _i, _i, _i, _d, _vp, _vp, _vp, _vp]),
    "moe_bias_update": (_i, [_vp, _i, ctypes.c_float, _vp, _vp, _vp]),
    "moe_capacity": (ctypes.c_int64, [_i, _i, _i, _d]),
    "moe_dispatch_noalloc": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_norm": (_i, [_vp, _vp, _vp, _i, _i, _f, _i, _i, _vp, _vp]),
    "moe_norm_residual": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _f, _i, _vp, _vp, _i, _i, _f, _i,
                               _vp, _vp, _vp]),
    "moe_route_grouped": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp,
                               _vp, _sz, _vp]),
    "moe_route_grouped_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "moe_linear": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "moe_linear_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "moe_linear_grouped": (_i, [_vp, _vp, _i, _i, _vp, _i, _i, _vp, _vp, _i, _vp, _i, _i, _i, _vp,
                                _vp, _sz, _vp]),
    "moe_linear_grouped_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "moe_linear_path": (_i, [_i, _i, _i, _i, _i, _i, _i, _vp]),
    "moe_quantize": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_quantize_weight": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "moe_linear_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "moe_linear_fp8_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "moe_linear_grouped_fp8": (_i, [_vp, _vp, _vp, _i, _i, _vp, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _i,
                                    _vp, _vp, _sz, _vp]),
    "moe_linear_grouped_fp8_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "moe_linear_fp8_path": (_i, [_i, _i, _i, _i, _i, _i, _vp]),
    "moe_layer_few": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                           _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_layer_few_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "moe_status_string": (ctypes.c_char_p, [_i]),
}


class MoELoadStats(ctypes.Structure):
    """Mirror of moe_load_stats_t."""
    _fields_ = [(n, ctypes.c_int64) for n in
                ["num_tokens", "assignments", "capacity", "max_load", "min_load", "dropped",
                 "num_stragglers", "gini_num", "gini_den"]] + \
               [(n, ctypes.c_double) for n in ["load_skew_ratio", "gini", "drop_rate"]]


STATS_BYTES = ctypes.sizeof(MoELoadStats)


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({moe_status_string(status)})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_mixture_experts_05_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


def _dev(t: torch.Tensor | None, name: str, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _want(t, name: str, shape, dtype=None):
    """Shape (and dtype) check of a tensor argument before any pointer reaches
    the library: the kernels index by the sizes passed with the pointers, so a
    mismatched tensor would be read or written out of bounds. None passes."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dims(t, name: str, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    return tuple(t.shape)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise ValueError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def moe_route_workspace_bytes(T: int, H: int, E: int, k: int, dtype_code: int) -> int:
    return lib().moe_route_workspace_bytes(T, H, E, k, dtype_code)


def moe_route(x, wg, bias, k: int, topk_idx=None, topk_w=None, ws=None, stream=None,
              prob_mean=None):
    """Top-k routing: returns (topk_idx int32 [T,k], topk_w fp32 [T,k]).

    prob_mean: optional fp32 [E] device tensor that receives the mean router
    probability of every expert over the T tokens."""
    T, H = _dims(x, "x", 2)
    E = _dims(wg, "wg", 2)[0]
    _want(wg, "wg", (E, H), x.dtype)
    _want(bias, "bias", (E,), torch.float32)
    _want(topk_idx, "topk_idx", (T, k), torch.int32)
    _want(topk_w, "topk_w", (T, k), torch.float32)
    _want(prob_mean, "prob_mean", (E,), torch.float32)
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    dt = _dtype_code(x)
    nbytes = moe_route_workspace_bytes(T, H, E, k, dt)
    if nbytes > 0:
        ws = _workspace(nbytes, x.device, ws)
    ws_ptr = _dev(ws, "ws") if ws is not None else None
    ws_len = ws.numel() if ws is not None else 0
    _check("moe_route", lib().moe_route(
        _dev(x, "x"), _dev(wg, "wg", x.dtype), _dev(bias, "bias", torch.float32), T, H, E, k, dt,
        _dev(topk_idx, "topk_idx", torch.int32), _dev(topk_w, "topk_w", torch.float32),
        _dev(prob_mean, "prob_mean", torch.float32), ws_ptr, ws_len, _stream(stream)))
    return topk_idx, topk_w


def moe_bias_update(counts, bias, gamma: float, load_frac=None, stream=None):
    """Dynamic routing-bias step in place on ``bias`` (fp32 [E]) from the expert
    counts (int32 [E]); writes the load fractions into ``load_frac`` if given.
    Returns load_frac."""
    E = _dims(counts, "counts", 1)[0]
    _want(counts, "counts", (E,), torch.int32)
    _want(bias, "bias", (E,), torch.float32)
    _want(load_frac, "load_frac", (E,), torch.float32)
    _check("moe_bias_update", lib().moe_bias_update(
        _dev(counts, "counts", torch.int32), E, float(gamma), _dev(bias, "bias", torch.float32),
        _dev(load_frac, "load_frac", torch.float32), _stream(stream)))
    return load_frac


def moe_dispatch_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib().moe_dispatch_workspace_bytes(T, E, k)


def moe_expert_ffn_workspace_bytes(rows, T, H, E, F, Fs, dtype_code) -> int:
    return lib().moe_expert_ffn_workspace_bytes(rows, T, H, E, F, Fs, dtype_code)


def _workspace(nbytes: int, device, ws=None):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def moe_capacity(T: int, k: int, E: int, capacity_factor: float) -> int:
    """Expert capacity, computed by the library (moe_capacity)."""
    cap = lib().moe_capacity(int(T), int(k), int(E), float(capacity_factor))
    if cap < 0:
        raise ValueError(f"moe_capacity: invalid arguments T={T} k={k} E={E} "
                         f"capacity_factor={capacity_factor}")
    return int(cap)


def moe_dispatch(topk_idx, x, E: int, out=None, ws=None, stream=None, capacity=None,
                 gather: bool = True):
    """Returns dict(counts, offsets, perm, inv, xs). With ``capacity`` (int >= 0)
    each expert keeps its first ``capacity`` assignments (moe_dispatch_capped).
    With ``gather=False`` no rows are copied and xs is None (for
    moe_expert_ffn_gather); a given ``out`` without "xs" (or xs None) does the same."""
    T, H = _dims(x, "x", 2)
    k = _dims(topk_idx, "topk_idx", 2)[1]
    _want(topk_idx, "topk_idx", (T, k), torch.int32)
    if out is not None:
        _want(out.get("counts"), "counts", (E,), torch.int32)
        _want(out.get("offsets"), "offsets", (E + 1,), torch.int32)
        _want(out.get("perm"), "perm", (T * k,), torch.int32)
        _want(out.get("inv"), "inv", (T * k,), torch.int32)
        _want(out.get("xs"), "xs", (T * k, H), x.dtype)
        for key in ["counts", "offsets", "perm", "inv"]:
            if out.get(key) is None:
                raise ValueError(f"out[{key!r}] is required")
    if capacity is not None and not 0 <= int(capacity) < 2 ** 31:
        raise ValueError(f"capacity {capacity} outside [0, 2^31)")
    dev = x.device
    if out is None:
        out = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm=torch.empty(T * k, dtype=torch.int32, device=dev),
                   inv=torch.empty(T * k, dtype=torch.int32, device=dev),
                   xs=torch.empty((T * k, H), dtype=x.dtype, device=dev) if gather else None)
    xs = out.get("xs")
    nbytes = moe_dispatch_workspace_bytes(T, E, k)
    ws = _workspace(nbytes, dev, ws)
    tail = (_dtype_code(x),
            _dev(out["counts"], "counts", torch.int32), _dev(out["offsets"], "offsets", torch.int32),
            _dev(out["perm"], "perm", torch.int32), _dev(out["inv"], "inv", torch.int32),
            _dev(xs, "xs", x.dtype), _dev(ws, "ws"), ws.numel(), _stream(stream))
    if capacity is None:
        _check("moe_dispatch", lib().moe_dispatch(
            _dev(topk_idx, "topk_idx", torch.int32), _dev(x, "x"), T, H, E, k, *tail))
    else:
        _check("moe_dispatch_capped", lib().moe_dispatch_capped(
            _dev(topk_idx, "topk_idx", torch.int32), _dev(x, "x"), T, H, E, k, int(capacity),
            *tail))
    return out


def moe_dispatch_noalloc(topk_idx, x, E: int, out=None, stream=None, gather: bool = True):
    """moe_dispatch on the library's fixed device scratch (no workspace): for
    callers that cannot allocate device memory. The same dict as moe_dispatch;
    ``out`` (preallocated outputs) avoids every allocation here too."""
    T, H = _dims(x, "x", 2)
    k = _dims(topk_idx, "topk_idx", 2)[1]
    _want(topk_idx, "topk_idx", (T, k), torch.int32)
    if out is not None:
        _want(out.get("counts"), "counts", (E,), torch.int32)
        _want(out.get("offsets"), "offsets", (E + 1,), torch.int32)
        _want(out.get("perm"), "perm", (T * k,), torch.int32)
        _want(out.get("inv"), "inv", (T * k,), torch.int32)
        _want(out.get("xs"), "xs", (T * k, H), x.dtype)
        for key in ["counts", "offsets", "perm", "inv"]:
            if out.get(key) is None:
                raise ValueError(f"out[{key!r}] is required")
    dev = x.device
    if out is None:
        out = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm=torch.empty(T * k, dtype=torch.int32, device=dev),
                   inv=torch.empty(T * k, dtype=torch.int32, device=dev),
                   xs=torch.empty((T * k, H), dtype=x.dtype, device=dev) if gather else None)
    _check("moe_dispatch_noalloc", lib().moe_dispatch_noalloc(
        _dev(topk_idx, "topk_idx", torch.int32), _dev(x, "x"), T, H, E, k, _dtype_code(x),
        _dev(out["counts"], "counts", torch.int32), _dev(out["offsets"], "offsets", torch.int32),
        _dev(out["perm"], "perm", torch.int32), _dev(out["inv"], "inv", torch.int32),
        _dev(out.get("xs"), "xs", x.dtype), _stream(stream)))
    return out


def moe_expert_ffn(xs, offsets, w1, w2, x=None, ws1=None, ws2=None, T=None, ys=None, ysh=None,
                   ws=None, stream=None):
    """Returns (ys [rows,H], ysh [T,H] or None)."""
    rows, H = _dims(xs, "xs", 2)
    E, F, _ = _dims(w1, "w1", 3)
    Fs = 0 if ws1 is None else _dims(ws1, "ws1", 2)[0]
    if T is None:
        T = x.shape[0] if x is not None else rows
    _want(offsets, "offsets", (E + 1,), torch.int32)
    _want(w1, "w1", (E, F, H), xs.dtype)
    _want(w2, "w2", (E, H, F), xs.dtype)
    _want(x, "x", (T, H), xs.dtype)
    if Fs > 0:
        if x is None or ws2 is None:
            raise ValueError("the shared expert needs x, ws1 and ws2")
        _want(ws1, "ws1", (Fs, H), xs.dtype)
        _want(ws2, "ws2", (H, Fs), xs.dtype)
        _want(ysh, "ysh", (T, H), xs.dtype)
    _want(ys, "ys", (rows, H), xs.dtype)
    dt = _dtype_code(xs)
    dev = xs.device
    if ys is None:
        ys = torch.empty((rows, H), dtype=xs.dtype, device=dev)
    if Fs > 0 and ysh is None:
        ysh = torch.empty((T, H), dtype=xs.dtype, device=dev)
    nbytes = moe_expert_ffn_workspace_bytes(rows, T, H, E, F, Fs, dt)
    ws = _workspace(nbytes, dev, ws)
    _check("moe_expert_ffn", lib().moe_expert_ffn(
        _dev(xs, "xs"), _dev(offsets, "offsets", torch.int32), rows, E, H, F,
        _dev(w1, "w1", xs.dtype), _dev(w2, "w2", xs.dtype), _dev(x, "x", xs.dtype),
        _dev(ws1, "ws1", xs.dtype), _dev(ws2, "ws2", xs.dtype), T, Fs, dt, _dev(ys, "ys", xs.dtype),
        _dev(ysh, "ysh", xs.dtype) if Fs > 0 else None, _dev(ws, "ws"), ws.numel(),
        _stream(stream)))
    return ys, (ysh if Fs > 0 else None)


def moe_expert_ffn_gather(x, perm, k: int, offsets, w1, w2, ws1=None, ws2=None, rows=None,
                          ys=None, ysh=None, ws=None, stream=None, gemm_events=None):
    """moe_expert_ffn reading routed row p from x[perm[p] // k] (no xs copy).
    Returns (ys [rows,H], ysh [T,H] or None); rows defaults to T*k.
    gemm_events: four torch.cuda.Event (timing enabled) that the library
    records right before and after the up and the down GEMM launches
    (moe_expert_ffn_gather_timed), or None."""
    T, H = _dims(x, "x", 2)
    E, F, _ = _dims(w1, "w1", 3)
    Fs = 0 if ws1 is None else _dims(ws1, "ws1", 2)[0]
    rows = T * k if rows is None else rows
    if not 1 <= rows <= T * k:
        raise ValueError(f"rows {rows} outside [1, T*k = {T * k}]")
    if _dims(perm, "perm", 1)[0] < rows or perm.dtype != torch.int32:
        raise ValueError(f"perm must be int32 with at least rows = {rows} entries")
    _want(offsets, "offsets", (E + 1,), torch.int32)
    _want(w1, "w1", (E, F, H), x.dtype)
    _want(w2, "w2", (E, H, F), x.dtype)
    if Fs > 0:
        if ws2 is None:
            raise ValueError("the shared expert needs ws1 and ws2")
        _want(ws1, "ws1", (Fs, H), x.dtype)
        _want(ws2, "ws2", (H, Fs), x.dtype)
        _want(ysh, "ysh", (T, H), x.dtype)
    _want(ys, "ys", (rows, H), x.dtype)
    dt = _dtype_code(x)
    dev = x.device
    if ys is None:
        ys = torch.empty((rows, H), dtype=x.dtype, device=dev)
    if Fs > 0 and ysh is None:
        ysh = torch.empty((T, H), dtype=x.dtype, device=dev)
    nbytes = moe_expert_ffn_workspace_bytes(rows, T, H, E, F, Fs, dt)
    ws = _workspace(nbytes, dev, ws)
    args = (_dev(x, "x"), _dev(perm, "perm", torch.int32), k, _dev(offsets, "offsets", torch.int32),
            rows, E, H, F, _dev(w1, "w1", x.dtype), _dev(w2, "w2", x.dtype),
            _dev(ws1, "ws1", x.dtype), _dev(ws2, "ws2", x.dtype), T, Fs, dt, _dev(ys, "ys", x.dtype),
            _dev(ysh, "ysh", x.dtype) if Fs > 0 else None, _dev(ws, "ws"), ws.numel(),
            _stream(stream))
    if gemm_events is None:
        _check("moe_expert_ffn_gather", lib().moe_expert_ffn_gather(*args))
    else:
        if len(gemm_events) != 4:
            raise ValueError("gemm_events takes four events (up before / after, down before / after)")
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        handles = (ctypes.c_void_p * 4)()
        for i, ev in enumerate(gemm_events):
            if not ev.cuda_event:
                ev.record(s)  # torch creates the HIP event on its first record
            handles[i] = ev.cuda_event
        _check("moe_expert_ffn_gather_timed", lib().moe_expert_ffn_gather_timed(*args, handles))
    return ys, (ysh if Fs > 0 else None)


def moe_combine(ys, inv, topk_w, ysh=None, out=None, stream=None):
    """Returns out [T,H]."""
    T, k = _dims(topk_w, "topk_w", 2)
    H = _dims(ys, "ys", 2)[1]
    _want(topk_w, "topk_w", (T, k), torch.float32)
    _want(ys, "ys", (T * k, H))
    _want(inv, "inv", (T * k,), torch.int32)
    _want(ysh, "ysh", (T, H), ys.dtype)
    _want(out, "out", (T, H), ys.dtype)
    if out is None:
        out = torch.empty((T, H), dtype=ys.dtype, device=ys.device)
    _check("moe_combine", lib().moe_combine(
        _dev(ys, "ys"), _dev(inv, "inv", torch.int32), _dev(topk_w, "topk_w", torch.float32),
        _dev(ysh, "ysh", ys.dtype), T, H, k, _dtype_code(ys), _dev(out, "out", ys.dtype),
        _stream(stream)))
    return out


def moe_load_stats(counts, T: int, k: int, capacity_factor: float, stats=None, overflow=None,
                   straggler_ids=None, stream=None, read_back: bool = True):
    """Enqueue the diagnostics; with read_back, synchronise and return a dict."""
    E = _dims(counts, "counts", 1)[0]
    _want(counts, "counts", (E,), torch.int32)
    if stats is not None and stats.numel() * stats.element_size() < STATS_BYTES:
        raise ValueError(f"stats must hold at least {STATS_BYTES} bytes")
    _want(overflow, "overflow", (E,), torch.int32)
    _want(straggler_ids, "straggler_ids", (E,), torch.int32)
    dev = counts.device
    if stats is None:
        stats = torch.empty(STATS_BYTES, dtype=torch.uint8, device=dev)
    if overflow is None:
        overflow = torch.empty(E, dtype=torch.int32, device=dev)
    if straggler_ids is None:
        straggler_ids = torch.empty(E, dtype=torch.int32, device=dev)
    _check("moe_load_stats", lib().moe_load_stats(
        _dev(counts, "counts", torch.int32), T, E, k, float(capacity_factor), _dev(stats, "stats"),
        _dev(overflow, "overflow", torch.int32), _dev(straggler_ids, "straggler_ids", torch.int32),
        _stream(stream)))
    if not read_back:
        return dict(stats=stats, overflow=overflow, straggler_ids=straggler_ids)
    return read_stats(stats, overflow, straggler_ids)


def read_stats(stats, overflow, straggler_ids) -> dict:
    """Synchronising copy of moe_load_stats' device outputs into a dict (the
    struct fields, overflow, the straggler ids and the -1 padding after them)."""
    raw = MoELoadStats.from_buffer_copy(bytes(stats.cpu().numpy().tobytes()[:STATS_BYTES]))
    d = {name: getattr(raw, name) for name, _ in MoELoadStats._fields_}
    d["overflow"] = overflow.cpu().tolist()
    ids = straggler_ids.cpu().tolist()
    d["straggler_ids"] = ids[: d["num_stragglers"]]
    d["straggler_tail"] = ids[d["num_stragglers"]:]
    return d


def moe_layer_forward(x, wg, bias, w1, w2, k: int, ws1=None, ws2=None, stream=None,
                      prob_mean=None, capacity=None, fused_gather: bool = True):
    """All five steps on one stream (no host synchronisation). Returns a dict.
    prob_mean (optional fp32 [E]) receives the mean router probabilities;
    capacity (optional int) drops each expert's assignments past it.
    fused_gather (default): dispatch copies no rows and the FFN reads x through
    perm (moe_expert_ffn_gather; xs is None); otherwise dispatch writes xs and
    moe_expert_ffn reads it. Both give bit-identical outputs."""
    E = wg.shape[0]
    idx, w = moe_route(x, wg, bias, k, stream=stream, prob_mean=prob_mean)
    d = moe_dispatch(idx, x, E, stream=stream, capacity=capacity, gather=not fused_gather)
    if fused_gather:
        ys, ysh = moe_expert_ffn_gather(x, d["perm"], k, d["offsets"], w1, w2, ws1=ws1, ws2=ws2,
                                        stream=stream)
    else:
        ys, ysh = moe_expert_ffn(d["xs"], d["offsets"], w1, w2, x=x, ws1=ws1, ws2=ws2,
                                 T=x.shape[0], stream=stream)
    out = moe_combine(ys, d["inv"], w, ysh, stream=stream)
    return dict(topk_idx=idx, topk_w=w, ys=ys, ysh=ysh, out=out, **d)


class MoELayerGraph:
    """The five calls captured once into a HIP graph (torch.cuda.CUDAGraph on ROCm)
    and replayed: one graph launch instead of ~10 kernel launches per layer,
    the decode-latency use of graph replay the lpqz.cn MoE blog describes (its
    section 4.3, graph capture of the per-token MoE inference).

    All buffers are allocated once here; ``run(x)`` copies x into the static
    input buffer and replays. The library never allocates, synchronises or
    clears memory with memset, so its launches are capture-safe.

    With ``drop``, dispatch enforces the expert capacity int(T*k/E*cf)
    (moe_dispatch_capped). With ``bias_gamma`` set (and a bias tensor given),
    every replay also ends
    with the dynamic-bias step on ``bias`` in place and writes the mean router
    probabilities ``prob_mean`` and load fractions ``load_frac``: the next
    replay routes with the updated bias.
    """

    def __init__(self, wg, bias, w1, w2, k: int, T: int, ws1=None, ws2=None,
                 capacity_factor: float = 1.25, bias_gamma: float | None = None,
                 drop: bool = False):
        E, H = wg.shape
        F = w1.shape[1]
        Fs = 0 if ws1 is None else ws1.shape[0]
        dev, dtype = wg.device, wg.dtype
        dt = _dtype_code(wg)
        self.k, self.T, self.cf = k, T, capacity_factor
        self.cap = moe_capacity(T, k, E, capacity_factor) if drop else None
        self.wg, self.bias, self.w1, self.w2, self.ws1, self.ws2 = wg, bias, w1, w2, ws1, ws2
        self.x = torch.zeros((T, H), dtype=dtype, device=dev)
        self.idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.dsp = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
                        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                        perm=torch.empty(T * k, dtype=torch.int32, device=dev),
                        inv=torch.empty(T * k, dtype=torch.int32, device=dev),
                        xs=None)  # the FFN reads x through perm
        self.ws_r = torch.empty(max(1, moe_route_workspace_bytes(T, H, E, k, dt)),
                                dtype=torch.uint8, device=dev)
        self.ws_d = torch.empty(max(1, moe_dispatch_workspace_bytes(T, E, k)), dtype=torch.uint8,
                                device=dev)
        self.ws_f = torch.empty(max(1, moe_expert_ffn_workspace_bytes(T * k, T, H, E, F, Fs, dt)),
                                dtype=torch.uint8, device=dev)
        self.ys = torch.empty((T * k, H), dtype=dtype, device=dev)
        self.ysh = torch.empty((T, H), dtype=dtype, device=dev) if Fs else None
        self.out = torch.empty((T, H), dtype=dtype, device=dev)
        self.stats = torch.empty(STATS_BYTES, dtype=torch.uint8, device=dev)
        self.overflow = torch.empty(E, dtype=torch.int32, device=dev)
        self.stragglers = torch.empty(E, dtype=torch.int32, device=dev)
        if bias_gamma is not None and bias is None:
            raise ValueError("bias_gamma needs a bias tensor to update")
        self.gamma = bias_gamma
        self.prob_mean = torch.empty(E, dtype=torch.float32, device=dev) if bias_gamma is not None else None
        self.load_frac = torch.empty(E, dtype=torch.float32, device=dev) if bias_gamma is not None else None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        saved = None if bias is None else bias.clone()
        with torch.cuda.stream(side):
            self._layer()  # one eager pass on a side stream before capture
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._layer()
        torch.cuda.synchronize()
        if saved is not None:
            bias.copy_(saved)  # the warm-up pass must not have moved the bias
            torch.cuda.synchronize()

    def _layer(self):
        moe_route(self.x, self.wg, self.bias, self.k, topk_idx=self.idx, topk_w=self.w,
                  ws=self.ws_r, prob_mean=self.prob_mean)
        moe_dispatch(self.idx, self.x, self.wg.shape[0], out=self.dsp, ws=self.ws_d,
                     capacity=self.cap)
        moe_expert_ffn_gather(self.x, self.dsp["perm"], self.k, self.dsp["offsets"], self.w1,
                              self.w2, ws1=self.ws1, ws2=self.ws2, ys=self.ys, ysh=self.ysh,
                              ws=self.ws_f)
        moe_combine(self.ys, self.dsp["inv"], self.w, self.ysh, out=self.out)
        moe_load_stats(self.dsp["counts"], self.T, self.k, self.cf, stats=self.stats,
                       overflow=self.overflow, straggler_ids=self.stragglers, read_back=False)
        if self.gamma is not None:
            moe_bias_update(self.dsp["counts"], self.bias, self.gamma, load_frac=self.load_frac)

    def run(self, x):
        """Copy x into the static input and replay; returns the static output tensor."""
        self.x.copy_(x)
        self.graph.replay()
        return self.out


# ---------------------------------------------------------------- around the layer
#
# Forward only, like the layer: no gradients flow through these calls. A call runs on
# the given stream, or the current stream of the tensors' device; outputs and
# workspaces that it allocates belong to that stream. Tensors made on another stream
# are the caller's to order.

# Handle of a device's current stream, and the current device. The public
# torch.cuda.current_stream() builds a Stream object, 2.8 us of a call that takes 7;
# torch's own generated code takes these.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
SCORES = {"softmax": 0, "sigmoid": 1}
ACTS = {"none": 0, "gelu": 1, "silu": 2, "geglu": 3, "swiglu": 4}
GATED_ACTS = ("geglu", "swiglu")


def _enum(table, value, name: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}")
    return code


def _shape(t, name: str, ndim: int):
    if isinstance(t, torch.Tensor) and t.dim() == ndim:
        return t.shape
    return _dims(t, name, ndim)  # raises


def _ptr(t, name: str, shape, dtype, device):
    """Address of a tensor argument after its checks: shape, type, the device of
    the call's first tensor, and contiguity. None passes."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _given(t, name: str):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _fits(*sizes):
    """Refuses sizes that a C int does not hold: ctypes would pass their low 32 bits."""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"sizes must fit 32 bits, got {max(sizes, key=abs)}")


def _ws(nbytes: int, device, ws):
    """(address, bytes) of the workspace: the caller's, or a new one."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        have = ws.numel() * ws.element_size()
        if have < nbytes:
            raise ValueError(f"workspace too small: {have} bytes, needs {nbytes}")
        if ws.device != device or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _other_stream(device, stream):
    """The stream a call has to switch to before it allocates and launches (the
    given one, or the current one of the tensors' device when that is not the
    current device), or None."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be GPU tensors, got {device}")
    if stream is None:
        return None if device.index == _current_device() else torch.cuda.current_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return None if stream == torch.cuda.current_stream() else stream


def moe_norm(x, weight=None, bias=None, eps: float = 1e-6, kind: str = "rms", out=None,
             stream=None):
    """Norm of every row of x [T,H]: "rms" or "layer", times weight, plus bias.

    bf16 or fp32, any H up to 16384; ``out`` may be x itself. Returns out."""
    T, H = _shape(x, "x", 2)
    _fits(T, H)
    dev, dtype = x.device, x.dtype
    dt, code = _dtype_code(x), _enum(NORM_KINDS, kind, "kind")
    xp = _ptr(x, "x", (T, H), dtype, dev)
    wp, bp = _ptr(weight, "weight", (H,), dtype, dev), _ptr(bias, "bias", (H,), dtype, dev)
    op = _ptr(out, "out", (T, H), dtype, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_norm(x, weight, bias, eps, kind, out)
    if out is None:
        out = torch.empty_like(x)
        op = out.data_ptr()
    _check("moe_norm", lib().moe_norm(xp, wp, bp, T, H, eps, code, dt, op,
                                      _raw_stream(dev.index)))
    return out


def moe_norm_residual(y, res, weight=None, bias=None, gate=None, scale: float = 1.0,
                      eps: float = 1e-6, kind: str = "rms", next_weight=None, next_bias=None,
                      next_kind: str = "none", res_out=None, next_out=None, stream=None):
    """h = res + scale * gate * norm(y), and the next block's norm of h, in one pass.

    y, res [T,H]; kind / next_kind "none", "rms" or "layer"; gate None, [T,1]
    (one value a row), [H] or [T,H]. Returns (h, norm of h or None). res_out may
    be res itself, next_out y itself."""
    T, H = _shape(y, "y", 2)
    _fits(T, H)
    dev, dtype, row = y.device, y.dtype, (H,)
    dt = _dtype_code(y)
    code, ncode = _enum(NORM_KINDS, kind, "kind"), _enum(NORM_KINDS, next_kind, "next_kind")
    if gate is None:
        mode, gshape = 0, None
    else:
        gshape = tuple(gate.shape) if isinstance(gate, torch.Tensor) else ()
        if gshape == (T, H):
            mode = 3
        elif gshape == (H,):
            mode = 2
        elif gshape == (T, 1):
            mode = 1
        else:
            raise ValueError(f"gate must have shape {(T, 1)}, {(H,)} or {(T, H)}, got {gshape}")
    if next_out is not None and ncode == 0:
        raise ValueError("next_out needs a next_kind")
    args = [_ptr(y, "y", (T, H), dtype, dev), code, _ptr(weight, "weight", row, dtype, dev),
            _ptr(bias, "bias", row, dtype, dev), _ptr(res, "res", (T, H), dtype, dev),
            _ptr(gate, "gate", gshape, dtype, dev), mode, scale, ncode,
            _ptr(next_weight, "next_weight", row, dtype, dev),
            _ptr(next_bias, "next_bias", row, dtype, dev)]
    rp = _ptr(res_out, "res_out", (T, H), dtype, dev)
    np_ = _ptr(next_out, "next_out", (T, H), dtype, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_norm_residual(y, res, weight, bias, gate, scale, eps, kind, next_weight,
                                     next_bias, next_kind, res_out, next_out)
    if res_out is None:
        res_out = torch.empty_like(y)
        rp = res_out.data_ptr()
    if next_out is None and ncode != 0:
        next_out = torch.empty_like(y)
        np_ = next_out.data_ptr()
    _check("moe_norm_residual", lib().moe_norm_residual(
        *args, T, H, eps, dt, rp, np_, _raw_stream(dev.index)))
    return res_out, next_out


def moe_route_grouped_workspace_bytes(T: int, H: int, E: int, k: int, dtype_code: int) -> int:
    _fits(T, H, E, k)
    return lib().moe_route_grouped_workspace_bytes(T, H, E, k, dtype_code)


def moe_route_grouped(x, wg, bias, k: int, score: str = "sigmoid", groups: int = 1,
                      topk_groups: int = 1, group_top: int = 2, renorm: bool = True,
                      scale: float = 1.0, topk_idx=None, topk_w=None, ws=None, stream=None):
    """Top-k routing with sigmoid or softmax scores, a bias (fp32 [E] or None) that
    moves the choice only, and the choice limited to the topk_groups best of
    ``groups`` groups of experts (by their ``group_top`` largest biased scores).
    Returns (topk_idx int32 [T,k], topk_w fp32 [T,k])."""
    T, H = _shape(x, "x", 2)
    E = _shape(wg, "wg", 2)[0]
    _fits(T, H, E, k, groups, topk_groups, group_top)
    dev, dtype = x.device, x.dtype
    dt, code = _dtype_code(x), _enum(SCORES, score, "score")
    xp, wp = _ptr(x, "x", (T, H), dtype, dev), _ptr(wg, "wg", (E, H), dtype, dev)
    bp = _ptr(bias, "bias", (E,), torch.float32, dev)
    ip = _ptr(topk_idx, "topk_idx", (T, k), torch.int32, dev)
    op = _ptr(topk_w, "topk_w", (T, k), torch.float32, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_route_grouped(x, wg, bias, k, score, groups, topk_groups, group_top, renorm,
                                     scale, topk_idx, topk_w, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_route_grouped_workspace_bytes(T, H, E, k, dt), dev, ws)
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        ip = topk_idx.data_ptr()
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        op = topk_w.data_ptr()
    _check("moe_route_grouped", L.moe_route_grouped(
        xp, wp, bp, T, H, E, k, code, groups, topk_groups, group_top, int(renorm), scale, dt, ip, op,
        wsp, wsn, _raw_stream(dev.index)))
    return topk_idx, topk_w


def moe_linear_workspace_bytes(M: int, N: int, K: int, act: str, dtype_code: int) -> int:
    _fits(M, N, K)
    return lib().moe_linear_workspace_bytes(M, N, K, _enum(ACTS, act, "act"), dtype_code)


def moe_linear(x, w, bias=None, act: str = "none", residual=None, y=None, ws=None, stream=None):
    """y = act(x . w^T + bias) + residual, everything after the product in fp32.

    x [M,K], w [N,K], bias [N], residual and y [M,N], all of one type (bf16 or
    fp32); act "none", "gelu" (erf) or "silu". Gated: act "geglu" or "swiglu"
    with w [2,N,K] and bias [2,N], y = act(gate half) * other half + residual.
    y may be residual itself. Returns y."""
    M, K = _shape(x, "x", 2)
    code = _enum(ACTS, act, "act")
    two = (2,) if code >= 3 else ()
    N = _shape(w, "w", 2 + len(two))[-2]
    _fits(M, N, K)
    dev, dtype = x.device, x.dtype
    dt = _dtype_code(x)
    xp, wp = _ptr(x, "x", (M, K), dtype, dev), _ptr(w, "w", (*two, N, K), dtype, dev)
    bp = _ptr(bias, "bias", (*two, N), dtype, dev)
    rp, yp = _ptr(residual, "residual", (M, N), dtype, dev), _ptr(y, "y", (M, N), dtype, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_linear(x, w, bias, act, residual, y, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_linear_workspace_bytes(M, N, K, code, dt), dev, ws)
    if y is None:
        y = x.new_empty((M, N))
        yp = y.data_ptr()
    _check("moe_linear", L.moe_linear(xp, wp, bp, code, rp, M, N, K, dt, yp, wsp, wsn,
                                      _raw_stream(dev.index)))
    return y


def moe_linear_grouped_workspace_bytes(E: int, rows: int, N: int, K: int, act: str,
                                       dtype_code: int) -> int:
    _fits(E, rows, N, K)
    return lib().moe_linear_grouped_workspace_bytes(E, rows, N, K, _enum(ACTS, act, "act"),
                                                    dtype_code)


LINEAR_PATHS = ("rows", "tiles", "256x128", "256x256")


def moe_linear_path(M: int, N: int, K: int, act: str, dtype_code: int, E: int | None = None):
    """(kernels, K slices) of a product of M rows, or with E of a grouped product of M
    buffer rows: "rows", "tiles", "256x128" or "256x256", and the slices of K (0 where
    the offsets decide). A host query; raises MoEError for sizes that are refused."""
    _fits(M, N, K, E or 1)
    n = ctypes.c_int(0)
    path = lib().moe_linear_path(1 if E is None else E, M, N, K, _enum(ACTS, act, "act"),
                                 int(E is not None), dtype_code, ctypes.byref(n))
    if path < 0:
        _check("moe_linear_path", path)
    return LINEAR_PATHS[path], n.value


def moe_linear_grouped(x, offsets, w, bias=None, act: str = "none", residual=None, perm=None,
                       k: int = 1, rows=None, y=None, ws=None, stream=None):
    """moe_linear over the experts' segments: buffer row p in [offsets[e],
    offsets[e+1]) takes w[e] and bias[e] (offsets int32 [E+1] from moe_dispatch).

    w [E,N,K] (gated: [E,2,N,K]), bias [E,N] ([E,2,N]). Without perm, x is the
    buffer [rows,K]; with perm (int32, from moe_dispatch of k experts a token) x is
    the token rows [T,K] and row p reads x[perm[p] // k]. rows (default: all of the
    buffer, T*k with perm) is an upper bound of offsets[E]; rows of y past
    offsets[E] are left as they were. Returns y [rows,N]."""
    T, K = _shape(x, "x", 2)
    code = _enum(ACTS, act, "act")
    two = (2,) if code >= 3 else ()
    dims = _shape(w, "w", 3 + len(two))
    E, N = dims[0], dims[-2]
    dev, dtype = x.device, x.dtype
    dt = _dtype_code(x)
    most = T if perm is None else T * k
    if rows is None:
        rows = most
    _fits(T, K, E, N, k, rows)
    if not 1 <= rows <= most:
        raise ValueError(f"rows {rows} outside [1, {most}]")
    if perm is not None and _shape(perm, "perm", 1)[0] < rows:
        raise ValueError(f"perm must have at least rows = {rows} entries")
    xp, wp = _ptr(x, "x", (T, K), dtype, dev), _ptr(w, "w", (E, *two, N, K), dtype, dev)
    fp = _ptr(offsets, "offsets", (E + 1,), torch.int32, dev)
    pp = None if perm is None else _ptr(perm, "perm", perm.shape, torch.int32, dev)
    bp = _ptr(bias, "bias", (E, *two, N), dtype, dev)
    rp, yp = _ptr(residual, "residual", (rows, N), dtype, dev), _ptr(y, "y", (rows, N), dtype, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_linear_grouped(x, offsets, w, bias, act, residual, perm, k, rows, y, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_linear_grouped_workspace_bytes(E, rows, N, K, code, dt), dev, ws)
    if y is None:
        y = x.new_empty((rows, N))
        yp = y.data_ptr()
    _check("moe_linear_grouped", L.moe_linear_grouped(
        xp, pp, k, T, fp, E, rows, wp, bp, code, rp, N, K, dt, yp, wsp, wsn,
        _raw_stream(dev.index)))
    return y


FP8 = torch.float8_e4m3fn  # 8-bit operands: 4 bits of exponent, 3 of mantissa, no infinities
FP8_BLOCK = 128            # elements of a scale block


def moe_quantize(x, q=None, scale=None, stream=None):
    """Rows x [rows,K] (bf16 or fp32) as float8_e4m3fn with one scale for each block of
    128 elements: x = q * scale. The scales are powers of two (one rounding), the least
    with |q| <= 448. K a multiple of 128. Returns (q [rows,K], scale fp32 [K/128,rows])."""
    rows, K = _shape(x, "x", 2)
    _fits(rows, K)
    dev, dtype = x.device, x.dtype
    dt = _dtype_code(x)
    sshape = (K // FP8_BLOCK, rows)
    xp = _ptr(x, "x", (rows, K), dtype, dev)
    qp = _ptr(q, "q", (rows, K), FP8, dev)
    sp = _ptr(scale, "scale", sshape, torch.float32, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_quantize(x, q, scale)
    if q is None:
        q = torch.empty((rows, K), dtype=FP8, device=dev)
        qp = q.data_ptr()
    if scale is None:
        scale = torch.empty(sshape, dtype=torch.float32, device=dev)
        sp = scale.data_ptr()
    _check("moe_quantize", lib().moe_quantize(xp, rows, K, dt, qp, sp, _raw_stream(dev.index)))
    return q, scale


def moe_quantize_weight(w, q=None, scale=None, stream=None):
    """Weights w [...,N,K] (bf16 or fp32) as float8_e4m3fn with one scale for each block of
    128 x 128. N a multiple of 64, K of 128. Returns (q [...,N,K], scale fp32
    [...,ceil(N/128),K/128])."""
    if not isinstance(w, torch.Tensor) or w.dim() < 2:
        raise ValueError("w must be a torch tensor of two dimensions or more")
    *lead, N, K = w.shape
    count = 1
    for n in lead:
        count *= n
    _fits(count, N, K)
    dev, dtype = w.device, w.dtype
    dt = _dtype_code(w)
    sshape = (*lead, -(-N // FP8_BLOCK), K // FP8_BLOCK)
    wp = _ptr(w, "w", w.shape, dtype, dev)
    qp = _ptr(q, "q", w.shape, FP8, dev)
    sp = _ptr(scale, "scale", sshape, torch.float32, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_quantize_weight(w, q, scale)
    if q is None:
        q = torch.empty(w.shape, dtype=FP8, device=dev)
        qp = q.data_ptr()
    if scale is None:
        scale = torch.empty(sshape, dtype=torch.float32, device=dev)
        sp = scale.data_ptr()
    _check("moe_quantize_weight", lib().moe_quantize_weight(wp, count, N, K, dt, qp, sp,
                                                            _raw_stream(dev.index)))
    return q, scale


def moe_linear_fp8_workspace_bytes(M: int, N: int, K: int, act: str) -> int:
    _fits(M, N, K)
    return lib().moe_linear_fp8_workspace_bytes(M, N, K, _enum(ACTS, act, "act"))


def moe_linear_fp8(x, x_scale, w, w_scale, bias=None, act: str = "none", residual=None, y=None,
                   ws=None, stream=None):
    """moe_linear of 8-bit operands with block scales; y in bf16.

    x [M,K] float8_e4m3fn with x_scale fp32 [K/128,M] (moe_quantize), w [N,K] (gated:
    [2,N,K]) with w_scale fp32 [ceil(N/128),K/128] ([2,...]; moe_quantize_weight, or
    a checkpoint's scales of any mantissa; a block's x_scale * w_scale has to stay within
    fp32); bias, residual and y bf16. K a multiple of 128, N of 64. y may be residual
    itself. Returns y."""
    M, K = _shape(x, "x", 2)
    code = _enum(ACTS, act, "act")
    two = (2,) if code >= 3 else ()
    N = _shape(w, "w", 2 + len(two))[-2]
    _fits(M, N, K)
    dev, bf16 = x.device, torch.bfloat16
    nkb, nnb = K // FP8_BLOCK, -(-N // FP8_BLOCK)
    xp, wp = _ptr(x, "x", (M, K), FP8, dev), _ptr(w, "w", (*two, N, K), FP8, dev)
    xsp = _ptr(_given(x_scale, "x_scale"), "x_scale", (nkb, M), torch.float32, dev)
    wsc = _ptr(_given(w_scale, "w_scale"), "w_scale", (*two, nnb, nkb), torch.float32, dev)
    bp = _ptr(bias, "bias", (*two, N), bf16, dev)
    rp, yp = _ptr(residual, "residual", (M, N), bf16, dev), _ptr(y, "y", (M, N), bf16, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_linear_fp8(x, x_scale, w, w_scale, bias, act, residual, y, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_linear_fp8_workspace_bytes(M, N, K, code), dev, ws)
    if y is None:
        y = torch.empty((M, N), dtype=bf16, device=dev)
        yp = y.data_ptr()
    _check("moe_linear_fp8", L.moe_linear_fp8(xp, xsp, wp, wsc, bp, code, rp, M, N, K, yp, wsp, wsn,
                                              _raw_stream(dev.index)))
    return y


def moe_linear_grouped_fp8_workspace_bytes(E: int, rows: int, N: int, K: int, act: str) -> int:
    _fits(E, rows, N, K)
    return lib().moe_linear_grouped_fp8_workspace_bytes(E, rows, N, K, _enum(ACTS, act, "act"))


FP8_PATHS = ("rows", "64x64", "128x128", "256x256")


def moe_linear_fp8_path(M: int, N: int, K: int, act: str, E: int | None = None):
    """(kernels, K slices) of an 8-bit product, as moe_linear_path: "rows", "64x64",
    "128x128" or "256x256"."""
    _fits(M, N, K, E or 1)
    n = ctypes.c_int(0)
    path = lib().moe_linear_fp8_path(1 if E is None else E, M, N, K, _enum(ACTS, act, "act"),
                                     int(E is not None), ctypes.byref(n))
    if path < 0:
        _check("moe_linear_fp8_path", path)
    return FP8_PATHS[path], n.value


def moe_linear_grouped_fp8(x, x_scale, offsets, w, w_scale, bias=None, act: str = "none",
                           residual=None, perm=None, k: int = 1, rows=None, y=None, ws=None,
                           stream=None):
    """moe_linear_fp8 over the experts' segments, as moe_linear_grouped.

    w [E,N,K] (gated: [E,2,N,K]) with w_scale [E,ceil(N/128),K/128] ([E,2,...]). Without
    perm, x is the buffer [rows,K] with x_scale [K/128,rows]; with perm x is the token
    rows [T,K] with x_scale [K/128,T], and row p reads row perm[p] // k. Returns y
    [rows,N] in bf16; its rows past offsets[E] are left as they were."""
    T, K = _shape(x, "x", 2)
    code = _enum(ACTS, act, "act")
    two = (2,) if code >= 3 else ()
    dims = _shape(w, "w", 3 + len(two))
    E, N = dims[0], dims[-2]
    dev, bf16 = x.device, torch.bfloat16
    most = T if perm is None else T * k
    if rows is None:
        rows = most
    _fits(T, K, E, N, k, rows)
    if not 1 <= rows <= most:
        raise ValueError(f"rows {rows} outside [1, {most}]")
    if perm is not None and _shape(perm, "perm", 1)[0] < rows:
        raise ValueError(f"perm must have at least rows = {rows} entries")
    if perm is None and rows != T:
        raise ValueError(f"rows {rows} without perm must be x's {T} (x_scale has that many columns)")
    nkb, nnb = K // FP8_BLOCK, -(-N // FP8_BLOCK)
    xp, wp = _ptr(x, "x", (T, K), FP8, dev), _ptr(w, "w", (E, *two, N, K), FP8, dev)
    xsp = _ptr(_given(x_scale, "x_scale"), "x_scale", (nkb, T), torch.float32, dev)
    wsc = _ptr(_given(w_scale, "w_scale"), "w_scale", (E, *two, nnb, nkb), torch.float32, dev)
    fp = _ptr(_given(offsets, "offsets"), "offsets", (E + 1,), torch.int32, dev)
    pp = None if perm is None else _ptr(perm, "perm", perm.shape, torch.int32, dev)
    bp = _ptr(bias, "bias", (E, *two, N), bf16, dev)
    rp, yp = _ptr(residual, "residual", (rows, N), bf16, dev), _ptr(y, "y", (rows, N), bf16, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_linear_grouped_fp8(x, x_scale, offsets, w, w_scale, bias, act, residual, perm,
                                          k, rows, y, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_linear_grouped_fp8_workspace_bytes(E, rows, N, K, code), dev, ws)
    if y is None:
        y = torch.empty((rows, N), dtype=bf16, device=dev)
        yp = y.data_ptr()
    _check("moe_linear_grouped_fp8", L.moe_linear_grouped_fp8(
        xp, xsp, pp, k, T, fp, E, rows, wp, wsc, bp, code, rp, N, K, yp, wsp, wsn,
        _raw_stream(dev.index)))
    return y


FEW_TOKENS = 64  # of moe_layer_few, at most
BIAS_MODES = {"choice": 0, "score": 1}


def moe_layer_few_workspace_bytes(T: int, H: int, E: int, k: int, F: int, Fs: int,
                                  dtype_code: int) -> int:
    _fits(T, H, E, k, F, Fs)
    return lib().moe_layer_few_workspace_bytes(T, H, E, k, F, Fs, dtype_code)


def moe_layer_few(x, wg, bias, w_up, w_down, k: int, score: str = "softmax",
                  bias_mode: str = "choice", groups: int = 1, topk_groups: int = 1,
                  group_top: int = 2, renorm: bool = True, scale: float = 1.0, act: str = "gelu",
                  b_up=None, b_down=None, ws_up=None, ws_down=None, out=None, topk_idx=None,
                  topk_w=None, ws=None, stream=None):
    """The whole layer for a few tokens (x [T,H], T <= 64) in two or three launches: routing,
    experts, shared expert and combine.

    Called one by one it is faster than the separate calls wherever the host bounds those
    (some 65 us a layer). Against a HIP graph of them it pays for experts of about 3 MB of
    weights or more (1024 x 512 gated, bf16) with up to 4 pairs of a token and an expert each
    (T * k / E); such a graph is up to 1.2 times as fast with 8 pairs an expert, 1.5 with 16,
    and 1.7 with smaller experts from 4 tokens on.

    Routing as moe_route_grouped; bias (fp32 [E] or None) moves the choice only
    (bias_mode "choice") or the scores themselves ("score", as moe_route). Experts as
    moe_block_forward: w_up [E,F,H] or, for a gated act, [E,2,F,H]; w_down [E,H,F];
    b_up [E,F] or [E,2,F], b_down [E,H]; ws_up, ws_down the same without E (the shared
    expert, no biases). moe_layer_forward's layer is act "gelu", bias_mode "score" and the
    other defaults. Returns (out [T,H], topk_idx int32 [T,k], topk_w fp32 [T,k])."""
    T, H = _shape(x, "x", 2)
    E = _shape(wg, "wg", 2)[0]
    code = _enum(ACTS, act, "act")
    two = (2,) if code >= 3 else ()
    F = _shape(w_up, "w_up", 3 + len(two))[-2]
    if (ws_up is None) != (ws_down is None):
        raise ValueError("the shared expert needs ws_up and ws_down")
    Fs = 0 if ws_up is None else _shape(ws_up, "ws_up", 2 + len(two))[-2]
    _fits(T, H, E, k, F, Fs, groups, topk_groups, group_top)
    dev, dtype = x.device, x.dtype
    dt, sc, bm = _dtype_code(x), _enum(SCORES, score, "score"), _enum(BIAS_MODES, bias_mode, "bias_mode")
    args = (_ptr(x, "x", (T, H), dtype, dev), _ptr(wg, "wg", (E, H), dtype, dev),
            _ptr(bias, "bias", (E,), torch.float32, dev), bm,
            _ptr(w_up, "w_up", (E, *two, F, H), dtype, dev),
            _ptr(_given(w_down, "w_down"), "w_down", (E, H, F), dtype, dev),
            _ptr(b_up, "b_up", (E, *two, F), dtype, dev), _ptr(b_down, "b_down", (E, H), dtype, dev),
            _ptr(ws_up, "ws_up", (*two, Fs, H), dtype, dev), _ptr(ws_down, "ws_down", (H, Fs), dtype, dev),
            T, H, E, k, F, Fs, code, sc, groups, topk_groups, group_top, int(renorm), scale, dt)
    op = _ptr(out, "out", (T, H), dtype, dev)
    ip = _ptr(topk_idx, "topk_idx", (T, k), torch.int32, dev)
    wp = _ptr(topk_w, "topk_w", (T, k), torch.float32, dev)
    other = _other_stream(dev, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_layer_few(x, wg, bias, w_up, w_down, k, score, bias_mode, groups, topk_groups,
                                 group_top, renorm, scale, act, b_up, b_down, ws_up, ws_down, out,
                                 topk_idx, topk_w, ws)
    L = lib()
    wsp, wsn, ws = _ws(L.moe_layer_few_workspace_bytes(T, H, E, k, F, Fs, dt), dev, ws)
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=dev)
        op = out.data_ptr()
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        ip = topk_idx.data_ptr()
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        wp = topk_w.data_ptr()
    _check("moe_layer_few", L.moe_layer_few(*args, op, ip, wp, wsp, wsn, _raw_stream(dev.index)))
    return out, topk_idx, topk_w


def moe_block_forward(h, wg, w_up, w_down, k: int, x=None, norm_weight=None, norm_bias=None,
                      norm: str = "rms", eps: float = 1e-6, route_bias=None,
                      score: str = "sigmoid", groups: int = 1, topk_groups: int = 1,
                      group_top: int = 2, renorm: bool = True, scale: float = 1.0,
                      act: str = "swiglu", b_up=None, b_down=None, ws_up=None, ws_down=None,
                      capacity=None, out_norm: str = "none", out_weight=None, out_bias=None,
                      gate=None, res_scale: float = 1.0, next_norm: str = "none",
                      next_weight=None, next_bias=None, stream=None, few: bool = False,
                      w_up_scale=None, w_down_scale=None, ws_up_scale=None, ws_down_scale=None):
    """A whole MoE block of a decoder on the residual stream h [T,H], on one stream
    without host synchronisation:

        x    = norm(h)                              (or given: the previous block's ``next``)
        idx, w = moe_route_grouped(x, wg, route_bias, k, ...)
        out  = sum_j w_j * expert_j(x) (+ shared expert(x)),
               expert(x) = act(x . w_up^T + b_up) . w_down^T + b_down
        res  = h + res_scale * gate * out_norm(out)
        next = next_norm(res)                       (None without a next_norm)

    w_up [E,F,H], or [E,2,F,H] for a gated act; w_down [E,H,F]; b_up [E,F] or
    [E,2,F], b_down [E,H]; ws_up, ws_down the same without E (no biases): the
    always-on shared expert. capacity (int) drops each expert's assignments past
    it. Returns a dict: res, next, and the steps' x, topk_idx, topk_w, counts,
    offsets, perm, inv, out.

    few=True runs route, experts and combine as moe_layer_few (T <= 64, no capacity; out
    sums the experts' rows before they are rounded; moe_layer_few says where it pays, in a
    MoEBlockGraph for large experts with few tokens each); counts, offsets, perm and inv
    are not made then.

    With w_up_scale and w_down_scale (moe_quantize_weight's, float8_e4m3fn weights, bf16 h
    and biases) the experts' products are moe_linear_grouped_fp8 of x and of the
    activated rows through moe_quantize; H and F are multiples of 128. ws_up_scale and
    ws_down_scale the same for the shared expert (moe_linear_fp8); each pair is given
    whole or not at all, and neither with few."""
    if (ws_up is None) != (ws_down is None):
        raise ValueError("the shared expert needs ws_up and ws_down")
    _dims(h, "h", 2)
    for up, down, name in ((w_up_scale, w_down_scale, "w"), (ws_up_scale, ws_down_scale, "ws")):
        if (up is None) != (down is None):
            raise ValueError(f"8-bit experts need {name}_up_scale and {name}_down_scale")
        if up is not None and few:
            raise ValueError("few takes no 8-bit experts")
        if up is not None and h.dtype != torch.bfloat16:
            raise ValueError(f"h must be torch.bfloat16 with 8-bit experts, got {h.dtype}")
    if ws_up_scale is not None and ws_up is None:
        raise ValueError("ws_up_scale without a shared expert")
    if few and capacity is not None:
        raise ValueError("few takes no capacity")
    other = _other_stream(h.device, stream)
    if other is not None:
        with torch.cuda.stream(other):
            return moe_block_forward(h, wg, w_up, w_down, k, x, norm_weight, norm_bias, norm, eps,
                                     route_bias, score, groups, topk_groups, group_top, renorm,
                                     scale, act, b_up, b_down, ws_up, ws_down, capacity, out_norm,
                                     out_weight, out_bias, gate, res_scale, next_norm, next_weight,
                                     next_bias, None, few, w_up_scale, w_down_scale, ws_up_scale,
                                     ws_down_scale)
    if x is None:
        x = moe_norm(h, norm_weight, norm_bias, eps, norm)
    if few:
        out, idx, w = moe_layer_few(x, wg, route_bias, w_up, w_down, k, score, "choice", groups,
                                    topk_groups, group_top, renorm, scale, act, b_up, b_down, ws_up,
                                    ws_down)
        d = {}
    else:
        idx, w = moe_route_grouped(x, wg, route_bias, k, score, groups, topk_groups, group_top, renorm,
                                   scale)
        d = moe_dispatch(idx, x, wg.shape[0], capacity=capacity, gather=False)
        if w_up_scale is not None or ws_up_scale is not None:
            x8 = moe_quantize(x)
        if w_up_scale is not None:
            a = moe_linear_grouped_fp8(*x8, d["offsets"], w_up, w_up_scale, b_up, act, perm=d["perm"], k=k)
            ys = moe_linear_grouped_fp8(*moe_quantize(a), d["offsets"], w_down, w_down_scale, b_down)
        else:
            a = moe_linear_grouped(x, d["offsets"], w_up, b_up, act, perm=d["perm"], k=k)
            ys = moe_linear_grouped(a, d["offsets"], w_down, b_down)
        ysh = None
        if ws_up_scale is not None:
            ysh = moe_linear_fp8(*x8, ws_up, ws_up_scale, act=act)
            ysh = moe_linear_fp8(*moe_quantize(ysh), ws_down, ws_down_scale)
        elif ws_up is not None:
            ysh = moe_linear(moe_linear(x, ws_up, act=act), ws_down)
        out = moe_combine(ys, d["inv"], w, ysh)
        del d["xs"]
    res, nxt = moe_norm_residual(out, h, out_weight, out_bias, gate, res_scale, eps, out_norm,
                                 next_weight, next_bias, next_norm)
    return dict(res=res, next=nxt, x=x, topk_idx=idx, topk_w=w, out=out, **d)


class MoEBlockGraph:
    """moe_block_forward for a fixed number of tokens T, captured once into a HIP
    graph and replayed (the decode-latency use of MoELayerGraph).

    Takes moe_block_forward's arguments after h, by keyword. ``run(h)`` copies h
    into the static input and replays; it returns (res, next), the static outputs,
    which the next run overwrites: runs on several streams are the caller's to order.
    ``state`` holds every step's static result. The weights and biases are read where
    they are: their owner may update them in place between runs."""

    def __init__(self, T: int, wg, w_up, w_down, k: int, **kw):
        if kw.get("x") is not None or kw.get("stream") is not None:
            raise ValueError("a captured block makes its own x and runs on the caller's current stream")
        dev = wg.device
        if dev.type != "cuda":
            raise ValueError("wg must be a GPU tensor")
        self.h = torch.zeros((T, wg.shape[1]), dtype=wg.dtype, device=dev)
        self.weights = (wg, w_up, w_down, kw)  # the graph reads them: kept alive with it
        call = lambda: moe_block_forward(self.h, wg, w_up, w_down, k, **kw)  # noqa: E731
        with torch.cuda.device(dev):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                call()  # one eager pass on a side stream before capture
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.state = call()
            torch.cuda.synchronize()

    def run(self, h):
        """Copy h (of the captured shape and type; host tensors are copied too) into the
        static input and replay; returns (res, next)."""
        if not isinstance(h, torch.Tensor):
            raise ValueError("h must be a torch tensor")
        _want(h, "h", self.h.shape, self.h.dtype)  # copy_ would broadcast and cast
        self.h.copy_(h)
        self.graph.replay()
        return self.state["res"], self.state["next"]
