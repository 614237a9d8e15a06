"""ctypes binding of libmtphead.so (include/mtp_head.h): argument marshalling only.

Each function has the name of the C entry point it calls and takes torch tensors where the C
function takes device (or host) pointers: the binding passes ``tensor.data_ptr()``, the
current CUDA stream (or the one given) and the sizes, and raises ``MTPError`` when the C call
returns a nonzero status. Every step of the computation runs in the library's CUDA kernels;
there is no fallback. If the shared library cannot be built or loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

W_BF16 = 0
W_FP8_E4M3 = 1
LOGITS_FP32 = 0
LOGITS_BF16 = 1

OK = 0
ERR_ARG = -1
ERR_SHAPE = -2
ERR_ALIGN = -3
ERR_WORKSPACE = -4
ERR_CUDA = -5
ERR_NONFINITE = -6
ERR_TOKEN_RANGE = -7
ERR_NOT_IMPLEMENTED = -8
ERR_TIMEOUT = -9

# name -> (restype, argtypes); mirrors include/mtp_head.h
P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
SIGNATURES = {
    "mtp_head_input_batched": (I, [P, P, P, P, P, P, P, P, I, I, I, F, P]),
    "mtp_head_input": (I, [P, P, P, P, P, P, P, P, I, I, F, P]),
    "mtp_head_logits_argmax_batched": (I, [P, P, P, P, I, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_logits_argmax": (I, [P, P, P, P, I, P, P, P, P, Z, I, I, F, P]),
    "mtp_head_logits_argmax_batched_noalloc": (I, [P, P, P, P, I, P, P, P, I, I, I, F, P]),
    "mtp_head_workspace_bytes": (Z, [I, I, I]),
    "mtp_head_forward_batched": (I, [P, P, P, P, P, P, P, I, P, P, P, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_forward_host": (I, [P, P, P, P, P, P, P, I, P, P, P, P, P, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_forward_host_args": (I, [P, P, P, P]),
    "mtp_head_quantize_fp8": (I, [P, P, P, P, I, I, P]),
    "mtp_head_context_rows": (I, [P, P, P, P, P, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_context_workspace_bytes": (Z, [I, I]),
    "mtp_head_logits_argmax_shard": (I, [P, P, P, P, I, I, I, P, P, P, P, P, Z, I, I, F, P]),
    "mtp_head_pick_combine": (I, [P, I, I, P, P, P]),
    "mtp_head_pick_key": (ctypes.c_int64, [F, ctypes.c_int32]),
    "mtp_head_pick_index": (ctypes.c_int32, [ctypes.c_int64]),
    "mtp_head_pick_value": (F, [ctypes.c_int64]),
    "mtp_head_set_wait_limit_ns": (ctypes.c_ulonglong, [ctypes.c_ulonglong]),
    "mtp_head_strerror": (ctypes.c_char_p, [I]),
    "mtp_head_fp4_padded": (I, [I]),
    "mtp_head_quantize_fp4": (I, [P, P, P, P, P, I, I, P]),
    "mtp_head_dequantize_fp4": (I, [P, P, P, P, I, I, P]),
    "mtp_head_logits_argmax_fp4": (I, [P, P, P, P, P, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_fp4_workspace_bytes": (Z, [I, I, I]),
    "mtp_head_linear_fp4": (I, [P, P, P, P, P, P, P, Z, I, I, I, P]),
    "mtp_head_linear_fp4_workspace_bytes": (Z, [I, I, I]),
    "mtp_head_context_rows_fp4": (I, [P, P, P, P, P, P, P, P, P, P, P, Z, I, I, I, F, P]),
    "mtp_head_context_fp4_workspace_bytes": (Z, [I, I]),
    "mtp_head_sample": (I, [P, I, ctypes.c_int64, P, P, P, P, P, P, P, P, P, I, I, P]),
    "mtp_head_verify": (I, [P, P, P, P, P, P, P, P, P, I, I, I, P]),
    "mtp_head_norm_residual": (I, [P, P, P, P, P, P, P, P, I, I, I, F, P]),
    "mtp_head_cache_write_fp4": (I, [P, L, P, L, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]),
    "mtp_head_cache_read_fp4": (I, [P, P, P, P, P, P, P, L, P, L, P, I, I, I, I, I, I, I, P]),
    "mtp_head_attention_fp4": (I, [P, L, P, P, P, P, P, P, P, L, P, P, P, Z, I, I, I, I, I, I, I, I, F, P]),
    "mtp_head_attention_fp4_workspace_bytes": (Z, [I, I, I, I, I, L]),
    "mtp_head_attention_prompt": (I, [P, L, P, L, P, L, P, P, L, P, P, I, I, I, I, I, F, P]),
}

_lib = None
_lock = threading.Lock()


class MTPError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: status {code}: {strerror(code)}")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load (building first if needed) libmtphead.so and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        lib_path = path or _build.build()
        if not os.path.exists(lib_path):
            raise RuntimeError(f"libmtphead.so not found at {lib_path}")
        lib = ctypes.CDLL(lib_path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def mtp_head_set_wait_limit_ns(ns: int) -> int:
    """Give-up time (ns) of the kernels' stage waits for later launches; returns the previous
    one. ns = 0: every stage wait gives up at once (the error path on demand)."""
    return int(load().mtp_head_set_wait_limit_ns(int(ns)))


def strerror(code: int) -> str:
    return load().mtp_head_strerror(int(code)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dev(t, name):
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _ptr(t)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(code: int, where: str) -> int:
    if code != OK:
        raise MTPError(code, where)
    return code


def mtp_head_workspace_bytes(B: int, H: int, V: int) -> int:
    return int(load().mtp_head_workspace_bytes(B, H, V))


def workspace(B: int, H: int, V: int, device=None) -> torch.Tensor:
    """A zero-filled workspace tensor for the output stage (reusable across calls)."""
    n = mtp_head_workspace_bytes(B, H, V)
    if n == 0:
        raise MTPError(ERR_SHAPE, "workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_input_batched(embed, enorm_w, hnorm_w, eh_proj, tokens, target_hidden, x_out,
                           status=None, eps: float = 1e-6, stream=None) -> None:
    V, H = embed.shape
    B = tokens.numel()
    _check(load().mtp_head_input_batched(
        _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"),
        _dev(eh_proj, "eh_proj"), _dev(tokens, "tokens"), _dev(target_hidden, "target_hidden"),
        _dev(x_out, "x_out"), _dev(status, "status"), B, H, V, eps, _stream(stream)),
        "mtp_head_input_batched")


def mtp_head_context_workspace_bytes(R: int, H: int) -> int:
    return int(load().mtp_head_context_workspace_bytes(R, H))


def context_workspace(R: int, H: int, device=None) -> torch.Tensor:
    """Scratch for mtp_head_context_rows (no initialisation needed)."""
    n = mtp_head_context_workspace_bytes(R, H)
    if n == 0:
        raise MTPError(ERR_SHAPE, "context_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_context_rows(embed, enorm_w, hnorm_w, eh_proj, tokens, target_hidden, x_out, ws=None,
                          status=None, eps: float = 1e-6, stream=None) -> None:
    V, H = embed.shape
    R = tokens.numel()
    _check(load().mtp_head_context_rows(
        _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"),
        _dev(eh_proj, "eh_proj"), _dev(tokens, "tokens"), _dev(target_hidden, "target_hidden"),
        _dev(x_out, "x_out"), _dev(status, "status"), _dev(ws, "workspace"),
        0 if ws is None else ws.numel() * ws.element_size(), R, H, V, eps, _stream(stream)),
        "mtp_head_context_rows")


def mtp_head_input(embed, enorm_w, hnorm_w, eh_proj, token, target_hidden, x_out, status=None,
                   eps: float = 1e-6, stream=None) -> None:
    V, H = embed.shape
    _check(load().mtp_head_input(
        _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"),
        _dev(eh_proj, "eh_proj"), _dev(token, "token"), _dev(target_hidden, "target_hidden"),
        _dev(x_out, "x_out"), _dev(status, "status"), H, V, eps, _stream(stream)),
        "mtp_head_input")


def mtp_head_logits_argmax_batched(x, final_norm_w, lm_head, row_scale, w_dtype: int, logits,
                                   draft, ws, status=None, eps: float = 1e-6, stream=None) -> None:
    V, H = lm_head.shape
    B = draft.numel()
    _check(load().mtp_head_logits_argmax_batched(
        _dev(x, "x"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"),
        _dev(row_scale, "row_scale"), int(w_dtype), _dev(logits, "logits"), _dev(draft, "draft"),
        _dev(status, "status"), _dev(ws, "workspace"), ws.numel() * ws.element_size(), B, H, V,
        eps, _stream(stream)),
        "mtp_head_logits_argmax_batched")


def mtp_head_logits_argmax(x, final_norm_w, lm_head, row_scale, w_dtype: int, logits, draft, ws,
                           status=None, eps: float = 1e-6, stream=None) -> None:
    V, H = lm_head.shape
    _check(load().mtp_head_logits_argmax(
        _dev(x, "x"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"),
        _dev(row_scale, "row_scale"), int(w_dtype), _dev(logits, "logits"), _dev(draft, "draft"),
        _dev(status, "status"), _dev(ws, "workspace"), ws.numel() * ws.element_size(), H, V, eps,
        _stream(stream)),
        "mtp_head_logits_argmax")


def mtp_head_logits_argmax_batched_noalloc(x, final_norm_w, lm_head, row_scale, w_dtype: int,
                                           logits, draft, status=None, eps: float = 1e-6,
                                           stream=None) -> None:
    """Output stage on the library's own fixed device scratch (no workspace argument): for
    callers that cannot allocate device memory. Calls that overlap on the GPU race on it."""
    V, H = lm_head.shape
    B = draft.numel()
    _check(load().mtp_head_logits_argmax_batched_noalloc(
        _dev(x, "x"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"),
        _dev(row_scale, "row_scale"), int(w_dtype), _dev(logits, "logits"), _dev(draft, "draft"),
        _dev(status, "status"), B, H, V, eps, _stream(stream)),
        "mtp_head_logits_argmax_batched_noalloc")


def mtp_head_logits_argmax_shard(x, final_norm_w, lm_head_shard, row_scale_shard, w_dtype: int, v0: int,
                                 logits, pick, draft, ws, status=None, eps: float = 1e-6, stream=None) -> None:
    """Output stage over the vocabulary rows [v0, v0 + n) (lm_head_shard holds those n rows):
    pick [B] int64 receives each sequence's exchange key; logits [B, n] and draft [B] (a global
    index) are optional."""
    n, H = lm_head_shard.shape
    B = pick.numel()
    _check(load().mtp_head_logits_argmax_shard(
        _dev(x, "x"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head_shard, "lm_head_shard"),
        _dev(row_scale_shard, "row_scale_shard"), int(w_dtype), int(v0), n, _dev(logits, "logits"),
        _dev(pick, "pick"), _dev(draft, "draft"), _dev(status, "status"), _dev(ws, "workspace"),
        ws.numel() * ws.element_size(), B, H, eps, _stream(stream)),
        "mtp_head_logits_argmax_shard")


def mtp_head_pick_combine(picks, draft, value=None, stream=None) -> None:
    """draft [B] (and value [B]) from the exchange keys picks [R, B] of R vocabulary shards."""
    B = draft.numel()
    R = picks.numel() // B
    _check(load().mtp_head_pick_combine(_dev(picks, "picks"), R, B, _dev(draft, "draft"), _dev(value, "value"),
                                        _stream(stream)),
           "mtp_head_pick_combine")


def mtp_head_pick_key(value: float, index: int) -> int:
    """The exchange key of (value, global index), computed on the host."""
    return int(load().mtp_head_pick_key(float(value), int(index)))


def mtp_head_pick_index(key: int) -> int:
    return int(load().mtp_head_pick_index(int(key)))


def mtp_head_pick_value(key: int) -> float:
    return float(load().mtp_head_pick_value(int(key)))


def mtp_head_forward_batched(embed, enorm_w, hnorm_w, eh_proj, final_norm_w, lm_head, row_scale,
                             w_dtype: int, tokens, target_hidden, x, logits, draft, ws,
                             status=None, eps: float = 1e-6, stream=None) -> None:
    V, H = embed.shape
    B = tokens.numel()
    _check(load().mtp_head_forward_batched(
        _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"),
        _dev(eh_proj, "eh_proj"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"),
        _dev(row_scale, "row_scale"), int(w_dtype), _dev(tokens, "tokens"),
        _dev(target_hidden, "target_hidden"), _dev(x, "x"), _dev(logits, "logits"),
        _dev(draft, "draft"), _dev(status, "status"), _dev(ws, "workspace"),
        ws.numel() * ws.element_size(), B, H, V, eps, _stream(stream)),
        "mtp_head_forward_batched")


def mtp_head_forward_host(embed, enorm_w, hnorm_w, eh_proj, final_norm_w, lm_head, row_scale,
                          w_dtype: int, tokens_host, hidden_host, tokens_dev, hidden_dev, x_dev,
                          draft_dev, draft_host, ws, status=None, eps: float = 1e-6,
                          stream=None) -> None:
    """Synchronous draft step from host buffers (tokens_host, hidden_host, draft_host are CPU
    tensors, pinned for asynchronous copies)."""
    V, H = embed.shape
    B = tokens_host.numel()
    for t, n in ((tokens_host, "tokens_host"), (hidden_host, "hidden_host"), (draft_host, "draft_host")):
        if t.is_cuda:
            raise ValueError(f"{n} must be a host tensor")
    _check(load().mtp_head_forward_host(
        _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"),
        _dev(eh_proj, "eh_proj"), _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"),
        _dev(row_scale, "row_scale"), int(w_dtype), _ptr(tokens_host), _ptr(hidden_host),
        _dev(tokens_dev, "tokens_dev"), _dev(hidden_dev, "hidden_dev"), _dev(x_dev, "x_dev"),
        _dev(draft_dev, "draft_dev"), _ptr(draft_host), _dev(status, "status"),
        _dev(ws, "workspace"), ws.numel() * ws.element_size(), B, H, V, eps, _stream(stream)),
        "mtp_head_forward_host")


class _HostStepArgs(ctypes.Structure):
    """mtp_host_step_args (include/mtp_head.h), field for field."""
    _fields_ = [("embed", P), ("enorm_w", P), ("hnorm_w", P), ("eh_proj", P), ("final_norm_w", P),
                ("lm_head", P), ("row_scale", P), ("w_dtype", I), ("tokens_dev", P), ("hidden_dev", P),
                ("x_dev", P), ("draft_dev", P), ("status", P), ("workspace", P), ("workspace_bytes", Z),
                ("B", I), ("H", I), ("V", I), ("eps", F), ("stream", P)]


class HostStep:
    """mtp_head_forward_host with its device buffers bound once: a call passes only the three host
    buffers (tensors, or their addresses as ints) to mtp_head_forward_host_args, so a synchronous
    draft step costs one four-argument ctypes call on the host. The bound tensors stay referenced
    for the object's lifetime."""

    def __init__(self, embed, enorm_w, hnorm_w, eh_proj, final_norm_w, lm_head, row_scale, w_dtype: int,
                 tokens_dev, hidden_dev, x_dev, draft_dev, ws, status=None, eps: float = 1e-6, stream=None):
        V, H = embed.shape
        B = tokens_dev.numel()
        self.B, self.H, self.V = B, H, V
        self._keep = (embed, enorm_w, hnorm_w, eh_proj, final_norm_w, lm_head, row_scale, tokens_dev,
                      hidden_dev, x_dev, draft_dev, ws, status, stream)
        self._fn = load().mtp_head_forward_host_args
        self._args = _HostStepArgs(
            _dev(embed, "embed"), _dev(enorm_w, "enorm_w"), _dev(hnorm_w, "hnorm_w"), _dev(eh_proj, "eh_proj"),
            _dev(final_norm_w, "final_norm_w"), _dev(lm_head, "lm_head"), _dev(row_scale, "row_scale"),
            int(w_dtype), _dev(tokens_dev, "tokens_dev"), _dev(hidden_dev, "hidden_dev"), _dev(x_dev, "x_dev"),
            _dev(draft_dev, "draft_dev"), _dev(status, "status"), _dev(ws, "workspace"),
            ws.numel() * ws.element_size(), B, H, V, float(eps), _stream(stream))
        self._addr = ctypes.addressof(self._args)

    def __call__(self, tokens_host, hidden_host, draft_host) -> None:
        t = tokens_host if isinstance(tokens_host, int) else tokens_host.data_ptr()
        h = hidden_host if isinstance(hidden_host, int) else hidden_host.data_ptr()
        d = draft_host if isinstance(draft_host, int) else draft_host.data_ptr()
        code = self._fn(self._addr, t, h, d)
        if code != OK:
            raise MTPError(code, "mtp_head_forward_host")


def mtp_head_quantize_fp8(w, q, row_scale, status, stream=None) -> None:
    V, H = w.shape
    _check(load().mtp_head_quantize_fp8(
        _dev(w, "w"), _dev(q, "q"), _dev(row_scale, "row_scale"), _dev(status, "status"), V, H,
        _stream(stream)),
        "mtp_head_quantize_fp8")


# ------------------------------------------------------------------ FP4 copies, sampling, acceptance
# These check every tensor (type, shape, layout, device) and launch on the tensors' own device.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _t(t, name, dtype, shape, dev, optional=False):
    """The address of a contiguous tensor of this type and shape on CUDA device ``dev``."""
    if t is None and optional:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _first(t, name, n):
    """The shape and CUDA device number of the tensor that decides both for a call."""
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.shape, t.get_device()


def _ws(t, dev):
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _call(dev, stream, name, *args):
    """The entry point on device ``dev``, on the given stream or that device's current one."""
    fn = getattr(_lib or load(), name)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            code = fn(*args, _stream(stream))
    else:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if code != OK:
        raise MTPError(code, name)


def mtp_head_fp4_padded(H: int) -> int:
    """Codes per row of the FP4 copy of an H-column matrix (0 for H outside the range)."""
    return int((_lib or load()).mtp_head_fp4_padded(H))


def fp4_empty(V: int, H: int, device=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Uninitialised (q, block_scale, row_scale) of the FP4 copy of a [V, H] matrix."""
    hp = mtp_head_fp4_padded(H)
    if hp == 0 or V < 1:
        raise MTPError(ERR_SHAPE, "fp4_empty")
    dev = device or "cuda"
    return (torch.empty((V, hp // 2), dtype=torch.uint8, device=dev),
            torch.empty((V, hp // 16), dtype=torch.uint8, device=dev),
            torch.empty(V, dtype=torch.float32, device=dev))


def _fp4(q, block_scale, row_scale, V, H, dev):
    hp = (H + 255) // 256 * 256  # mtp_head_fp4_padded (the library checks the range)
    return (_t(q, "q", _U8, (V, hp // 2), dev), _t(block_scale, "block_scale", _U8, (V, hp // 16), dev),
            _t(row_scale, "row_scale", _F32, (V,), dev))


def mtp_head_quantize_fp4(w, q, block_scale, row_scale, status, stream=None) -> None:
    """The FP4 copy (q, block_scale, row_scale) of w [V, H] BF16."""
    (V, H), dev = _first(w, "w", 2)
    _call(dev, stream, "mtp_head_quantize_fp4", _t(w, "w", _BF16, (V, H), dev),
          *_fp4(q, block_scale, row_scale, V, H, dev), _t(status, "status", _I32, (1,), dev), V, H)


def mtp_head_dequantize_fp4(q, block_scale, row_scale, w, stream=None) -> None:
    """w [V, H] BF16: the matrix that an FP4 copy stands for."""
    (V, H), dev = _first(w, "w", 2)
    _call(dev, stream, "mtp_head_dequantize_fp4", *_fp4(q, block_scale, row_scale, V, H, dev),
          _t(w, "w", _BF16, (V, H), dev), V, H)


def mtp_head_fp4_workspace_bytes(B: int, H: int, V: int) -> int:
    return int(load().mtp_head_fp4_workspace_bytes(B, H, V))


def fp4_workspace(B: int, H: int, V: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for mtp_head_logits_argmax_fp4 (reusable across calls)."""
    n = mtp_head_fp4_workspace_bytes(B, H, V)
    if n == 0:
        raise MTPError(ERR_SHAPE, "fp4_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_logits_argmax_fp4(x, final_norm_w, q, block_scale, row_scale, logits, draft, ws, status=None,
                               eps: float = 1e-6, stream=None) -> None:
    """Output stage over the FP4 copy of lm_head; logits [B, V] optional, draft [B]."""
    (B, H), dev = _first(x, "x", 2)
    (V,), _ = _first(row_scale, "row_scale", 1)
    _call(dev, stream, "mtp_head_logits_argmax_fp4", _t(x, "x", _BF16, (B, H), dev),
          _t(final_norm_w, "final_norm_w", _BF16, (H,), dev), *_fp4(q, block_scale, row_scale, V, H, dev),
          _t(logits, "logits", _F32, (B, V), dev, True), _t(draft, "draft", _I32, (B,), dev),
          _t(status, "status", _I32, (1,), dev, True), *_ws(ws, dev), B, H, V, eps)


def mtp_head_linear_fp4_workspace_bytes(R: int, N: int, K: int) -> int:
    return int(load().mtp_head_linear_fp4_workspace_bytes(R, N, K))


def linear_fp4_workspace(R: int, N: int, K: int, device=None) -> torch.Tensor:
    """Scratch for mtp_head_linear_fp4 (no initialisation needed)."""
    n = mtp_head_linear_fp4_workspace_bytes(R, N, K)
    if n == 0:
        raise MTPError(ERR_SHAPE, "linear_fp4_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_linear_fp4(x, q, block_scale, row_scale, y, ws, status=None, stream=None) -> None:
    """y [R, N] = rows of x [R, K], quantised to FP4, times the FP4 copy of a [N, K] matrix."""
    (R, K), dev = _first(x, "x", 2)
    (N,), _ = _first(row_scale, "row_scale", 1)
    _call(dev, stream, "mtp_head_linear_fp4", _t(x, "x", _BF16, (R, K), dev),
          *_fp4(q, block_scale, row_scale, N, K, dev), _t(y, "y", _BF16, (R, N), dev),
          _t(status, "status", _I32, (1,), dev, True), *_ws(ws, dev), R, N, K)


def mtp_head_context_fp4_workspace_bytes(R: int, H: int) -> int:
    return int(load().mtp_head_context_fp4_workspace_bytes(R, H))


def context_fp4_workspace(R: int, H: int, device=None) -> torch.Tensor:
    """Scratch for mtp_head_context_rows_fp4 (no initialisation needed)."""
    n = mtp_head_context_fp4_workspace_bytes(R, H)
    if n == 0:
        raise MTPError(ERR_SHAPE, "context_fp4_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_context_rows_fp4(embed, enorm_w, hnorm_w, eh_q, eh_block_scale, eh_row_scale, tokens, target_hidden,
                              x_out, ws, status=None, eps: float = 1e-6, stream=None) -> None:
    """The input stage of R rows with an FP4 copy of eh_proj."""
    (V, H), dev = _first(embed, "embed", 2)
    (R,), _ = _first(tokens, "tokens", 1)
    _call(dev, stream, "mtp_head_context_rows_fp4", _t(embed, "embed", _BF16, (V, H), dev),
          _t(enorm_w, "enorm_w", _BF16, (H,), dev), _t(hnorm_w, "hnorm_w", _BF16, (H,), dev),
          *_fp4(eh_q, eh_block_scale, eh_row_scale, H, 2 * H, dev), _t(tokens, "tokens", _I32, (R,), dev),
          _t(target_hidden, "target_hidden", _BF16, (R, H), dev), _t(x_out, "x_out", _BF16, (R, H), dev),
          _t(status, "status", _I32, (1,), dev, True), *_ws(ws, dev), R, H, V, eps)


def mtp_head_sample(logits, u=None, token=None, prob=None, probs=None, temperature=None, top_k=None, top_p=None,
                    min_p=None, status=None, stream=None) -> None:
    """One token per row of logits [R, V] (fp32 or BF16; the rows may be strided) from u [R]. The
    parameters are [R] tensors or None; token, prob [R] and probs [R, V] are outputs, each optional."""
    (R, V), dev = _first(logits, "logits", 2)
    if logits.dtype not in (_F32, _BF16):
        raise ValueError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    ld = logits.stride(0) if R > 1 else V
    if (V > 1 and logits.stride(1) != 1) or ld < V:
        raise ValueError("logits: each row must be contiguous, and the rows must not overlap")
    r = (R,)
    _call(dev, stream, "mtp_head_sample", logits.data_ptr(), LOGITS_BF16 if logits.dtype is _BF16 else LOGITS_FP32, ld,
          _t(temperature, "temperature", _F32, r, dev, True), _t(top_k, "top_k", _I32, r, dev, True),
          _t(top_p, "top_p", _F32, r, dev, True), _t(min_p, "min_p", _F32, r, dev, True), _t(u, "u", _F32, r, dev, True),
          _t(token, "token", _I32, r, dev, True), _t(prob, "prob", _F32, r, dev, True),
          _t(probs, "probs", _F32, (R, V), dev, True), _t(status, "status", _I32, (1,), dev, True), R, V)


def mtp_head_verify(target_probs, draft_probs, draft_tokens, u, tokens, accepted, prob=None, draft_len=None,
                    status=None, stream=None) -> None:
    """Drafts [B, D] accepted against target_probs [B, D + 1, V]; draft_probs [B, D, V], or None for
    greedy drafts. tokens [B, D + 1], accepted [B] and prob [B] (optional) are outputs. u [B, D + 1] is
    independent of the numbers that drew the drafts."""
    (B, D1, V), dev = _first(target_probs, "target_probs", 3)
    D = D1 - 1
    _call(dev, stream, "mtp_head_verify", _t(target_probs, "target_probs", _F32, (B, D1, V), dev),
          _t(draft_probs, "draft_probs", _F32, (B, D, V), dev, True), _t(draft_tokens, "draft_tokens", _I32, (B, D), dev),
          _t(draft_len, "draft_len", _I32, (B,), dev, True), _t(u, "u", _F32, (B, D1), dev),
          _t(tokens, "tokens", _I32, (B, D1), dev), _t(accepted, "accepted", _I32, (B,), dev),
          _t(prob, "prob", _F32, (B,), dev, True), _t(status, "status", _I32, (1,), dev, True), B, D, V)


# ------------------------------------------------------------------ the attention half of a draft layer
def mtp_head_norm_residual(x, w, delta=None, total=None, y=None, q=None, q_scale=None, status=None, group: int = 0,
                           eps: float = 1e-6, stream=None) -> None:
    """total [R, H] = x + delta, y [R, H] = its norm with weight w [H], q [R, H] the E4M3 codes of y with
    q_scale [R] (group 0) or [R, ceil(H / 128)] (group 128). total, y and q are outputs, each optional."""
    (R, H), dev = _first(x, "x", 2)
    n = (R, H)
    scales = (R,) if group == 0 else (R, -(-H // group)) if group > 0 else None
    _call(dev, stream, "mtp_head_norm_residual", _t(x, "x", _BF16, n, dev), _t(delta, "delta", _BF16, n, dev, True),
          _t(w, "w", _BF16, (H,), dev), _t(total, "total", _BF16, n, dev, True), _t(y, "y", _BF16, n, dev, True),
          _t(q, "q", _U8, n, dev, True), _t(q_scale, "q_scale", _F32, scales, dev, True),
          _t(status, "status", _I32, (1,), dev, True), R, H, group, eps)


def cache_empty(pages: int, page: int, heads: int, head_dim: int, device=None):
    """Zero-filled (q, block_scale, row_scale) of a paged FP4 cache."""
    if pages < 1 or page < 16 or heads < 1 or head_dim < 16 or head_dim % 16:
        raise MTPError(ERR_SHAPE, "cache_empty")
    dev = device or "cuda"
    return (torch.zeros((pages, 2, heads, page, head_dim // 2), dtype=torch.uint8, device=dev),
            torch.zeros((pages, 2, heads, page, head_dim // 16), dtype=torch.uint8, device=dev),
            torch.zeros((pages, 2, heads, page), dtype=torch.float32, device=dev))


def _cache(q, block_scale, row_scale):
    """The addresses of a cache, its sizes (pages, heads, page, head_dim) and its device."""
    (pages, two, heads, page, half), dev = _first(q, "q", 5)
    if two != 2:
        raise ValueError("q must have shape (pages, 2, heads, page, head_dim / 2)")
    at = (_t(q, "q", _U8, (pages, 2, heads, page, half), dev),
          _t(block_scale, "block_scale", _U8, (pages, 2, heads, page, half // 8), dev),
          _t(row_scale, "row_scale", _F32, (pages, 2, heads, page), dev))
    return at, pages, heads, page, 2 * half, dev


def _rows_of_heads(t, name, shape, dev):
    """The address and row stride of a BF16 tensor [..., heads, head_dim] whose rows may lie apart: its
    heads dense, the rows at equal distances."""
    if (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr(), shape[-2] * shape[-1]
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    heads, dim = shape[-2:]
    st = t.stride()
    dense = (dim == 1 or st[-1] == 1) and (heads == 1 or st[-2] == dim)
    ld = heads * dim
    if len(shape) == 3:
        ld = st[0] if shape[0] > 1 else ld
    else:
        if shape[1] > 1:
            ld = st[1]
            dense = dense and (shape[0] == 1 or st[0] == shape[1] * ld)
        elif shape[0] > 1:
            ld = st[0]
    if not dense or ld < heads * dim:
        raise ValueError(f"{name}: a row's heads must be dense, and its rows at equal distances")
    return t.data_ptr(), ld


def mtp_head_cache_write_fp4(k, v, row_start, position, block_table, q, block_scale, row_scale, status=None,
                             stream=None) -> None:
    """Rows k, v [T, heads, head_dim] (BF16, the rows may lie apart) into the cache: sequence b's rows
    row_start[b] .. row_start[b + 1] at its positions from position[b] on."""
    at, pages, heads, page, D, dev = _cache(q, block_scale, row_scale)
    (T, _, _), _ = _first(k, "k", 3)
    (B, max_pages), _ = _first(block_table, "block_table", 2)
    shape = (T, heads, D)
    _call(dev, stream, "mtp_head_cache_write_fp4", *_rows_of_heads(k, "k", shape, dev), *_rows_of_heads(v, "v", shape, dev),
          _t(row_start, "row_start", _I32, (B + 1,), dev), _t(position, "position", _I32, (B,), dev),
          _t(block_table, "block_table", _I32, (B, max_pages), dev), *at, _t(status, "status", _I32, (1,), dev, True),
          T, B, heads, D, pages, page, max_pages)


def mtp_head_cache_read_fp4(q, block_scale, row_scale, row_start, position, block_table, k, v, status=None,
                            stream=None) -> None:
    """The rows that a write of the same arguments filled, back as BF16 into k, v [T, heads, head_dim]."""
    at, pages, heads, page, D, dev = _cache(q, block_scale, row_scale)
    (T, _, _), _ = _first(k, "k", 3)
    (B, max_pages), _ = _first(block_table, "block_table", 2)
    shape = (T, heads, D)
    _call(dev, stream, "mtp_head_cache_read_fp4", *at, _t(row_start, "row_start", _I32, (B + 1,), dev),
          _t(position, "position", _I32, (B,), dev), _t(block_table, "block_table", _I32, (B, max_pages), dev),
          *_rows_of_heads(k, "k", shape, dev), *_rows_of_heads(v, "v", shape, dev),
          _t(status, "status", _I32, (1,), dev, True), T, B, heads, D, pages, page, max_pages)


def mtp_head_attention_fp4_workspace_bytes(B: int, Q: int, q_heads: int, kv_heads: int, head_dim: int,
                                           max_len: int) -> int:
    return int(load().mtp_head_attention_fp4_workspace_bytes(B, Q, q_heads, kv_heads, head_dim, max_len))


def attention_fp4_workspace(B: int, Q: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int,
                            device=None) -> torch.Tensor:
    """A zero-filled workspace for mtp_head_attention_fp4 (max_len: max_pages * page), reusable across calls
    of these sizes."""
    n = mtp_head_attention_fp4_workspace_bytes(B, Q, q_heads, kv_heads, head_dim, max_len)
    if n == 0:
        raise MTPError(ERR_SHAPE, "attention_fp4_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def mtp_head_attention_fp4(query, q, block_scale, row_scale, block_table, length, out, ws, rows=None, lse=None,
                           scale: float | None = None, status=None, stream=None) -> None:
    """out [B, Q, q_heads, head_dim] = attention of query (the same shape, BF16, rows may lie apart) over each
    sequence's pages; length [B] counts the query rows' own tokens, rows [B] (optional) how many of the Q rows
    a sequence has; lse [B, Q, q_heads] optional. scale: 1 / sqrt(head_dim) unless given."""
    at, pages, heads, page, D, dev = _cache(q, block_scale, row_scale)
    (B, Q, hq, _), _ = _first(query, "query", 4)
    (_, max_pages), _ = _first(block_table, "block_table", 2)
    shape = (B, Q, hq, D)
    _call(dev, stream, "mtp_head_attention_fp4", *_rows_of_heads(query, "query", shape, dev), *at,
          _t(block_table, "block_table", _I32, (B, max_pages), dev), _t(length, "length", _I32, (B,), dev),
          _t(rows, "rows", _I32, (B,), dev, True), *_rows_of_heads(out, "out", shape, dev),
          _t(lse, "lse", _F32, (B, Q, hq), dev, True), _t(status, "status", _I32, (1,), dev, True), *_ws(ws, dev),
          B, Q, hq, heads, D, pages, page, max_pages, D ** -0.5 if scale is None else scale)


def mtp_head_attention_prompt(q, k, v, row_start, out, lse=None, scale: float | None = None, status=None,
                              stream=None) -> None:
    """out [T, q_heads, head_dim] = causal attention of q (the same shape) over k, v [T, kv_heads, head_dim] within
    each sequence row_start[b] .. row_start[b + 1] (BF16; rows may lie apart); lse [T, q_heads] optional. scale:
    1 / sqrt(head_dim) unless given."""
    (T, hq, D), dev = _first(q, "q", 3)
    (_, heads, _), _ = _first(k, "k", 3)
    (B1,), _ = _first(row_start, "row_start", 1)
    _call(dev, stream, "mtp_head_attention_prompt", *_rows_of_heads(q, "q", (T, hq, D), dev),
          *_rows_of_heads(k, "k", (T, heads, D), dev), *_rows_of_heads(v, "v", (T, heads, D), dev),
          _t(row_start, "row_start", _I32, (B1,), dev), *_rows_of_heads(out, "out", (T, hq, D), dev),
          _t(lse, "lse", _F32, (T, hq), dev, True), _t(status, "status", _I32, (1,), dev, True), T, B1 - 1, hq, heads, D,
          D ** -0.5 if scale is None else scale)
