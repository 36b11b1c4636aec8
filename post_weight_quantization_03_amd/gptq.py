"""Python binding of libgptq (ctypes): argument marshalling for the C ABI in include/gptq.h.

Every step of the quantizer runs in the HIP library; this module only checks tensor
shapes, dtypes and devices, allocates outputs and workspaces with PyTorch on the current
device, and passes raw pointers and the current HIP stream.  It raises if the shared
library has not been built: there is no fallback path.

Names follow the C ABI: ``accumulate_hessian``, ``prepare_hinv``, ``quantize_layer``,
``pack_int4``.  Tensors may carry a leading batch dimension (independent problems, e.g.
mixture-of-experts layers).  ``moe_*`` route tokens to experts and ``fp8_*`` serve layers in
8 bits; no call records a gradient.

``stream`` is the torch stream a call runs on (None: the current one).  Its inputs have to be
ready there; what the call allocates comes from that stream's memory.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgptq.so")
_lib = None

GPTQ_OK, GPTQ_ERR_INVALID_ARG, GPTQ_ERR_NOT_SPD, GPTQ_ERR_HIP, GPTQ_ERR_WORKSPACE, GPTQ_ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
GPTQ_ERR_TOO_LARGE = -6
NOALLOC_SCRATCH_BYTES = 64 << 20
WS_HESSIAN, WS_PREPARE, WS_QUANTIZE, WS_W4A16_REPACK, WS_W4A16 = 0, 1, 2, 3, 4
WS_FP8_MATMUL, WS_FP8_GROUPED, WS_MOE_GROUP = 5, 6, 7

EXPORTED = ("gptq_accumulate_hessian", "gptq_prepare_hinv", "gptq_quantize_layer", "gptq_quantize_layer_noalloc",
            "gptq_accumulate_hessian_grouped", "gptq_pack_int4", "gptq_w4a16_repack", "gptq_w4a16_matmul",
            "gptq_fp8_quantize", "gptq_fp8_matmul", "gptq_fp8_matmul_grouped", "gptq_moe_route",
            "gptq_moe_group_tokens", "gptq_moe_combine",
            "gptq_workspace_size", "gptq_status_string", "gptq_version", "gptq_timing_enable", "gptq_timing_read")


class GptqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class NotSPDError(GptqError):
    pass


class _Params(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group_size", ctypes.c_int), ("block_size", ctypes.c_int),
                ("damp", ctypes.c_float), ("act_order", ctypes.c_int), ("sym", ctypes.c_int),
                ("static_groups", ctypes.c_int)]


class _RouteParams(ctypes.Structure):
    _fields_ = [("scoring", ctypes.c_int), ("n_groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("group_score", ctypes.c_int), ("top_k", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("scale", ctypes.c_float)]


@dataclasses.dataclass(frozen=True)
class Params:
    """Quantizer knobs: bits, group_size (-1 = per row), block_size (128), damp, act_order,
    sym (symmetric grid), static_groups (groups of original columns fitted up front)."""

    bits: int = 4
    group_size: int = 128
    block_size: int = 128
    damp: float = 0.01
    act_order: bool = False
    sym: bool = False
    static_groups: bool = False

    def c(self) -> _Params:
        return _Params(self.bits, self.group_size, self.block_size, self.damp, int(self.act_order), int(self.sym),
                       int(self.static_groups))

    def n_groups(self, d_in: int) -> int:
        return 1 if self.group_size == -1 else d_in // self.group_size


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded libgptq.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m post_weight_quantization_03_amd.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.gptq_accumulate_hessian.argtypes = [i32, i32, i64, i32, vp, i64, i64, vp, i64, vp, vp, vp, sz, vp]
    L.gptq_accumulate_hessian_grouped.argtypes = [i32, i32, i64, i64, i32, vp, i64, vp, vp, i64, vp, vp, vp, sz, vp]
    L.gptq_prepare_hinv.argtypes = [i32, i32, vp, i64, vp, ctypes.POINTER(_Params), vp, i64, vp, vp, vp, sz, vp]
    L.gptq_quantize_layer.argtypes = [i32, i32, i32, i32, vp, i64, i64, vp, i64, vp, vp, ctypes.POINTER(_Params),
                                      vp, vp, vp, vp, vp, sz, vp]
    L.gptq_quantize_layer_noalloc.argtypes = [i32, i32, i32, i32, vp, i64, i64, vp, i64, vp, vp,
                                              ctypes.POINTER(_Params), vp, vp, vp, vp, vp]
    L.gptq_pack_int4.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.gptq_w4a16_repack.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.gptq_w4a16_matmul.argtypes = [i32, i32, i32, i32, i32, vp, i64, vp, vp, vp, vp, vp, i64, vp, sz, vp]
    L.gptq_fp8_quantize.argtypes = [i32, i64, i32, i32, vp, i64, i64, i32, i32, vp, vp, i64, i64, i64, vp]
    L.gptq_fp8_matmul.argtypes = [i64, i32, i32, i32, vp, i64, i32, vp, i64, i64, vp, vp, i32, vp, i64, vp, sz, vp]
    L.gptq_fp8_matmul_grouped.argtypes = [i32, i64, i64, i32, i32, i32, vp, i64, i32, vp, i64, i64, vp, vp, vp, vp,
                                          i32, vp, i64, vp, sz, vp]
    L.gptq_moe_route.argtypes = [i64, i32, i32, vp, i64, vp, ctypes.POINTER(_RouteParams), vp, vp, vp]
    L.gptq_moe_group_tokens.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.gptq_moe_combine.argtypes = [i64, i32, i64, i32, i32, vp, i64, vp, vp, vp, i64, vp]
    L.gptq_workspace_size.argtypes = [i32, i32, i32, i32, i64, ctypes.POINTER(_Params)]
    L.gptq_workspace_size.restype = sz
    L.gptq_status_string.argtypes = [i32]
    L.gptq_status_string.restype = ctypes.c_char_p
    L.gptq_version.argtypes = []
    L.gptq_version.restype = ctypes.c_char_p
    L.gptq_timing_enable.argtypes = [i32]
    L.gptq_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    for name in ("gptq_accumulate_hessian", "gptq_accumulate_hessian_grouped", "gptq_prepare_hinv", "gptq_quantize_layer", "gptq_quantize_layer_noalloc",
                 "gptq_pack_int4", "gptq_w4a16_repack", "gptq_w4a16_matmul", "gptq_timing_enable",
                 "gptq_timing_read", "gptq_fp8_quantize", "gptq_fp8_matmul", "gptq_fp8_matmul_grouped",
                 "gptq_moe_route", "gptq_moe_group_tokens", "gptq_moe_combine"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().gptq_status_string(status).decode()


def _check(status: int, what: str):
    if status == GPTQ_ERR_NOT_SPD:
        raise NotSPDError(status, what)
    if status != GPTQ_OK:
        raise GptqError(status, what)


_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _tensors(v):
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (tuple, list, dict)):
        for x in v.values() if isinstance(v, dict) else v:
            yield from _tensors(x)


def _on(stream, call, *args):
    """``call(*args)`` with ``stream`` as the current one, so that also the call's own tensors come
    from that stream's memory: a block freed on the caller's stream may still have work queued
    there, which the other stream would not wait for.  The caching allocator is told that the
    caller's tensors are in use on that stream and the results on the caller's: they may be freed
    before the work queued there is done."""
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return call(*args)
    used = list(_tensors(args))
    if any(t.device != stream.device for t in used):
        raise ValueError("stream and tensors must be on one GPU")
    with torch.cuda.stream(stream):
        result = call(*args)
    for t in used:
        t.record_stream(stream)
    for t in _tensors(result):
        t.record_stream(current)
    return result


def _batched(t: torch.Tensor, nd: int) -> torch.Tensor:
    return t.unsqueeze(0) if t.dim() == nd else t


def workspace_size(which: int, batch: int, d_out: int, d_in: int, n_tokens_hint: int = 0,
                   params: Params | None = None) -> int:
    p = (params or Params()).c()
    return int(lib().gptq_workspace_size(which, batch, d_out, d_in, n_tokens_hint, ctypes.byref(p)))


def _workspace(nbytes: int, device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None and workspace.numel() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def new_hessian(d_in: int, batch: int | None = None, device="cuda"):
    """Zeroed (H fp32, diag_key fp64, n_seen int64) accumulators."""
    shp = () if batch is None else (batch,)
    return (torch.zeros(*shp, d_in, d_in, dtype=torch.float32, device=device),
            torch.zeros(*shp, d_in, dtype=torch.float64, device=device),
            torch.zeros(*(shp or (1,)), dtype=torch.int64, device=device))


def accumulate_hessian(X: torch.Tensor, H: torch.Tensor, diag_key: torch.Tensor, n_seen: torch.Tensor,
                       workspace: torch.Tensor | None = None, stream=None) -> None:
    """H += 2 X^T X, diag_key += 2 sum x^2 (fp64), n_seen += n for token-major X [(batch,) n, d_in]."""
    if stream is not None:
        return _on(stream, accumulate_hessian, X, H, diag_key, n_seen, workspace)
    Xb = _batched(X, 2)
    Hb = _batched(H, 2)
    batch, n, d_in = Xb.shape
    if X.dtype not in _DT or H.dtype != torch.float32 or diag_key.dtype != torch.float64 or n_seen.dtype != torch.int64:
        raise TypeError("X must be fp32/bf16/fp16, H fp32, diag_key fp64, n_seen int64")
    if Hb.shape != (batch, d_in, d_in) or diag_key.numel() != batch * d_in or n_seen.numel() < batch:
        raise ValueError("shape mismatch between X, H, diag_key, n_seen")
    if Xb.stride(2) != 1 or not Hb.is_contiguous() or not diag_key.is_contiguous():
        raise ValueError("X rows must be contiguous; H and diag_key contiguous")
    ws = _workspace(workspace_size(WS_HESSIAN, batch, 0, d_in, n), X.device, workspace)
    _check(lib().gptq_accumulate_hessian(batch, d_in, n, _DT[X.dtype], Xb.data_ptr(), Xb.stride(1),
                                         Xb.stride(0) if batch > 1 else n * Xb.stride(1), Hb.data_ptr(),
                                         d_in * d_in, diag_key.data_ptr(), n_seen.data_ptr(), ws.data_ptr(),
                                         ws.numel(), _stream()), "gptq_accumulate_hessian")


def accumulate_hessian_grouped(X: torch.Tensor, token_offsets: torch.Tensor, H: torch.Tensor, diag_key: torch.Tensor,
                               n_seen: torch.Tensor, max_tokens: int, workspace: torch.Tensor | None = None,
                               stream=None) -> None:
    """Per-problem token ranges of one buffer: problem e accumulates rows token_offsets[e] ..
    token_offsets[e + 1] - 1 of token-major X [total, d_in] (at most ``max_tokens`` rows each,
    the largest count the caller expects); n_seen[e] += the rows it took."""
    if stream is not None:
        return _on(stream, accumulate_hessian_grouped, X, token_offsets, H, diag_key, n_seen, max_tokens, workspace)
    total, d_in = X.shape
    batch = token_offsets.numel() - 1
    Hb = _batched(H, 2)
    if X.dtype not in _DT or H.dtype != torch.float32 or diag_key.dtype != torch.float64 or n_seen.dtype != torch.int64:
        raise TypeError("X must be fp32/bf16/fp16, H fp32, diag_key fp64, n_seen int64")
    if token_offsets.dtype != torch.int64 or not token_offsets.is_contiguous() or batch < 1:
        raise ValueError("token_offsets must be contiguous int64 [batch + 1]")
    if Hb.shape != (batch, d_in, d_in) or diag_key.numel() != batch * d_in or n_seen.numel() < batch:
        raise ValueError("shape mismatch between token_offsets, H, diag_key, n_seen")
    if X.stride(1) != 1 or not Hb.is_contiguous() or not diag_key.is_contiguous():
        raise ValueError("X rows must be contiguous; H and diag_key contiguous")
    ws = _workspace(workspace_size(WS_HESSIAN, batch, 0, d_in, max_tokens), X.device, workspace)
    _check(lib().gptq_accumulate_hessian_grouped(batch, d_in, total, max_tokens, _DT[X.dtype], X.data_ptr(),
                                                 X.stride(0), token_offsets.data_ptr(), Hb.data_ptr(), d_in * d_in,
                                                 diag_key.data_ptr(), n_seen.data_ptr(), ws.data_ptr(), ws.numel(),
                                                 _stream()), "gptq_accumulate_hessian_grouped")


class HessianHook:
    """Calibration hook on a ``torch.nn.Linear`` ("GPTQ Architecture, in depth", "The
    algorithm in code": a hook records each linear layer's inputs batch by batch): every
    forward call adds its input, flattened to token-major [tokens, in_features], to H,
    diag_key and n_seen on the stream the forward runs on.  ``remove()`` detaches it.

    H holds the unnormalised 2 sum x x^T (the running mean of the pages differs by 1/n, and
    the quantizer's results do not depend on that scale); one H serves every weight that
    reads the same input (e.g. the q, k and v projections)."""

    def __init__(self, module: torch.nn.Module, in_features: int | None = None, device=None):
        d_in = in_features if in_features is not None else module.in_features
        dev = device if device is not None else next(module.parameters()).device
        self.H, self.diag_key, self.n_seen = new_hessian(d_in, None, dev)
        self._handle = module.register_forward_pre_hook(self._hook)

    def _hook(self, module, args):
        x = args[0]
        accumulate_hessian(x.reshape(-1, x.shape[-1]), self.H, self.diag_key, self.n_seen)

    def remove(self) -> None:
        self._handle.remove()


def prepare_hinv(H: torch.Tensor, diag_key: torch.Tensor, params: Params, workspace: torch.Tensor | None = None,
                 stream=None):
    """-> (U fp32 [(batch,) d_in, d_in], perm int32 [(batch,) d_in], dead uint8 [(batch,) d_in]).
    Raises NotSPDError if the damped Hessian has no Cholesky factor."""
    if stream is not None:
        return _on(stream, prepare_hinv, H, diag_key, params, workspace)
    Hb = _batched(H, 2)
    batch, d_in, _ = Hb.shape
    if not Hb.is_contiguous() or not diag_key.is_contiguous():
        raise ValueError("H and diag_key must be contiguous")
    shp = H.shape[:-1]
    U = torch.empty(*H.shape, dtype=torch.float32, device=H.device)
    perm = torch.empty(*shp, dtype=torch.int32, device=H.device)
    dead = torch.empty(*shp, dtype=torch.uint8, device=H.device)
    ws = _workspace(workspace_size(WS_PREPARE, batch, 0, d_in, 0, params), H.device, workspace)
    p = params.c()
    _check(lib().gptq_prepare_hinv(batch, d_in, Hb.data_ptr(), d_in * d_in, diag_key.data_ptr(), ctypes.byref(p),
                                   U.data_ptr(), d_in * d_in, perm.data_ptr(), dead.data_ptr(), ws.data_ptr(),
                                   ws.numel(), _stream()), "gptq_prepare_hinv")
    return U, perm, dead


def quantize_layer(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, dead: torch.Tensor, params: Params,
                   workspace: torch.Tensor | None = None, stream=None):
    """-> (codes uint8 [(b,) d_out, d_in] original order, scales fp32 [(b,) n_groups, d_out],
    zeros uint8 [(b,) n_groups, d_out], g_idx int32 [(b,) d_in])."""
    if stream is not None:
        return _on(stream, quantize_layer, W, U, perm, dead, params, workspace)
    Wb = _batched(W, 2)
    batch, d_out, d_in = Wb.shape
    if W.dtype not in _DT:
        raise TypeError("W must be fp32/bf16/fp16")
    if Wb.stride(2) != 1 or not U.is_contiguous() or not perm.is_contiguous() or not dead.is_contiguous():
        raise ValueError("W rows, U, perm and dead must be contiguous")
    ng = params.n_groups(d_in)
    lead = W.shape[:-2]
    codes = torch.empty(*lead, d_out, d_in, dtype=torch.uint8, device=W.device)
    scales = torch.empty(*lead, ng, d_out, dtype=torch.float32, device=W.device)
    zeros = torch.empty(*lead, ng, d_out, dtype=torch.uint8, device=W.device)
    g_idx = torch.empty(*lead, d_in, dtype=torch.int32, device=W.device)
    ws = _workspace(workspace_size(WS_QUANTIZE, batch, d_out, d_in, 0, params), W.device, workspace)
    p = params.c()
    _check(lib().gptq_quantize_layer(batch, d_out, d_in, _DT[W.dtype], Wb.data_ptr(), Wb.stride(1),
                                     Wb.stride(0) if batch > 1 else d_out * Wb.stride(1), U.data_ptr(),
                                     d_in * d_in, perm.data_ptr(), dead.data_ptr(), ctypes.byref(p),
                                     codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), g_idx.data_ptr(),
                                     ws.data_ptr(), ws.numel(), _stream()), "gptq_quantize_layer")
    return codes, scales, zeros, g_idx


def quantize_layer_noalloc(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, dead: torch.Tensor, params: Params,
                           out=None, stream=None):
    """gptq_quantize_layer_noalloc: the same results as :func:`quantize_layer` with the
    library's fixed device scratch instead of a workspace.  ``out`` = (codes, scales,
    zeros, g_idx) preallocated by the caller (shapes as returned by quantize_layer);
    without it they are allocated here, but the C call itself never allocates."""
    if stream is not None:
        return _on(stream, quantize_layer_noalloc, W, U, perm, dead, params, out)
    Wb = _batched(W, 2)
    batch, d_out, d_in = Wb.shape
    if W.dtype not in _DT:
        raise TypeError("W must be fp32/bf16/fp16")
    if Wb.stride(2) != 1 or not U.is_contiguous() or not perm.is_contiguous() or not dead.is_contiguous():
        raise ValueError("W rows, U, perm and dead must be contiguous")
    ng = params.n_groups(d_in)
    lead = W.shape[:-2]
    if out is None:
        out = (torch.empty(*lead, d_out, d_in, dtype=torch.uint8, device=W.device),
               torch.empty(*lead, ng, d_out, dtype=torch.float32, device=W.device),
               torch.empty(*lead, ng, d_out, dtype=torch.uint8, device=W.device),
               torch.empty(*lead, d_in, dtype=torch.int32, device=W.device))
    codes, scales, zeros, g_idx = out
    want = [((*lead, d_out, d_in), torch.uint8), ((*lead, ng, d_out), torch.float32),
            ((*lead, ng, d_out), torch.uint8), ((*lead, d_in), torch.int32)]
    for t, (shape, dt) in zip(out, want):
        if tuple(t.shape) != tuple(shape) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"output tensor must be contiguous {dt} of shape {shape}")
    p = params.c()
    _check(lib().gptq_quantize_layer_noalloc(batch, d_out, d_in, _DT[W.dtype], Wb.data_ptr(), Wb.stride(1),
                                             Wb.stride(0) if batch > 1 else d_out * Wb.stride(1), U.data_ptr(),
                                             d_in * d_in, perm.data_ptr(), dead.data_ptr(), ctypes.byref(p),
                                             codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), g_idx.data_ptr(),
                                             _stream()), "gptq_quantize_layer_noalloc")
    return codes, scales, zeros, g_idx


def pack_int4(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, stream=None):
    """-> (qweight int32 [(b,) d_in/8, d_out], qzeros int32 [(b,) n_groups, d_out/8],
    scales fp16 [(b,) n_groups, d_out])."""
    if stream is not None:
        return _on(stream, pack_int4, codes, scales, zeros)
    cb = _batched(codes, 2)
    batch, d_out, d_in = cb.shape
    ng = scales.shape[-2]
    if not (codes.is_contiguous() and scales.is_contiguous() and zeros.is_contiguous()):
        raise ValueError("codes, scales and zeros must be contiguous")
    lead = codes.shape[:-2]
    qweight = torch.empty(*lead, d_in // 8, d_out, dtype=torch.int32, device=codes.device)
    qzeros = torch.empty(*lead, ng, d_out // 8, dtype=torch.int32, device=codes.device)
    sf16 = torch.empty(*lead, ng, d_out, dtype=torch.float16, device=codes.device)
    _check(lib().gptq_pack_int4(batch, d_out, d_in, ng, codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                qweight.data_ptr(), qzeros.data_ptr(), sf16.data_ptr(), _stream()),
           "gptq_pack_int4")
    return qweight, qzeros, sf16


TIME_SYRK, TIME_LAZY_GEMM, TIME_SWEEP, TIME_PACK, TIME_W4A16 = 0, 1, 2, 3, 4


def w4a16_repack(qweight: torch.Tensor, g_idx: torch.Tensor, n_groups: int, workspace: torch.Tensor | None = None,
                 stream=None):
    """Serving layout of a packed layer: (qweight_s int32 [(b,) d_in/8, d_out], order int32
    [(b,) d_in]) with the inputs sorted by group.  Raises GptqError on a malformed g_idx."""
    if stream is not None:
        return _on(stream, w4a16_repack, qweight, g_idx, n_groups, workspace)
    qb = _batched(qweight, 2)
    batch, rows8, d_out = qb.shape
    d_in = rows8 * 8
    if qweight.dtype != torch.int32 or g_idx.dtype != torch.int32 or g_idx.numel() != batch * d_in:
        raise TypeError("qweight and g_idx must be int32, g_idx [(b,) d_in]")
    if not qweight.is_contiguous() or not g_idx.is_contiguous():
        raise ValueError("qweight and g_idx must be contiguous")
    qs = torch.empty_like(qweight)
    order = torch.empty_like(g_idx)
    ws = _workspace(workspace_size(WS_W4A16_REPACK, batch, d_out, d_in), qweight.device, workspace)
    _check(lib().gptq_w4a16_repack(batch, d_out, d_in, n_groups, qweight.data_ptr(), g_idx.data_ptr(), qs.data_ptr(),
                                   order.data_ptr(), ws.data_ptr(), ws.numel(), _stream()), "gptq_w4a16_repack")
    return qs, order


def w4a16_matmul(X: torch.Tensor, qweight_s: torch.Tensor, qzeros: torch.Tensor, scales_f16: torch.Tensor,
                 order: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y fp32 [m, d_out] = X What^T from the packed tensors (X [m, d_in] bf16 / fp16).
    ``order`` from :func:`w4a16_repack`, or None when qweight is in input order with
    contiguous groups."""
    if stream is not None:
        return _on(stream, w4a16_matmul, X, qweight_s, qzeros, scales_f16, order, out, workspace)
    m, d_in = X.shape
    d_out = qweight_s.shape[-1]
    n_groups = scales_f16.shape[0]
    if X.dtype not in (torch.bfloat16, torch.float16) or X.stride(1) != 1:
        raise TypeError("X must be bf16 or fp16 with contiguous rows")
    if qweight_s.dtype != torch.int32 or qzeros.dtype != torch.int32 or scales_f16.dtype != torch.float16:
        raise TypeError("qweight and qzeros int32, scales fp16")
    if not (qweight_s.is_contiguous() and qzeros.is_contiguous() and scales_f16.is_contiguous()):
        raise ValueError("packed tensors must be contiguous")
    if order is not None and (order.dtype != torch.int32 or order.numel() != d_in or not order.is_contiguous()):
        raise ValueError("order must be contiguous int32 [d_in]")
    Y = out if out is not None else torch.empty(m, d_out, dtype=torch.float32, device=X.device)
    gsz = -1 if n_groups == 1 else d_in // n_groups
    ws = _workspace(workspace_size(WS_W4A16, 1, d_out, d_in, m, Params(group_size=gsz)), X.device, workspace)
    _check(lib().gptq_w4a16_matmul(m, d_out, d_in, n_groups, _DT[X.dtype], X.data_ptr(), X.stride(0),
                                   qweight_s.data_ptr(), None if order is None else order.data_ptr(), qzeros.data_ptr(),
                                   scales_f16.data_ptr(), Y.data_ptr(), Y.stride(0), ws.data_ptr(), ws.numel(),
                                   _stream()), "gptq_w4a16_matmul")
    return Y


E4M3, E8M0 = 3, 4
_SDT = {torch.float32: 0, torch.float8_e8m0fnu: E8M0}
_FP8_BLOCK = 128


def _run(what: str, tensors, *args) -> None:
    """The library's call ``what`` with ``args`` and a stream handle, for tensors (or None) of
    one GPU, with that GPU as the current device, on its current stream.  The first of
    ``tensors`` is not None.  Small calls last a few microseconds, so this path creates no Stream
    object (2.8 us of a 12.9 us call)."""
    device = tensors[0].get_device()
    if device < 0:
        raise ValueError("tensors must be on a GPU")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors must be on one GPU")
    fn = getattr(_lib or lib(), what)
    if device == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream())
    if status != GPTQ_OK:
        _check(status, what)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(which: int, batch: int, d_out: int, d_in: int, hint: int) -> int:
    return workspace_size(which, batch, d_out, d_in, hint)


def _scratch(which, batch, d_out, d_in, hint, device, workspace) -> torch.Tensor | None:
    """The caller's workspace if it is large enough, else a new one; None where the call needs none."""
    nbytes = _workspace_bytes(which, batch, d_out, d_in, hint)
    if nbytes <= 256:   # the size of a workspace that nothing is kept in
        return None
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if _bytes(workspace) >= nbytes:
            return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


@functools.lru_cache(maxsize=256)
def _route_params(*values) -> _RouteParams:
    return _RouteParams(*values)


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.stride(-1) != 1 or (
            len(shape) > 1 and shape[0] > 1 and out.stride(0) < shape[-1]):
        raise ValueError(f"out must be {dtype} of shape {tuple(shape)} with contiguous rows")
    return out


def _row_stride(t: torch.Tensor) -> int:
    """Elements between rows; the row length where there is one row (its stride says nothing)."""
    rows, cols = t.shape[-2:]
    return t.stride()[-2] if rows > 1 else cols


def fp8_quantize(X: torch.Tensor, block_rows: int = 1, scale_dtype: torch.dtype = torch.float32, stream=None):
    """-> (q float8_e4m3fn of X's shape, scales [(b,) ceil(rows / block_rows), ceil(cols / 128)]):
    X [(b,) rows, cols] fp32/bf16/fp16 in blocks of block_rows x 128, q = X / scale rounded to
    nearest even, scale = max|X| / 448 (fp32) or the power of two at or above it
    (``scale_dtype`` float8_e8m0fnu).  block_rows 1 for activations, 128 for weights.  The
    scales of activations are stored block by block (stride 1 along the rows), as the products
    read them."""
    if stream is not None:
        return _on(stream, fp8_quantize, X, block_rows, scale_dtype)
    if X.dtype not in _DT or scale_dtype not in _SDT:
        raise TypeError("X must be fp32/bf16/fp16, scale_dtype float32 or float8_e8m0fnu")
    if block_rows not in (1, _FP8_BLOCK) or X.dim() not in (2, 3):
        raise ValueError("X must be [(batch,) rows, cols], block_rows 1 or 128")
    Xb = _batched(X, 2)
    batch, rows, cols = Xb.shape
    if cols < 16 or cols % 16 or batch < 1:
        raise ValueError("cols must be a positive multiple of 16")
    if Xb.stride(2) != 1:
        raise ValueError("X rows must be contiguous")
    rb, cb = -(-rows // block_rows), -(-cols // _FP8_BLOCK)
    ld_row, ld_block = (1, max(rb, 1)) if block_rows == 1 else (cb, 1)
    q = torch.empty(X.shape, dtype=torch.float8_e4m3fn, device=X.device)
    if X.dim() == 2:
        S = torch.empty_strided((rb, cb), (ld_row, ld_block), dtype=scale_dtype, device=X.device)
    else:
        S = torch.empty_strided((batch, rb, cb), (rb * cb, ld_row, ld_block), dtype=scale_dtype, device=X.device)
    _run("gptq_fp8_quantize", (X, q, S), batch, rows, cols, _DT[X.dtype], X.data_ptr(), _row_stride(Xb),
         Xb.stride(0), block_rows, _SDT[scale_dtype], q.data_ptr(), S.data_ptr(), ld_row, ld_block, rb * cb)
    return q, S


def _fp8_operands(X, x_scales, qweight, w_scales, out_dtype):
    """Checks shared by the dense and the grouped product; -> the scales' type code."""
    if qweight.dtype != torch.float8_e4m3fn or w_scales.dtype not in _SDT or out_dtype not in _DT:
        raise TypeError("qweight must be float8_e4m3fn, scales fp32 or float8_e8m0fnu, out_dtype fp32/bf16/fp16")
    d_out, d_in = qweight.shape[-2:]
    blocks = -(-d_in // _FP8_BLOCK)
    if d_in < 16 or d_in % 16 or d_out < 1:
        raise ValueError("d_in must be a positive multiple of 16")
    if X.dim() != 2 or X.shape[1] != d_in or X.stride(1) != 1:
        raise ValueError("X must be [rows, d_in] with contiguous rows")
    if w_scales.shape != (*qweight.shape[:-2], -(-d_out // _FP8_BLOCK), blocks):
        raise ValueError("w_scales must be [(batch,) ceil(d_out / 128), ceil(d_in / 128)]")
    if not (qweight.is_contiguous() and w_scales.is_contiguous()):
        raise ValueError("qweight and w_scales must be contiguous")
    if X.dtype == torch.float8_e4m3fn:
        if x_scales is None or x_scales.dtype != w_scales.dtype:
            raise TypeError("x_scales must come with float8_e4m3fn X, of the type of w_scales")
        if x_scales.shape != (X.shape[0], blocks):
            raise ValueError("x_scales must be [rows, ceil(d_in / 128)]")
        if x_scales.numel() and (x_scales.stride(0) < 1 or x_scales.stride(1) < 1):
            raise ValueError("x_scales must not be an expanded tensor")
    elif X.dtype in (torch.bfloat16, torch.float16):
        if x_scales is not None:
            raise TypeError("x_scales belong to float8_e4m3fn X")
    else:
        raise TypeError("X must be float8_e4m3fn, bf16 or fp16")
    return _SDT[w_scales.dtype]


def _fp8_scales(x_scales):
    """Pointer and strides of the scales of 8-bit activations."""
    if x_scales is None:
        return None, 0, 0
    sr, sb = x_scales.stride()
    return x_scales.data_ptr(), max(sr, 1), max(sb, 1)


def fp8_matmul(X: torch.Tensor, qweight: torch.Tensor, w_scales: torch.Tensor, x_scales: torch.Tensor | None = None,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, d_out] = X What^T with e4m3 weights [d_out, d_in] and the scales of their 128 x 128
    blocks (:func:`fp8_quantize` with block_rows 128).  X [m, d_in] is float8_e4m3fn with
    ``x_scales`` [m, ceil(d_in / 128)], or bf16 / fp16, then rounded first as
    :func:`fp8_quantize` does.  ``out_dtype`` float32 has fp32 sums; for 16-bit types the 8-bit
    matrix instructions cut products at 2^-13 of the largest of 8, which fp16 can show."""
    if stream is not None:
        return _on(stream, fp8_matmul, X, qweight, w_scales, x_scales, out_dtype, out, workspace)
    if qweight.dim() != 2:
        raise ValueError("qweight must be [d_out, d_in]")
    sdt = _fp8_operands(X, x_scales, qweight, w_scales, out_dtype)
    (m, d_in), d_out = X.shape, qweight.shape[0]
    Y = _out(out, (m, d_out), out_dtype, X.device)
    ws = None if X.dtype == torch.float8_e4m3fn else _scratch(WS_FP8_MATMUL, 1, d_out, d_in, m, X.device, workspace)
    _run("gptq_fp8_matmul", (X, qweight, w_scales, x_scales, Y, ws), m, d_out, d_in, _DT.get(X.dtype, E4M3),
         X.data_ptr(), _row_stride(X), sdt, *_fp8_scales(x_scales), qweight.data_ptr(), w_scales.data_ptr(),
         _DT[out_dtype], Y.data_ptr(), _row_stride(Y), _ptr(ws),
         _bytes(ws))
    return Y


def fp8_matmul_grouped(X: torch.Tensor, qweight: torch.Tensor, w_scales: torch.Tensor, token_offsets: torch.Tensor,
                       row_index: torch.Tensor | None = None, x_scales: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts' products: row p of Y [n_rows, d_out], token_offsets[e] <= p <
    token_offsets[e + 1], is row row_index[p] of X (row p without ``row_index``) times
    expert e's weights qweight [experts, d_out, d_in]; operands otherwise as in
    :func:`fp8_matmul`.  ``token_offsets`` int64 [experts + 1] and ``row_index`` int32 [n_rows]
    come from :func:`moe_group_tokens`.  Rows outside every range are not written."""
    if stream is not None:
        return _on(stream, fp8_matmul_grouped, X, qweight, w_scales, token_offsets, row_index, x_scales,
                   out_dtype, out, workspace)
    if qweight.dim() != 3 or qweight.shape[0] < 1:
        raise ValueError("qweight must be [experts, d_out, d_in]")
    sdt = _fp8_operands(X, x_scales, qweight, w_scales, out_dtype)
    (x_rows, d_in), (experts, d_out) = X.shape, qweight.shape[:2]
    if token_offsets.dtype != torch.int64 or not token_offsets.is_contiguous() or token_offsets.shape != (experts + 1,):
        raise ValueError("token_offsets must be contiguous int64 [experts + 1]")
    if row_index is not None and (row_index.dtype != torch.int32 or row_index.dim() != 1 or
                                  not row_index.is_contiguous()):
        raise ValueError("row_index must be contiguous int32 [n_rows]")
    n_rows = x_rows if row_index is None else row_index.numel()
    Y = _out(out, (n_rows, d_out), out_dtype, X.device)
    ws = None if X.dtype == torch.float8_e4m3fn else _scratch(WS_FP8_GROUPED, experts, d_out, d_in, x_rows, X.device,
                                                              workspace)
    _run("gptq_fp8_matmul_grouped", (X, qweight, w_scales, token_offsets, row_index, x_scales, Y, ws), experts,
         x_rows, n_rows, d_out, d_in, _DT.get(X.dtype, E4M3), X.data_ptr(), _row_stride(X), sdt,
         *_fp8_scales(x_scales), qweight.data_ptr(), w_scales.data_ptr(), token_offsets.data_ptr(),
         _ptr(row_index), _DT[out_dtype], Y.data_ptr(), _row_stride(Y),
         _ptr(ws), _bytes(ws))
    return Y


_SCORING, _GROUP_SCORE = {"softmax": 0, "sigmoid": 1}, {"max": 0, "top2": 1}


def moe_route(logits: torch.Tensor, top_k: int, bias: torch.Tensor | None = None, scoring: str = "softmax",
              n_groups: int = 1, top_groups: int | None = None, group_score: str = "max", renormalize: bool = True,
              scale: float = 1.0, stream=None):
    """-> (ids int32 [tokens, top_k], weights fp32 [tokens, top_k]) from router logits [tokens,
    experts] (fp32/bf16/fp16): the ``top_k`` largest of softmax or sigmoid scores + ``bias``
    (fp32 [experts]) among the experts of the ``top_groups`` best of ``n_groups`` groups
    (ranked by their best choice value or the sum of their two best), in descending order,
    equal values by index; weights are ``scale`` times the scores without bias, divided by
    their sum with ``renormalize``.  Logits or biases of -inf or NaN take an expert out; ids
    are -1 (weight 0) where none is left."""
    if stream is not None:
        return _on(stream, moe_route, logits, top_k, bias, scoring, n_groups, top_groups, group_score,
                   renormalize, scale)
    if logits.dtype not in _DT or (bias is not None and bias.dtype != torch.float32):
        raise TypeError("logits must be fp32/bf16/fp16, bias fp32")
    if logits.dim() != 2 or logits.shape[1] < 1 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [tokens, experts] with contiguous rows")
    tokens, experts = logits.shape
    if bias is not None and (bias.shape != (experts,) or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous [experts]")
    if scoring not in _SCORING or group_score not in _GROUP_SCORE:
        raise ValueError("scoring must be 'softmax' or 'sigmoid', group_score 'max' or 'top2'")
    p = _route_params(_SCORING[scoring], n_groups, n_groups if top_groups is None else top_groups,
                      _GROUP_SCORE[group_score], top_k, int(renormalize), scale)
    ids = torch.empty((tokens, max(top_k, 0)), dtype=torch.int32, device=logits.device)
    weights = torch.empty_like(ids, dtype=torch.float32)
    _run("gptq_moe_route", (logits, bias, ids, weights), tokens, experts, _DT[logits.dtype], logits.data_ptr(),
         _row_stride(logits), _ptr(bias), ctypes.byref(p), ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_group_tokens(ids: torch.Tensor, n_experts: int, workspace: torch.Tensor | None = None, stream=None):
    """-> (token_offsets int64 [n_experts + 1], row_index int32 [tokens * top_k], place int32
    [tokens, top_k]): the choices ids [tokens, top_k] sorted by expert, in token order inside an
    expert.  ``token_offsets`` are the experts' ranges that accumulate_hessian_grouped and
    fp8_matmul_grouped take, ``row_index`` the token at each position (-1 behind the last
    range), ``place`` the position of each choice (-1 for an id outside [0, n_experts))."""
    if stream is not None:
        return _on(stream, moe_group_tokens, ids, n_experts, workspace)
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 2 or not ids.is_contiguous() or ids.shape[1] < 1 or not 1 <= n_experts <= 1024:
        raise ValueError("ids must be contiguous [tokens, top_k], n_experts 1..1024")
    tokens, k = ids.shape
    offsets = torch.empty(n_experts + 1, dtype=torch.int64, device=ids.device)
    rows = torch.empty(tokens * k, dtype=torch.int32, device=ids.device)
    place = torch.empty_like(ids)
    ws = _scratch(WS_MOE_GROUP, 1, n_experts, k, tokens, ids.device, workspace)
    _run("gptq_moe_group_tokens", (ids, offsets, rows, place, ws), tokens, k, n_experts, ids.data_ptr(),
         offsets.data_ptr(), rows.data_ptr(), place.data_ptr(), _ptr(ws), _bytes(ws))
    return offsets, rows, place


def moe_combine(Y: torch.Tensor, place: torch.Tensor, weights: torch.Tensor, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """out [tokens, d] (Y's type) = sum over j of weights[:, j] * Y[place[:, j]]: every token's
    expert outputs, summed in fp32 in the order of its choices; a place outside Y adds
    nothing."""
    if stream is not None:
        return _on(stream, moe_combine, Y, place, weights, out)
    if Y.dtype not in _DT or place.dtype != torch.int32 or weights.dtype != torch.float32:
        raise TypeError("Y must be fp32/bf16/fp16, place int32, weights fp32")
    if Y.dim() != 2 or Y.shape[1] < 1 or Y.stride(1) != 1:
        raise ValueError("Y must be [rows, d] with contiguous rows")
    if place.dim() != 2 or place.shape[1] < 1 or weights.shape != place.shape or not (
            place.is_contiguous() and weights.is_contiguous()):
        raise ValueError("place and weights must be contiguous [tokens, top_k]")
    (tokens, k), (rows, d) = place.shape, Y.shape
    res = _out(out, (tokens, d), Y.dtype, Y.device)
    _run("gptq_moe_combine", (Y, place, weights, res), tokens, k, rows, d, _DT[Y.dtype], Y.data_ptr(),
         _row_stride(Y), place.data_ptr(), weights.data_ptr(), res.data_ptr(), _row_stride(res))
    return res


def timing_enable(on: bool = True, kinds=None) -> None:
    """Start/stop recording HIP events around the launches of the timed kernel classes
    (``kinds``: an iterable of TIME_* values, all of them when None)."""
    mask = 0
    if on:
        mask = -1 if kinds is None else sum(1 << k for k in set(kinds))
    _check(lib().gptq_timing_enable(mask), "gptq_timing_enable")


def timing_read(which: int = TIME_SYRK):
    """(summed kernel milliseconds, launches) of one timed class since its previous read."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
    _check(lib().gptq_timing_read(which, ctypes.byref(ms), ctypes.byref(n)), "gptq_timing_read")
    return ms.value, n.value


def gptq_layer(W: torch.Tensor, X_chunks, params: Params, stream=None):
    """Whole layer: accumulate H over the chunks (taken from X_chunks with ``stream`` as the current
    one), prepare U, quantize.  Returns a dict."""
    if stream is not None:
        return _on(stream, gptq_layer, W, X_chunks, params)
    lead = W.shape[:-2]
    d_in = W.shape[-1]
    H, key, n = new_hessian(d_in, lead[0] if lead else None, W.device)
    for Xc in X_chunks:
        accumulate_hessian(Xc, H, key, n)
    U, perm, dead = prepare_hinv(H, key, params)
    codes, scales, zeros, g_idx = quantize_layer(W, U, perm, dead, params)
    return dict(H=H, diag_key=key, n_seen=n, U=U, perm=perm, dead=dead, codes=codes, scales=scales,
                zeros=zeros, g_idx=g_idx)
