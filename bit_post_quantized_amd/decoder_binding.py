"""ctypes binding of include/svdq_decoder.h, with the same function names, in the manner of
``serve_binding``: every function checks its device tensors (dtype, shape, device, size), passes
their pointers, the sizes and a HIP stream to the library and raises ``SvdqError`` on a nonzero
status.  ``decoder`` holds the objects a serving program keeps.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import binding
from .binding import SVDQ_OUT_BF16, SVDQ_OUT_FP32, _Args, _out_dtype
from .serve_binding import _OnDevice

_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGNATURES = {
    "svdq_decoder_version": ([], _I),
    "svdq_rms_norm": ([_P, _I, _L, _P, _I, _P, _P, _I, _I, _F, _P, _P, _P, _P], _I),
    "svdq_quantize_rows": ([_P, _I, _L, _P, _I, _I, _P, _P, _P], _I),
    "svdq_w8a8_container_bytes": ([_I, _I], _Z),
    "svdq_pack_w8a8": ([_P, _I, _I, _P, _P], _I),
    "svdq_w8a8_workspace_bytes": ([_I, _I, _I], _Z),
    "svdq_w8a8_gemm": ([_P] * 5 + [_I] * 3 + [_P, _I, _P, _P], _I),
    "svdq_rope": ([_P, _L, _I, _P, _L] + [_I] * 6 + [_P, _P, _F, _P, _L, _P, _L, _P], _I),
    "svdq_sample_workspace_bytes": ([_I, _I], _Z),
    "svdq_sample": ([_P, _I, _L, _I, _I] + [_P] * 9, _I),
}
EXPORTED = tuple(_SIGNATURES)

_BF16, _F32, _F64 = torch.bfloat16, torch.float32, torch.float64
_I8, _I32 = torch.int8, torch.int32

_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """The built library with this header's functions declared (``binding.load``)."""
    global _lib
    if _lib is None:
        lib = binding.load()
        for name, (argtypes, restype) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = lib
    return _lib


def _call(fn: str, a: _Args, args, stream) -> None:
    for kind, v in zip(_SIGNATURES[fn][0], args):
        if kind is _I and not -1 << 31 <= v < 1 << 31:  # (ctypes would drop the upper bits)
            raise ValueError(f"{fn}: {v} does not fit 32 bits")
    with _OnDevice(a.device):
        status = getattr(load(), fn)(*args, a.stream(stream))
    binding._check(fn, status)


def _dtype(fn: str, t: torch.Tensor, name: str) -> int:
    if t.dtype == _F32:
        return SVDQ_OUT_FP32
    if t.dtype == _BF16:
        return SVDQ_OUT_BF16
    raise ValueError(f"{fn}: {name} must be bfloat16 or float32 (got {t.dtype})")


def _strided(a: _Args, t: torch.Tensor, name: str, inner: tuple) -> tuple:
    """A [rows, *inner] tensor whose rows are contiguous and may stand apart: (pointer, row stride)."""
    size, want = 1, []
    for n in reversed(inner):
        want.insert(0, size)
        size *= n
    got = t.stride()[1:]
    if tuple(t.shape[1:]) != tuple(inner) or any(n > 1 and g != w for n, g, w in zip(inner, got, want)):
        raise ValueError(f"{a.fn}: {name} must be [rows, {', '.join(map(str, inner))}] with contiguous rows "
                         f"(got {tuple(t.shape)}, strides {tuple(t.stride())})")
    if not t.is_cuda:
        raise ValueError(f"{a.fn}: {name} must be a device tensor")
    if a.device is None:
        a.device = t.device
    elif t.device != a.device:
        raise ValueError(f"{a.fn}: {name} is on {t.device}, other arguments on {a.device}")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else size


def svdq_decoder_version() -> int:
    return load().svdq_decoder_version()


def svdq_rms_norm(x: torch.Tensor, residual: Optional[torch.Tensor], residual_out: Optional[torch.Tensor],
                  gamma: Optional[torch.Tensor], eps: float, y: Optional[torch.Tensor],
                  codes: Optional[torch.Tensor], scales: Optional[torch.Tensor], stream=None) -> None:
    """x bf16 or fp32 [M, K] (rows may stand apart), residual bf16 or fp32 [M, K], gamma fp32 [K] ->
    residual_out (of residual's dtype), y bf16 [M, K], codes int8 [M, K] with scales fp32 [M]."""
    fn = "svdq_rms_norm"
    a = _Args(fn)
    M, K = x.shape
    xp, xs = _strided(a, x, "x", (K,))
    kind = SVDQ_OUT_BF16 if residual is None else _dtype(fn, residual, "residual")
    size = 4 if kind == SVDQ_OUT_FP32 else 2
    stream_dtype = None if residual is None else residual.dtype
    args = (xp, _dtype(fn, x, "x"), xs, a(residual, size * M * K, "residual", None, (M, K)), kind,
            a(residual_out, size * M * K, "residual_out", stream_dtype, (M, K)),
            a(gamma, 4 * K, "gamma", _F32, (K,)), M, K, float(eps), a(y, 2 * M * K, "y", _BF16, (M, K)),
            a(codes, M * K, "codes", _I8, (M, K)), a(scales, 4 * M, "scales", _F32, (M,)))
    _call(fn, a, args, stream)


def svdq_quantize_rows(x: torch.Tensor, factor: Optional[torch.Tensor], codes: torch.Tensor,
                       scales: torch.Tensor, stream=None) -> None:
    """x bf16 or fp32 [M, K] (rows may stand apart), factor fp32 [K] -> codes int8 [M, K], scales
    fp32 [M]."""
    fn = "svdq_quantize_rows"
    a = _Args(fn)
    M, K = x.shape
    xp, xs = _strided(a, x, "x", (K,))
    args = (xp, _dtype(fn, x, "x"), xs, a(factor, 4 * K, "factor", _F32, (K,)), M, K,
            a(codes, M * K, "codes", _I8, (M, K)), a(scales, 4 * M, "scales", _F32, (M,)))
    _call(fn, a, args, stream)


def svdq_w8a8_container_bytes(N: int, K: int) -> int:
    """Bytes of svdq_w8a8_gemm's weight container for N columns of K codes."""
    return load().svdq_w8a8_container_bytes(N, K)


def svdq_pack_w8a8(codes: torch.Tensor, container: torch.Tensor, stream=None) -> None:
    """codes int8 [N, K] -> container int8 [svdq_w8a8_container_bytes(N, K)]."""
    fn = "svdq_pack_w8a8"
    N, K = codes.shape
    a = _Args(fn)
    args = (a(codes, N * K, "codes", _I8), N, K,
            a(container, svdq_w8a8_container_bytes(N, K), "container", _I8))
    _call(fn, a, args, stream)


@functools.lru_cache(maxsize=4096)
def svdq_w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().svdq_w8a8_workspace_bytes(M, N, K)


def svdq_w8a8_gemm(qx: torch.Tensor, sx: torch.Tensor, container: torch.Tensor, sw: torch.Tensor,
                   bias: Optional[torch.Tensor], Y: torch.Tensor, workspace: Optional[torch.Tensor],
                   stream=None) -> None:
    """qx int8 [M, K], sx fp32 [M], container (from svdq_pack_w8a8), sw fp32 [N], bias bf16 [N] ->
    Y [M, N], bf16 or fp32."""
    fn = "svdq_w8a8_gemm"
    M, K = qx.shape
    N = Y.shape[1]
    out = _out_dtype(fn, Y)
    a = _Args(fn)
    args = (a(qx, M * K, "qx", _I8), a(sx, 4 * M, "sx", _F32, (M,)),
            a(container, svdq_w8a8_container_bytes(N, K), "container", _I8), a(sw, 4 * N, "sw", _F32, (N,)),
            a(bias, 2 * N, "bias", _BF16, (N,)), M, N, K, a(Y, Y.element_size() * M * N, "Y", None, (M, N)),
            out, a(workspace, svdq_w8a8_workspace_bytes(M, N, K), "workspace"))
    _call(fn, a, args, stream)


def svdq_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
              interleaved: bool, scale: float, q_out: torch.Tensor, k_out: Optional[torch.Tensor],
              stream=None) -> None:
    """q [rows, heads, dim] and k [rows, kv_heads, dim] bf16 or fp32 (rows may stand apart),
    positions int32 [rows], freqs fp64 [rot_dim / 2] -> q_out, k_out bf16 (rows may stand apart)."""
    fn = "svdq_rope"
    a = _Args(fn)
    rows, heads, dim = q.shape
    qp, qs = _strided(a, q, "q", (heads, dim))
    qop, qos = _strided(a, q_out, "q_out", (heads, dim))
    kp = kop = None
    kv = ks = kos = 0
    outs = [("q_out", q_out)]
    if k is None and k_out is not None:
        raise ValueError(f"{fn}: k_out needs k")
    if k is not None:
        if k_out is None:
            raise ValueError(f"{fn}: k needs k_out")
        kv = k.shape[1]
        kp, ks = _strided(a, k, "k", (kv, dim))
        kop, kos = _strided(a, k_out, "k_out", (kv, dim))
        outs.append(("k_out", k_out))
        if k.dtype != q.dtype:
            raise ValueError(f"{fn}: q and k must have the same dtype (got {q.dtype}, {k.dtype})")
        if k.shape[0] != rows:
            raise ValueError(f"{fn}: q and k must have the same rows (got {rows}, {k.shape[0]})")
    for name, t in outs:
        if t.dtype != _BF16:
            raise ValueError(f"{fn}: {name} must be {_BF16} (got {t.dtype})")
        if t.shape[0] != rows:
            raise ValueError(f"{fn}: {name} must have {rows} rows (got {t.shape[0]})")
    args = (qp, qs, heads, kp, ks, kv, _dtype(fn, q, "q"), rows, dim, 2 * freqs.shape[0], int(interleaved),
            a(positions, 4 * rows, "positions", _I32, (rows,)), a(freqs, 8 * freqs.shape[0], "freqs", _F64),
            float(scale), qop, qos, kop, kos)
    _call(fn, a, args, stream)


@functools.lru_cache(maxsize=4096)
def svdq_sample_workspace_bytes(rows: int, vocab: int) -> int:
    return load().svdq_sample_workspace_bytes(rows, vocab)


def svdq_sample(logits: torch.Tensor, temperature: torch.Tensor, uniform: torch.Tensor,
                top_k: Optional[torch.Tensor], top_p: Optional[torch.Tensor], min_p: Optional[torch.Tensor],
                tokens: torch.Tensor, share: Optional[torch.Tensor], workspace: torch.Tensor,
                stream=None) -> None:
    """logits bf16 or fp32 [rows, vocab] (rows may stand apart), temperature and uniform fp32 [rows],
    top_k int32 [rows], top_p and min_p fp32 [rows] -> tokens int32 [rows], share fp32 [rows]."""
    fn = "svdq_sample"
    a = _Args(fn)
    rows, vocab = logits.shape
    p, stride = _strided(a, logits, "logits", (vocab,))
    args = (p, _dtype(fn, logits, "logits"), stride, rows, vocab,
            a(temperature, 4 * rows, "temperature", _F32, (rows,)), a(uniform, 4 * rows, "uniform", _F32, (rows,)),
            a(top_k, 4 * rows, "top_k", _I32, (rows,)), a(top_p, 4 * rows, "top_p", _F32, (rows,)),
            a(min_p, 4 * rows, "min_p", _F32, (rows,)), a(tokens, 4 * rows, "tokens", _I32, (rows,)),
            a(share, 4 * rows, "share", _F32, (rows,)),
            a(workspace, svdq_sample_workspace_bytes(rows, vocab), "workspace"))
    _call(fn, a, args, stream)
