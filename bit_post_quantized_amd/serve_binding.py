"""ctypes binding of the decoding step's C ABI (include/svdq_serve.h), with the same function
names, in the manner of ``binding``: every function checks its device tensors (dtype, shape,
device, size), passes their pointers, the sizes and a HIP stream to the library and raises
``SvdqError`` on a nonzero status.  ``serve`` holds the objects a serving program keeps.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import binding
from .binding import SVDQ_OUT_BF16, SVDQ_OUT_FP32, _Args, _out_dtype

_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGNATURES = {
    "svdq_serve_version": ([], _I),
    "svdq_w4a16_container_bytes": ([_I, _I], _Z),
    "svdq_pack_w4a16": ([_P, _P, _I, _I, _P, _P], _I),
    "svdq_w4a16_workspace_bytes": ([_I] * 5, _Z),
    "svdq_w4a16_gemv": ([_P] * 6 + [_I] * 4 + [_P, _I, _P, _P], _I),
    "kv_block_plan": ([_P, _P, _I, _P, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P], _I),
    "kv_block_release": ([_P, _P, _I, _P, _I, _I, _P, _I, _P, _P, _P, _P], _I),
    "kv_block_append": ([_P, _P, _L, _L, _P] + [_I] * 5 + [_P] * 5, _I),
    "kv_block_read": ([_P] + [_I] * 5 + [_P] * 7, _I),
    "kv_block_attention_workspace_bytes": ([_I] * 8, _Z),
    "kv_block_attention": ([_P, _L, _P, _P, _P, _P, _P, _I, _P, _P] + [_I] * 9 + [_F, _P, _P, _P],
                           _I),
}
EXPORTED = tuple(_SIGNATURES)

_BF16, _F32, _F16 = torch.bfloat16, torch.float32, torch.float16
_U8, _I32, _I64 = torch.uint8, torch.int32, torch.int64

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


class _OnDevice:
    """The device that a call's tensors are on is made the current one for the launch."""

    def __init__(self, device: Optional[torch.device]):
        self._other = None
        if device is not None and device.index is not None and torch.cuda.is_available() \
                and device.index != torch.cuda.current_device():
            self._other = torch.cuda.device(device)

    def __enter__(self):
        if self._other is not None:
            self._other.__enter__()

    def __exit__(self, *exc):
        if self._other is not None:
            self._other.__exit__(*exc)


def _call(fn: str, a: _Args, args, stream) -> None:
    for kind, v in zip(_SIGNATURES[fn][0], args):
        if kind is _I and not -1 << 31 <= v < 1 << 31:  # (ctypes would drop the upper bits)
            raise ValueError(f"{fn}: {v} does not fit 32 bits")
    with _OnDevice(a.device):
        status = getattr(load(), fn)(*args, a.stream(stream))
    binding._check(fn, status)


def svdq_serve_version() -> int:
    return load().svdq_serve_version()


@functools.lru_cache(maxsize=1024)
def svdq_w4a16_workspace_bytes(M: int, N: int, K: int, r: int, out_dtype: int) -> int:
    return load().svdq_w4a16_workspace_bytes(M, N, K, r, out_dtype)


def svdq_w4a16_container_bytes(N: int, K: int) -> int:
    """Bytes of svdq_w4a16_gemv's weight container for N columns of K codes."""
    return load().svdq_w4a16_container_bytes(N, K)


def svdq_pack_w4a16(wq: torch.Tensor, w_scales: torch.Tensor, container: torch.Tensor,
                    stream=None) -> None:
    """wq uint8 [N, K/2], w_scales fp16 [K/64, N] (from svdq_pack_weights) -> container uint8
    [svdq_w4a16_container_bytes(N, K)]."""
    fn = "svdq_pack_w4a16"
    N, half_k = wq.shape
    K = 2 * half_k
    a = _Args(fn)
    args = (a(wq, N * half_k, "wq", _U8), a(w_scales, 2 * (K // 64) * N, "w_scales", _F16, (K // 64, N)),
            N, K, a(container, svdq_w4a16_container_bytes(N, K), "container", _U8))
    _call(fn, a, args, stream)


def svdq_w4a16_gemv(X: torch.Tensor, inv_lambda: torch.Tensor, L1p: Optional[torch.Tensor],
                    container: torch.Tensor, L2p: Optional[torch.Tensor],
                    bias: Optional[torch.Tensor], r: int, Y: torch.Tensor,
                    workspace: Optional[torch.Tensor], stream=None) -> None:
    """X bf16 [M, K] (M <= 64), inv_lambda fp32 [K], L1p bf16 [r, K], container (from
    svdq_pack_w4a16), L2p bf16 [N, r], bias bf16 [N] -> Y [M, N], bf16 or fp32."""
    fn = "svdq_w4a16_gemv"
    M, K = X.shape
    N = Y.shape[1]
    out = _out_dtype(fn, Y)
    need = svdq_w4a16_workspace_bytes(M, N, K, r, out)
    a = _Args(fn)
    args = (a(X, 2 * M * K, "X", _BF16, (M, K)), a(inv_lambda, 4 * K, "inv_lambda", _F32, (K,)),
            a(L1p, 2 * r * K, "L1p", _BF16, (r, K)),
            a(container, svdq_w4a16_container_bytes(N, K), "container", _U8),
            a(L2p, 2 * N * r, "L2p", _BF16, (N, r)), a(bias, 2 * N, "bias", _BF16, (N,)),
            M, N, K, r, a(Y, Y.element_size() * M * N, "Y", None, (M, N)), out,
            a(workspace, need, "workspace"))
    _call(fn, a, args, stream)


def kv_block_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_tables: torch.Tensor,
                  block_size: int, free_blocks: torch.Tensor, free_count: torch.Tensor,
                  cu_rows: torch.Tensor, seq_lens: torch.Tensor, positions: torch.Tensor,
                  slots: torch.Tensor, status: torch.Tensor, free_count_out: torch.Tensor,
                  stream=None) -> None:
    """Lengths int32 [requests], block_tables int32 [requests, width] (in and out), free_blocks
    int32 [capacity], free_count int32 [1] -> cu_rows int32 [requests + 1], seq_lens and status
    int32 [requests], positions int32 [rows], slots int64 [rows], free_count_out int32 [1]."""
    fn = "kv_block_plan"
    n, width = block_tables.shape
    rows, cap = slots.shape[0], free_blocks.shape[0]
    a = _Args(fn)
    args = (a(ctx_lens, 4 * n, "ctx_lens", _I32, (n,)), a(new_lens, 4 * n, "new_lens", _I32, (n,)),
            n, a(block_tables, 4 * n * width, "block_tables", _I32), width, block_size,
            a(free_blocks, 4 * cap, "free_blocks", _I32, (cap,)), cap,
            a(free_count, 4, "free_count", _I32, (1,)), a(cu_rows, 4 * (n + 1), "cu_rows", _I32, (n + 1,)),
            a(seq_lens, 4 * n, "seq_lens", _I32, (n,)), rows,
            a(positions, 4 * rows, "positions", _I32, (rows,)), a(slots, 8 * rows, "slots", _I64, (rows,)),
            a(status, 4 * n, "status", _I32, (n,)),
            a(free_count_out, 4, "free_count_out", _I32, (1,)))
    _call(fn, a, args, stream)


def kv_block_release(seq_lens: torch.Tensor, done: torch.Tensor, block_tables: torch.Tensor,
                     block_size: int, free_blocks: torch.Tensor, free_count: torch.Tensor,
                     seq_lens_out: torch.Tensor, free_count_out: torch.Tensor,
                     stream=None) -> None:
    """seq_lens int32 [requests], done uint8 [requests], block_tables and free_blocks in and out
    -> seq_lens_out int32 [requests], free_count_out int32 [1]."""
    fn = "kv_block_release"
    n, width = block_tables.shape
    cap = free_blocks.shape[0]
    a = _Args(fn)
    args = (a(seq_lens, 4 * n, "seq_lens", _I32, (n,)), a(done, n, "done", _U8, (n,)), n,
            a(block_tables, 4 * n * width, "block_tables", _I32), width, block_size,
            a(free_blocks, 4 * cap, "free_blocks", _I32, (cap,)), cap,
            a(free_count, 4, "free_count", _I32, (1,)),
            a(seq_lens_out, 4 * n, "seq_lens_out", _I32, (n,)),
            a(free_count_out, 4, "free_count_out", _I32, (1,)))
    _call(fn, a, args, stream)


def _cache_args(a: _Args, k_codes, v_codes, k_scale, v_scale):
    """(num_blocks, heads, block_size, dim) of a cache and its four pointers."""
    num, heads, bs, dim = k_codes.shape
    n = num * heads
    return (num, heads, bs, dim), (
        a(k_codes, n * bs * dim, "k_codes", _U8), a(v_codes, n * bs * dim, "v_codes", _U8, (num, heads, dim, bs)),
        a(k_scale, 4 * n, "k_scale", _F32, (num, heads)), a(v_scale, 4 * n, "v_scale", _F32, (num, heads)))


def _strided(a: _Args, t: torch.Tensor, name: str, heads: int, dim: int) -> tuple:
    """A bf16 [rows, heads, dim] tensor whose rows may stand apart: (pointer, row stride)."""
    if tuple(t.shape[1:]) != (heads, dim) or t.stride(2) != 1 or t.stride(1) != dim:
        raise ValueError(f"{a.fn}: {name} must be [rows, {heads}, {dim}] with contiguous rows "
                         f"(got {tuple(t.shape)}, strides {tuple(t.stride())})")
    rows = t.shape[0]
    stride = t.stride(0) if rows > 1 else heads * dim
    if t.dtype != _BF16:
        raise ValueError(f"{a.fn}: {name} must be {_BF16} (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{a.fn}: {name} must be a device tensor")
    if a.device is None:
        a.device = t.device
    elif t.device != a.device:
        raise ValueError(f"{a.fn}: {name} is on {t.device}, other arguments on {a.device}")
    return t.data_ptr(), stride


def kv_block_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_codes: torch.Tensor,
                    v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                    stream=None) -> None:
    """k, v bf16 [rows, heads, dim] (rows may be slices of a fused projection), slots int64
    [rows]; the cache is written in place."""
    fn = "kv_block_append"
    a = _Args(fn)
    (num, heads, bs, dim), cache = _cache_args(a, k_codes, v_codes, k_scale, v_scale)
    rows = slots.shape[0]
    if k.shape[0] != rows or v.shape[0] != rows:
        raise ValueError(f"{fn}: k, v and slots must have the same rows (got {k.shape[0]}, "
                         f"{v.shape[0]}, {rows})")
    kp, ks = _strided(a, k, "k", heads, dim)
    vp, vs = _strided(a, v, "v", heads, dim)
    args = (kp, vp, ks, vs, a(slots, 8 * rows, "slots", _I64, (rows,)), rows, heads, dim, bs, num,
            *cache)
    _call(fn, a, args, stream)


def kv_block_read(slots: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, k_out: torch.Tensor,
                  v_out: torch.Tensor, stream=None) -> None:
    """slots int64 [rows] -> k_out, v_out bf16 [rows, heads, dim]."""
    fn = "kv_block_read"
    a = _Args(fn)
    (num, heads, bs, dim), cache = _cache_args(a, k_codes, v_codes, k_scale, v_scale)
    rows = slots.shape[0]
    n = rows * heads * dim
    args = (a(slots, 8 * rows, "slots", _I64, (rows,)), rows, heads, dim, bs, num, *cache,
            a(k_out, 2 * n, "k_out", _BF16, (rows, heads, dim)),
            a(v_out, 2 * n, "v_out", _BF16, (rows, heads, dim)))
    _call(fn, a, args, stream)


@functools.lru_cache(maxsize=4096)
def kv_block_attention_workspace_bytes(requests: int, rows: int, max_rows: int, heads: int,
                                       kv_heads: int, dim: int, width: int,
                                       block_size: int) -> int:
    return load().kv_block_attention_workspace_bytes(requests, rows, max_rows, heads, kv_heads,
                                                     dim, width, block_size)


def kv_block_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                       k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                       seq_lens: torch.Tensor, cu_rows: torch.Tensor, max_rows: int, causal: bool,
                       sm_scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor],
                       stream=None) -> None:
    """q bf16 [rows, heads, dim] (rows may stand apart), the cache, block_tables int32
    [requests, width], seq_lens int32 [requests], cu_rows int32 [requests + 1] -> out bf16
    [rows, heads, dim]."""
    fn = "kv_block_attention"
    a = _Args(fn)
    (num, kv_heads, bs, dim), cache = _cache_args(a, k_codes, v_codes, k_scale, v_scale)
    rows, heads = q.shape[0], q.shape[1]
    n, width = block_tables.shape
    qp, qs = _strided(a, q, "q", heads, dim)
    need = kv_block_attention_workspace_bytes(n, rows, max_rows, heads, kv_heads, dim, width, bs)
    args = (qp, qs, *cache, a(block_tables, 4 * n * width, "block_tables", _I32), width,
            a(seq_lens, 4 * n, "seq_lens", _I32, (n,)), a(cu_rows, 4 * (n + 1), "cu_rows", _I32, (n + 1,)),
            n, rows, max_rows, heads, kv_heads, dim, bs, num, int(causal), float(sm_scale),
            a(out, 2 * rows * heads * dim, "out", _BF16, (rows, heads, dim)),
            a(workspace, need, "workspace"))
    _call(fn, a, args, stream)
