"""What a decoding step needs between its projections, as a serving program uses it: objects that keep
weights, checked once, over the entry points of include/svdq_decoder.h.

    h8, res = norm.rows8(x, res)                  # RMSNorm: residual added, codes and row scales
    qkv = linear(h8)                              # Linear8: 8-bit codes on both sides
    rope(q, k, plan.positions)                    # Rope: q and k in place, positions of the block plan
    cache.append(k, v, plan.slots)                # serve.BlockCache, as before
    tokens, share = sample(logits, temperature, uniform, top_k, top_p, min_p)

Every call runs on the current stream of its tensors' device and allocates from torch's caching
allocator unless the caller gives the outputs and the workspace; all of them can be captured into
a graph.  As in ``serve``, a call that passes a few comparisons goes straight to the library, and
what does not goes through ``decoder_binding``, which names what is wrong.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding
from . import decoder_binding as B
from .serve import _here, _is, _stream

_BF16, _F32, _F64, _I8, _I32, _U8 = (torch.bfloat16, torch.float32, torch.float64, torch.int8,
                                     torch.int32, torch.uint8)
_CODE = {_BF16: B.SVDQ_OUT_BF16, _F32: B.SVDQ_OUT_FP32}


def _rows_of(t: torch.Tensor, dtype: torch.dtype, rows: int, heads: int, dim: int, device: torch.device) -> bool:
    """A [rows, heads, dim] tensor whose rows may stand apart."""
    return (t.dtype is dtype and t.shape == (rows, heads, dim) and t.device == device
            and t.stride()[1:] == (dim, 1))


@dataclass
class Rows8:
    """Rows in 8 bits: the value at [m, k] is codes[m, k] scales[m]."""
    codes: torch.Tensor    # int8 [M, K]
    scales: torch.Tensor   # fp32 [M]

    @classmethod
    def empty(cls, M: int, K: int, device="cuda") -> "Rows8":
        return cls(torch.empty(M, K, dtype=_I8, device=device), torch.empty(M, dtype=_F32, device=device))


class RMSNorm:
    """y = h / sqrt(mean(h^2) + eps) gamma of h = x + residual (``svdq_rms_norm``); gamma fp32 [K].
    A smoothing factor of the projection behind it is folded into gamma.  Gamma's memory is checked and bound
    when the object is made, and anew when another tensor is assigned to ``gamma``."""

    def __init__(self, gamma: torch.Tensor, eps: float = 1e-6):
        self.gamma, self.eps = gamma, float(eps)
        self._call = B.load().svdq_rms_norm

    @property
    def gamma(self) -> torch.Tensor:
        return self._gamma

    @gamma.setter
    def gamma(self, gamma: torch.Tensor):
        a, K = binding._Args("RMSNorm"), gamma.shape[0]
        self._pointer = a(gamma, 4 * K, "gamma", _F32, (K,))
        self._gamma = gamma.detach()   # (holds the memory, whatever becomes of the tensor's own)
        self.K, self.device = K, a.device

    def _run(self, x, residual, residual_out, y, codes, scales, good):
        """``good``: the outputs are as they should be."""
        M, K, dev, code = x.shape[0], self.K, self.device, _CODE.get(x.dtype)
        res = out = kind = 0
        if residual is not None:
            kind = _CODE.get(residual.dtype)
            good = good and kind is not None and _is(residual, residual.dtype, (M, K), dev)
            res, out = residual.data_ptr(), residual_out.data_ptr()
        if good and code is not None and _is(x, x.dtype, (M, K), dev) and _here(dev):
            status = self._call(x.data_ptr(), code, K, res, kind, out, self._pointer, M, K, self.eps,
                                None if y is None else y.data_ptr(), None if codes is None else codes.data_ptr(),
                                None if codes is None else scales.data_ptr(), _stream(dev))
            if status:
                binding._check("svdq_rms_norm", status)
        else:
            B.svdq_rms_norm(x, residual, residual_out, self._gamma, self.eps, y, codes, scales)

    def _stream_out(self, x, residual, residual_out):
        """(where x + residual goes, whether it is as it should be)"""
        if residual is None:
            if residual_out is not None:
                raise ValueError("RMSNorm: residual_out needs a residual")
            return None, True
        if residual_out is None:
            return torch.empty(residual.shape, dtype=residual.dtype, device=residual.device), True
        return residual_out, _is(residual_out, residual.dtype, x.shape, self.device)

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None):
        """x bf16 or fp32 [M, K], residual bf16 or fp32 [M, K] -> (y bf16 [M, K], x + residual in the
        residual's dtype; None without one).  ``residual_out`` may be ``residual``."""
        residual_out, good = self._stream_out(x, residual, residual_out)
        if out is None:
            out = torch.empty(x.shape, dtype=_BF16, device=x.device)
        else:
            good = good and _is(out, _BF16, x.shape, self.device)
        self._run(x, residual, residual_out, out, None, None, good)
        return out, residual_out

    def rows8(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, out: Optional[Rows8] = None,
              residual_out: Optional[torch.Tensor] = None):
        """The same in 8 bits: (Rows8, x + residual)."""
        residual_out, good = self._stream_out(x, residual, residual_out)
        if out is None:
            out = Rows8.empty(*x.shape, device=x.device)
        else:
            good = (good and _is(out.codes, _I8, x.shape, self.device)
                    and _is(out.scales, _F32, x.shape[:1], self.device))
        self._run(x, residual, residual_out, None, out.codes, out.scales, good)
        return out, residual_out


def quantize_rows(x: torch.Tensor, factor: Optional[torch.Tensor] = None, out: Optional[Rows8] = None) -> Rows8:
    """x bf16 or fp32 [M, K], times factor fp32 [K], in 8 bits with a scale for each row
    (``svdq_quantize_rows``): activations that no norm precedes, or a weight [N, K]."""
    if out is None:
        out = Rows8.empty(*x.shape, device=x.device)
    (M, K), dev, code = x.shape, x.device, _CODE.get(x.dtype)
    if (dev.type == "cuda" and code is not None and _is(x, x.dtype, (M, K), dev) and _is(out.codes, _I8, (M, K), dev)
            and _is(out.scales, _F32, (M,), dev) and (factor is None or _is(factor, _F32, (K,), dev)) and _here(dev)):
        status = B.load().svdq_quantize_rows(x.data_ptr(), code, K, None if factor is None else factor.data_ptr(), M, K,
                                             out.codes.data_ptr(), out.scales.data_ptr(), _stream(dev))
        if status:
            binding._check("svdq_quantize_rows", status)
    else:
        B.svdq_quantize_rows(x, factor, out.codes, out.scales)
    return out


class Linear8:
    """Y = sx sw (qx qw^T) + bias for any number of rows (``svdq_w8a8_gemm``).  The weight's codes int8
    [N, K] and scales fp32 [N] (``quantize_rows`` of the weight, or ``from_weight``) are checked and
    laid out when the object is made; the codes are not kept."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: Optional[torch.Tensor] = None):
        N, K = codes.shape
        self.N, self.K = N, K
        a = binding._Args("svdq_w8a8_gemm")
        self.container = torch.empty(B.svdq_w8a8_container_bytes(N, K), dtype=_I8, device=codes.device)
        B.svdq_pack_w8a8(codes, self.container)
        self._weights = (a(self.container, 0, "container"), a(scales, 4 * N, "sw", _F32, (N,)),
                         a(bias, 2 * N, "bias", _BF16, (N,)))
        # (detached: holds the memory, whatever becomes of the tensors' own)
        self._held = (self.container.detach(), scales.detach(), None if bias is None else bias.detach())
        self.device = a.device
        self._call = B.load().svdq_w8a8_gemm

    @classmethod
    def from_weight(cls, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    factor: Optional[torch.Tensor] = None) -> "Linear8":
        """W bf16 or fp32 [N, K], times factor fp32 [K] (the smoothing that the activations were divided
        by)."""
        w = quantize_rows(W, factor)
        return cls(w.codes, w.scales, bias)

    def __call__(self, x: Rows8, out: Optional[torch.Tensor] = None, out_dtype=_BF16,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Rows8 of [M, K] -> [M, N], bf16 or fp32."""
        codes, dev, N = x.codes, self.device, self.N
        M = codes.shape[0]
        good = _is(codes, _I8, (M, self.K), dev) and _is(x.scales, _F32, (M,), dev) and _here(dev)
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=codes.device)
        else:
            good = good and _is(out, out.dtype, (M, N), dev)
        need = B.svdq_w8a8_workspace_bytes(M, N, self.K)
        if workspace is not None:
            good = good and workspace.device == dev and workspace.is_contiguous() and workspace.nbytes >= need
        elif need:
            workspace = torch.empty(need, dtype=_U8, device=codes.device)
        code = _CODE.get(out.dtype)
        if good and code is not None:
            status = self._call(codes.data_ptr(), x.scales.data_ptr(), *self._weights, M, N, self.K, out.data_ptr(),
                                code, None if workspace is None else workspace.data_ptr(), _stream(dev))
            if status:
                binding._check("svdq_w8a8_gemm", status)
        else:
            if codes.shape[1:] != (self.K,):
                raise ValueError(f"Linear8: codes must have shape {(M, self.K)} (got {tuple(codes.shape)})")
            B.svdq_w8a8_gemm(codes, x.scales, *self._held, out, workspace)
        return out


def rope_frequencies(rot_dim: int, base: float = 10000.0, factor: float = 1.0, original: Optional[int] = None,
                     low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """Frequencies fp64 [rot_dim / 2] in radians per position, base^(-2 i / rot_dim), for contexts
    ``factor`` times as long as trained: all divided by it (positions interpolated), or, with the trained
    length ``original``, by parts as in YaRN (Peng et al. 2023): those that make at least ``high`` turns
    in it stay, those of at most ``low`` turns are divided, in between linearly in the turns.  (A model whose
    configuration goes linearly over the channels in between, not over their turns, needs frequencies of its
    own: ``Rope`` takes any.)"""
    i = torch.arange(rot_dim // 2, dtype=_F64)
    f = float(base) ** (-2.0 * i / rot_dim)
    if original is None:
        f = f / factor
    else:
        stay = ((original * f / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (stay + (1.0 - stay) / factor)
    return f.to(device)


class Rope:
    """Rotary positions (``svdq_rope``) with the frequencies fp64 [rot_dim / 2]; channels from rot_dim on
    are left as they are.  ``scale`` multiplies what is rotated (a factor of a scheme for long contexts).
    The frequencies' memory is checked and bound when the object is made, and anew when another tensor is
    assigned to ``freqs``."""

    def __init__(self, freqs: torch.Tensor, interleaved: bool = False, scale: float = 1.0):
        self.freqs = freqs
        self.interleaved, self.scale = bool(interleaved), float(scale)
        self._call = B.load().svdq_rope

    @property
    def freqs(self) -> torch.Tensor:
        return self._freqs

    @freqs.setter
    def freqs(self, freqs: torch.Tensor):
        a, pairs = binding._Args("Rope"), freqs.shape[0]
        self._pointer = a(freqs, 8 * pairs, "freqs", _F64, (pairs,))
        self._freqs = freqs.detach()   # (holds the memory, whatever becomes of the tensor's own)
        self.rot_dim, self.device = 2 * pairs, a.device

    def __call__(self, q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
        """q [rows, heads, dim] and k [rows, kv_heads, dim] (slices of a fused projection need no copy),
        positions int32 [rows] -> (q_out, k_out) in bf16: in place where they are bf16 and no output is
        given, new tensors where they are fp32."""
        if q_out is None:
            q_out = q if q.dtype is _BF16 else torch.empty(q.shape, dtype=_BF16, device=q.device)
        if k_out is None and k is not None:
            k_out = k if k.dtype is _BF16 else torch.empty(k.shape, dtype=_BF16, device=k.device)
        rows, heads, dim = q.shape
        dev, code = self.device, _CODE.get(q.dtype)
        kv = 0 if k is None else k.shape[1]
        if (code is not None and _rows_of(q, q.dtype, rows, heads, dim, dev) and _rows_of(q_out, _BF16, rows, heads, dim, dev)
                and (k_out is None if k is None else
                     _rows_of(k, q.dtype, rows, kv, dim, dev) and _rows_of(k_out, _BF16, rows, kv, dim, dev))
                and _is(positions, _I32, (rows,), dev) and _here(dev)):
            one = rows <= 1   # (the strides of a single row say nothing)
            wide, narrow = heads * dim, kv * dim
            status = self._call(q.data_ptr(), wide if one else q.stride(0), heads, None if k is None else k.data_ptr(),
                                narrow if one or k is None else k.stride(0), kv, code, rows, dim, self.rot_dim,
                                1 if self.interleaved else 0, positions.data_ptr(), self._pointer, self.scale,
                                q_out.data_ptr(), wide if one else q_out.stride(0),
                                None if k is None else k_out.data_ptr(),
                                narrow if one or k is None else k_out.stride(0), _stream(dev))
            if status:
                binding._check("svdq_rope", status)
        else:
            B.svdq_rope(q, k, positions, self._freqs, self.interleaved, self.scale, q_out, k_out)
        return q_out, k_out


def sample(logits: torch.Tensor, temperature: torch.Tensor, uniform: torch.Tensor,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
           share: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """logits bf16 or fp32 [rows, vocab], temperature and uniform fp32 [rows], top_k int32 [rows], top_p
    and min_p fp32 [rows] (None: no such limit) -> (tokens int32 [rows], the tokens' share of what the
    limits left, fp32 [rows]); see ``svdq_sample``."""
    rows, vocab = logits.shape
    dev = logits.device
    good = True
    if tokens is None:
        tokens = torch.empty(rows, dtype=_I32, device=dev)
    else:
        good = _is(tokens, _I32, (rows,), dev)
    if share is None:
        share = torch.empty(rows, dtype=_F32, device=dev)
    else:
        good = good and _is(share, _F32, (rows,), dev)
    need = B.svdq_sample_workspace_bytes(rows, vocab)
    if workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=dev)
    else:
        good = good and workspace.device == dev and workspace.is_contiguous() and workspace.nbytes >= need
    if (good and dev.type == "cuda" and logits.dtype in _CODE and (logits.stride(1) == 1 or vocab == 1)
            and _is(temperature, _F32, (rows,), dev) and _is(uniform, _F32, (rows,), dev)
            and (top_k is None or _is(top_k, _I32, (rows,), dev))
            and (top_p is None or _is(top_p, _F32, (rows,), dev))
            and (min_p is None or _is(min_p, _F32, (rows,), dev)) and _here(dev)):
        status = B.load().svdq_sample(
            logits.data_ptr(), _CODE[logits.dtype], logits.stride(0) if rows > 1 else vocab, rows, vocab, temperature.data_ptr(),
            uniform.data_ptr(), None if top_k is None else top_k.data_ptr(), None if top_p is None else top_p.data_ptr(),
            None if min_p is None else min_p.data_ptr(), tokens.data_ptr(), share.data_ptr(), workspace.data_ptr(),
            _stream(dev))
        if status:
            binding._check("svdq_sample", status)
    else:
        B.svdq_sample(logits, temperature, uniform, top_k, top_p, min_p, tokens, share, workspace)
    return tokens, share
