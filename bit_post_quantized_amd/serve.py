"""The decoding step as a serving program uses it: objects that keep weights, cache and tables,
checked once, over the entry points of include/svdq_serve.h.

    planner = BlockPlanner(block_tables, free_blocks, block_size=16, rows=64)
    p = planner.plan(ctx_lens, new_lens, free_count)      # slots, positions, lengths
    qkv = qkv_linear(x)                                   # DecodeLinear: 4-bit weights
    cache.append(k, v, p.slots)                           # BlockCache: codes and block scales
    o = cache.attention(q, block_tables, p.seq_lens, p.cu_rows, max_rows=1)

Every call runs on the current stream of its tensors' device and allocates from torch's caching
allocator unless the caller gives the outputs and the workspace; all of them can be captured into
a graph.

A decoding step is many small launches, so the host's share counts.  The tensors an object keeps
are checked when it is made and their pointers kept; a call checks its own tensors in a few
comparisons and passes them on, and whatever does not pass goes through ``serve_binding``, which
names what is wrong.  (Plans of 8 requests one after the other: 5.9 us each, 13.3 through the
checks of ``serve_binding``.)
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding, layer
from . import serve_binding as B

_BF16, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)


def _is(t: torch.Tensor, dtype: torch.dtype, shape: tuple, device: torch.device) -> bool:
    """A contiguous tensor of just this dtype, shape and device."""
    return t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()


def _rows(t: torch.Tensor, shape: tuple, device: torch.device) -> bool:
    """A bf16 [rows, heads, dim] tensor whose rows may stand apart."""
    return (t.dtype is _BF16 and t.shape == shape and t.device == device
            and t.stride()[1:] == (shape[2], 1))


def _here(device: torch.device) -> bool:
    """Whether `device` is the current one (the raw calls below launch there)."""
    return torch._C._cuda_getDevice() == device.index


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


class DecodeLinear:
    """The SVDQuant linear of ``layer.PackedWeights`` (nibble container) for up to 64 rows, with
    the activations kept at 16 bits (``svdq_w4a16_gemv``).  The weights are checked, laid out for
    it (``svdq_pack_w4a16``; ``pw.wq`` is not kept) and bound when the object is made."""

    def __init__(self, pw: layer.PackedWeights):
        if pw.e3m2:
            raise ValueError("DecodeLinear reads the nibble container (e3m2=False)")
        self.K, self.N, self.rank = K, N, r = pw.K, pw.N, pw.rank
        if tuple(pw.wq.shape) != (N, K // 2):
            raise ValueError(f"DecodeLinear: wq must have shape {(N, K // 2)} (got {tuple(pw.wq.shape)})")
        self.container = torch.empty(B.svdq_w4a16_container_bytes(N, K), dtype=_U8, device=pw.wq.device)
        B.svdq_pack_w4a16(pw.wq, pw.w_scales, self.container)
        a = binding._Args("svdq_w4a16_gemv")
        l1, l2 = (pw.L1p, pw.L2p) if r else (None, None)
        self._weights = (a(pw.inv_lambda, 4 * K, "inv_lambda", _F32, (K,)),
                         a(l1, 2 * r * K, "L1p", _BF16, (r, K)), a(self.container, 0, "container"),
                         a(l2, 2 * N * r, "L2p", _BF16, (N, r)),
                         a(pw.bias, 2 * N, "bias", _BF16, (N,)))
        self._held = (pw.inv_lambda, l1, self.container, l2, pw.bias)
        self.device = a.device
        self._call = B.load().svdq_w4a16_gemv

    def __call__(self, X: torch.Tensor, out: Optional[torch.Tensor] = None, out_dtype=_BF16,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """X bf16 [M, K], M <= 64 -> [M, N], bf16 or fp32."""
        M, N, dev = X.shape[0], self.N, self.device
        good = _is(X, _BF16, (M, self.K), dev) and _here(dev)  # (and what is allocated here with it)
        if out is None:
            out = X.new_empty((M, N), dtype=out_dtype)
        else:
            good = good and _is(out, out.dtype, (M, N), dev)
        code = B.SVDQ_OUT_FP32 if out.dtype is _F32 else B.SVDQ_OUT_BF16
        need = B.svdq_w4a16_workspace_bytes(M, N, self.K, self.rank, code)
        if workspace is None:
            workspace = X.new_empty(need, dtype=_U8)
        else:
            good = good and (workspace.device == dev and workspace.is_contiguous()
                             and workspace.nbytes >= need)
        if good and (code or out.dtype is _BF16):
            status = self._call(X.data_ptr(), *self._weights, M, N, self.K, self.rank,
                                out.data_ptr(), code, workspace.data_ptr(), _stream(dev))
            if status:
                binding._check("svdq_w4a16_gemv", status)
        else:
            B.svdq_w4a16_gemv(X, *self._held, self.rank, out, workspace)
        return out


@dataclass
class SlotPlan:
    """What ``kv_block_plan`` writes for one step (see svdq_serve.h)."""
    cu_rows: torch.Tensor     # int32 [requests + 1]
    seq_lens: torch.Tensor    # int32 [requests]
    positions: torch.Tensor   # int32 [rows]
    slots: torch.Tensor       # int64 [rows]
    status: torch.Tensor      # int32 [requests]
    free_count: torch.Tensor  # int32 [1]
    _outputs: tuple = ()      # their pointers, in the call's order


class BlockPlanner:
    """Block tables and slot maps of a batch (``kv_block_plan``, ``kv_block_release``).

    ``block_tables`` int32 [requests, width] and ``free_blocks`` int32 [capacity] are the
    caller's and updated in place.  ``plan`` and ``release`` write one of five sets of outputs,
    the oldest that none of their own arguments is the beginning of, so the outputs of one call can
    be the next call's arguments; a plan stays valid until the second call after it.  A captured
    call writes the set that its capture chose at every replay, whatever was called in between: give
    a captured step a planner of its own.
    """

    def __init__(self, block_tables: torch.Tensor, free_blocks: torch.Tensor, block_size: int,
                 rows: int):
        self.block_tables, self.free_blocks = block_tables, free_blocks
        self.block_size, self.rows = block_size, rows
        self.requests, self.width = n, width = block_tables.shape
        self.device = dev = block_tables.device
        a = binding._Args("kv_block_plan")
        cap = free_blocks.shape[0]
        self._tables = (n, a(block_tables, 4 * n * width, "block_tables", _I32), width, block_size,
                        a(free_blocks, 4 * cap, "free_blocks", _I32, (cap,)), cap)
        self._call = B.load().kv_block_plan
        if max(rows, n, width, cap) >= 1 << 30:
            raise ValueError(f"BlockPlanner: {rows} rows, tables of {n} x {width} or {cap} free blocks are too many")

        def i32(*shape):
            return torch.empty(*shape, dtype=_I32, device=dev)

        self._plans = []
        for _ in range(5):
            p = SlotPlan(i32(n + 1), i32(n), i32(rows),
                         torch.empty(rows, dtype=_I64, device=dev), i32(n), i32(1))
            p._outputs = (p.cu_rows.data_ptr(), p.seq_lens.data_ptr(), rows, p.positions.data_ptr(),
                          p.slots.data_ptr(), p.status.data_ptr(), p.free_count.data_ptr())
            self._plans.append(p)

    def _other(self, a: int, b: int, count: int) -> SlotPlan:
        """The oldest set that is not an argument's (lengths at a and b, free count at count), which
        becomes the newest: of the four older ones at most three are, so it is never the set of the
        call before.  (Without requests the lengths are nowhere.)"""
        plans = self._plans
        if not self.requests:
            a = b = count
        for i in range(4):
            o = plans[i]._outputs
            if not (count in o or a in o or b in o):
                break
        plans.append(plans.pop(i))
        return plans[4]

    def plan(self, ctx_lens: torch.Tensor, new_lens: torch.Tensor,
             free_count: torch.Tensor) -> SlotPlan:
        ctx, new, dev, n = ctx_lens.data_ptr(), new_lens.data_ptr(), self.device, self.requests
        count = free_count.data_ptr()
        p = self._other(ctx, new, count)
        if (_is(ctx_lens, _I32, (n,), dev) and _is(new_lens, _I32, (n,), dev)
                and _is(free_count, _I32, (1,), dev) and _here(dev)):
            status = self._call(ctx, new, *self._tables, count, *p._outputs,
                                _stream(dev))
            if status:
                binding._check("kv_block_plan", status)
        else:
            B.kv_block_plan(ctx_lens, new_lens, self.block_tables, self.block_size,
                            self.free_blocks, free_count, p.cu_rows, p.seq_lens, p.positions,
                            p.slots, p.status, p.free_count)
        return p

    def release(self, seq_lens: torch.Tensor, done: torch.Tensor, free_count: torch.Tensor):
        """Gives back the blocks of the requests with ``done`` (uint8) set: (lengths, free
        count), of the set of outputs that the arguments are not part of."""
        p = self._other(seq_lens.data_ptr(), done.data_ptr(), free_count.data_ptr())
        B.kv_block_release(seq_lens, done, self.block_tables, self.block_size, self.free_blocks,
                           free_count, p.seq_lens, p.free_count)
        return p.seq_lens, p.free_count


class BlockCache:
    """A layer's K and V in blocks of tokens, held in 8 bits with a scale for each block and
    head (``kv_block_append``, ``kv_block_read``, ``kv_block_attention``)."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.num_blocks, self.kv_heads, self.block_size, self.dim = k_codes.shape
        self.device = k_codes.device
        self._arrays = (k_codes, v_codes, k_scale, v_scale)
        a = binding._Args("BlockCache")
        _, self._pointers = B._cache_args(a, *self._arrays)
        lib = B.load()
        self._append, self._read, self._attend = (lib.kv_block_append, lib.kv_block_read,
                                                  lib.kv_block_attention)

    @classmethod
    def empty(cls, num_blocks: int, block_size: int, kv_heads: int, dim: int, device="cuda"):
        """A cache of uninitialized blocks (a block needs none before its first append)."""
        return cls(torch.empty(num_blocks, kv_heads, block_size, dim, dtype=torch.uint8, device=device),
                   torch.empty(num_blocks, kv_heads, dim, block_size, dtype=torch.uint8, device=device),
                   torch.empty(num_blocks, kv_heads, dtype=torch.float32, device=device),
                   torch.empty(num_blocks, kv_heads, dtype=torch.float32, device=device))

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
        """k, v bf16 [rows, kv_heads, dim] (slices of a fused projection need no copy) into
        ``slots`` int64 [rows] (-1: no token)."""
        dev, rows = self.device, slots.shape[0]
        shape = (rows, self.kv_heads, self.dim)
        if (rows > 1 and _rows(k, shape, dev) and _rows(v, shape, dev)
                and _is(slots, _I64, (rows,), dev) and _here(dev)):
            status = self._append(k.data_ptr(), v.data_ptr(), k.stride(0), v.stride(0),
                                  slots.data_ptr(), rows, self.kv_heads, self.dim, self.block_size,
                                  self.num_blocks, *self._pointers, _stream(dev))
            if status:
                binding._check("kv_block_append", status)
        else:
            B.kv_block_append(k, v, slots, *self._arrays)

    def read(self, slots: torch.Tensor, k_out: Optional[torch.Tensor] = None,
             v_out: Optional[torch.Tensor] = None):
        """The values at ``slots``, bf16 [rows, kv_heads, dim] each; rows without a token keep
        what the outputs held (0 where they are allocated here)."""
        dev, rows = self.device, slots.shape[0]
        shape = (rows, self.kv_heads, self.dim)
        if k_out is None:
            k_out = torch.zeros(shape, dtype=_BF16, device=slots.device)
        if v_out is None:
            v_out = torch.zeros(shape, dtype=_BF16, device=slots.device)
        if (_is(k_out, _BF16, shape, dev) and _is(v_out, _BF16, shape, dev)
                and _is(slots, _I64, (rows,), dev) and _here(dev)):
            status = self._read(slots.data_ptr(), rows, self.kv_heads, self.dim, self.block_size,
                                self.num_blocks, *self._pointers, k_out.data_ptr(),
                                v_out.data_ptr(), _stream(dev))
            if status:
                binding._check("kv_block_read", status)
        else:
            B.kv_block_read(slots, *self._arrays, k_out, v_out)
        return k_out, v_out

    def attention(self, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  cu_rows: torch.Tensor, max_rows: int, causal: bool = True,
                  sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """q bf16 [rows, heads, dim] -> [rows, heads, dim]; sm_scale 1/sqrt(dim) by default.

        ``max_rows`` chooses the kernel for all requests, so a batch of decoding requests and
        prompts is faster as a call for each kind (63 requests decoding before up to 8192 tokens
        and a prompt of 500 rows: 765 us in one call, 168 in two)."""
        shape, dev = q.shape, self.device
        rows, heads, dim = shape
        n, width = block_tables.shape
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(dim)
        if out is None:
            out = torch.zeros(shape, dtype=_BF16, device=q.device)
        need = B.kv_block_attention_workspace_bytes(n, rows, max_rows, heads, self.kv_heads, dim,
                                                    width, self.block_size)
        if workspace is None and need:
            workspace = q.new_empty(need, dtype=_U8)
        if (rows > 1 and dim == self.dim and max_rows < 1 << 31 and _rows(q, shape, dev) and _is(out, _BF16, shape, dev)
                and _is(block_tables, _I32, (n, width), dev) and _is(seq_lens, _I32, (n,), dev)
                and _is(cu_rows, _I32, (n + 1,), dev) and _here(dev)
                and (workspace is None or workspace.device == dev and workspace.is_contiguous()
                     and workspace.nbytes >= need)):
            status = self._attend(q.data_ptr(), q.stride(0), *self._pointers,
                                  block_tables.data_ptr(), width, seq_lens.data_ptr(),
                                  cu_rows.data_ptr(), n, rows, max_rows, heads, self.kv_heads, dim,
                                  self.block_size, self.num_blocks, 1 if causal else 0, sm_scale,
                                  out.data_ptr(),
                                  None if workspace is None else workspace.data_ptr(),
                                  _stream(dev))
            if status:
                binding._check("kv_block_attention", status)
        else:
            B.kv_block_attention(q, *self._arrays, block_tables, seq_lens, cu_rows, max_rows,
                                 causal, sm_scale, out, workspace)
        return out
