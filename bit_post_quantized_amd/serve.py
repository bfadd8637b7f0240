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
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import layer
from . import serve_binding as B


class DecodeLinear:
    """The SVDQuant linear of ``layer.PackedWeights`` (nibble container) for up to 64 rows, with
    the activations kept at 16 bits (``svdq_w4a16_gemv``)."""

    def __init__(self, pw: layer.PackedWeights):
        if pw.e3m2:
            raise ValueError("DecodeLinear reads the nibble container (e3m2=False)")
        self.pw = pw
        self._l1 = pw.L1p if pw.rank else None
        self._l2 = pw.L2p if pw.rank else None

    def __call__(self, X: torch.Tensor, out: Optional[torch.Tensor] = None,
                 out_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None
                 ) -> torch.Tensor:
        """X bf16 [M, K], M <= 64 -> [M, N]."""
        pw = self.pw
        M = X.shape[0]
        if out is None:
            out = torch.empty(M, pw.N, dtype=out_dtype, device=X.device)
        if workspace is None:
            code = B.SVDQ_OUT_FP32 if out.dtype == torch.float32 else B.SVDQ_OUT_BF16
            workspace = torch.empty(B.svdq_w4a16_workspace_bytes(M, pw.N, pw.K, pw.rank, code),
                                    dtype=torch.uint8, device=X.device)
        B.svdq_w4a16_gemv(X, pw.inv_lambda, self._l1, pw.wq, pw.w_scales, self._l2, pw.bias,
                          pw.rank, out, workspace)
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


class BlockPlanner:
    """Block tables and slot maps of a batch (``kv_block_plan``, ``kv_block_release``).

    ``block_tables`` int32 [requests, width] and ``free_blocks`` int32 [capacity] are the
    caller's and updated in place.  ``plan`` writes one of two sets of outputs, the one that its
    own arguments are not part of, so the ``seq_lens`` and ``free_count`` of one step can be the
    next step's arguments; a plan stays valid until the second call after it.
    """

    def __init__(self, block_tables: torch.Tensor, free_blocks: torch.Tensor, block_size: int,
                 rows: int):
        self.block_tables, self.free_blocks = block_tables, free_blocks
        self.block_size, self.rows = block_size, rows
        n, dev = block_tables.shape[0], block_tables.device

        def i32(*shape):
            return torch.empty(*shape, dtype=torch.int32, device=dev)

        self._plans = [SlotPlan(i32(n + 1), i32(n), i32(rows),
                                torch.empty(rows, dtype=torch.int64, device=dev), i32(n), i32(1))
                       for _ in range(2)]

    def _other(self, lens: torch.Tensor, free_count: torch.Tensor) -> SlotPlan:
        used = (lens.data_ptr(), free_count.data_ptr())
        free = [p for p in self._plans
                if not (lens.numel() and p.seq_lens.data_ptr() == used[0])
                and p.free_count.data_ptr() != used[1]]
        if not free:
            raise ValueError("lengths and free count must come from the same plan")
        return free[0]

    def plan(self, ctx_lens: torch.Tensor, new_lens: torch.Tensor,
             free_count: torch.Tensor) -> SlotPlan:
        p = self._other(ctx_lens, free_count)
        B.kv_block_plan(ctx_lens, new_lens, self.block_tables, self.block_size, self.free_blocks,
                        free_count, p.cu_rows, p.seq_lens, p.positions, p.slots, p.status,
                        p.free_count)
        return p

    def release(self, seq_lens: torch.Tensor, done: torch.Tensor, free_count: torch.Tensor):
        """Gives back the blocks of the requests with ``done`` (uint8) set: (lengths, free
        count), of the set of outputs that the arguments are not part of."""
        p = self._other(seq_lens, free_count)
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
        self._arrays = (k_codes, v_codes, k_scale, v_scale)

    @classmethod
    def empty(cls, num_blocks: int, block_size: int, kv_heads: int, dim: int, device="cuda"):
        """A cache of uninitialized blocks (a block needs none before its first append)."""
        return cls(torch.empty(num_blocks, kv_heads, block_size, dim, dtype=torch.uint8, device=device),
                   torch.empty(num_blocks, kv_heads, dim, block_size, dtype=torch.uint8, device=device),
                   torch.empty(num_blocks, kv_heads, dtype=torch.float32, device=device),
                   torch.empty(num_blocks, kv_heads, dtype=torch.float32, device=device))

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
        """k, v bf16 [rows, kv_heads, dim] into ``slots`` int64 [rows] (-1: no token)."""
        B.kv_block_append(k, v, slots, *self._arrays)

    def read(self, slots: torch.Tensor, k_out: Optional[torch.Tensor] = None,
             v_out: Optional[torch.Tensor] = None):
        """The values at ``slots``, bf16 [rows, kv_heads, dim] each; rows without a token keep
        what the outputs held (0 where they are allocated here)."""
        shape = (slots.shape[0], self.kv_heads, self.dim)
        if k_out is None:
            k_out = torch.zeros(shape, dtype=torch.bfloat16, device=slots.device)
        if v_out is None:
            v_out = torch.zeros(shape, dtype=torch.bfloat16, device=slots.device)
        B.kv_block_read(slots, *self._arrays, k_out, v_out)
        return k_out, v_out

    def attention(self, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  cu_rows: torch.Tensor, max_rows: int, causal: bool = True,
                  sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """q bf16 [rows, heads, dim] -> [rows, heads, dim]; sm_scale 1/sqrt(dim) by default."""
        rows, heads, dim = q.shape
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(dim)
        if out is None:
            out = torch.zeros(rows, heads, dim, dtype=torch.bfloat16, device=q.device)
        if workspace is None:
            need = B.kv_block_attention_workspace_bytes(
                block_tables.shape[0], rows, max_rows, heads, self.kv_heads, dim,
                block_tables.shape[1], self.block_size)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        B.kv_block_attention(q, *self._arrays, block_tables, seq_lens, cu_rows, max_rows, causal,
                             sm_scale, out, workspace)
        return out
