"""Oracle of the decoding step: few-row linear, block plan, block-scaled 8-bit cache, attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__`` for the page short names).

Plain loops and fp64, from the definitions in include/svdq_serve.h; the contract's fp32 roundings
(the block scale, the quotient before rounding to a code) are NumPy's IEEE float32.
"""
from __future__ import annotations

import numpy as np

from .numerics import bf16_to_bits, decode_bf16, round_bf16


# ------------------------------------------------------------------------------------ linear
def linear(x_bits, inv_lambda, l1, codes, w_scales, l2, bias):
    """(Y, A) fp64 [M, N]: the layer and the sum of its terms' magnitudes (for error bounds).

    x_bits bf16 [M, K]; l1 [K, r] and l2 [r, N] exact values; codes int [N, K]; w_scales [G, N]."""
    xh = (decode_bf16(x_bits).astype(np.float32) * np.asarray(inv_lambda, np.float32)[None, :]).astype(np.float64)
    w = codes.astype(np.float64) * np.repeat(np.asarray(w_scales, np.float64).T, 64, axis=1)  # [N, K]
    y, a = xh @ w.T, np.abs(xh) @ np.abs(w).T
    if l1.shape[1]:
        y = y + (xh @ l1) @ l2
        a = a + (np.abs(xh) @ np.abs(l1)) @ np.abs(l2)
    if bias is not None:
        y, a = y + bias[None, :], a + np.abs(bias)[None, :]
    return y, a


# -------------------------------------------------------------------------------------- plan
def plan(ctx, new, tables, bs, free, count, rows):
    """The step's bookkeeping, request by request; tables is a copy that is returned."""
    tables = np.array(tables, dtype=np.int64)
    width = tables.shape[1]
    stack = [int(x) for x in free[:min(max(count, 0), len(free))]]
    dry = False
    cu, seq, status = [0], [], []
    pos = np.zeros(rows, np.int64)
    slots = np.full(rows, -1, np.int64)
    for b in range(len(ctx)):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        end, held = -(-(c + n) // bs), -(-c // bs)
        first = cu[-1]
        cu.append(first + n)
        need = end - held
        if end > width:
            st = 2
        elif first + n > rows:
            st = 3
        else:
            dry = dry or need > len(stack)
            st = 1 if need > 0 and dry else 0
        if st == 0:
            for j in range(held, end):
                tables[b, j] = stack.pop()
        seq.append(c if st else c + n)
        status.append(st)
        for i in range(n):
            if first + i < rows:
                pos[first + i] = c + i
                if st == 0:
                    slots[first + i] = tables[b, (c + i) // bs] * bs + (c + i) % bs
    return dict(tables=tables, cu=np.array(cu), seq=np.array(seq), positions=pos, slots=slots,
                status=np.array(status), free_count=len(stack))


# ------------------------------------------------------------------------------------- cache
class Cache:
    """codes [num, H, bs, D] (c, not c + 128) and scale [num, H] fp32 of one of K and V."""

    def __init__(self, codes, scale):
        self.codes = np.array(codes, dtype=np.int64)
        self.scale = np.array(scale, dtype=np.float32)

    def append(self, x, slots):
        """x exact values [T, H, D] of bf16 inputs; one block and head at a time."""
        num, H, bs, D = self.codes.shape
        t = 0
        slots = [int(s) for s in slots]
        while t < len(slots):
            s = slots[t]
            if not 0 <= s < num * bs:
                t += 1
                continue
            n = 1
            while t + n < len(slots) and slots[t + n] == s + n and (s + n) % bs:
                n += 1
            b, off = divmod(s, bs)
            for h in range(H):
                v = x[t:t + n, h].astype(np.float32)
                old = np.float32(0) if off == 0 else self.scale[b, h]
                new = np.maximum(old, np.float32(np.abs(v).max()) / np.float32(127))  # (a NaN stays one)
                if off > 0 and new > old:
                    ratio = np.float32(old / new)
                    was = self.codes[b, h, :off].astype(np.float32)
                    self.codes[b, h, :off] = np.rint(was * ratio).astype(np.int64)
                if 0 < new < np.inf:
                    q = np.clip(np.rint(v / new), -127, 127).astype(np.int64)
                else:
                    q = np.zeros_like(v, dtype=np.int64)
                self.codes[b, h, off:off + n] = q
                self.scale[b, h] = new
            t += n

    def values(self, slots):
        """bf16 bits [T, H, D] of the values at valid slots."""
        bs = self.codes.shape[2]
        b, o = np.asarray(slots) // bs, np.asarray(slots) % bs
        v = self.codes[b, :, o].astype(np.float32) * self.scale[b][:, :, None]
        return bf16_to_bits(round_bf16(v.astype(np.float64)))


# --------------------------------------------------------------------------------- attention
def attention(q, k_codes, k_scale, v_codes, v_scale, tables, seq, cu, causal, sm_scale, max_rows):
    """(out, bound, written): fp64 [T, heads, D]; bound[t, h, d] the sum of the weighted value
    magnitudes times a row's relative weight error per unit (see the tests); written [T] marks the
    rows the call writes.  k_codes, v_codes [num, KV, bs, D] hold c."""
    T, heads, D = q.shape
    num, KV, bs, _ = k_codes.shape
    g = heads // KV
    out = np.zeros((T, heads, D))
    mag = np.zeros((T, heads, D))
    top = np.zeros((T, heads))
    written = np.zeros(T, bool)
    for b in range(len(seq)):
        n = cu[b + 1] - cu[b]
        length = min(max(int(seq[b]), 0), tables.shape[1] * bs)
        ids = [int(x) for x in tables[b, :-(-length // bs)]] if length else []
        good = np.repeat([0 <= i < num for i in ids], bs)[:length].astype(bool)
        ids = [i if 0 <= i < num else 0 for i in ids]
        for h in range(KV):
            if length:
                k = (k_codes[ids, h] * k_scale[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:length]
                v = (v_codes[ids, h] * v_scale[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:length]
            for i in range(min(n, max_rows)):
                t = cu[b] + i
                written[t] = True
                lim = length if not causal else min(length, max(length - n + i + 1, 0))
                seen = good[:lim] if length else np.zeros(0, bool)
                if not seen.any():
                    continue
                kk, vv = k[:lim][seen], v[:lim][seen]
                for e in range(h * g, (h + 1) * g):
                    s = sm_scale * (kk @ q[t, e])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[t, e] = w @ vv
                    mag[t, e] = w @ np.abs(vv)
                    top[t, e] = abs(sm_scale) * (np.abs(kk) @ np.abs(q[t, e])).max()
    return out, mag, top, written
