"""The operators together, as a decoding program runs them: plan, fused projection on 4-bit
weights, append, attention, output projection; prompts first, then one token at a time, eager and
captured, against a step-by-step fp64 model that shares only the weights and the inputs."""
import math

import numpy as np
import pytest
import torch

from bit_post_quantized_amd import serve
from oracle import serve as osv
from tests.serve_cases import bf16_values, host64, host_cache, to_dev, to_dev_bf16
from tests.test_gpu_serve_linear import make

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, BS, HID = 4, 2, 64, 16, 256


class Step:
    def __init__(self, requests, num, width, rows):
        self.qkv_pw, self.out_pw = make(1, 1, HID, (HEADS + 2 * KV) * DIM, 16, True)[1], \
            make(2, 1, HEADS * DIM, HID, 16, False)[1]
        self.qkv, self.o = serve.DecodeLinear(self.qkv_pw), serve.DecodeLinear(self.out_pw)
        self.cache = serve.BlockCache.empty(num, BS, KV, DIM)
        i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
        self.tables = i32(np.full((requests, width), -1))
        self.planner = serve.BlockPlanner(self.tables, i32(np.arange(num)[::-1].copy()), BS, rows)
        self.seq, self.count = i32(np.zeros(requests)), i32([num])

    def __call__(self, x, new, max_rows):
        p = self.planner.plan(self.seq, new, self.count)
        qkv = self.qkv(x).view(x.shape[0], HEADS + 2 * KV, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        self.cache.append(k, v, p.slots)
        a = self.cache.attention(q, self.tables, p.seq_lens, p.cu_rows, max_rows)
        y = self.o(a.view(x.shape[0], HEADS * DIM))
        return p, qkv, a, y


def test_prompts_then_tokens(gpu_lib):
    rng = np.random.default_rng(0)
    n, rows = 3, 48
    s = Step(n, 24, 8, rows)
    past = [(np.zeros((0, KV, DIM)), np.zeros((0, KV, DIM))) for _ in range(n)]
    for step, new in enumerate([[20, 7, 17], [1, 1, 1], [1, 0, 1], [5, 1, 1]] + [[1, 1, 1]] * 12):
        x = to_dev_bf16(bf16_values(rng, rows, HID))
        p, qkv, a, y = s(x, to_dev(np.array(new), torch.int32), max(new))
        torch.cuda.synchronize()
        assert p.status.cpu().tolist() == [0] * n
        s.seq, s.count = p.seq_lens, p.free_count
        qkv, got = host64(qkv), host64(a)
        kc, ks, vc, vs = host_cache(s.cache)
        tables, cu = s.tables.cpu().numpy(), np.concatenate([[0], np.cumsum(new)])
        want, mag, top, written = osv.attention(qkv[:, :HEADS], kc, ks, vc, vs, tables,
                                                p.seq_lens.cpu().numpy(), cu, True, 1 / math.sqrt(DIM), 99)
        tol = 2.0 ** -8 * np.abs(want) + (2 * (2 * DIM + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -20)[:, :, None] * mag
        assert (np.abs(got - want) <= tol)[written].all(), step
        # the cache holds every token so far, each off by its block's step (and by half a step for
        # each time the block's scale grew, at most 16 tokens' worth)
        for b in range(n):
            k0, v0 = past[b]
            past[b] = (np.concatenate([k0, qkv[cu[b]:cu[b + 1], HEADS:HEADS + KV]]),
                       np.concatenate([v0, qkv[cu[b]:cu[b + 1], HEADS + KV:]]))
            for x0, codes, scale in ((past[b][0], kc, ks), (past[b][1], vc, vs)):
                ids = tables[b, :-(-len(x0) // BS)]
                val = (codes[ids] * scale[ids][:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, KV, DIM)[:len(x0)]
                step_of = np.repeat(scale[ids], BS, axis=0)[:len(x0)][:, :, None]
                assert (np.abs(val - x0) <= 0.5 * (BS + 1) * step_of * 1.001).all()
        assert np.isfinite(host64(y)[:sum(new)]).all()


def test_captured_decoding_equals_eager(gpu_lib):
    """One captured step, replayed with new lengths, tables and inputs, against eager steps on a
    twin; the program's own eager work runs between the replays."""
    rng = np.random.default_rng(1)
    n = 4
    eager, cap = Step(n, 20, 5, n), Step(n, 20, 5, n)
    x = torch.zeros(n, HID, dtype=torch.bfloat16, device="cuda")
    new = torch.ones(n, dtype=torch.int32, device="cuda")
    seq, count = torch.zeros_like(new), torch.full((1,), 20, dtype=torch.int32, device="cuda")
    cap.seq, cap.count = seq, count
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p, _, a, y = cap(x, new, 1)
        seq.copy_(p.seq_lens)
        count.copy_(p.free_count)
    for step in range(20):
        xs = to_dev_bf16(bf16_values(rng, n, HID))
        add = to_dev((rng.random(n) < 0.8).astype(np.int32))
        x.copy_(xs)
        new.copy_(add)
        g.replay()
        pe, _, ae, ye = eager(xs, add, 1)
        eager.seq, eager.count = pe.seq_lens, pe.free_count
        torch.cuda.synchronize()
        live = int(add.sum())
        assert torch.equal(seq, pe.seq_lens) and torch.equal(count, pe.free_count)
        assert torch.equal(cap.tables, eager.tables)
        assert torch.equal(p.slots, pe.slots)
        assert torch.equal(a[:live], ae[:live]) and torch.equal(y[:live], ye[:live]), step


def test_two_batches_at_once_on_two_streams(gpu_lib):
    """Two programs with their own cache and tables on two streams at a time give what they give
    one after the other."""
    rng = np.random.default_rng(2)
    xs = [[to_dev_bf16(bf16_values(rng, 2, HID)) for _ in range(6)] for _ in range(2)]
    new = torch.ones(2, dtype=torch.int32, device="cuda")

    def program(i):
        s, ys = Step(2, 8, 4, 2), []
        for x in xs[i]:
            p, _, _, y = s(x, new, 1)
            s.seq, s.count = p.seq_lens, p.free_count
            ys.append(y)
        return s, ys

    want = [program(i)[1] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            got.append(program(i))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(want[i], got[i][1]):
            assert torch.equal(a, b)
