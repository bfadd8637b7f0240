"""A whole decoding step as a serving program runs it: plan, norm to 8 bits, 8-bit projection, rotary
positions, append, attention, 8-bit output projection, norm to 16 bits, vocabulary projection on 4-bit
weights, sampling; prompts first, then one token at a time, eager and captured, each operator against
its 64-bit form on the inputs it got."""
import math

import numpy as np
import pytest
import torch

from bit_post_quantized_amd import decoder, serve
from oracle import decoder as od
from oracle import serve as osv
from tests.serve_cases import bf16_values, host64, host_cache, to_dev, to_dev_bf16
from tests.test_gpu_decoder_norm import check as check_norm
from tests.test_gpu_decoder_norm import check8
from tests.test_gpu_decoder_rope import check as check_rope
from tests.test_gpu_serve_linear import check as check_linear
from tests.test_gpu_serve_linear import make

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, BS, HID, VOCAB = 4, 2, 64, 16, 256, 999


class Step:
    def __init__(self, requests, num, width, rows, seed=1):
        rng = np.random.default_rng(seed)
        self.embed = to_dev_bf16(bf16_values(rng, VOCAB, HID))
        self.gamma = [(1 + 0.2 * rng.standard_normal(HID)).astype(np.float32) for _ in range(2)]
        self.norms = [decoder.RMSNorm(to_dev(g), 1e-6) for g in self.gamma]
        self.w = [od.quantize_rows(bf16_values(rng, n, k, scale=k ** -0.5), None)
                  for n, k in (((HEADS + 2 * KV) * DIM, HID), (HID, HEADS * DIM))]
        self.qkv, self.o = (decoder.Linear8(to_dev(c), to_dev(s)) for c, s in self.w)
        _, pw, self.head_ref = make(2, 1, HID, VOCAB, 16, False)
        self.head = serve.DecodeLinear(pw)
        self.rope = decoder.Rope(decoder.rope_frequencies(DIM, 1e4, 4.0, original=64))
        self.cache = serve.BlockCache.empty(num, BS, KV, DIM)
        i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
        self.tables = i32(np.full((requests, width), -1))
        self.planner = serve.BlockPlanner(self.tables, i32(np.arange(num)[::-1].copy()), BS, rows)
        self.seq, self.count = i32(np.zeros(requests)), i32([num])
        self.t, self.k, self.p = (to_dev(np.full(rows, v, d)) for v, d in ((0.8, np.float32), (50, np.int32), (0.95, np.float32)))

    def __call__(self, ids, new, max_rows, u):
        r = {}
        rows = ids.shape[0]
        r["plan"] = p = self.planner.plan(self.seq, new, self.count)
        r["x"] = x = self.embed[ids.long()]
        r["h"], _ = self.norms[0].rows8(x)
        r["qkv"] = self.qkv(r["h"])
        qkv = r["qkv"].clone().view(rows, HEADS + 2 * KV, DIM)
        q, k = self.rope(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], p.positions)
        r["turned"] = qkv
        self.cache.append(k, qkv[:, HEADS + KV:], p.slots)
        r["a"] = a = self.cache.attention(q, self.tables, p.seq_lens, p.cu_rows, max_rows)
        r["a8"] = decoder.quantize_rows(a.view(rows, HEADS * DIM))
        r["o"] = self.o(r["a8"])
        r["y"], r["res"] = self.norms[1](r["o"], x)
        r["logits"] = self.head(r["y"], out_dtype=torch.float32)
        r["tokens"], r["share"] = decoder.sample(r["logits"], self.t, u, self.k, self.p)
        return r


def test_prompts_then_tokens(gpu_lib):
    rng = np.random.default_rng(0)
    n, rows = 3, 48
    s = Step(n, 24, 8, rows)
    ids = to_dev(rng.integers(0, VOCAB, rows).astype(np.int32))
    for step, new in enumerate([[20, 7, 17], [1, 1, 1], [1, 0, 1], [5, 1, 1]] + [[1, 1, 1]] * 8):
        u = rng.random(rows).astype(np.float32)
        r = s(ids, to_dev(np.array(new), torch.int32), max(new), to_dev(u))
        torch.cuda.synchronize()
        p = r["plan"]
        assert p.status.cpu().tolist() == [0] * n
        s.seq, s.count = p.seq_lens, p.free_count
        live = sum(new)
        x = host64(r["x"])
        check8(r["h"], od.rms_norm(x, None, s.gamma[0], np.float32(1e-6))[1], HID)
        h = r["h"].codes.cpu().numpy(), r["h"].scales.cpu().numpy()
        assert np.array_equal(host64(r["qkv"]), od.linear8(*h, *s.w[0], None, True))
        qkv = host64(r["qkv"]).reshape(rows, HEADS + 2 * KV, DIM)
        turned, pos = host64(r["turned"]), p.positions.cpu().numpy()
        check_rope(turned[:, :HEADS + KV], qkv[:, :HEADS + KV], pos, s.rope.freqs.cpu().numpy(), False, 1.0)
        assert np.array_equal(turned[:, HEADS + KV:], qkv[:, HEADS + KV:])
        kc, ks, vc, vs = host_cache(s.cache)
        cu = np.concatenate([[0], np.cumsum(new)])
        want, mag, top, written = osv.attention(turned[:, :HEADS], kc, ks, vc, vs, s.tables.cpu().numpy(),
                                                p.seq_lens.cpu().numpy(), cu, True, 1 / math.sqrt(DIM), 99)
        tol = 2.0 ** -8 * np.abs(want) + (2 * (2 * DIM + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -20)[:, :, None] * mag
        a = host64(r["a"])
        assert (np.abs(a - want) <= tol)[written].all(), step
        codes, scales = od.quantize_rows(a.reshape(rows, -1), None)
        assert np.array_equal(r["a8"].codes.cpu().numpy(), codes) and np.array_equal(r["a8"].scales.cpu().numpy(), scales)
        assert np.array_equal(host64(r["o"]), od.linear8(codes, scales, *s.w[1], None, True))
        check_norm(host64(r["y"]), od.rms_norm(host64(r["o"]), x, s.gamma[1], np.float32(1e-6))[1], HID)
        logits = r["logits"].double().cpu().numpy()
        check_linear(logits, *s.head_ref(host64(r["y"])), HID, True)
        tokens = r["tokens"].cpu().numpy()
        for b in range(live):
            assert tokens[b] == od.sample_row(logits[b], float(np.float32(0.8)), float(u[b]), 50, float(np.float32(0.95)))[0]
        # the next tokens are the ones drawn for each request's last row
        last = np.maximum(cu[1:] - 1, 0)
        ids = to_dev(rng.integers(0, VOCAB, rows).astype(np.int32))
        ids[:n] = r["tokens"][to_dev(last)]


def test_captured_decoding_equals_eager(gpu_lib):
    """One captured step, replayed with new lengths, tokens and numbers, against eager steps on a twin;
    the program's own eager work runs between the replays."""
    rng = np.random.default_rng(1)
    n = 4
    eager, cap = Step(n, 20, 5, n), Step(n, 20, 5, n)
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    u = torch.zeros(n, device="cuda")
    new = torch.ones(n, dtype=torch.int32, device="cuda")
    seq, count = torch.zeros_like(new), torch.full((1,), 20, dtype=torch.int32, device="cuda")
    cap.seq, cap.count = seq, count
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = cap(ids, new, 1, u)
        seq.copy_(r["plan"].seq_lens)
        count.copy_(r["plan"].free_count)
        ids.copy_(r["tokens"])
    ids_e = torch.zeros_like(ids)
    ids.zero_()
    for step in range(12):
        us, add = to_dev(rng.random(n).astype(np.float32)), to_dev((rng.random(n) < 0.8).astype(np.int32))
        u.copy_(us)
        new.copy_(add)
        g.replay()
        e = eager(ids_e, add, 1, us)
        eager.seq, eager.count = e["plan"].seq_lens, e["plan"].free_count
        torch.cuda.synchronize()
        live = int(add.sum())
        assert torch.equal(seq, eager.seq) and torch.equal(cap.tables, eager.tables)
        for k in ("qkv", "turned", "a", "o", "y", "res", "logits", "tokens", "share"):
            assert torch.equal(r[k][:live], e[k][:live]), (step, k)
        ids_e = e["tokens"].clone()
        ids_e[live:] = 0
        ids[live:] = 0


def test_two_programs_on_two_streams(gpu_lib):
    rng = np.random.default_rng(2)
    us = [[to_dev(rng.random(2).astype(np.float32)) for _ in range(5)] for _ in range(2)]
    new = torch.ones(2, dtype=torch.int32, device="cuda")

    def program(i):
        s, out, ids = Step(2, 8, 4, 2, seed=i), [], torch.zeros(2, dtype=torch.int32, device="cuda")
        for u in us[i]:
            r = s(ids, new, 1, u)
            s.seq, s.count = r["plan"].seq_lens, r["plan"].free_count
            ids = r["tokens"]
            out += [r["logits"], r["tokens"], r["share"]]
        return s, out

    want = [program(i)[1] for i in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, st in enumerate([torch.cuda.Stream() for _ in range(2)]):
        with torch.cuda.stream(st):
            got.append(program(i))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(want[i], got[i][1]):
            assert torch.equal(a, b)


def test_calls_on_a_stream_that_is_not_current(gpu_lib):
    """The bindings take a stream; what runs on it does not wait for the current one's work."""
    from bit_post_quantized_amd import decoder_binding as DB
    x = torch.randn(33, 512, device="cuda").to(torch.bfloat16)
    want = decoder.quantize_rows(x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = decoder.Rows8.empty(33, 512)
    DB.svdq_quantize_rows(x, None, out.codes, out.scales, stream=st)
    st.synchronize()
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
