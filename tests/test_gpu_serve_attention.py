"""kv_block_attention against fp64 attention over the exact values of the cache.

Bounds, for a row with weights w and values v: a score's fp32 error is at most (2 D + 4) 2^-24
times sm_scale sum_d |q_d K_td| (a matrix step may truncate, hence 2 per product; the queries and
codes are exact) plus the factor's and the FMA's roundings, 4 * 2^-24 of the score; exp2 adds 2^-22.
A weight enters the product rounded to fp16, 2^-11 relative. Weights and their sum both carry the
score error, so the output is off by at most 2 (score error) + 2^-11 + 2^-20 of sum_t w_t |v_t|, and
the store rounds by 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

from bit_post_quantized_amd import serve
from oracle import serve as osv
from tests.serve_cases import bf16_values, dev_cache, host64, random_cache, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def batch(seed, seq, rows, heads, kv_heads, dim, bs, width=None, extra=0, spare=3):
    """Ragged requests over a random pool: seq tokens cached and rows query rows each."""
    rng = np.random.default_rng(seed)
    need = [-(-s // bs) for s in seq]
    width = max(max(need), 1) if width is None else width
    num = sum(need) + spare
    ids = rng.permutation(num)
    tables = np.full((len(seq), width), -1)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = ids[at:at + k]
        at += k
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    q = bf16_values(rng, int(cu[-1]) + extra, heads, dim)
    return dict(q=q, cache=random_cache(rng, num, kv_heads, bs, dim), tables=tables, seq=np.array(seq),
                cu=cu, unused=ids[at:])


def run(c, causal, sm_scale, max_rows=None, cache=None, q=None, workspace=None):
    q = to_dev_bf16(c["q"]) if q is None else q
    out = torch.full((c["q"].shape[0],) + tuple(q.shape[1:]), 99.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: to_dev(a, torch.int32)  # noqa: E731
    most = int(np.diff(c["cu"]).max(initial=1)) if max_rows is None else max_rows
    (dev_cache(*c["cache"]) if cache is None else cache).attention(
        q, i32(c["tables"]), i32(c["seq"]), i32(c["cu"]), max(most, 1), causal=causal,
        sm_scale=sm_scale, out=out, workspace=workspace)
    torch.cuda.synchronize()
    return host64(out)


def check(c, got, causal, sm_scale, max_rows=1 << 30):
    want, mag, top, written = osv.attention(c["q"], *c["cache"], c["tables"], c["seq"], c["cu"],
                                            causal, sm_scale, max_rows)
    D = c["q"].shape[2]
    err = (2 * (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -20)[:, :, None] * mag
    tol = 2.0 ** -8 * np.abs(want) + err
    bad = np.abs(got - want)[written] > tol[written]
    assert not bad.any(), float((np.abs(got - want)[written] / np.maximum(tol[written], 1e-30)).max())
    assert (got[~written] == 99.0).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("seq,rows,heads,kv_heads,dim,bs", [
    ([1], [1], 1, 1, 64, 16),
    ([1, 2, 15, 16, 17, 31, 33], [1] * 7, 2, 1, 64, 16),
    ([63, 64, 65, 127, 128, 129], [1] * 6, 4, 4, 128, 32),
    ([0, 255, 0, 256, 257, 0], [1] * 6, 8, 2, 128, 64),
    ([511, 513, 1], [1] * 3, 6, 2, 64, 128),
    ([1000, 3, 700], [1, 1, 1], 16, 1, 128, 16),          # 16 query heads to one cached head
    ([300, 40], [1, 1], 34, 2, 64, 16),                   # 17: a second row tile with one row
    ([300, 40], [1, 1], 128, 1, 128, 32),                 # 128 to one
    ([5, 100, 333, 64], [5, 1, 7, 2], 8, 4, 64, 16),      # draft tokens, a prompt without a cache
    ([40, 200, 3], [40, 17, 0], 4, 2, 128, 16),           # no rows for a request
    ([7, 90, 128, 0], [20, 90, 33, 5], 6, 3, 64, 32),     # more rows than tokens: empty rows
    ([600, 130], [300, 129], 3, 1, 64, 64),               # chunks of a prompt
    ([450], [450], 2, 2, 128, 128),
])
def test_matches_the_oracle(gpu_lib, seq, rows, heads, kv_heads, dim, bs, causal):
    c = batch(sum(seq) + heads, seq, rows, heads, kv_heads, dim, bs)
    sm = 1.0 / math.sqrt(dim)
    check(c, run(c, causal, sm), causal, sm)


@pytest.mark.parametrize("bs,dim", [(16, 64), (16, 128), (32, 64), (64, 128), (128, 64), (128, 128)])
def test_long_rows_split_over_workgroups(gpu_lib, bs, dim):
    c = batch(bs + dim, [9000, 1, 4097, 300], [2, 1, 1, 1], 8, 2, dim, bs, width=9600 // bs)
    sm = 1.0 / math.sqrt(dim)
    for causal in (False, True):
        check(c, run(c, causal, sm), causal, sm)


@pytest.mark.parametrize("seq,rows,heads,kv_heads,dim,bs,width", [
    ([20000, 77], [5, 2], 8, 1, 64, 64, 320), ([20000, 77], [5, 2], 8, 1, 128, 16, 1250),   # 40 rows: 64 to a workgroup
    ([2100, 900], [5, 4], 8, 1, 64, 128, 17), ([2100, 900], [4, 5], 8, 1, 128, 32, 66),
    ([5000, 64], [100, 64], 1, 1, 64, 16, 320), ([5000, 64], [100, 64], 2, 1, 128, 64, 80),  # 128
    ([9000], [33], 34, 2, 64, 128, 71), ([4096], [150], 3, 3, 128, 16, 256),
])
def test_many_rows_split_over_workgroups(gpu_lib, seq, rows, heads, kv_heads, dim, bs, width):
    from bit_post_quantized_amd import serve_binding as SB
    assert SB.kv_block_attention_workspace_bytes(len(seq), sum(rows), max(rows), heads, kv_heads, dim, width, bs)
    c = batch(sum(seq) + dim, seq, rows, heads, kv_heads, dim, bs, width=width)
    sm = 1.0 / math.sqrt(dim)
    for causal in (False, True):
        check(c, run(c, causal, sm), causal, sm)


def test_many_short_requests_under_a_wide_table(gpu_lib):
    # 300 requests: no cut for the workgroups' sake, but chunks of 16384 tokens under this table
    rng = np.random.default_rng(6)
    seq = [int(x) for x in rng.integers(0, 40, 300)]
    seq[17] = 17000
    c = batch(9, seq, [1] * 300, 2, 1, 64, 128, width=400)
    check(c, run(c, True, 0.125), True, 0.125)


@pytest.mark.parametrize("seq,rows,heads,kv_heads,dim,bs,width", [
    ([0] * 5 + [1] + [0] * 3, [1] * 9, 2, 1, 64, 16, 600),               # one unit each, mostly of nothing
    ([5000], [0], 1, 1, 128, 16, 400), ([0], [1], 1, 1, 128, 16, 400),
    ([300, 5000, 255, 256, 257, 0, 4000], [1, 0, 2, 0, 1, 1, 3], 8, 2, 64, 32, 256),
    ([16384, 9, 700], [1, 1, 1], 32, 2, 64, 128, 200),                   # two row tiles
    ([4097, 4096, 8192], [4, 4, 4], 4, 1, 128, 16, 600),
    ([20000, 3, 3, 3, 900], [2, 1, 2, 1, 2], 6, 3, 128, 64, 400),
    ([513] * 40, [1] * 40, 4, 4, 64, 16, 512),
])
def test_few_rows_in_equal_shares(gpu_lib, seq, rows, heads, kv_heads, dim, bs, width):
    from bit_post_quantized_amd import serve_binding as SB
    assert sum(rows) == 0 or SB.kv_block_attention_workspace_bytes(
        len(seq), sum(rows), max(max(rows), 1), heads, kv_heads, dim, width, bs)
    c = batch(sum(seq) + bs, seq, rows, heads, kv_heads, dim, bs, width=width, extra=2)
    for causal in (False, True):
        check(c, run(c, causal, 0.1), causal, 0.1)


@pytest.mark.parametrize("n,heads,dim,bs,width", [(40, 8, 128, 16, 1500), (300, 11, 64, 64, 300), (4100, 33, 64, 128, 40)])
def test_uneven_requests_of_drafts(gpu_lib, n, heads, dim, bs, width):
    # more than 16 (32) rows x heads each, chunks of a long table; some without rows, some without tokens
    rng = np.random.default_rng(n)
    rows = rng.integers(1, 6, n) * (rng.random(n) < 0.8)
    rows[:3] = 5 if n < 1000 else 1
    if n > 1000:
        rows[3:] = 0
        rows[rng.integers(3, n, 30)] = 1
    seq = rng.integers(0, 50, n)
    seq[[1, n // 2]] = min(17000, width * bs), 4100
    c = batch(n, [int(x) for x in seq], [int(x) for x in rows], heads, 1, dim, bs, width=width)
    check(c, run(c, True, 0.1), True, 0.1)


@pytest.mark.parametrize("n,kv_heads,width", [(700, 3, 200), (4096, 1, 300), (4097, 1, 300)])
def test_many_uneven_requests(gpu_lib, n, kv_heads, width):
    # shares of thousands of requests, several to a thread that adds them up; one more and none is cut
    rng = np.random.default_rng(n)
    seq, rows = rng.integers(0, 60, n), rng.integers(0, 3, n)
    seq[rng.integers(0, n, 3)] = [9000, 3000, 12000]
    c = batch(n, [int(x) for x in seq], [int(x) for x in rows], 2 * kv_heads, kv_heads, 64, 64, width=width)
    check(c, run(c, True, 0.125), True, 0.125)


@pytest.mark.parametrize("seq,rows,heads,kv_heads,dim,bs,width", [
    ([9000, 50, 4096], [1, 1, 1], 8, 2, 128, 16, 600), ([9000, 50, 4096], [4, 3, 4], 8, 2, 64, 16, 600),
    ([300] * 70, [1] * 70, 2, 1, 64, 128, 64), ([20000, 30], [5, 5], 16, 1, 128, 64, 320),
    ([5000, 600], [70, 64], 2, 1, 64, 16, 320), ([5000, 600], [70, 64], 2, 1, 128, 16, 320),
])
def test_the_workspace_holds_what_it_says(gpu_lib, seq, rows, heads, kv_heads, dim, bs, width):
    from bit_post_quantized_amd import serve_binding as SB
    c = batch(sum(seq) + width, seq, rows, heads, kv_heads, dim, bs, width=width)
    need = SB.kv_block_attention_workspace_bytes(len(seq), sum(rows), max(rows), heads, kv_heads, dim, width, bs)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    check(c, run(c, True, 0.1, workspace=ws[:need]), True, 0.1)
    assert need > 0 and (ws[need:] == 0xA5).all()


def test_shares_follow_the_lengths_in_a_graph(gpu_lib):
    c = batch(92, [6000, 3000, 0, 900], [1, 2, 1, 1], 8, 2, 128, 16, width=700)
    c["tables"][3, :] = c["tables"][0, :]
    cache = dev_cache(*c["cache"])
    i32 = lambda a: to_dev(a, torch.int32)  # noqa: E731
    q, tables, seq, cu = to_dev_bf16(c["q"]), i32(c["tables"]), i32(c["seq"]), i32(c["cu"])
    out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attention(q, tables, seq, cu, 2, sm_scale=0.1, out=out)
    for lens in ([6000, 3000, 0, 900], [1, 0, 0, 0], [6000, 5, 1, 6000], [0, 0, 0, 0], [300, 3000, 4000, 1]):
        seq.copy_(i32(np.array(lens)))
        g.replay()
        eager = cache.attention(q, tables, seq, cu, 2, sm_scale=0.1)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), lens
        check(dict(c, seq=np.array(lens)), host64(eager), True, 0.1)


def test_split_rows_with_bad_entries_on_two_streams_and_in_a_graph(gpu_lib):
    c = batch(91, [6000, 700], [6, 6], 8, 1, 64, 32, width=200)
    c["tables"][0, 40:75], c["tables"][1, 3] = -1, 10 ** 6
    cache = dev_cache(*c["cache"])
    i32 = lambda a: to_dev(a, torch.int32)  # noqa: E731
    q, tables, seq, cu = to_dev_bf16(c["q"]), i32(c["tables"]), i32(c["seq"]), i32(c["cu"])
    first = cache.attention(q, tables, seq, cu, 6, sm_scale=0.125)
    check(c, host64(first), True, 0.125)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs += [cache.attention(q, tables, seq, cu, 6, sm_scale=0.125) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    out, g = torch.zeros_like(first), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attention(q, tables, seq, cu, 6, sm_scale=0.125, out=out)
    for lens in ([6000, 700], [5, 0], [700, 6000], [6000, 700]):
        seq.copy_(i32(np.array(lens)))
        g.replay()
        eager = cache.attention(q, tables, seq, cu, 6, sm_scale=0.125)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), lens
    assert torch.equal(out, first)


def test_sharp_flat_and_signed_scores(gpu_lib):
    c = batch(77, [700, 260], [3, 1], 4, 2, 64, 16)
    for sm in (3.0, 0.0, 1e-20, -0.2):
        check(c, run(c, True, sm), True, sm)


def test_scales_of_very_different_blocks(gpu_lib):
    # V scales from 1e-12 to 1e12 and blocks of zero scale (whose codes are zero)
    c = batch(78, [640, 100], [2, 1], 4, 2, 128, 16)
    kc, ks, vc, vs = c["cache"]
    rng = np.random.default_rng(0)
    vs[:] = (10.0 ** rng.uniform(-12, 12, vs.shape)).astype(np.float32)
    zero = rng.random(vs.shape) < 0.2
    vs[zero], vc[zero] = 0.0, 0
    zero = rng.random(ks.shape) < 0.2
    ks[zero], kc[zero] = 0.0, 0
    sm = 0.1
    check(c, run(c, True, sm), True, sm)


def test_queries_of_any_magnitude(gpu_lib):
    c = batch(79, [100, 50, 70], [1, 1, 1], 4, 2, 64, 16)
    c["q"][0] *= 2.0 ** 60
    c["q"][1] *= 2.0 ** -60
    c["q"][2] = 0.0
    kc, ks, vc, vs = c["cache"]
    ks *= np.float32(2.0 ** -60)
    check(c, run(c, False, 0.125), False, 0.125)


def test_what_lies_behind_a_sequence_is_not_read(gpu_lib):
    """Blocks no sequence holds, and table entries behind one, have NaN scales and any codes; rows
    behind the last request and rows past max_rows keep what they held."""
    c = batch(80, [33, 0, 130], [2, 1, 4], 4, 2, 64, 32, width=6, extra=3)
    kc, ks, vc, vs = c["cache"]
    for b in c["unused"]:
        ks[b], vs[b] = np.nan, np.inf
    c["tables"][0, 2:] = c["unused"][0]           # stale entries of an earlier sequence
    c["tables"][1, :] = c["unused"][1]
    sm = 0.125
    check(c, run(c, True, sm), True, sm)
    check(c, run(c, True, sm, max_rows=2), True, sm, max_rows=2)


def test_bad_table_entries_are_left_out(gpu_lib):
    c = batch(81, [200, 64, 20], [1, 2, 1], 4, 2, 64, 16)
    num = c["cache"][0].shape[0]
    c["tables"][0, 3], c["tables"][0, 7] = -1, num
    c["tables"][1, 0], c["tables"][2, :2] = -(1 << 31), 2 ** 31 - 1
    for causal in (False, True):
        check(c, run(c, causal, 0.125), causal, 0.125)


def test_lengths_outside_the_table_are_clamped(gpu_lib):
    c = batch(82, [64, 48], [1, 1], 2, 1, 64, 16)
    got = run(dict(c, seq=np.array([2 ** 31 - 1, -5])), False, 0.125)
    check(dict(c, seq=np.array([64, 0])), got, False, 0.125)


def test_non_finite_queries_stay_in_their_row(gpu_lib):
    c = batch(83, [200, 90], [2, 2], 8, 2, 64, 16)
    q = to_dev_bf16(c["q"])
    q[1, 3, 5], q[2, 0, 0] = float("nan"), float("inf")
    got = run(c, True, 0.125, q=q)
    assert np.isnan(got[1, 3]).all() and np.isnan(got[2, 0]).any()
    keep = dict(c)
    want, mag, top, _ = osv.attention(c["q"], *c["cache"], c["tables"], c["seq"], c["cu"], True, 0.125, 99)
    sel = np.ones(got.shape[:2], bool)
    sel[1, 3] = sel[2, 0] = False
    tol = 2.0 ** -8 * np.abs(want) + (2 * (2 * 64 + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -20)[:, :, None] * mag
    assert (np.abs(got - want) <= tol)[sel].all()
    assert keep is not c


def test_strided_queries_and_a_shared_workspace(gpu_lib):
    c = batch(84, [3000, 100], [1, 1], 4, 2, 128, 16)
    fused = torch.zeros(2, 9, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:6] = to_dev_bf16(c["q"])
    cache = dev_cache(*c["cache"])
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    sm = 0.09
    for _ in range(2):
        check(c, run(c, True, sm, cache=cache, q=fused[:, 2:6], workspace=ws), True, sm)
    d = batch(85, [700, 5000], [3, 1], 8, 1, 64, 64)
    check(d, run(d, False, sm, workspace=ws), False, sm)


def test_a_long_flat_row(gpu_lib):
    # 150 000 tokens of equal weight 1 and one far ahead: small weights are not lost in fp16
    n = 150000
    c = batch(86, [n], [1], 2, 1, 64, 128)
    kc, ks, vc, vs = c["cache"]
    kc[:] = 0
    vc[:] = np.abs(vc)
    kc[c["tables"][0, 5], 0, 7, 0] = 100
    ks[:] = 0.01
    c["q"][:] = 0.0
    c["q"][0, :, 0] = [8.0, 12.0]         # scores 8 and 12 against 0
    check(c, run(c, False, 1.0), False, 1.0)


def test_same_bits_on_another_stream_and_in_a_graph(gpu_lib):
    c = batch(87, [900, 300, 0], [1, 1, 1], 8, 2, 128, 16, width=64)
    cache = dev_cache(*c["cache"])
    i32 = lambda a: to_dev(a, torch.int32)  # noqa: E731
    q, tables, seq, cu = to_dev_bf16(c["q"]), i32(c["tables"]), i32(c["seq"]), i32(c["cu"])
    first = cache.attention(q, tables, seq, cu, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(cache.attention(q, tables, seq, cu, 1), first)
    torch.cuda.synchronize()
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attention(q, tables, seq, cu, 1, out=out)
    for lens in ([900, 300, 0], [30, 1, 0], [899, 0, 0]):   # the lengths live on the device
        seq.copy_(i32(np.array(lens)))
        g.replay()
        eager = cache.attention(q, tables, seq, cu, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), lens


def test_attention_refusals(gpu_lib):
    c = batch(88, [64], [1], 4, 2, 64, 16)
    cache = dev_cache(*c["cache"])
    i32 = lambda a: to_dev(a, torch.int32)  # noqa: E731
    q, tables, seq, cu = to_dev_bf16(c["q"]), i32(c["tables"]), i32(c["seq"]), i32(c["cu"])
    with pytest.raises(RuntimeError, match="heads"):
        cache.attention(q[:, :3].contiguous(), tables, seq, cu, 1)
    with pytest.raises(RuntimeError, match="sm_scale"):
        cache.attention(q, tables, seq, cu, 1, sm_scale=float("inf"))
    with pytest.raises(RuntimeError, match="max_rows"):
        cache.attention(q, tables, seq, cu, 0)
    with pytest.raises(ValueError, match="fit 32 bits"):   # 2^32 + 1 is not 1
        cache.attention(q, tables, seq, cu, (1 << 32) + 1)
    with pytest.raises(ValueError, match="seq_lens must be"):
        cache.attention(q, tables, seq.long(), cu, 1)
    with pytest.raises(ValueError, match="cu_rows must have shape"):
        cache.attention(q, tables, seq, cu[:1], 1)
    with pytest.raises(ValueError, match="q must be"):
        cache.attention(q[..., :32], tables, seq, cu, 1)
    none = cache.attention(q[:0], tables, seq, torch.zeros_like(cu), 1)
    assert none.shape[0] == 0
