"""NaN and infinities in what a decoding step is given: they stay in their row, or in their block
and head, and finite values beside them keep the bits they would have had."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import serve
from oracle import serve as osv
from oracle.numerics import bf16_to_bits, decode_bf16
from tests.serve_cases import bf16_values, dev_cache, host64, host_cache, random_cache, to_dev, to_dev_bf16
from tests.test_gpu_serve_attention import batch, run

pytestmark = pytest.mark.gpu

NAN, NAN_ALL_ONES, INF, NEG_INF = 0x7FC0, 0xFFFF, 0x7F80, 0xFF80


def from_bits(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


# ------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("bad", [NAN, NAN_ALL_ONES, INF, NEG_INF])
@pytest.mark.parametrize("bs,dim", [(16, 64), (16, 128), (64, 128), (128, 64), (128, 128)])
def test_append_keeps_a_bad_value_in_its_block_and_head(gpu_lib, bs, dim, bad):
    # a single token and a run of three (short runs), a whole block and a tail that begins inside
    # one (long runs); the bad value in the first, an inner or the last row of each, in K or V
    heads, num = 3, 9
    runs = [(1, bs - 1, 1), (2, 0, 1), (3, 2, 3), (4, 0, bs), (5, 3, bs - 3), (6, 0, 3), (7, bs - 12, 12)]
    slots = np.concatenate([np.arange(b * bs + o, b * bs + o + n) for b, o, n in runs])
    rng = np.random.default_rng(bs + dim)
    kc, ks, vc, vs = random_cache(rng, num, heads, bs, dim)
    first = np.cumsum([0] + [n for *_, n in runs])
    for is_v in (False, True):
        for which in range(3):
            x = [bf16_to_bits(bf16_values(rng, len(slots), heads, dim, scale=40.0)) for _ in "kv"]
            hit = []
            for i, (b, _, n) in enumerate(runs):
                head = (i + which) % heads
                x[is_v][first[i] + (0, n // 2, n - 1)[which], head, (5, dim - 1, 0)[which]] = bad
                hit.append((b, head))
            cache, ok, ov = dev_cache(kc, ks, vc, vs), osv.Cache(kc, ks), osv.Cache(vc, vs)
            cache.append(from_bits(x[0]), from_bits(x[1]), to_dev(slots))
            ok.append(decode_bf16(x[0]), slots)
            ov.append(decode_bf16(x[1]), slots)
            torch.cuda.synchronize()
            got = host_cache(cache)
            for g, w in zip(got, (ok.codes, ok.scale, ov.codes, ov.scale)):
                np.testing.assert_array_equal(g, w)
            scale = got[3 if is_v else 1]
            lost = np.zeros_like(scale, dtype=bool)
            lost[tuple(np.array(hit).T)] = True
            np.testing.assert_array_equal(np.isfinite(scale), ~lost)
            # every token of such a block and head reads as NaN, also after another token of it
            every = np.arange(num * bs)
            read = host64(cache.read(to_dev(every))[int(is_v)]).reshape(num, bs, heads, dim)
            for b, o, n in runs:
                assert np.isnan(read[b, :o + n, lost[b]]).all()
            assert np.isfinite(read.transpose(0, 2, 1, 3)[~lost]).all()
            b = runs[2][0]
            one = to_dev_bf16(bf16_values(rng, 1, heads, dim))
            cache.append(one, one, to_dev(np.array([b * bs + 5])))
            more = host_cache(cache)[3 if is_v else 1]
            np.testing.assert_array_equal(np.isfinite(more[b]), ~lost[b])
            cache.append(one, one, to_dev(np.array([b * bs])))      # begun anew
            assert np.isfinite(host_cache(cache)[3 if is_v else 1][b]).all()


# --------------------------------------------------------------------------------- attention
SHAPES = [
    ([200, 90], [2, 2], 8, 2, 64, 16, None),            # few rows
    ([300, 40], [1, 1], 34, 2, 64, 16, None),           # two tiles of them
    ([9000, 50, 4096], [4, 1, 2], 8, 2, 128, 16, 600),  # in equal shares
    ([600, 130], [300, 129], 3, 1, 64, 64, None),       # eight waves
    ([450, 90], [450, 33], 2, 2, 128, 16, None),        # two row tiles
    ([200, 150], [20, 17], 2, 2, 64, 32, None),         # one
    ([20000, 77], [5, 2], 8, 1, 128, 64, 320),          # chunks, joined per row
    ([5000, 64], [100, 64], 2, 1, 128, 16, 320),        # chunks, joined by lanes
]


def tolerance(c, want, mag, top):
    D = c["q"].shape[2]
    err = (2 * (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -20)[:, :, None] * mag
    return 2.0 ** -8 * np.abs(want) + err


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][0]}x{s[1][0]}x{s[2]}x{s[4]}")
def test_a_bad_query_stays_in_its_row(gpu_lib, shape):
    seq, rows, heads, kv_heads, dim, bs, width = shape
    c = batch(sum(seq) + 1, seq, rows, heads, kv_heads, dim, bs, width=width)
    bits = bf16_to_bits(c["q"])
    hit = [(0, heads - 1, NAN, 5), (rows[0] - 1, 0, NAN_ALL_ONES, 0), (rows[0], heads // 2, INF, dim - 1)]
    for t, h, bad, d in hit:
        bits[t, h, d] = bad
    got = run(c, True, 0.125, q=from_bits(bits))
    want, mag, top, _ = osv.attention(c["q"], *c["cache"], c["tables"], c["seq"], c["cu"], True, 0.125, 1 << 30)
    keep = np.ones(got.shape[:2], bool)
    for t, h, bad, _ in hit:
        assert np.isnan(got[t, h]).all() if bad in (NAN, NAN_ALL_ONES) else not np.isfinite(got[t, h]).any(), (t, h)
        keep[t, h] = False
    assert (np.abs(got - want) <= tolerance(c, want, mag, top))[keep].all()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][0]}x{s[1][0]}x{s[2]}x{s[4]}")
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_bad_block_is_seen_by_its_rows_only(gpu_lib, shape, value):
    # the last block of each request is bad in one cached head: its last row sees it, rows whose
    # causal limit ends before it, and the other head's, do not
    seq, rows, heads, kv_heads, dim, bs, width = shape
    for which in (1, 3):                              # K's scales, then V's
        c = batch(sum(seq) + 2, seq, rows, heads, kv_heads, dim, bs, width=width)
        kc, ks, vc, vs = c["cache"]
        good = (kc, ks.copy(), vc, vs.copy())
        for b, s in enumerate(seq):
            last = c["tables"][b, -(-s // bs) - 1]
            c["cache"][which][last, 0] = value
            kc[last, 0], vc[last, 0] = 0, 0           # as an append leaves it: NaN whatever the code
        got = run(c, True, 0.125)
        want, mag, top, _ = osv.attention(c["q"], *good, c["tables"], c["seq"], c["cu"], True, 0.125, 1 << 30)
        sees = np.zeros(got.shape[:2], bool)
        for b, s in enumerate(seq):
            for i in range(rows[b]):
                sees[c["cu"][b] + i, :heads // kv_heads] = s - rows[b] + i >= (-(-s // bs) - 1) * bs
        assert sees.any() and np.isnan(got[sees]).all()
        assert (np.abs(got - want) <= tolerance(c, want, mag, top))[~sees].all()


# ------------------------------------------------------------------------------------ linear
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [NAN, 0x7FFF, NAN_ALL_ONES])
@pytest.mark.parametrize("M,K,N,r", [(3, 256, 50, 16), (20, 64 * 70, 33, 0), (1, 64 * 129, 40, 32)])
def test_a_nan_of_any_payload_makes_its_row_nan(gpu_lib, M, K, N, r, bad, dtype):
    from tests.test_gpu_serve_linear import check, make
    x, pw, ref = make(M + K, M, K, N, r, True)
    bits = bf16_to_bits(x)
    bits[M - 1, 7] = bad
    y = host64(serve.DecodeLinear(pw)(from_bits(bits), out_dtype=dtype))
    assert np.isnan(y[M - 1]).all()
    want, mag = ref(x)
    check(y[:M - 1], want[:M - 1], mag[:M - 1], K, dtype == torch.float32)


def test_a_nan_bias_makes_its_column_nan(gpu_lib):
    from tests.test_gpu_serve_linear import make
    for K in (128, 64 * 70):
        x, pw, _ = make(K, 20, K, 33, 16, True)
        pw.bias[5:7] = from_bits(np.array([0x7FFF, 0xFFFF], np.uint16))
        y = host64(serve.DecodeLinear(pw)(to_dev_bf16(x)))
        assert np.isnan(y[:, 5:7]).all() and np.isfinite(np.delete(y, (5, 6), 1)).all()
