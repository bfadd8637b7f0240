"""The decoding step at the ends of its sizes and magnitudes."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import serve
from oracle.numerics import decode_bf16, round_bf16
from tests.serve_cases import bf16_values, dev_cache, host64, host_bits, random_cache, to_dev, to_dev_bf16
from tests.test_gpu_serve_attention import batch, check, run
from tests.test_gpu_serve_blocks import check_append

pytestmark = pytest.mark.gpu

LARGEST = float(decode_bf16(np.array([0x7F7F], np.uint16))[0])


# --------------------------------------------------------------------------------- read-back
@pytest.mark.parametrize("peak", [2.0 ** -133, 3e-39, 1e-30, 1.0, 2.0 ** 120, 2.0 ** 127, LARGEST])
@pytest.mark.parametrize("bs,dim", [(16, 64), (64, 128)])
def test_read_back_of_extreme_magnitudes(gpu_lib, bs, dim, peak):
    rng = np.random.default_rng(3)
    x = rng.uniform(-1, 1, (3 * bs + 5, 2, dim)) * peak
    x[::7, 0, 3], x[1::5, 1, 9] = peak, -peak
    x = round_bf16(x)
    slots = np.arange(bs, 4 * bs + 5)
    cache, ok, ov = check_append(9, 6, 2, bs, dim, list(slots), x=x)
    for order in (slots, rng.permutation(slots)):      # runs of 16 slots, and none
        k, v = cache.read(to_dev(order))
        np.testing.assert_array_equal(host_bits(k), ok.values(order))
        np.testing.assert_array_equal(host_bits(v), ov.values(order))
        assert np.isfinite(host64(k)).all() and (host64(k) != 0).any()


# --------------------------------------------------------------------------------- attention
def test_rows_of_a_request_that_the_batch_cuts_off(gpu_lib):
    # the last request has more rows than q holds: those that there are keep their causal limit
    for seq, rows, have, heads, dim in (([300, 90], [1, 9], 5, 2, 64), ([90, 500], [40, 300], 200, 1, 128)):
        c = batch(sum(seq), seq, rows, heads, 1, dim, 16)
        full = run(c, True, 0.125)
        check(c, full, True, 0.125)
        got = run(dict(c, q=c["q"][:have]), True, 0.125, max_rows=max(rows))
        np.testing.assert_array_equal(got, full[:have])


@pytest.mark.parametrize("kv_heads,heads,rows,dim,bs", [(1, 8, 5, 64, 128), (4, 32, 5, 128, 128), (1, 1, 64, 64, 64)])
def test_drafts_before_more_tokens_than_a_join_has_parts_for(gpu_lib, kv_heads, heads, rows, dim, bs):
    """More than 1024 x 4096 tokens under a wider table, whose entries repeat a few blocks: equal
    tokens count as often as the table names them.  The last blocks weigh most.  To the bounds of
    test_gpu_serve_attention come the sums of 1024 parts and of a part's tokens, 2^-15."""
    n, sm = 1024 * 4096 + 70001, 0.25
    rng = np.random.default_rng(dim + kv_heads)
    kc, ks, vc, vs = random_cache(rng, 7, kv_heads, bs, dim)
    ks[:] = np.float32(1 / 400)
    kc[:, :, :, 0] = 0
    kc[4:, :, :, 0] = 127
    used = -(-n // bs)
    table = np.full((1, used + 9000), -1)
    table[0, :used] = np.arange(used) % 4
    table[0, used - 600:used] = 4 + np.arange(600) % 3
    q = bf16_values(rng, rows, heads, dim)
    q[:, :, 0] = 40.0
    cache = dev_cache(kc, ks, vc, vs)
    i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
    for causal in (True, False):
        out = cache.attention(to_dev_bf16(q), i32(table), i32([n]), i32([0, rows]), rows, causal=causal, sm_scale=sm)
        got = host64(out)
        for i in range(rows):
            seen = n - rows + i + 1 if causal else n
            count = np.zeros((7, bs))
            np.add.at(count, table[0, :seen // bs], 1.0)
            count[table[0, seen // bs], :seen % bs] += 1.0
            for h in range(heads):
                k = (kc[:, h * kv_heads // heads] * ks[:, h * kv_heads // heads, None, None].astype(np.float64)).reshape(-1, dim)
                v = (vc[:, h * kv_heads // heads] * vs[:, h * kv_heads // heads, None, None].astype(np.float64)).reshape(-1, dim)
                s = sm * (k @ q[i, h])
                w = count.reshape(-1) * np.exp(s - s.max())
                w /= w.sum()
                top = sm * (np.abs(k) @ np.abs(q[i, h])).max()
                err = 2 * (2 * dim + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -15
                assert np.all(np.abs(got[i, h] - w @ v) <= 2.0 ** -8 * np.abs(w @ v) + err * (w @ np.abs(v))), (causal, i, h)


# ------------------------------------------------------------------------------------ linear
@pytest.mark.parametrize("power", [-100, -112, -118, -124])
def test_linear_of_a_few_tiny_activations(gpu_lib, power):
    """22 bits of every activation of a row of tiny ones (fp32 output): the bound of
    test_gpu_serve_linear, where two terms meet eight roundings or fewer (adding zeros is exact; half of
    the 2^-21 is theirs), each of 2^-149 at most below the normal range, where a matrix step may
    truncate and four of them come before a sum of its own size."""
    from tests.test_gpu_serve_linear import make
    rng = np.random.default_rng(8)
    K = 512
    x = np.zeros((24, K))
    for m in range(24):
        x[m, rng.integers(0, K, 1 + m % 2)] = rng.uniform(1, 2, 1 + m % 2) * 2.0 ** power
    x, pw, ref = make(power + 200, 24, K, 40, 0, False, x=round_bf16(x))
    y = host64(serve.DecodeLinear(pw)(to_dev_bf16(x), out_dtype=torch.float32))
    want, mag = ref(x)
    tol = 2.0 ** -24 * np.abs(want) + (2.0 ** -21 + 4 * 2.0 ** -24) * mag + 4 * 2.0 ** -149
    assert np.all(np.abs(y - want) <= tol), float((np.abs(y - want) / tol).max())
