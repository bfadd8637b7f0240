"""NaN and infinities in what a decoding step is given: they stay in their row, or in their block
and head, and finite values beside them keep the bits they would have had."""
import numpy as np
import pytest
import torch

from oracle import serve as osv
from oracle.numerics import bf16_to_bits, decode_bf16
from tests.serve_cases import bf16_values, dev_cache, host64, host_cache, random_cache, to_dev, to_dev_bf16

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
            # every value of such a block and head reads as NaN, also after another token of it
            every = np.arange(num * bs)
            read = host64(cache.read(to_dev(every))[int(is_v)]).reshape(num, bs, heads, dim)
            assert np.isnan(read.transpose(0, 2, 1, 3)[lost]).all()
            assert np.isfinite(read.transpose(0, 2, 1, 3)[~lost]).all()
            b = runs[2][0]
            one = to_dev_bf16(bf16_values(rng, 1, heads, dim))
            cache.append(one, one, to_dev(np.array([b * bs + 5])))
            more = host_cache(cache)[3 if is_v else 1]
            np.testing.assert_array_equal(np.isfinite(more[b]), ~lost[b])
            cache.append(one, one, to_dev(np.array([b * bs])))      # begun anew
            assert np.isfinite(host_cache(cache)[3 if is_v else 1][b]).all()
