"""kv_block_attention over V scales that an append can make: subnormal, zero, far apart.

Bounds, beside those of test_gpu_serve_attention (a score's error, 2^-11 of a weight, the store's
2^-8): a weight carries its block's V scale through log2, whose value and sum with the score are at
most 2^8, so each of the three roundings there is at most 2^-17 and they move a weight by
3 ln 2 2^-17 < 2^-15.  A weight is held to 2^-25 where the row's largest is 2^10 or more, which is
2^-35 of the largest weight times scale for each of n tokens' codes.  A block whose scale is under
2^-80 of the largest may count as one of 2^-80, 2^-64 of the largest value at most in all.  Outputs
below bf16's normal range are off by half its smallest step, 2^-134."""
import numpy as np
import pytest

from oracle import serve as osv
from tests.test_gpu_serve_attention import batch, run

pytestmark = pytest.mark.gpu

# every kernel: few rows whole and in equal shares, more rows of 64 and 128 channels, cut into
# chunks that either join adds
SHAPES = [
    ([640, 100], [2, 1], 4, 2, 128, 16, None),
    ([300, 40], [1, 1], 34, 2, 64, 16, None),
    ([9000, 50, 4096], [1, 1, 1], 8, 2, 128, 16, 600),
    ([300] * 70, [1] * 70, 2, 1, 64, 128, 64),
    ([600, 130], [300, 129], 3, 1, 64, 64, None),
    ([450, 90], [450, 33], 2, 2, 128, 16, None),
    ([200, 150], [20, 17], 2, 2, 64, 32, None),
    ([20000, 77], [5, 2], 8, 1, 128, 64, 320),
    ([5000, 64], [100, 64], 2, 1, 128, 16, 320),
]


def check(c, got, causal, sm_scale):
    want, mag, top, written = osv.attention(c["q"], *c["cache"], c["tables"], c["seq"], c["cu"],
                                            causal, sm_scale, 1 << 30)
    D = c["q"].shape[2]
    used = c["cache"][3][c["tables"][c["tables"] >= 0]]
    err = (2 * (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -11 + 2.0 ** -15)[:, :, None] * mag
    tol = 2.0 ** -8 * np.abs(want) + err + max(c["seq"]) * 127 * 2.0 ** -35 * mag.max(axis=2, keepdims=True)
    tol += 2.0 ** -64 * 127 * float(used.max()) + 2.0 ** -134
    assert np.isfinite(got[written]).all()
    bad = np.abs(got - want)[written] > tol[written]
    assert not bad.any(), float((np.abs(got - want) / tol)[written].max())
    return want


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][0]}x{s[1][0]}x{s[2]}x{s[4]}")
@pytest.mark.parametrize("kind", ["subnormal", "one", "small", "zeros", "zeros_beside_small", "all"])
def test_v_scales_of_every_size(gpu_lib, shape, kind):
    seq, rows, heads, kv_heads, dim, bs, width = shape
    c = batch(sum(seq) + dim + len(kind), seq, rows, heads, kv_heads, dim, bs, width=width)
    kc, ks, vc, vs = c["cache"]
    rng = np.random.default_rng(7)
    some = rng.random(vs.shape) < 0.3
    if kind == "subnormal":            # blocks appended from values near 1e-40
        vs[:] = (2.0 ** rng.uniform(-148, -127, vs.shape)).astype(np.float32)
    elif kind == "one":                # a few such blocks among ordinary ones
        vs[some] = np.float32(2.0 ** -140)
    elif kind == "small":
        vs[:] = (10.0 ** rng.uniform(-36, -9, vs.shape)).astype(np.float32)
    elif kind == "zeros":
        vs[:], vc[:] = 0.0, 0
    elif kind == "zeros_beside_small":  # zero blocks of high scores hide nothing of the others
        vs[:] = np.float32(1e-11)
        vs[some], vc[some] = 0.0, 0
        ks[some] *= 8.0
    else:
        vs[:] = (2.0 ** rng.uniform(-140, 121, vs.shape)).astype(np.float32)
        vs[some], vc[some] = 0.0, 0
    for causal in (True, False):
        want = check(c, run(c, causal, 0.1), causal, 0.1)
        assert (want != 0).any() == (kind != "zeros")


@pytest.mark.parametrize("order", [1, -1])
def test_scales_that_grow_or_shrink_along_a_sequence(gpu_lib, order):
    # block after block 2^18 larger (or smaller): sums follow the unit of the largest scale
    for dim, rows, heads in ((64, 1, 4), (128, 40, 2), (64, 200, 1)):
        c = batch(dim + rows, [320], [rows], heads, 1, dim, 32)
        for k, b in enumerate(c["tables"][0]):
            c["cache"][3][b] = np.float32(2.0 ** (order * (18 * k - 81)))
        for causal in (True, False):
            check(c, run(c, causal, 0.1), causal, 0.1)
