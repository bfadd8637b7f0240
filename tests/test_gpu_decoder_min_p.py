"""svdq_sample where min-p's border is among the smallest weights.  Weights are whole numbers, so
w >= least holds from 2^40 exp(x) = least - 1/2 on, up to 0.7 in x before least itself; with a top-p
whose limit lies farther down, what is between the two stays and can be drawn."""
import math

import numpy as np
import pytest

from tests.test_gpu_decoder_sample import check

pytestmark = pytest.mark.gpu

VOCAB, TOP = 104000, 50000


def at_a_bin(least):
    """The first least weight >= `least` of which a multiple of 28.5 / 2048 in x divides what rounds up."""
    for n in range(least, 16 * least):
        edge = math.floor(-math.log((n - 0.25) / 2.0 ** 40) * 2048 / 28.5) * -28.5 / 2048
        if 0.6 < 2.0 ** 40 * math.exp(edge) - (n - 1) < 0.9:
            return n
    raise AssertionError("no such weight")


@pytest.mark.parametrize("temperature", [1.0, 0.37])
@pytest.mark.parametrize("least", [1, 2, 3, 11, at_a_bin(500), at_a_bin(20000)])
def test_border_among_the_smallest_weights(gpu_lib, least, temperature):
    border = math.log((least - 0.5) / 2.0 ** 40)
    x = np.full(VOCAB, -40.0)
    # at the front what rounds up to `least`, and a little more; far behind it the largest; then, for top-p's limit,
    # more of what min-p takes away than 2^-24 of the sum (weights of 1 are not taken away by 1)
    x[:3000] = np.linspace(border + 1e-3 / least, math.log((least + 0.2) / 2.0 ** 40), 3000)
    x[TOP] = 0.0
    x[TOP + 1:TOP + 48001] = math.log(0.8 * (least - 0.5) / 2.0 ** 40) if least > 1 else border + 1e-4
    x[3000:50000] = x[TOP + 1]
    z = np.tile((x * temperature).astype(np.float32).astype(np.float64), (5, 1))
    u = np.array([0.0, 1e-10, 3e-9, 0.5, 0.99999994], np.float32)
    full = lambda v, d=np.float32: np.full(5, v, d)  # noqa: E731
    t, p, m = full(temperature), full(0.99999994), full(least / 2.0 ** 40)
    check(z, t, u, p=p, m=m)
    check(z, t, u, p=p, m=np.nextafter(m, np.float32(0)))
    check(z, t, u, m=m)
    check(z, t, u, k=full(2500, np.int32), p=p, m=m)
