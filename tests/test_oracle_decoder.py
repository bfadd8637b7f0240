"""The oracle of the operators between the projections, pinned by hand and by invariants."""
import math

import numpy as np
import pytest

from oracle import decoder as od


def test_norm_by_hand():
    h, y = od.rms_norm([[3.0, 4.0]], [[0.0, 0.0]], [2.0, 1.0], 0.0)
    assert h.tolist() == [[3.0, 4.0]]
    assert np.allclose(y, [[6 / math.sqrt(12.5), 4 / math.sqrt(12.5)]])
    _, y = od.rms_norm([[0.0, 0.0]], None, None, 0.0)
    assert y.tolist() == [[0.0, 0.0]]
    q, s = od.rows8(np.array([[127.0, -63.4, 0.0], [0.0, 0.0, 0.0]]))
    assert s.tolist() == [1.0, 0.0] and q.tolist() == [[127.0, -63.4, 0.0], [0.0, 0.0, 0.0]]


def test_rows_by_hand():
    c, s = od.quantize_rows([[254.0, -1.0, 3.0], [0.0, 0.0, 0.0], [math.inf, 1.0, 2.0]], [0.5, 1.0, 1.0])
    assert c.tolist() == [[127, -1, 3], [0, 0, 0], [0, 0, 0]] and s.tolist() == [1.0, 0.0, math.inf]
    c, s = od.quantize_rows([[1.0, math.nan]], None)
    assert c.tolist() == [[0, 0]] and math.isnan(s[0])


def test_product_by_hand():
    y = od.linear8([[1, -2], [127, 127]], [0.5, 2.0], [[3, 4], [127, 127]], [2.0, 1.0], [1.0, 0.0], False)
    assert y.tolist() == [[0.5 * -5 * 2 + 1, 0.5 * -127], [2 * 127 * 7 * 2 + 1, 2.0 * 2 * 127 * 127]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_by_the_angle(interleaved):
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    out, mag = od.rope(x, [1], [math.pi / 2, 0.0], interleaved, 2.0)
    if interleaved:
        assert np.allclose(out[0, 0], [-4, 2, 6, 8, 5, 6, 7, 8]) and mag[0, 0].tolist() == [6, 6, 14, 14, 0, 0, 0, 0]
    else:
        assert np.allclose(out[0, 0], [-6, 4, 2, 8, 5, 6, 7, 8]) and mag[0, 0].tolist() == [8, 12, 8, 12, 0, 0, 0, 0]


def test_sample_by_hand():
    z = [0.0, math.log(2.0), -math.inf, math.log(2.0)]      # weights 1 : 2 : 0 : 2
    assert od.weights(z, 1.0) == [1 << 39, 1 << 40, 0, 1 << 40]
    draw = lambda u, **k: od.sample_row(z, 1.0, u, **k)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.19, 0.21, 0.59, 0.61, 0.999)] == [0, 0, 1, 1, 3, 3]
    assert [draw(u, top_k=2) for u in (0.0, 0.49, 0.51)] == [1, 1, 3]
    assert [draw(u, top_k=1) for u in (0.0, 0.99)] == [1, 1]
    assert [draw(u, top_p=0.4) for u in (0.0, 0.99)] == [1, 1]       # 0.4 of the sum is reached by the first
    assert [draw(u, top_p=0.41) for u in (0.0, 0.99)] == [1, 3]
    assert [draw(u, min_p=0.6) for u in (0.0, 0.99)] == [1, 3]
    assert draw(0.9, top_p=0.0) == 1 and draw(0.9, min_p=5.0) == 3
    assert od.sample_row(z, 0.0, 0.9) == (1, 1.0) and od.sample_row([-math.inf] * 3, 1.0, 0.5) == (-1, 0.0)
    assert od.sample_row([0.0, math.nan], 1.0, 0.5) == (-1, 0.0)
    assert od.sample_row([0.0, math.inf, math.inf], 1.0, 0.6) == (2, 0.5)


def test_sample_shares_are_the_weights():
    rng = np.random.default_rng(0)
    z = rng.standard_normal(50) * 2
    p = np.exp(z / 0.7)
    p /= p.sum()
    edges = np.cumsum(p)
    for u in rng.random(200):
        token, share = od.sample_row(z, 0.7, u)
        assert token == int(np.searchsorted(edges, u, side="right")) and abs(share - p[token]) < 1e-11
