"""Pins of the decoding step's oracle: hand examples, closed forms and invariants."""
import numpy as np

from oracle import serve as osv
from oracle.numerics import bf16_to_bits, decode_bf16, round_bf16


def test_linear_against_a_triple_loop():
    rng = np.random.default_rng(0)
    x = round_bf16(rng.standard_normal((2, 128)))
    inv = rng.random(128).astype(np.float32)
    codes = rng.integers(-8, 8, (3, 128))
    ws = rng.random((2, 3)).astype(np.float16)
    l1, l2, b = rng.standard_normal((128, 16)), rng.standard_normal((16, 3)), rng.standard_normal(3)
    y, a = osv.linear(bf16_to_bits(x), inv, l1, codes, ws, l2, b)
    for m in range(2):
        xh = [float(np.float32(x[m, k]) * inv[k]) for k in range(128)]
        for n in range(3):
            want = b[n] + sum(xh[k] * codes[n, k] * float(ws[k // 64, n]) for k in range(128))
            want += sum(sum(xh[k] * l1[k, j] for k in range(128)) * l2[j, n] for j in range(16))
            assert abs(y[m, n] - want) < 1e-10 and a[m, n] >= abs(want) - 1e-10


def test_plan_by_hand():
    # blocks of 16; request 0 fills its block exactly, 1 starts a block, 2 finds the list empty,
    # 3 needs no block, 4 is wider than its table
    got = osv.plan([10, 16, 0, 5, 47], [6, 1, 3, 2, 2], [[4, -1, -1], [2, -1, -1], [-1] * 3, [7, -1, -1],
                                                       [1, 3, 5]], 16, [9, 8], 1, 20)
    assert got["status"].tolist() == [0, 0, 1, 0, 2] and got["free_count"] == 0
    assert got["tables"][1].tolist() == [2, 9, -1] and got["tables"][2].tolist() == [-1] * 3
    assert got["cu"].tolist() == [0, 6, 7, 10, 12, 14] and got["seq"].tolist() == [16, 17, 0, 7, 47]
    assert got["slots"].tolist() == [4 * 16 + i for i in range(10, 16)] + [9 * 16] + [-1] * 3 + [7 * 16 + 5, 7 * 16 + 6] + [-1] * 8
    assert got["positions"].tolist()[:14] == list(range(10, 16)) + [16, 0, 1, 2, 5, 6, 47, 48]


def test_append_by_hand():
    c = osv.Cache(np.zeros((2, 1, 16, 4), int), np.full((2, 1), np.nan))
    c.append(np.array([[[127.0, 1.0, -1.5, 0.5]]]), [16])
    assert c.scale[1, 0] == 1 and c.codes[1, 0, 0].tolist() == [127, 1, -2, 0]       # ties to even
    c.append(np.array([[[254.0, 3.0, -254.0, 1.0]]]), [17])                          # the scale doubles
    assert c.scale[1, 0] == 2 and c.codes[1, 0, 0].tolist() == [64, 0, -1, 0]
    assert c.codes[1, 0, 1].tolist() == [127, 2, -127, 0] and np.isnan(c.scale[0, 0])
    c.append(np.array([[[2.0, 0.0, 0.0, 0.0]]]), [18])                               # and stays
    assert c.scale[1, 0] == 2 and c.codes[1, 0, 2].tolist() == [1, 0, 0, 0]
    c.append(np.zeros((1, 1, 4)), [16])                                              # a block begun anew
    assert c.scale[1, 0] == 0 and c.codes[1, 0, 0].tolist() == [0] * 4
    assert decode_bf16(c.values([17])).tolist() == [[[0.0] * 4]]


def test_append_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = round_bf16(rng.standard_normal((40, 2, 64)))
    c = osv.Cache(np.zeros((3, 2, 16, 64), int), np.zeros((3, 2)))
    c.append(x, np.arange(40))
    s = np.repeat(c.scale.astype(np.float64), 16, axis=0)[:40]
    val = c.codes.transpose(0, 2, 1, 3).reshape(48, 2, 64)[:40] * s[:, :, None]
    # half a step of the quotient, whose own fp32 rounding and that of s / amax each move a quotient
    # of up to 127 by at most 127 * 2^-24 < 2^-17
    assert (np.abs(val - x) <= (0.5 + 2.0 ** -16) * s[:, :, None]).all()
    assert (np.abs(c.codes).max(axis=(2, 3)) == 127).all()


def test_attention_closed_forms():
    # equal scores give the mean; one score far ahead gives its value; causal rows see their prefix
    num, bs, D = 3, 16, 64
    kc, vc = np.zeros((num, 1, bs, D), int), np.arange(num * bs)[:, None].repeat(D, 1).reshape(num, 1, bs, D)
    one = np.ones((num, 1), np.float32)
    q = np.ones((4, 1, D))
    tables, seq, cu = np.array([[2, 0], [-1, 1]]), [20, 18], [0, 2, 4]
    out, mag, top, written = osv.attention(q, kc, one, vc, one, tables, seq, cu, False, 1.0, 9)
    assert np.allclose(out[0], (sum(range(32, 48)) + 0 + 1 + 2 + 3) / 20)
    assert np.allclose(out[2], (16 + 17) / 2)          # the block outside the pool is left out
    out, *_ = osv.attention(q, kc, one, vc, one, tables, seq, cu, True, 1.0, 9)
    assert np.allclose(out[0], (sum(range(32, 48)) + 0 + 1 + 2) / 19) and np.allclose(out[1], mag[1])
    kc[0, 0, 3, 0] = 127
    out, *_ = osv.attention(q, kc, one, vc, one, tables, seq, cu, True, 1.0, 1)
    assert np.allclose(out[0], (sum(range(32, 48)) + 3) / 19)   # token 19 is hidden from row 0
    out, *_, written = osv.attention(q, kc, one, vc, one, tables, seq, cu, False, 1.0, 1)
    assert np.allclose(out[0], 3.0) and written.tolist() == [True, False, True, False]
