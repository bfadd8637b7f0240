"""svdq_rope against fp64.

Bounds.  The angle is off by |t| 2^-51 (the product and the frequency in half turns), its remainder by
2^-25 half turns; sine and cosine are within 4 steps of fp32, the factor, the two products and their
sum add 4 roundings: (2^-20 + |t| 2^-51) (|a| + |b|) |scale| covers them twofold.  The store rounds by
2^-8 of the value; copied channels are exact (bf16) or rounded once."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import decoder
from oracle import decoder as od
from oracle.numerics import round_bf16
from tests.serve_cases import bf16_values, host64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def check(got, x, pos, freqs, inter, scale):
    want, mag = od.rope(x, pos, freqs, inter, scale)
    t = np.abs(np.asarray(pos, np.float64)).max(initial=0) * np.abs(freqs).max()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + t * 2.0 ** -51) * mag + 2.0 ** -133
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
    rest = slice(2 * len(freqs), None)
    assert np.array_equal(got[:, :, rest], round_bf16(x[:, :, rest]))


def case(seed, rows, heads, kv, dim, rot, x32, far):
    rng = np.random.default_rng(seed)
    shape = (rows, heads + 2 * kv, dim)
    x = rng.standard_normal(shape).astype(np.float32).astype(np.float64) if x32 else bf16_values(rng, *shape)
    pos = rng.integers(0, far, rows).astype(np.int32)
    return x, to_dev(x.astype(np.float32)) if x32 else to_dev_bf16(x), pos, decoder.rope_frequencies(rot, 10000.0)


@pytest.mark.parametrize("x32", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,heads,kv,dim,rot,far", [
    (1, 1, 1, 16, 16, 1), (1, 32, 8, 128, 128, 131072), (3, 5, 1, 64, 32, 1 << 20), (17, 6, 3, 96, 96, 4096),
    (64, 8, 2, 128, 64, 1 << 24), (5, 2, 2, 1024, 1024, 100), (9, 3, 1, 136, 48, 2 ** 31 - 1)])
def test_matches(gpu_lib, rows, heads, kv, dim, rot, far, inter, x32):
    x, xd, pos, freqs = case(rows + dim, rows, heads, kv, dim, rot, x32, far)
    rope = decoder.Rope(freqs, inter, 1.25)
    keep = xd.clone()
    q_out = torch.full((rows, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((rows, kv, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k = rope(xd[:, :heads], xd[:, heads:heads + kv], to_dev(pos), q_out, k_out)
    torch.cuda.synchronize()
    assert q is q_out and k is k_out and torch.equal(xd, keep)
    f = freqs.cpu().numpy()
    check(host64(q), x[:, :heads], pos, f, inter, 1.25)
    check(host64(k), x[:, heads:heads + kv], pos, f, inter, 1.25)


@pytest.mark.parametrize("rows", [1, 20, 5000, 9001])
def test_in_place_on_a_fused_projection(gpu_lib, rows):
    x, xd, pos, freqs = case(rows, rows, 4, 2, 64, 64, False, 5000)
    rope, p = decoder.Rope(freqs), to_dev(pos)
    want_q, want_k = rope(xd[:, :4], xd[:, 4:6], p, torch.empty_like(xd[:, :4]).contiguous(),
                          torch.empty(rows, 2, 64, dtype=torch.bfloat16, device="cuda"))
    v = xd[:, 6:].clone()
    q, k = rope(xd[:, :4], xd[:, 4:6], p)
    assert torch.equal(xd[:, :4], want_q) and torch.equal(xd[:, 4:6], want_k) and torch.equal(xd[:, 6:], v)
    some = sorted({0, rows // 2, rows - 1})
    check(host64(want_q)[some], x[some, :4], pos[some], freqs.cpu().numpy(), False, 1.0)


def test_negative_positions_turn_back_and_q_alone(gpu_lib):
    x, xd, pos, freqs = case(1, 12, 4, 1, 64, 64, True, 1000)
    rope, p = decoder.Rope(freqs), to_dev(pos)
    q = xd[:, :4]
    q1, none = rope(q, None, p)
    assert none is None and q1.dtype is torch.bfloat16
    back, _ = rope(q1.float(), None, -p)
    # two roundings to bf16 of each of the pair, and the sines' error
    assert np.all(np.abs(host64(back) - x[:, :4]) <= 3 * 2.0 ** -8 * np.abs(x[:, :4]).max())
    check(host64(q1), x[:, :4], pos, freqs.cpu().numpy(), False, 1.0)
    empty = rope(xd[:0, :4], xd[:0, 4:5], p[:0])
    assert empty[0].shape == (0, 4, 64)


def test_non_finite_channels_stay_in_their_pair(gpu_lib):
    x, xd, pos, freqs = case(2, 6, 2, 1, 64, 32, False, 100)
    xd[3, 1, 5] = float("nan")
    xd[4, 0, 60] = float("inf")
    q, _ = decoder.Rope(freqs)(xd[:, :2], None, to_dev(pos), torch.empty(6, 2, 64, dtype=torch.bfloat16, device="cuda"))
    bad = (~torch.isfinite(q)).nonzero().cpu().tolist()
    assert bad == [[3, 1, 5], [3, 1, 21], [4, 0, 60]]


def test_more_rows_than_workgroups(gpu_lib):
    rows = (1 << 22) + 5
    x = torch.randn(64, 1, 16, device="cuda").to(torch.bfloat16).repeat((rows + 63) // 64, 1, 1)[:rows]
    pos = (torch.arange(rows, device="cuda") % 64).to(torch.int32)
    rope = decoder.Rope(decoder.rope_frequencies(16))
    few, _ = rope(x[:64].clone(), None, pos[:64])
    all_, _ = rope(x.contiguous().clone(), None, pos)
    n = rows // 64
    assert torch.equal(all_[:n * 64].view(n, 64, 1, 16), few[None].expand(n, 64, 1, 16))


def test_frequencies_for_long_contexts():
    f = decoder.rope_frequencies(64, 1e4, device="cpu").numpy()
    assert np.allclose(f, 1e4 ** (-np.arange(32) / 32))
    assert np.allclose(decoder.rope_frequencies(64, 1e4, 4.0, device="cpu").numpy(), f / 4)
    g = decoder.rope_frequencies(64, 1e4, 4.0, original=4096, device="cpu").numpy()
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4)
    assert np.all(np.diff(g) < 0) and np.all((g <= f) & (g >= f / 4 * (1 - 1e-12)))
