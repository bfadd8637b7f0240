"""svdq_rms_norm and svdq_quantize_rows against fp64.

Bounds.  h is one fp32 rounding, as in the oracle.  A row's sum of squares has at most
n = K / 64 + 40 roundings on a term's way (a thread's chain and the tree), all of the same sign, and
the root halves them; the division by K, eps, the root, its reciprocal and the two products are 6
more: r = (n / 2 + 6) 2^-24 of y.  The store rounds once more, by 2^-8 of y (bf16; subnormal results
by 2^-134).  A scale is off by r and two roundings; a code by half a step and what y / s is off, 127
times that."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import decoder
from oracle import decoder as od
from oracle.numerics import bf16_to_bits, round_bf16
from tests.serve_cases import bf16_values, host64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def rel(K):
    return ((K / 64 + 40) / 2 + 6) * 2.0 ** -24


def dev(values, fp32):
    return to_dev(values.astype(np.float32)) if fp32 else to_dev_bf16(values)


def values(rng, fp32, *shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float32).astype(np.float64) if fp32 \
        else bf16_values(rng, *shape, scale=scale)


def check(y, want, K):
    tol = (rel(K) + 2.0 ** -8) * np.abs(want) + 2.0 ** -133
    assert np.all(np.abs(y - want) <= tol), float((np.abs(y - want) / tol).max())


def check8(r8, want, K):
    q, s = od.rows8(want)
    got = r8.scales.double().cpu().numpy()
    assert np.all(np.abs(got - s) <= s * (rel(K) + 2.0 ** -23) + 2.0 ** -149)
    codes = r8.codes.cpu().numpy()
    assert np.all(np.abs(codes - q) <= 0.5 + 127 * 2 * (rel(K) + 2.0 ** -22))
    assert np.abs(codes.astype(int)).max() <= 127


@pytest.mark.parametrize("x32,r32", [(False, False), (False, True), (True, False), (True, True), (False, None), (True, None)])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (5, 504), (4, 512), (9, 520), (7, 1024), (2, 1032), (6, 2048),
                                 (3, 2056), (2, 4096), (5, 5120), (3, 8192), (2, 8200), (2, 16384), (3, 16392), (2, 40000)])
def test_matches(gpu_lib, M, K, x32, r32):
    rng = np.random.default_rng(M * 1000 + K)
    x = values(rng, x32, M, K)
    r = None if r32 is None else values(rng, r32, M, K, scale=3.0)
    gamma = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    norm = decoder.RMSNorm(to_dev(gamma), 1e-5)
    rd = None if r is None else dev(r, r32)
    y, ro = norm(dev(x, x32), rd)
    r8, ro8 = norm.rows8(dev(x, x32), rd)
    torch.cuda.synchronize()
    h, want = od.rms_norm(x, r, gamma, np.float32(1e-5))
    check(host64(y), want, K)
    check8(r8, want, K)
    if r is None:
        assert ro is None and ro8 is None
    else:
        assert ro.dtype == rd.dtype and torch.equal(ro, ro8)
        assert np.array_equal(ro.double().cpu().numpy(), h if r32 else round_bf16(h))


@pytest.mark.parametrize("K", [256, 4096, 24576])
def test_in_place_residual_and_strided_rows(gpu_lib, K):
    rng = np.random.default_rng(K)
    wide = to_dev_bf16(bf16_values(rng, 6, K + 64))
    x, r = wide[:, 32:32 + K], to_dev_bf16(bf16_values(rng, 6, K))
    norm = decoder.RMSNorm(torch.ones(K, device="cuda"))
    want, wr = norm(x.contiguous(), r)
    keep = wide.clone()
    y, ro = norm(x, r, residual_out=r)
    assert ro is r and torch.equal(y, want) and torch.equal(r, wr) and torch.equal(wide, keep)
    a, b = decoder.quantize_rows(x), decoder.quantize_rows(x.contiguous())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("K", [64, 1024, 4096, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_any_magnitude(gpu_lib, K, eps):
    rng = np.random.default_rng(K + 1)
    x = rng.standard_normal((8, K)) * np.array([1e-38, 1e-30, 1e-22, 1e-12, 1e15, 1e25, 1e37, 1.0])[:, None]
    x = x.astype(np.float32).astype(np.float64)
    x[7] = 0.0
    norm = decoder.RMSNorm(torch.ones(K, device="cuda"), eps)
    y, _ = norm(to_dev(x.astype(np.float32)))
    r8, _ = norm.rows8(to_dev(x.astype(np.float32)))
    _, want = od.rms_norm(x, None, None, np.float32(eps))
    # (elements that the scaling makes subnormal, 2^-126 of the row's largest, keep 2^-24 of 2^-126)
    check(host64(y), want, K)
    live = np.abs(want).max(axis=1) > 1e-30
    check8(decoder.Rows8(r8.codes[torch.from_numpy(live).cuda()], r8.scales[torch.from_numpy(live).cuda()]), want[live], K)
    assert (r8.codes[7] == 0).all() and r8.scales[7] == 0


@pytest.mark.parametrize("K", [512, 4096, 20000])
def test_a_non_finite_row_stays_alone(gpu_lib, K):
    rng = np.random.default_rng(K + 2)
    x = bf16_values(rng, 9, K)
    bits = bf16_to_bits(x)
    bits[2, K - 1], bits[5, 3] = 0x7FC1, 0xFF80
    xd = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    norm = decoder.RMSNorm(torch.ones(K, device="cuda"))
    y, r8 = norm(xd)[0], norm.rows8(xd)[0]
    keep = [i for i in range(9) if i not in (2, 5)]
    want = od.rms_norm(x, None, None, np.float32(1e-6))[1][keep]
    check(host64(y)[keep], want, K)
    check8(decoder.Rows8(r8.codes[keep], r8.scales[keep]), want, K)
    assert torch.isnan(y[2]).all() and torch.isnan(y[5, 3])
    assert torch.isnan(r8.scales[[2, 5]]).all() and (r8.codes[[2, 5]] == 0).all()
    q = decoder.quantize_rows(xd)
    assert torch.isnan(q.scales[2]) and torch.isinf(q.scales[5]) and (q.codes[[2, 5]] == 0).all()


@pytest.mark.parametrize("x32", [False, True])
@pytest.mark.parametrize("M,K", [(1, 8), (4, 512), (5, 1000), (3, 4096), (2, 16384), (2, 30000)])
def test_quantized_rows_are_exact(gpu_lib, M, K, x32):
    rng = np.random.default_rng(M + K)
    x = values(rng, x32, M, K, scale=5.0)
    x[0, :] *= 1e-20 if x32 else 1.0
    x = x.astype(np.float32).astype(np.float64) if x32 else x
    factor = np.exp(rng.standard_normal(K)).astype(np.float32)
    for f in (None, factor):
        r8 = decoder.quantize_rows(dev(x, x32), None if f is None else to_dev(f))
        codes, scales = od.quantize_rows(x, f)
        assert np.array_equal(r8.scales.cpu().numpy(), scales)
        assert np.array_equal(r8.codes.cpu().numpy(), codes)


def test_quantized_rows_whose_scale_is_subnormal(gpu_lib):
    x = np.zeros((3, 16), np.float32)
    x[0, :3], x[1, :3], x[2, :2] = [1e-38, -3e-39, 2e-40], [1.4e-45, 0, -1.4e-45], [3.4e38, -1e38]
    r8 = decoder.quantize_rows(to_dev(x))
    codes, scales = od.quantize_rows(x, None)
    assert np.array_equal(r8.scales.cpu().numpy(), scales) and np.array_equal(r8.codes.cpu().numpy(), codes)


def test_no_rows_guards_and_many_rows(gpu_lib):
    norm = decoder.RMSNorm(torch.ones(64, device="cuda"))
    y, _ = norm(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert tuple(y.shape) == (0, 64)
    guard = torch.full((5, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    norm(x, out=guard[1:4])
    assert (guard[0] == 9).all() and (guard[4] == 9).all() and torch.equal(guard[1:4], norm(x)[0])
    # more rows than one launch has workgroups for
    many = torch.randn(64, 8, device="cuda").to(torch.bfloat16).repeat(1 << 17, 1)[: (1 << 23) - 3]
    few = decoder.quantize_rows(many[:64])
    all_ = decoder.quantize_rows(many)
    n = many.shape[0] // 64
    assert torch.equal(all_.codes[:n * 64].view(n, 64, 8), few.codes[None].expand(n, 64, 8))
    assert torch.equal(all_.scales[:n * 64].view(n, 64), few.scales[None].expand(n, 64))


def test_rows_past_two_gib(gpu_lib):
    """[70001, 16384]: offsets past 2^31 bytes in x, the residual, the codes' 2^30 elements and y."""
    M, K = 70001, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(K, device="cuda")
    norm = decoder.RMSNorm(gamma)
    y, _ = norm(x)
    h8, res = norm.rows8(x, x)
    for rows in (slice(0, 2), slice(32767, 32770), slice(65535, 65538), slice(M - 2, M)):
        part = x[rows].contiguous()
        assert torch.equal(y[rows], norm(part)[0])
        p8, pres = norm.rows8(part, part)
        assert torch.equal(h8.codes[rows], p8.codes) and torch.equal(h8.scales[rows], p8.scales)
        assert torch.equal(res[rows], pres)
