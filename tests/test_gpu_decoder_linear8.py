"""svdq_w8a8_gemm against whole numbers: the sums are exact and every rounding after them is named, so
the outputs are compared bit for bit."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import decoder
from bit_post_quantized_amd import decoder_binding as DB
from oracle import decoder as od
from tests.serve_cases import bf16_values, host64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def make(seed, M, K, N, bias, full=False):
    rng = np.random.default_rng(seed)
    if full:
        qx, qw = (rng.choice([-128, 127], (n, K)).astype(np.int8) for n in (M, N))
    else:
        qx, qw = (np.clip(np.rint(rng.standard_normal((n, K)) * 40), -127, 127).astype(np.int8) for n in (M, N))
    sx, sw = ((0.5 + rng.random(n)).astype(np.float32) / 100 for n in (M, N))
    return qx, sx, qw, sw, bf16_values(rng, N) if bias else None


def run(case, dtype, **more):
    qx, sx, qw, sw, b = case
    lin = decoder.Linear8(to_dev(qw), to_dev(sw), None if b is None else to_dev_bf16(b))
    return lin(decoder.Rows8(to_dev(qx), to_dev(sx)), out_dtype=dtype, **more)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,bias", [
    (1, 64, 1, False), (1, 64, 16, True), (1, 4096, 200, True), (2, 128, 17, True), (3, 320, 15, False),
    (15, 192, 100, True), (16, 1024, 33, False), (17, 64 * 17, 48, True), (31, 64 * 33, 95, False), (32, 128, 1000, True),
    (33, 512, 130, False), (48, 64 * 7, 4, True), (49, 64 * 65, 50, False), (63, 384, 129, True), (64, 2048, 72, False),
    (5, 256, 9000, True), (40, 64 * 5, 17000, False), (64, 64, 33000, True),
    (65, 64, 1, True), (65, 192, 127, False), (100, 64 * 9, 128, True), (128, 128, 129, False), (129, 64 * 31, 257, True),
    (200, 64 * 64, 300, False), (257, 64 * 3, 1000, True), (500, 64 * 40, 130, True), (255, 64 * 100, 64, False),
    (3000, 64 * 3, 5000, True), (4097, 128, 4095, False), (70, 64 * 150, 20, True),
    (4099, 64, 4104, True), (4200, 64 * 5, 4001, True), (4352, 64 * 4, 4096, False), (16400, 64 * 7, 1020, True),
])
def test_matches_bit_for_bit(gpu_lib, M, K, N, bias, dtype):
    case = make(M * 7919 + K + N, M, K, N, bias)
    y = run(case, dtype)
    torch.cuda.synchronize()
    assert y.dtype == dtype and tuple(y.shape) == (M, N)
    assert np.array_equal(host64(y), od.linear8(*case, dtype == torch.bfloat16))


@pytest.mark.parametrize("M", [3, 70])
def test_the_longest_sums_do_not_overflow(gpu_lib, M):
    K = 64 * 2047
    case = make(5, M, K, 20, False, full=True)
    case[0][0], case[2][0] = -128, -128       # 128 * 128 * K, just under 2^31
    assert np.array_equal(host64(run(case, torch.float32)), od.linear8(*case, False))


@pytest.mark.parametrize("M", [20, 300])
def test_rows_without_a_finite_scale_stay_alone(gpu_lib, M):
    qx, sx, qw, sw, b = make(7, M, 256, 50, True)
    sx[3], sx[M - 1], sx[5] = np.nan, np.inf, 0.0
    qx[M - 1] = 0
    y = host64(run((qx, sx, qw, sw, b), torch.float32))
    with np.errstate(invalid="ignore"):
        want = od.linear8(qx, sx, qw, sw, b, False)
    assert np.isnan(y[[3, M - 1]]).all() and np.array_equal(y, want, equal_nan=True)


@pytest.mark.parametrize("M,N", [(3, 37), (90, 131), (300, 260)])
def test_no_rows_and_guarded_outputs(gpu_lib, M, N):
    case = make(13, M, 320, N, True)
    guard = torch.full((M + 2, N), 7.0, dtype=torch.float32, device="cuda")
    inner = torch.empty(M * N + 8, device="cuda").fill_(7.0)
    run(case, torch.float32, out=inner[4:4 + M * N].view(M, N))
    guard[1:-1] = inner[4:4 + M * N].view(M, N)
    assert (inner[:4] == 7).all() and (inner[4 + M * N:] == 7).all()
    assert np.array_equal(host64(guard[1:-1]), od.linear8(*case, False))
    qx, sx, qw, sw, b = case
    assert tuple(run((qx[:0], sx[:0], qw, sw, b), torch.bfloat16).shape) == (0, N)


def test_workspace_needs_no_initialization_and_serves_other_sizes(gpu_lib):
    cases = [make(17 + i, M, K, N, True) for i, (M, K, N) in
             enumerate([(100, 64 * 40, 200), (300, 64 * 64, 100), (70, 64 * 30, 500)])]
    need = [DB.svdq_w8a8_workspace_bytes(c[0].shape[0], c[2].shape[0], c[0].shape[1]) for c in cases]
    assert max(need) > 0
    ws = torch.full((max(need) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for c in cases * 2:
        assert np.array_equal(host64(run(c, torch.float32, workspace=ws[:max(need)])), od.linear8(*c, False))
    assert (ws[max(need):] == 0xFF).all()


def test_from_weight_and_rows_of_activations(gpu_lib):
    rng = np.random.default_rng(3)
    W, x = bf16_values(rng, 96, 256), bf16_values(rng, 10, 256)
    f = np.exp(0.5 * rng.standard_normal(256)).astype(np.float32)
    lin = decoder.Linear8.from_weight(to_dev_bf16(W), factor=to_dev(f))
    y = lin(decoder.quantize_rows(to_dev_bf16(x), to_dev((1 / f).astype(np.float32))), out_dtype=torch.float32)
    qw, sw = od.quantize_rows(W, f)
    qx, sx = od.quantize_rows(x, (1 / f).astype(np.float32))
    assert np.array_equal(host64(y), od.linear8(qx, sx, qw, sw, None, False))
    # half a step of either side in every product
    want, mag = x @ W.T, (np.abs(x / f) @ (0.5 * np.repeat(sw[:, None], 256, 1)).T + 0.5 * sx[:, None] * np.abs(W * f).sum(1)[None, :]
                          + 0.25 * 256 * sx[:, None] * sw[None, :])
    assert np.all(np.abs(host64(y) - want) <= mag * 1.0001)


def test_captured_and_replayed(gpu_lib):
    case = make(23, 120, 64 * 40, 200, True)
    qx, sx, qw, sw, b = case
    lin = decoder.Linear8(to_dev(qw), to_dev(sw), to_dev_bf16(b))
    x = decoder.Rows8(to_dev(qx), to_dev(sx))
    lin(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lin(x)
    for i in range(3):
        q2 = np.roll(qx, i, axis=0)
        x.codes.copy_(to_dev(q2))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host64(y), od.linear8(q2, sx, qw, sw, b, True)), i
        assert torch.equal(lin(x), y)


def on_device(x, w, dtype, bias=None):
    """The same as the oracle, with the sums from a product in 64-bit floats (whole numbers under 2^31: exact)."""
    acc = x.codes.double() @ w.codes.double().t().contiguous()
    y = (acc.float() * x.scales[:, None]) * w.scales[None, :]
    if bias is not None:
        y = y + bias.float()[None, :]
    return y.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [
    # each tile and division, N odd and even, the last tiles nearly empty
    (129, 64 * 53, 4440), (144, 64 * 57, 4101), (4097, 64 * 65, 132), (4360, 64 * 66, 135), (4532, 64 * 35, 1),
    (2196, 64 * 66, 33), (1000, 64 * 128, 1000), (4758, 64, 792), (1999, 64 * 33, 4095), (2000, 64 * 12, 4096),
    (4101, 64 * 92, 129), (4205, 64 * 96, 132), (2337, 64, 3331), (5000, 64 * 7, 5001),
])
def test_tiles_and_divisions(gpu_lib, M, K, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + N)

    def rows(n):
        return decoder.Rows8(torch.randint(-127, 128, (n, K), generator=g, device="cuda").to(torch.int8),
                             0.5 + torch.rand(n, generator=g, device="cuda"))

    x, w = rows(M), rows(N)
    bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) * 1e4
    guard = torch.full((M * N + 128,), 7.0, dtype=dtype, device="cuda")
    decoder.Linear8(w.codes, w.scales, bias)(x, out=guard[64:-64].view(M, N))
    assert torch.equal(guard[64:-64].view(M, N), on_device(x, w, dtype, bias))
    assert (guard[:64] == 7).all() and (guard[-64:] == 7).all()
    assert torch.equal(decoder.Linear8(w.codes, w.scales)(x, out_dtype=dtype), on_device(x, w, dtype))


@pytest.mark.parametrize("M,N", [(66001, 33000), (40, (1 << 24) - 5), (20000, 65601)])
def test_results_past_two_gib(gpu_lib, M, N):
    K = 64
    g = torch.Generator(device="cuda").manual_seed(N)
    x = decoder.Rows8(torch.randint(-127, 128, (M, K), generator=g, device="cuda").to(torch.int8),
                      0.5 + torch.rand(M, generator=g, device="cuda"))
    w = decoder.Rows8(torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8),
                      0.5 + torch.rand(N, generator=g, device="cuda"))
    dtype = torch.float32 if M == 20000 else torch.bfloat16
    y = decoder.Linear8(w.codes, w.scales)(x, out_dtype=dtype)
    for first in range(0, M, 8192):
        part = decoder.Rows8(x.codes[first:first + 8192], x.scales[first:first + 8192])
        assert torch.equal(y[first:first + 8192], on_device(part, w, dtype)), first
