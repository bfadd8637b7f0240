"""svdq_w4a16_gemv against the fp64 layer.

Bounds.  An activation enters with relative error at most u = 2^-11 (fp16, bf16 output) or 2^-21
(an fp16 pair, fp32 output); its products with 4-bit codes are exact; the fp32 sums have at most
2 * 64 + G + 64 roundings on a term's way (a matrix step may truncate, hence 2 per product; one
FMA per group; the waves, T's slices and the epilogue), each 2^-24 of the sum of magnitudes A;
the store rounds once, by eps / 2 relative."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import layer, serve
from bit_post_quantized_amd import serve_binding as SB
from oracle import serve as osv
from oracle.numerics import bf16_to_bits, round_bf16
from tests.serve_cases import bf16_values, host64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def make(seed, M, K, N, r, bias, x=None):
    rng = np.random.default_rng(seed)
    x = bf16_values(rng, M, K) if x is None else x
    hot = rng.random(K) < 0.02
    if x is not None:
        x = round_bf16(x * np.where(hot, 16.0, 1.0))
    inv = (np.where(hot, 0.1, 1.0) * np.exp(0.3 * rng.standard_normal(K))).astype(np.float32)
    codes = np.clip(np.rint(rng.standard_normal((N, K)) * 2.5), -8, 7).astype(np.int64)
    ws = (np.exp(0.2 * rng.standard_normal((K // 64, N))) * 0.3 / np.sqrt(K)).astype(np.float16)
    l1, l2 = bf16_values(rng, K, r, scale=K ** -0.5), bf16_values(rng, r, N, scale=max(r, 1) ** -0.5)
    b = bf16_values(rng, N) if bias else None
    u = codes & 15
    wq = (u[:, 0::2] | (u[:, 1::2] << 4)).astype(np.uint8)
    pw = layer.PackedWeights(K=K, N=N, rank=r, inv_lambda=to_dev(inv), L1p=to_dev_bf16(l1.T.copy()),
                             L2p=to_dev_bf16(l2.T.copy()), wq=to_dev(wq), w_scales=to_dev(ws),
                             bias=None if b is None else to_dev_bf16(b))
    return x, pw, lambda v: osv.linear(bf16_to_bits(v), inv, l1, codes, ws.astype(np.float64), l2, b)


def check(y, ref, mag, K, fp32):
    steps = 2 * 64 + K // 64 + 64
    tol = (2.0 ** -24 if fp32 else 2.0 ** -8) * np.abs(ref) + \
        ((2.0 ** -21 if fp32 else 2.0 ** -11) + steps * 2.0 ** -24) * mag
    assert np.all(np.abs(y - ref) <= tol), float((np.abs(y - ref) / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,r,bias", [
    (1, 64, 1, 0, False), (1, 64, 16, 16, True), (1, 4096, 200, 32, True), (1, 12288, 65, 16, False),
    (2, 128, 17, 0, True), (3, 320, 15, 48, False), (7, 1024, 1000, 32, True), (8, 576, 33, 128, True),
    (9, 256, 31, 16, False), (15, 192, 100, 0, False), (16, 4096, 48, 32, True), (17, 704, 130, 64, True),
    (31, 128, 64, 16, False), (32, 2048, 95, 32, True), (33, 512, 16, 128, False), (48, 64, 7, 0, True),
    (49, 1088, 50, 112, True), (63, 384, 129, 32, False), (64, 4096, 72, 128, True),
    (5, 64 * 33, 4100, 32, True),
    # K beyond what a workgroup holds of X: read again (one row tile) or cut over workgroups
    (3, 64 * 129, 40, 32, True), (16, 64 * 150, 33, 128, False), (17, 64 * 65, 130, 48, True),
    (24, 64 * 131, 50, 0, True), (33, 64 * 33, 600, 16, False), (40, 64 * 97, 17, 112, True),
    (64, 64 * 1100, 20, 64, True), (64, 64 * 40, 4100, 128, False),
])
def test_matches_the_layer(gpu_lib, M, K, N, r, bias, dtype):
    x, pw, ref = make(M * 7919 + K + N, M, K, N, r, bias)
    y = serve.DecodeLinear(pw)(to_dev_bf16(x), out_dtype=dtype)
    torch.cuda.synchronize()
    assert y.dtype == dtype and tuple(y.shape) == (M, N)
    check(host64(y), *ref(x), K, dtype == torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_activations_of_any_magnitude(gpu_lib, dtype):
    # rows from 1e-30 to 1e30, a row of zeros and groups of zeros: a scale per (row, group)
    rng = np.random.default_rng(3)
    x = bf16_values(rng, 6, 256)
    x *= np.array([1e-30, 1e30, 70000.0, 1.0, 0.0, 1e-6])[:, None]
    x[3, 64:128] = 0.0
    x[3, 128:192] *= 1e6
    x = round_bf16(x)
    x, pw, ref = make(5, 6, 256, 40, 16, False, x=x)
    y = serve.DecodeLinear(pw)(to_dev_bf16(x), out_dtype=dtype)
    check(host64(y), *ref(x), 256, dtype == torch.float32)


def test_a_non_finite_row_stays_alone(gpu_lib):
    x, pw, ref = make(11, 20, 256, 50, 16, True)
    bits = bf16_to_bits(x)
    bits[4, 7], bits[18, 200] = 0x7FC0, 0x7F80
    xd = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    y = host64(serve.DecodeLinear(pw)(xd))
    keep = [i for i in range(20) if i not in (4, 18)]
    want, mag = ref(x)
    check(y[keep], want[keep], mag[keep], 256, False)
    assert np.isnan(y[4]).all() and not np.isfinite(y[18]).any()


def test_no_rows_and_guarded_outputs(gpu_lib):
    x, pw, ref = make(13, 3, 128, 37, 16, True)
    lin = serve.DecodeLinear(pw)
    assert tuple(lin(to_dev_bf16(x)[:0]).shape) == (0, 37)
    guard = torch.full((5, 37), 7.0, dtype=torch.bfloat16, device="cuda")
    lin(to_dev_bf16(x), out=guard[1:4])
    assert (guard[0] == 7).all() and (guard[4] == 7).all()
    check(host64(guard[1:4]), *ref(x), 128, False)


def test_workspace_needs_no_initialization_and_serves_other_sizes(gpu_lib):
    cases = [make(17 + i, M, K, N, r, True) for i, (M, K, N, r) in
             enumerate([(9, 512, 100, 32), (1, 128, 60, 16), (33, 256, 20, 64)])]
    need = max(SB.svdq_w4a16_workspace_bytes(c[0].shape[0], c[1].N, c[1].K, c[1].rank, 0) for c in cases)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [(serve.DecodeLinear(pw)(to_dev_bf16(x), workspace=ws), ref(x), pw.K) for x, pw, ref in cases * 2]
    for y, r, K in outs:
        check(host64(y), *r, K, False)


def test_same_bits_every_time_on_streams_and_in_graphs(gpu_lib):
    x, pw, ref = make(23, 4, 1024, 300, 32, True)
    lin = serve.DecodeLinear(pw)
    xd = to_dev_bf16(x)
    first = lin(xd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = lin(xd)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    buf, out = xd.clone(), torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin(buf, out=out)
    for k in range(3):
        buf.copy_(xd * (k + 1))
        g.replay()
        eager = lin(buf)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k
    assert lin(xd).equal(first)
    check(host64(first), *ref(x), 1024, False)


def test_same_bits_and_guards_where_k_is_cut(gpu_lib):
    x, pw, ref = make(24, 30, 64 * 70, 45, 32, True)
    lin, xd = serve.DecodeLinear(pw), to_dev_bf16(x)
    first = lin(xd)
    check(host64(first), *ref(x), pw.K, False)
    need = SB.svdq_w4a16_workspace_bytes(30, 45, pw.K, 32, 0)
    ws = torch.full((need + 32,), 0x7F, dtype=torch.uint8, device="cuda")
    guard = torch.full((32, 45), 7.0, dtype=torch.bfloat16, device="cuda")
    buf = torch.empty_like(xd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin(buf, out=guard[1:31], workspace=ws[:need])
    for k in range(3):
        buf.copy_(xd * 2 ** k)
        g.replay()
        eager = lin(buf)
        torch.cuda.synchronize()
        assert torch.equal(guard[1:31], eager) and torch.equal(lin(xd), first), k
    assert (guard[0] == 7).all() and (guard[31] == 7).all() and (ws[need:] == 0x7F).all()


@pytest.mark.parametrize("N,K", [(16, 512), (1, 64), (50, 704), (33, 1024)])
def test_container_layout(gpu_lib, N, K):
    rng = np.random.default_rng(N)
    wq = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    ws = rng.integers(0, 1 << 15, (K // 64, N)).astype(np.uint16)
    G, segs, tiles = K // 64, -(-K // 512), -(-N // 16)
    got = torch.full((SB.svdq_w4a16_container_bytes(N, K),), 0xEE, dtype=torch.uint8, device="cuda")
    SB.svdq_pack_w4a16(to_dev(wq), to_dev(ws.view(np.float16)), got)
    want = np.zeros((tiles, segs, 4352), np.uint8)
    for n in range(N):
        for g in range(G):
            unit = want[n // 16, g // 8]
            for j in range(4):
                at = (g % 8) // 2 * 1024 + (16 * j + n % 16) * 16 + g % 2 * 8
                unit[at:at + 8] = wq[n, 32 * g + 8 * j:32 * g + 8 * j + 8]
            at = 4096 + (n % 16) * 16 + g % 8 * 2
            unit[at:at + 2] = ws[g, n:n + 1].view(np.uint8)
    np.testing.assert_array_equal(got.cpu().numpy(), want.reshape(-1))


def test_refusals(gpu_lib):
    x, pw, _ = make(29, 2, 128, 32, 16, False)
    lin = serve.DecodeLinear(pw)
    with pytest.raises(RuntimeError, match="M must be <= 64"):
        lin(torch.zeros(65, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="X must be"):
        lin(torch.zeros(2, 128, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="inv_lambda must have shape"):  # K of X against the weights
        lin(torch.zeros(2, 192, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="X must be contiguous"):
        lin(torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")[:, ::2])
    with pytest.raises(ValueError, match="workspace holds"):
        lin(to_dev_bf16(x), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="Y must be bfloat16 or float32"):
        lin(to_dev_bf16(x), out=torch.empty(2, 32, dtype=torch.float16, device="cuda"))
