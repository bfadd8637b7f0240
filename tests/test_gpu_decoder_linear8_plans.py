"""svdq_w8a8_gemm through every kernel, tile and division of K that it can choose, bit for bit.  That
SHAPES reach all of them is checked without a GPU, by the choice itself (test_w8a8_plan_cpu.py)."""
import pytest
import torch

from bit_post_quantized_amd import decoder
from tests.test_gpu_decoder_linear8 import on_device

pytestmark = pytest.mark.gpu

# (rows, K, columns): columns odd, even and whole pieces of 16 bytes; units of K that neither the waves nor the shares
# divide, fewer of them than waves, and ordinary projections
SHAPES = [
    # up to 64 rows, the weights in whole units: tiles of 16 rows by tiles of 16 columns
    (1, 64, 1), (16, 64 * 19, 1001), (1, 64, 16425), (13, 64 * 9, 17001), (16, 64 * 64, 16400), (1, 64 * 67, 17325),
    (16, 64 * 65, 16376), (1, 8192, 28672),
    (17, 64, 3), (31, 64 * 17, 1000), (29, 320, 8180), (18, 704, 8261), (32, 64, 8184), (27, 1216, 16374), (17, 2624, 16371),
    (17, 64 * 41, 16949),
    (33, 64, 5), (47, 64 * 21, 333), (44, 320, 8189), (40, 448, 8189), (48, 64, 8184), (42, 3648, 16374), (33, 7488, 16580),
    (49, 64, 7), (64, 64 * 13, 1000), (64, 320, 8181), (61, 448, 8177), (49, 832, 8465), (50, 320, 16380), (51, 448, 16372),
    # the same rows in the smallest tile, undivided and divided
    (17, 64, 4272), (64, 64 * 5, 33001), (24, 8192, 28672), (19, 5824, 16203), (33, 5824, 16208), (17, 9856, 7999),
    (63, 9856, 7000), (17, 22400, 13), (39, 13696, 40), (64, 16384, 1024),
    # more rows: 64 x 128
    (65, 64, 1), (65, 64, 127), (74, 3904, 4410), (74, 3712, 4533), (65, 2112, 1), (130, 2048, 264), (66, 4160, 1),
    (65, 4288, 256),
    # 128 x 128
    (65, 64, 16451), (2000, 64 * 5, 4095), (1324, 19776, 1291), (113, 19776, 15747), (65, 3776, 4478), (66, 4032, 4347),
    (65, 6848, 2054), (67, 7232, 2064),
    # 128 x 256
    (65, 64, 32930), (65, 16320, 17054), (66, 9792, 8386), (65, 9664, 8677), (67, 13120, 4394), (69, 14784, 4107),
    # 256 x 256
    (193, 64, 32985), (300, 8192, 28672), (197, 13120, 16431), (194, 14272, 16583), (194, 13504, 8726), (193, 14144, 9153),
    (200, 15680, 4165), (257, 16192, 3240), (1618, 15872, 525),
]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_every_choice(gpu_lib, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M * 31 + N)

    def rows(n):
        return decoder.Rows8(torch.randint(-127, 128, (n, K), generator=g, device="cuda").to(torch.int8),
                             0.5 + torch.rand(n, generator=g, device="cuda"))

    x, w = rows(M), rows(N)
    bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) * 1e4
    linear, plain = decoder.Linear8(w.codes, w.scales, bias), decoder.Linear8(w.codes, w.scales)
    for dtype in (torch.bfloat16, torch.float32):
        guard = torch.full((M * N + 128,), 7.0, dtype=dtype, device="cuda")
        linear(x, out=guard[64:-64].view(M, N))
        assert torch.equal(guard[64:-64].view(M, N), on_device(x, w, dtype, bias))
        assert (guard[:64] == 7).all() and (guard[-64:] == 7).all()
        assert torch.equal(plain(x, out_dtype=dtype), on_device(x, w, dtype))
