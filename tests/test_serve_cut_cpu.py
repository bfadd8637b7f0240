"""How the attention over the block cache cuts a batch, from the sizes of its workspace (no GPU)."""
import os

import pytest

from bit_post_quantized_amd import binding
from bit_post_quantized_amd import serve_binding as SB

MOST_PARTS = 1024   # of a row that the join of few rows can take


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run python -m bit_post_quantized_amd.build)")
    return SB.load()


def chunks(lib, n, rows, max_rows, heads, kv, dim, width, bs):
    """Parts per row of a batch with more rows than the few-rows kernel takes (0: not cut)."""
    per = rows * heads * (dim + 4) * 4
    size = lib.kv_block_attention_workspace_bytes(n, rows, max_rows, heads, kv, dim, width, bs)
    assert size % per == 0
    return size // per


def test_no_row_has_more_parts_than_a_join_takes(lib):
    cut = 0
    for n in (1, 2, 3, 5, 7, 8, 64, 700, 4096):
        for kv in (1, 2, 4, 7, 8):
            for max_rows, group in ((5, 8), (33, 1), (17, 2), (64, 1), (65, 1), (500, 3)):
                for dim in (64, 128):
                    if max_rows * group <= (32 if dim == 64 else 16):
                        continue
                    for bs in (16, 128):
                        for tokens in (256, 4096, 10000, 131072, 1 << 22, (1 << 22) + 64, 1 << 23, 1 << 26, 1 << 30):
                            width = -(-tokens // bs)
                            if n * width >= 1 << 31:
                                continue
                            k = chunks(lib, n, n * max_rows, max_rows, kv * group, kv, dim, width, bs)
                            assert k <= MOST_PARTS, (n, kv, max_rows, group, dim, bs, tokens, k)
                            cut += k > 1
    assert cut > 1000
