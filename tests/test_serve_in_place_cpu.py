"""Plans over their own arguments are refused before anything is launched (no GPU)."""
import pytest

from bit_post_quantized_amd import binding
from bit_post_quantized_amd import serve_binding as SB

CTX, NEW, COUNT = 0x10000, 0x20000, 0x30000


@pytest.mark.parametrize("seq,status", [(CTX, 0x70000), (NEW, 0x70000), (0x60000, CTX), (0x60000, NEW)])
def test_a_plan_over_its_lengths_is_refused(seq, status):
    lib = SB.load()
    got = lib.kv_block_plan(CTX, NEW, 2, 0x40000, 4, 16, 0x50000, 8, COUNT, 0x80000, seq, 4, 0x90000,
                            0xA0000, status, 0xB0000, None)
    assert got == binding.SVDQ_EINVAL and b"seq_lens and status" in lib.svdq_last_error()
