"""What the decoder's objects keep of a caller's tensors: the memory itself, and the one that a call is
given.  Stand-ins for device tensors; the library's entry points are replaced and nothing is launched."""
import gc

import pytest
import torch

from bit_post_quantized_amd import decoder
from bit_post_quantized_amd import decoder_binding as DB
from tests.test_decoder_abi_cpu import Rows

BF16, F32, F64, I8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32


class Memory:
    """A device allocation: gone when nothing refers to it."""
    at, alive = 0x100000, set()

    def __init__(self):
        Memory.at += 0x10000
        self.pointer = Memory.at
        Memory.alive.add(self.pointer)

    def __del__(self):
        Memory.alive.discard(self.pointer)


class Held(Rows):
    """A stand-in that refers to its memory, as a tensor does to its storage."""

    def __init__(self, shape, dtype, memory=None):
        super().__init__(shape, dtype)
        self.memory = memory or Memory()

    def data_ptr(self):
        return self.memory.pointer

    def detach(self):
        return Held(self.shape, self.dtype, self.memory)


@pytest.fixture
def calls(monkeypatch):
    """The arguments that reach the library, from the fast path and from the checked one."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append(args) or 0

    real = DB.load()
    monkeypatch.setattr(DB, "load", lambda: Lib())
    monkeypatch.setattr(decoder, "_here", lambda dev: True)
    monkeypatch.setattr(decoder, "_stream", lambda dev: 0)
    monkeypatch.setattr(DB._Args, "stream", lambda self, stream: 0)
    for name in ("svdq_w8a8_workspace_bytes", "svdq_w8a8_container_bytes"):
        monkeypatch.setattr(DB, name, getattr(real, name))
    return seen


@pytest.fixture(params=[True, False], ids=["fast", "checked"])
def fast(request, monkeypatch):
    if not request.param:
        monkeypatch.setattr(decoder, "_is", lambda *a: False)
        monkeypatch.setattr(decoder, "_rows_of", lambda *a: False)
    return request.param


def norm_gamma(norm, calls):
    x, y = Held([3, norm.K], BF16), Held([3, norm.K], BF16)
    norm._run(x, None, None, y, None, None, True)
    return calls[-1][6]


def rope_freqs(rope, calls):
    q, out = Held([3, 4, 64], BF16), Held([3, 4, 64], BF16)
    rope(q, None, Held([3], I32), out)
    return calls[-1][12]


OBJECTS = [(decoder.RMSNorm, "gamma", norm_gamma, ([64], F32), ([128], F32)),
           (decoder.Rope, "freqs", rope_freqs, ([32], F64), ([16], F64))]


@pytest.mark.parametrize("make,name,used,first,second", OBJECTS, ids=["RMSNorm", "Rope"])
def test_an_assigned_tensor_is_the_one_used(calls, fast, make, name, used, first, second):
    o, other = make(Held(*first)), Held(*second)
    setattr(o, name, other)
    gc.collect()
    assert used(o, calls) == other.memory.pointer
    assert other.memory.pointer in Memory.alive and getattr(o, name).data_ptr() == other.memory.pointer
    with pytest.raises(ValueError, match=f"{name} must be"):
        setattr(o, name, Held(second[0], I32))
    assert used(o, calls) == other.memory.pointer


@pytest.mark.parametrize("make,name,used,first,second", OBJECTS, ids=["RMSNorm", "Rope"])
def test_memory_that_a_tensor_gives_up_is_kept(calls, fast, make, name, used, first, second):
    t = Held(*first)
    o = make(t)
    t.memory = Memory()        # (what `t.data = ...` does, a module's move to another type among them)
    del t
    gc.collect()
    assert used(o, calls) in Memory.alive


def test_the_linears_scales_and_bias_are_kept(calls, monkeypatch):
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device=None: empty(n, dtype=dtype) if device is None
                        else Held([n], dtype))
    scales, bias = Held([16], F32), Held([16], BF16)
    linear = decoder.Linear8(Held([16, 64], I8), scales, bias)
    want = [scales.memory.pointer, bias.memory.pointer]
    scales.memory, bias.memory = Memory(), Memory()
    gc.collect()
    assert [t.data_ptr() for t in linear._held[1:]] == want == list(linear._weights[1:])
    assert set(want) <= Memory.alive


def test_the_planners_tables_are_kept_and_the_same_for_plan_and_release(monkeypatch):
    from bit_post_quantized_amd import serve
    empty, seen = torch.empty, []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append(args) or 0

    monkeypatch.setattr(serve.B, "load", lambda: Lib())
    monkeypatch.setattr(serve.B._Args, "stream", lambda self, stream: 0)
    monkeypatch.setattr(torch, "empty", lambda *n, dtype, device=None: empty(*n, dtype=dtype) if device is None
                        else Held(n, dtype))
    for name, value in (("_here", True), ("_stream", 0)):
        monkeypatch.setattr(serve, name, lambda dev, value=value: value)
    tables, free = Held([4, 8], I32), Held([32], I32)
    want = [tables.memory.pointer, free.memory.pointer]
    planner = serve.BlockPlanner(tables, free, 16, 40)
    for name in ("block_tables", "free_blocks"):
        with pytest.raises(AttributeError):
            setattr(planner, name, Held([4, 8], I32))
    tables.memory, free.memory = Memory(), Memory()
    gc.collect()
    planner.plan(Held([4], I32), Held([4], I32), Held([1], I32))
    planner.release(Held([4], I32), Held([4], torch.uint8), Held([1], I32))
    assert set(want) <= Memory.alive and len(seen) == 2
    assert all(pointer in call for call in seen for pointer in want)


def test_an_output_of_keys_without_keys_is_refused(calls, fast):
    rope = decoder.Rope(Held([32], F64))
    q, pos = Held([3, 4, 64], BF16), Held([3], I32)
    with pytest.raises(ValueError, match="k_out needs k"):
        rope(q, None, pos, q, Held([3, 2, 64], BF16))
    assert not calls
    assert rope(q, None, pos) == (q, None) and len(calls) == 1
