"""Which set of outputs a BlockPlanner call writes (no GPU: the sets are tuples of made-up pointers)."""
import itertools

import pytest

from bit_post_quantized_amd import serve


def planner(requests=3):
    p = object.__new__(serve.BlockPlanner)
    p.requests = requests
    p._plans = []
    for k in range(5):
        at = 0x1000 * (k + 1)
        empty = requests == 0    # (an empty tensor's pointer is 0)
        p._plans.append(serve.SlotPlan(*[None] * 6, _outputs=(
            at, 0 if empty else at + 0x100, 7, at + 0x200, at + 0x300, 0 if empty else at + 0x400, at + 0x500)))
    return p


SEQ, STATUS, COUNT = 1, 5, 6   # places in the outputs


def test_the_call_before_and_the_arguments_are_left_alone():
    own = 0xF0000
    for lens, new, count in itertools.product(range(-1, 5), repeat=3):   # -1: the caller's own
        for field in (SEQ, STATUS):
            p = planner()
            sets = [s._outputs for s in p._plans]
            args = (own if lens < 0 else sets[lens][SEQ], own if new < 0 else sets[new][field],
                    own if count < 0 else sets[count][COUNT])
            got = p._other(*args)
            assert got._outputs not in [sets[k] for k in (lens, new, count) if k >= 0], (lens, new, count)
            assert got._outputs != sets[4] and p._plans[4] is got
            free = [s for k, s in enumerate(sets[:4]) if k not in (lens, new, count)]
            assert got._outputs == free[0]


def test_sets_take_turns_without_requests():
    p = planner(0)
    seen = [p._other(0, 0, 0xF0000)._outputs for _ in range(10)]
    assert len(set(seen)) == 5 and seen[:5] == seen[5:]


@pytest.mark.parametrize("ahead", [1, 2])
def test_a_plan_outlives_the_next_call(ahead):
    p = planner()
    last = p._other(1, 2, 3)
    for _ in range(ahead):
        now = p._other(last._outputs[SEQ], last._outputs[STATUS], last._outputs[COUNT])
        assert now is not last
