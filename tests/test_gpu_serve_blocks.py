"""The block cache: plan, release, append and read-back, exact against the oracle."""
import numpy as np
import pytest
import torch

from bit_post_quantized_amd import serve
from bit_post_quantized_amd import serve_binding as SB
from oracle import serve as osv
from oracle.numerics import decode_bf16
from tests.serve_cases import (bf16_values, dev_cache, host64, host_bits, host_cache, random_cache,
                               to_dev, to_dev_bf16)

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------------- plan
def plan_case(seed, n, max_ctx, max_new, bs, width, free, count=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, max_ctx + 1, n)
    new = rng.integers(0, max_new + 1, n)
    held = -(-ctx // bs)
    ids = rng.permutation(int(held.sum()) + free + 3)
    tables = np.full((n, width), -7)
    at = 0
    for b in range(n):
        k = min(int(held[b]), width)
        tables[b, :k] = ids[at:at + k]
        at += held[b]
    return ctx, new, tables, ids[at:at + free], free if count is None else count


def run_plan(ctx, new, tables, bs, free, count, rows):
    i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
    t, f = i32(tables), i32(free)
    p = serve.BlockPlanner(t, f, bs, rows).plan(i32(ctx), i32(new), i32([count]))
    torch.cuda.synchronize()
    return dict(tables=t, cu=p.cu_rows, seq=p.seq_lens, positions=p.positions, slots=p.slots,
                status=p.status, free_count=p.free_count), f


def same(got, want):
    for k, v in want.items():
        np.testing.assert_array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(v).reshape(-1), err_msg=k)


@pytest.mark.parametrize("n,max_ctx,max_new,bs,width,free,rows", [
    (1, 0, 1, 16, 1, 1, 1), (1, 100, 300, 16, 30, 40, 300), (8, 4096, 1, 16, 300, 9, 8),
    (5, 1000, 40, 128, 9, 10, 256), (64, 500, 3, 32, 17, 30, 200), (300, 2000, 30, 64, 33, 200, 9000),
    (1023, 64, 2, 16, 6, 500, 2500), (1024, 64, 2, 16, 6, 5000, 2500), (1025, 64, 2, 16, 6, 100, 2500),
    (3000, 300, 4, 16, 20, 4000, 9000),           # three chunks of requests
    (40, 300, 100, 16, 20, 400, 1500),            # tables too narrow for some, rows for the last
    (10, 50, 5, 16, 4, 0, 60),                    # an empty free list
    (4, 10, 70000, 64, 1200, 5000, 200000),       # long prompts over many row ranges
])
def test_plan_matches_the_oracle(gpu_lib, n, max_ctx, max_new, bs, width, free, rows):
    for seed in range(3):
        case = plan_case(seed * 101 + n, n, max_ctx, max_new, bs, width, free)
        ctx, new, tables, pool, count = case
        pool = pool if len(pool) else np.array([0])
        want = osv.plan(ctx, new, tables, bs, pool, count, rows)
        got, f = run_plan(ctx, new, tables, bs, pool, count, rows)
        same(got, want)
        np.testing.assert_array_equal(f.cpu().numpy(), pool)


def test_plan_of_nothing_and_odd_counts(gpu_lib):
    # no requests; no rows; negative lengths count as 0; a count past the list is the list
    got, _ = run_plan([], [], np.zeros((0, 4)), 16, [5, 6], 2, 3)
    same(got, dict(cu=[0], positions=[0, 0, 0], slots=[-1, -1, -1], free_count=[2]))
    got, _ = run_plan([3, -5, 4], [-1, 2, 0], np.zeros((3, 2)), 16, [5, 6], 99, 4)
    same(got, osv.plan([3, -5, 4], [-1, 2, 0], np.zeros((3, 2)), 16, [5, 6], 99, 4))
    got, _ = run_plan([3, 0], [0, 0], np.ones((2, 1)), 16, [5], -3, 0)
    same(got, dict(cu=[0, 0, 0], seq=[3, 0], status=[0, 0], free_count=[0]))


def test_plan_with_lengths_at_the_ends_of_their_type(gpu_lib):
    big = 2 ** 31 - 1
    ctx, new = [5, big, 0, 7], [2, big, big, 1]
    got, _ = run_plan(ctx, new, np.full((4, 3), 2), 16, [9, 8], 2, 20)
    assert got["status"].cpu().tolist() == [0, 2, 2, 3]
    assert got["slots"].cpu().tolist()[:2] == [2 * 16 + 5, 2 * 16 + 6]
    assert all(s == -1 for s in got["slots"].cpu().tolist()[2:])
    assert got["free_count"].cpu().tolist() == [2]


def test_steps_in_a_row_and_release_keep_every_block_once(gpu_lib):
    # plans whose lengths and counts feed the next one, with requests that finish and begin again
    rng = np.random.default_rng(5)
    n, width, bs, num, rows = 12, 6, 16, 40, 64
    i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
    tables, free = i32(np.full((n, width), -1)), i32(rng.permutation(num))
    planner = serve.BlockPlanner(tables, free, bs, rows)
    seq, count = i32(np.zeros(n)), i32([num])
    for step in range(30):
        new = rng.integers(0, 8, n)
        before = (seq.cpu().numpy(), tables.cpu().numpy(), free.cpu().numpy(), int(count))
        p = planner.plan(seq, i32(new), count)
        want = osv.plan(before[0], new, before[1], bs, before[2], before[3], rows)
        same(dict(tables=tables, cu=p.cu_rows, seq=p.seq_lens, positions=p.positions, slots=p.slots,
                  status=p.status, free_count=p.free_count), want)
        seq, count = p.seq_lens, p.free_count
        done = (rng.random(n) < 0.15) | (seq.cpu().numpy() > 80)
        seq, count = planner.release(seq, to_dev(done.astype(np.uint8)), count)
        t, s, c = tables.cpu().numpy(), seq.cpu().numpy(), int(count)
        held = [t[b, j] for b in range(n) for j in range(-(-s[b] // bs))]
        assert sorted(held + list(free.cpu().numpy()[:c])) == list(range(num)), step
        assert (s[done] == 0).all() and (t[done] == -1).all()


def test_a_plan_outlives_the_next_call(gpu_lib):
    """Arguments of the caller's own, of the last plan, of an older one, or of two plans at once:
    the plan before a call still holds what it held after it."""
    i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
    own = i32([3, 40]), i32([1, 1]), i32([6])
    planner = serve.BlockPlanner(i32(np.zeros((2, 8))), i32(np.arange(6)), 16, 4)
    plans = [planner.plan(*own)]
    for k in range(12):
        last, older = plans[-1], plans[-2 if k else -1]
        lens = (own[0], last.seq_lens, older.seq_lens, last.seq_lens)[k % 4]
        count = (own[2], last.free_count, older.free_count, older.free_count)[k % 4]
        held = [t.clone() for t in (last.cu_rows, last.seq_lens, last.positions, last.slots, last.status, last.free_count)]
        args = lens.clone(), count.clone()
        plans.append(planner.plan(lens, own[1], count))
        now = (last.cu_rows, last.seq_lens, last.positions, last.slots, last.status, last.free_count)
        assert all(torch.equal(a, b) for a, b in zip(held, now)), k
        assert torch.equal(args[0], lens) and torch.equal(args[1], count), k
        assert torch.equal(plans[-1].seq_lens, args[0] + 1), k


def test_release_keeps_to_the_free_list(gpu_lib):
    i32 = lambda a: to_dev(np.asarray(a), torch.int32)  # noqa: E731
    tables, free = i32([[1, 2, 3], [4, 5, 6], [7, 8, 9]]), i32([10, 0, 0])
    seq_out, out = i32([0, 0, 0]), i32([0])
    SB.kv_block_release(i32([40, 20, 99]), to_dev(np.array([1, 0, 1], np.uint8)), tables, 16, free,
                        i32([1]), seq_out, out)
    assert free.cpu().tolist() == [10, 1, 2] and out.cpu().tolist() == [3]
    assert seq_out.cpu().tolist() == [0, 20, 0]
    assert tables.cpu().tolist() == [[-1] * 3, [4, 5, 6], [-1] * 3]


# ----------------------------------------------------------------------------------- append
def check_append(seed, num, heads, bs, dim, slots, scale=1.0, strided=False, x=None, rounds=1):
    """Appends at `slots` to a random cache and compares the whole cache with the oracle's."""
    rng = np.random.default_rng(seed)
    kc, ks, vc, vs = random_cache(rng, num, heads, bs, dim)
    cache = dev_cache(kc, ks, vc, vs)
    ok, ov = osv.Cache(kc, ks), osv.Cache(vc, vs)
    for _ in range(rounds):
        k = bf16_values(rng, len(slots), heads, dim, scale=scale) if x is None else x
        v = bf16_values(rng, len(slots), heads, dim, scale=scale) if x is None else x
        if strided:   # slices of a fused projection
            fused = torch.zeros(len(slots), 3 * heads + 1, dim, dtype=torch.bfloat16, device="cuda")
            fused[:, 1:heads + 1], fused[:, 2 * heads + 1:] = to_dev_bf16(k), to_dev_bf16(v)
            cache.append(fused[:, 1:heads + 1], fused[:, 2 * heads + 1:], to_dev(np.asarray(slots, np.int64)))
        else:
            cache.append(to_dev_bf16(k), to_dev_bf16(v), to_dev(np.asarray(slots, np.int64)))
        ok.append(k, slots)
        ov.append(v, slots)
    torch.cuda.synchronize()
    gk, gks, gv, gvs = host_cache(cache)
    np.testing.assert_array_equal(gks, ok.scale)
    np.testing.assert_array_equal(gvs, ov.scale)
    np.testing.assert_array_equal(gk, ok.codes)
    np.testing.assert_array_equal(gv, ov.codes)
    return cache, ok, ov


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_append_runs_of_every_kind(gpu_lib, bs, dim):
    # whole blocks, a prompt's tail, single tokens at a block's first, inner and last place, rows
    # without a token before, between and behind, and one run for each length around the tiles
    slots = [-1] + list(range(2 * bs, 3 * bs)) + list(range(5 * bs, 5 * bs + bs // 2 + 1)) + [-1, -5]
    slots += [7 * bs, 8 * bs + 3, 9 * bs + bs - 1] + [(1 << 40)] + list(range(10 * bs + 5, 10 * bs + 11))
    slots += [14 * bs] + list(range(11 * bs + 1, 12 * bs)) + list(range(12 * bs, 13 * bs)) + [-1]
    check_append(bs + dim, 15, 3, bs, dim, slots)
    check_append(bs + dim + 1, 14, 2, bs, dim, slots, scale=30.0, strided=True)


@pytest.mark.parametrize("heads", [1, 2, 8, 13])
def test_append_one_token_at_a_time(gpu_lib, heads):
    # a block filled token by token: the scale grows and the earlier codes are taken along
    num, bs, dim = 4, 16, 64
    rng = np.random.default_rng(heads)
    cache = serve.BlockCache(torch.full((num, heads, bs, dim), 255, dtype=torch.uint8, device="cuda"),
                             torch.full((num, heads, dim, bs), 255, dtype=torch.uint8, device="cuda"),
                             torch.full((num, heads), float("nan"), device="cuda"),
                             torch.full((num, heads), float("nan"), device="cuda"))
    ok = osv.Cache(np.full((num, heads, bs, dim), 127), np.full((num, heads), np.nan))
    ov = osv.Cache(np.full((num, heads, bs, dim), 127), np.full((num, heads), np.nan))
    for t in range(20):
        slots = np.array([(1 + t // bs) * bs + t % bs])
        k, v = bf16_values(rng, 1, heads, dim, scale=1 + t), bf16_values(rng, 1, heads, dim, scale=2.0)
        cache.append(to_dev_bf16(k), to_dev_bf16(v), to_dev(slots))
        ok.append(k, slots)
        ov.append(v, slots)
    at = np.array([bs + i for i in range(20)])
    kr, vr = cache.read(to_dev(at))
    np.testing.assert_array_equal(host_bits(kr), ok.values(at))
    np.testing.assert_array_equal(host_bits(vr), ov.values(at))
    assert torch.isnan(cache.k_scale[0]).all() and (cache.k_codes[0] == 255).all()


@pytest.mark.parametrize("scale", [0.0, 1e-40, 3e-38, 1e-30, 1e30])
def test_append_of_extreme_magnitudes(gpu_lib, scale):
    rng = np.random.default_rng(9)
    x = bf16_values(rng, 40, 2, 64) * scale
    from oracle.numerics import round_bf16
    x = round_bf16(x)
    check_append(9, 4, 2, 16, 64, list(range(16, 56)), x=x)


def test_append_many_rows_and_blocks_of_a_long_cache(gpu_lib):
    rng = np.random.default_rng(2)
    order = rng.permutation(70)
    slots = np.concatenate([np.arange(b * 32, b * 32 + 32) for b in order[:60]] + [[-1] * 9])
    check_append(3, 70, 4, 32, 128, list(slots), rounds=2)


def test_cache_past_four_gib(gpu_lib):
    # block offsets beyond 2^32 bytes: the last blocks of two code arrays of 8.6 GB
    num, heads, bs, dim = 2 ** 17 + 3, 8, 64, 128
    cache = serve.BlockCache.empty(num, bs, heads, dim)
    assert (num - 1) * heads * bs * dim > 2 ** 33
    rng = np.random.default_rng(1)
    k, v = bf16_values(rng, bs, heads, dim), bf16_values(rng, bs, heads, dim)
    for b in (num - 1, 0, 2 ** 15, 2 ** 16 + 1):
        slots = to_dev(np.arange(b * bs, b * bs + bs))
        cache.append(to_dev_bf16(k), to_dev_bf16(v), slots)
        kr, vr = cache.read(slots)
        # half a code step (amax / 127 at most), then bf16's half step of a value <= amax
        for got, x in ((kr, k), (vr, v)):
            off, amax = float(np.abs(host64(got) - x).max()), float(np.abs(x).max())
            assert off <= amax * (0.5 / 127 + 2.0 ** -8) * (1 + 2.0 ** -8)
        i32 = lambda *v: to_dev(np.array(v), torch.int32)  # noqa: E731
        out = cache.attention(to_dev_bf16(k[-1:]), i32([b]), i32(bs), i32(0, 1), 1)
        # the same row in shares of a wide table, and 40 times over (the kernel of more rows)
        wide = cache.attention(to_dev_bf16(k[-1:]), i32([b] + [-1] * 150), i32(bs), i32(0, 1), 1)
        many = cache.attention(to_dev_bf16(k[-1:]).repeat(40, 1, 1), i32([b]), i32(bs), i32(0, 40), 40, causal=False)
        s = np.einsum("hd,thd->ht", k[-1], host64(kr)) / np.sqrt(dim)
        w = np.exp(s - s.max(1, keepdims=True))
        want = np.einsum("ht,thd->hd", w / w.sum(1, keepdims=True), host64(vr))
        # weights and values as read back, each rounded to bf16 (2^-8), against the codes' own: the
        # scores (up to 11 here) are off by 2^-8 of sum |q k|, so compare loosely, by largest value
        amax = float(np.abs(v).max())
        for o in (out, wide, many):
            assert float(np.abs(host64(o) - want).max()) <= 2.0 ** -4 * amax
    del cache
    torch.cuda.empty_cache()


def test_read_any_order_repeats_and_gaps(gpu_lib):
    rng = np.random.default_rng(4)
    for bs, dim in ((16, 64), (128, 128), (64, 64)):
        kc, ks, vc, vs = random_cache(rng, 5, 3, bs, dim)
        cache = dev_cache(kc, ks, vc, vs)
        slots = rng.integers(0, 5 * bs, 333)
        slots[10], slots[11], slots[332] = -1, 5 * bs, -(1 << 50)
        live = (slots >= 0) & (slots < 5 * bs)
        k = torch.full((333, 3, dim), 3.0, dtype=torch.bfloat16, device="cuda")
        v = torch.full((333, 3, dim), 4.0, dtype=torch.bfloat16, device="cuda")
        cache.read(to_dev(slots), k, v)
        np.testing.assert_array_equal(host_bits(k)[live], osv.Cache(kc, ks).values(slots[live]))
        np.testing.assert_array_equal(host_bits(v)[live], osv.Cache(vc, vs).values(slots[live]))
        assert (host64(k)[~live] == 3).all() and (host64(v)[~live] == 4).all()
    k, v = cache.read(to_dev(np.zeros(0, np.int64)))
    assert k.shape[0] == 0
    assert np.all(decode_bf16(host_bits(cache.read(to_dev(np.array([-1])))[0])) == 0)


def test_append_refusals(gpu_lib):
    cache = serve.BlockCache.empty(4, 16, 2, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="same rows"):
        cache.append(x, x[:2], s)
    with pytest.raises(ValueError, match="k must be"):
        cache.append(x.half(), x, s)
    with pytest.raises(ValueError, match="slots must be"):
        cache.append(x, x, s.int())
    with pytest.raises(ValueError, match="contiguous rows"):
        cache.append(torch.zeros(3, 64, 2, dtype=torch.bfloat16, device="cuda").transpose(1, 2), x, s)
    with pytest.raises(RuntimeError, match="k_stride"):
        cache.append(torch.zeros(3, 132, dtype=torch.bfloat16, device="cuda")[:, :128].view(3, 2, 64), x, s)
    with pytest.raises(RuntimeError, match="16-byte aligned"):
        cache.append(torch.zeros(388, dtype=torch.bfloat16, device="cuda")[4:].view(3, 2, 64), x, s)
    cache.append(x[:0], x[:0], s[:0])
