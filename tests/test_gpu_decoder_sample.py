"""svdq_sample against whole-number arithmetic: tokens have to be equal.  (A weight may differ by a unit,
2^-40 of the largest, where two exponentials round apart; a number drawn that near a border is not among
these.)  A share is rounded to fp32 once, 2^-24 of it, and off by those units: 2^-23 and 2^-30."""
import math

import numpy as np
import pytest
import torch

from bit_post_quantized_amd import decoder
from bit_post_quantized_amd import decoder_binding as DB
from oracle import decoder as od
from oracle.numerics import round_bf16
from tests.serve_cases import to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def settings(rng, rows, kind):
    t = (0.4 + rng.random(rows)).astype(np.float32)
    u = rng.random(rows).astype(np.float32)
    k = p = m = None
    if kind in ("k", "both", "all"):
        k = rng.integers(-1, 60, rows).astype(np.int32)
    if kind in ("p", "both", "all"):
        p = rng.choice([0.0, 0.3, 0.9, 0.999, 1.0, 1.5], rows).astype(np.float32)
    if kind in ("m", "all"):
        m = rng.choice([0.0, 0.02, 0.3, 1.0, 2.0], rows).astype(np.float32)
    if kind == "all":
        t[rng.random(rows) < 0.2] = 0.0
    return t, u, k, p, m


def run(z, t, u, k=None, p=None, m=None, bf16=False, **more):
    d = lambda a: None if a is None else to_dev(a)  # noqa: E731
    zd = z if isinstance(z, torch.Tensor) else to_dev_bf16(z) if bf16 else to_dev(np.asarray(z, np.float32))
    tokens, share = decoder.sample(zd, d(t), d(u), d(k), d(p), d(m), **more)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), share.cpu().numpy()


def check(z, t, u, k=None, p=None, m=None, bf16=False):
    tokens, share = run(z, t, u, k, p, m, bf16)
    for b in range(len(z)):
        want, s = od.sample_row(z[b], float(t[b]), float(u[b]), 0 if k is None else int(k[b]),
                                1.0 if p is None else float(p[b]), 0.0 if m is None else float(m[b]))
        assert tokens[b] == want, (b, tokens[b], want)
        assert abs(share[b] - s) <= 2.0 ** -23 * s + 2.0 ** -30, (b, share[b], s)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "both", "all"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 63), (4, 1000), (40, 1025), (2, 5000), (7, 20011)])
def test_matches(gpu_lib, rows, vocab, kind, bf16):
    rng = np.random.default_rng(rows * 31 + vocab)
    z = rng.standard_normal((rows, vocab)) * 2.5
    z[rng.random((rows, vocab)) < 0.05] = -math.inf
    z[:, 0] = 1.0
    z = round_bf16(z) if bf16 else z.astype(np.float32).astype(np.float64)
    check(z, *settings(rng, rows, kind), bf16=bf16)


@pytest.mark.parametrize("kind", ["none", "k", "p", "all"])
def test_many_numbers_on_one_row(gpu_lib, kind):
    """Every border of a short row is met from both sides."""
    rng = np.random.default_rng(3)
    z = np.tile((rng.standard_normal(12) * 1.5).astype(np.float32).astype(np.float64), (600, 1))
    t, u, k, p, m = settings(rng, 600, kind)
    t[:], u = 0.8, ((np.arange(600) + 0.5) / 600).astype(np.float32)
    check(z, t, u, k, p, m)


@pytest.mark.parametrize("vocab", [17, 3000, 9000])
def test_equal_logits_go_by_index(gpu_lib, vocab):
    # more equal elements than a row's list holds, too
    rows = 8
    z = np.zeros((rows, vocab))
    z[1, vocab // 2] = -0.0
    z[2, ::2] = 1.0
    z[3, 1:] = 0.5
    t, u = np.ones(rows, np.float32), np.linspace(0, 0.9999, rows).astype(np.float32)
    check(z, t, u)
    check(z, t, u, k=np.full(rows, max(vocab // 3, 1), np.int32))
    check(z, t, u, p=np.full(rows, 0.7, np.float32))
    check(z, t, u, k=np.full(rows, vocab // 2 + 1, np.int32), p=np.full(rows, 0.5, np.float32), m=np.full(rows, 0.5, np.float32))
    check(z, np.zeros(rows, np.float32), u)


def test_limits_wider_than_the_list(gpu_lib):
    rng = np.random.default_rng(5)
    rows, vocab = 6, 30000
    z = (rng.standard_normal((rows, vocab)) * 0.3).astype(np.float32).astype(np.float64)
    t, u = np.ones(rows, np.float32), rng.random(rows).astype(np.float32)
    k = np.array([2047, 2048, 2049, 8000, 29999, 30000], np.int32)
    check(z, t, u, k=k)
    check(z, t, u, k=k, p=np.full(rows, 0.8, np.float32))
    check(z * 0.01, t, u, p=np.linspace(0.1, 0.99, rows).astype(np.float32))
    check(z, t * 50, u, p=np.linspace(0.1, 0.99, rows).astype(np.float32), m=np.full(rows, 0.98, np.float32))


def test_ends_of_the_settings(gpu_lib):
    rng = np.random.default_rng(6)
    z = np.tile((rng.standard_normal(500) * 3).astype(np.float32).astype(np.float64), (12, 1))
    t = np.array([1e-45, 1e-6, 0.02, 1e6, np.inf, 1, 1, 1, 1, -1, np.nan, 1], np.float32)
    u = np.array([0.5, 0.5, 0.5, 0.5, 0.5, -1, 1, 2, np.nan, 0.5, 0.5, 0.99999994], np.float32)
    check(z, t, u)
    p = np.array([0, -1, 1e-45, 0.99999994, np.nan, 1, 2, 0.5, 0.5, 0.5, 0.5, 1e-3], np.float32)
    check(z, t, u, p=p)
    check(z, t, u, k=np.array([1, -5, 2 ** 31 - 1, 500, 499, 501, 0, -2 ** 31, 3, 3, 3, 2], np.int32), p=p)
    check(z, t, u, m=np.array([1, 2, np.inf, np.nan, -1, 1e-45, 0.999, 0.5, 0.5, 0.5, 0.5, 0.5], np.float32))


def test_rows_without_a_token_and_infinite_logits(gpu_lib):
    inf = math.inf
    z = np.zeros((7, 2500))
    z[0] = -inf
    z[1, 2400] = np.nan
    z[2, [5, 2000]] = inf
    z[3, 7:] = -inf
    z[4, 0], z[4, 1], z[4, 2] = 3.4e38, -3.4e38, np.nan
    z[5, :] = -inf
    z[5, 2499] = -3e38
    z[6, 1] = 3e38
    u = np.full(7, 0.75, np.float32)
    for t in (0.0, 1.0):
        for k, p in ((None, None), (3, None), (None, 0.9), (3, 0.9)):
            check(z, np.full(7, t, np.float32), u, None if k is None else np.full(7, k, np.int32),
                  None if p is None else np.full(7, p, np.float32))


@pytest.mark.parametrize("rows,vocab", [(1, 1 << 22), (3, 200001), (600, 3000)])
def test_large_vocabularies_and_batches(gpu_lib, rows, vocab):
    """Against the same definition in torch's 64-bit operations (the oracle's lists are too slow)."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randn(rows, vocab, generator=g, device="cuda") * 2
    u = torch.rand(rows, generator=g, device="cuda")
    k = torch.full((rows,), 40, dtype=torch.int32, device="cuda")
    p = torch.full((rows,), 0.9, device="cuda")
    t = torch.full((rows,), 0.9, device="cuda")
    w = torch.round(torch.exp((z.double() - z.double().amax(1, keepdim=True)) / t.double()[:, None]) * 2.0 ** 40).to(torch.int64)
    order = torch.sort(z, dim=1, descending=True, stable=True)[1]
    sw = torch.gather(w, 1, order)
    for limits in ((None, None), (k, None), (None, p), (k, p)):
        stay = torch.ones_like(sw, dtype=torch.bool)
        if limits[0] is not None:
            stay[:, 40:] = False
        if limits[1] is not None:
            kw = torch.where(stay, sw, 0)
            stay &= (torch.cumsum(kw, 1) - kw).double() < p.double()[:, None] * kw.sum(1, keepdim=True).double()
        kept = torch.zeros_like(w).scatter_(1, order, torch.where(stay, sw, 0))
        total = kept.sum(1)
        at = torch.floor(total.double() * u.double()).to(torch.int64)
        want = (torch.cumsum(kept, 1) <= at[:, None]).sum(1)
        tokens, _ = decoder.sample(z, t, u, *limits)
        assert torch.equal(tokens.long(), want)


def test_strided_rows_guards_and_any_workspace(gpu_lib):
    rng = np.random.default_rng(8)
    wide = to_dev_bf16(round_bf16(rng.standard_normal((5, 3003)) * 3))
    z = wide[:, 1:3002]                       # rows at odd elements
    t, u, k, p, m = settings(rng, 5, "both")
    want = run(z.contiguous(), t, u, k, p)
    guard = torch.full((7,), -7, dtype=torch.int32, device="cuda")
    need = DB.svdq_sample_workspace_bytes(5, 3001)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = run(z, t, u, k, p, tokens=guard[1:6], workspace=ws[:need])
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert guard[0] == -7 and guard[6] == -7 and (ws[need:] == 0xFF).all()
    none = decoder.sample(z[:0], to_dev(t[:0]), to_dev(u[:0]))
    assert none[0].shape == (0,)


def test_captured_and_replayed(gpu_lib):
    rng = np.random.default_rng(9)
    z = to_dev((rng.standard_normal((4, 6000)) * 2).astype(np.float32))
    t, u, k, p, m = (None if a is None else to_dev(a) for a in settings(rng, 4, "all"))
    decoder.sample(z, t, u, k, p, m)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tokens, share = decoder.sample(z, t, u, k, p, m)
    for i in range(4):
        z.copy_(to_dev((rng.standard_normal((4, 6000)) * (1 + i)).astype(np.float32)))
        u.copy_(to_dev(rng.random(4).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        want = decoder.sample(z, t, u, k, p, m)
        assert torch.equal(tokens, want[0]) and torch.equal(share, want[1]), i


@pytest.mark.parametrize("bf16", [False, True])
def test_counts_between_the_parts_and_the_list(gpu_lib, bf16):
    """Top-k from fewer elements than a row has parts to more than its list holds, with top-p and min-p."""
    rng = np.random.default_rng(11)
    k = np.array([1, 63, 64, 65, 255, 256, 257, 300, 511, 512, 513, 700, 1000, 2047, 2049, 4000], np.int32)
    z = rng.standard_normal((len(k), 40009)) * np.linspace(0.5, 4, len(k))[:, None]
    z = round_bf16(z) if bf16 else z.astype(np.float32).astype(np.float64)
    t, u, _, _, _ = settings(rng, len(k), "none")
    check(z, t, u, k=k, bf16=bf16)
    check(z, t, u, k=k, p=np.full(len(k), 0.9, np.float32), bf16=bf16)
    check(z, t, u, k=k, p=np.full(len(k), 0.99, np.float32), m=np.full(len(k), 0.01, np.float32), bf16=bf16)


@pytest.mark.parametrize("bf16", [False, True])
def test_more_rows_than_are_done_at_a_time(gpu_lib, bf16):
    rng = np.random.default_rng(12)
    z = rng.standard_normal((4099, 130)) * 2
    z = round_bf16(z) if bf16 else z.astype(np.float32).astype(np.float64)
    check(z, *settings(rng, len(z), "all"), bf16=bf16)


def test_rows_past_two_gib(gpu_lib):
    """Logits whose rows stand far apart: the last one begins past 2^32 bytes."""
    far = 1 << 29
    store = torch.full((2 * far + 1000,), float("nan"), device="cuda")
    rng = np.random.default_rng(13)
    z = (rng.standard_normal((3, 1000)) * 2).astype(np.float32)
    logits = store.as_strided((3, 1000), (far, 1))
    logits.copy_(to_dev(z))
    t, u, k, p, m = settings(rng, 3, "both")
    tokens, share = run(logits, t, u, k, p)
    want, _ = run(z, t, u, k, p)
    assert (tokens == want).all() and (tokens >= 0).all()


def test_greedy_takes_the_first_of_the_largest(gpu_lib):
    """In every place of chunk and part, next to one that is hardly smaller, and to its equals behind."""
    rng = np.random.default_rng(14)
    vocab = 9001
    at = np.concatenate([[0, 1, 7, 8, 2047, 2048, 2049, 4095, 4096, vocab - 2, vocab - 1], rng.integers(0, vocab, 40)])
    z = np.minimum(rng.standard_normal((len(at), vocab)), 3).astype(np.float32)
    for b, i in enumerate(at):
        z[b, i] = 4.0
        z[b, min(i + 1 + b % 5, vocab - 1)] = 4.0 if i + 1 + b % 5 < vocab else z[b, vocab - 1]
        if i:
            z[b, i - 1] = np.nextafter(np.float32(4), np.float32(0))
    tokens, share = run(z, np.zeros(len(at), np.float32), np.full(len(at), 0.5, np.float32))
    assert (tokens == at).all() and (share == 1).all()
