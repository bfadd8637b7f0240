"""The operators between a decoding step's projections, as cases that can be timed and checked: the
root-mean-square norm with the residual's addition (to 16 bits, or to 8 with a scale for each row),
the product of 8-bit integers with scales for each row and column, rotary positions, and sampling
from logits with given random numbers.

``run`` computes a case in plain torch operations (``own`` false) or through the framework's
entry points (``own`` true); ``exact`` computes it in 64 bits from the definitions.

Definitions:

  norm     h = x + residual, residual' = h rounded to its type, y = h / sqrt(mean(h^2) + eps) gamma;
           in 8 bits: s = fl32(max |y| / 127) of the row, c = clamp(rne(fl32(y / s)), -127, 127)
  linear8  Y[m, n] = sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n]
  rope     pairs (a, b) of the first rot_dim channels of a head, channels i and i + rot_dim / 2, or
           2 i and 2 i + 1 (interleaved), become scale (a cos t - b sin t, a sin t + b cos t),
           t = position freqs[i]; the other channels stay
  sample   w_i = rne(2^40 exp((z_i - max z) / temperature)), whole numbers. In the order of falling
           z (the lower index first among equals) the first top_k stay; of these, each before which
           less than top_p of their sum stands; of these, those with w_i >= min_p 2^40. The token is
           the first in the vocabulary's order up to and with which more than floor(u W) of the
           remaining sum W stands. Temperature 0: the first largest logit.
"""
import math

import torch

own = False

DEV = "cuda"
UNIT = 40


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token before a projection in 8 bits: the smallest call, where the launch is what counts
        dict(name="norm_1x4096_q8", op="norm", rows=1, hidden=4096, x="bf16", residual="bf16", out="q8"),
        # a batch that decodes, with a residual stream in fp32, before a projection in 16 bits
        dict(name="norm_200x5120_bf16", op="norm", rows=200, hidden=5120, x="fp32", residual="fp32", out="bf16"),
        # prompts before a projection in 8 bits
        dict(name="norm_16384x8192_q8", op="norm", rows=16384, hidden=8192, x="bf16", residual="bf16", out="q8"),
        # one token through a square projection
        dict(name="linear8_1x4096x4096", op="linear8", rows=1, k=4096, n=4096, bias=True, out="bf16"),
        # a batch that decodes through a wide up-projection: the weights' bytes
        dict(name="linear8_40x8192x28672", op="linear8", rows=40, k=8192, n=28672, bias=False, out="bf16"),
        # a chunk of a prompt through a down-projection, accumulated further in fp32
        dict(name="linear8_500x12288x4096_f32", op="linear8", rows=500, k=12288, n=4096, bias=True, out="fp32"),
        # prompts through a wide projection: the matrix units' rate
        dict(name="linear8_8192x8192x12288", op="linear8", rows=8192, k=8192, n=12288, bias=False, out="bf16"),
        # a batch that decodes at far positions, q and k slices of a fused projection
        dict(name="rope_64_decode", op="rope", rows=64, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, x="bf16", far=131072),
        # prompts, half of each head rotated, pairs side by side
        dict(name="rope_20000_prompts", op="rope", rows=20000, heads=24, kv_heads=8, dim=128, rot=64, interleaved=True, x="bf16", far=32768),
        # one request's next token out of a large vocabulary
        dict(name="sample_1x131072", op="sample", rows=1, vocab=131072, logits="fp32", limits="both"),
        # a batch of requests, each with settings of its own
        dict(name="sample_64x131072", op="sample", rows=64, vocab=131072, logits="fp32", limits="mixed"),
        # many short requests over a smaller vocabulary of odd size, logits in 16 bits
        dict(name="sample_300x32001_bf16", op="sample", rows=300, vocab=32001, logits="bf16", limits="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear8", "linear8", "rope", "sample"))
    if op == "norm":
        hidden = 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, min(20000, (1 << 27) // hidden)), hidden=hidden,
                    x=rng.choice(("bf16", "bf16", "fp32")), residual=rng.choice(("bf16", "bf16", "fp32", "none")),
                    out=rng.choice(("bf16", "q8", "q8")))
    if op == "linear8":
        k = 64 * _log(rng, 1, 256)
        n = _log(rng, 1, 30000)
        rows = rng.choice((_log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 65, 8192)))
        rows = max(1, min(rows, (1 << 39) // (k * n)))
        return dict(op=op, rows=rows, k=k, n=n, bias=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "fp32")))
    if op == "rope":
        dim = rng.choice((64, 96, 128, 192, 256))
        kv = rng.choice((1, 2, 4, 8))
        heads = kv * rng.choice((1, 2, 3, 4, 6, 8))
        rot = dim if rng.random() < 0.6 else 16 * rng.randint(1, dim // 16)
        return dict(op=op, rows=_log(rng, 1, min(20000, (1 << 26) // (dim * (heads + kv)))), heads=heads, kv_heads=kv,
                    dim=dim, rot=rot, interleaved=rng.random() < 0.4, x=rng.choice(("bf16", "bf16", "fp32")),
                    far=rng.choice((2048, 32768, 1 << 20)))
    vocab = _log(rng, 500, 200000)
    return dict(op=op, rows=_log(rng, 1, min(512, (1 << 23) // vocab)), vocab=vocab,
                logits=rng.choice(("fp32", "fp32", "bf16")), limits=rng.choice(("none", "both", "mixed", "mixed")))


# ----------------------------------------------------------------------------------- inputs
def _prepare_norm(case, g):
    M, K = case["rows"], case["hidden"]
    hot = torch.where(_rand(g, K) < 0.01, 12.0, 1.0)     # a few channels of a residual stream are large
    s = dict(x=_randn(g, M, K).to(_type(case["x"])), gamma=(1.0 + 0.2 * _randn(g, K)) / hot.sqrt(), eps=1e-6,
             residual=None if case["residual"] == "none" else (3.0 * _randn(g, M, K) * hot).to(_type(case["residual"])))
    if own:
        from bit_post_quantized_amd import decoder
        s["norm"] = decoder.RMSNorm(s["gamma"], s["eps"])
    return s


def _prepare_linear8(case, g):
    M, K, N = case["rows"], case["k"], case["n"]

    def codes(rows):                                     # a row's largest value is 127
        c = torch.empty(rows, K, dtype=torch.int8, device=DEV)
        step = max(1, (1 << 27) // K)
        for r in range(0, rows, step):
            c[r:r + step] = (_randn(g, min(step, rows - r), K) * 32.0).round_().clamp_(-127, 127)
        return c

    s = dict(qx=codes(M), sx=(2.0 + _rand(g, M)) / 127.0, qw=codes(N), sw=(3.0 + _rand(g, N)) / (127.0 * math.sqrt(K)),
             bias=_randn(g, N).to(torch.bfloat16) if case["bias"] else None)
    if own:
        from bit_post_quantized_amd import decoder
        s["linear"] = decoder.Linear8(s["qw"], s["sw"], s["bias"])
        s["rows8"] = decoder.Rows8(s["qx"], s["sx"])
    return s


def _prepare_rope(case, g):
    M, H, KV, D, rot = (case[x] for x in ("rows", "heads", "kv_heads", "dim", "rot"))
    qkv = _randn(g, M, H + 2 * KV, D).to(_type(case["x"]))   # q and k are slices of a fused projection
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    s = dict(q=qkv[:, :H], k=qkv[:, H:H + KV], positions=(_rand(g, M).double() * case["far"]).to(torch.int32),
             freqs=10000.0 ** (-2.0 * i / rot), rot=rot, interleaved=case["interleaved"], scale=1.1 if case["far"] > 32768 else 1.0,
             q_out=torch.empty(M, H, D, dtype=torch.bfloat16, device=DEV),
             k_out=torch.empty(M, KV, D, dtype=torch.bfloat16, device=DEV))
    if own:
        from bit_post_quantized_amd import decoder
        s["rope"] = decoder.Rope(s["freqs"], interleaved=s["interleaved"], scale=s["scale"])
    return s


def _prepare_sample(case, g):
    M, V = case["rows"], case["vocab"]
    z = _randn(g, M, V) * (1.0 + 2.0 * _rand(g, M, 1))   # from flat rows to ones of a few likely tokens
    z = z + torch.where(_rand(g, M, V) < 20.0 / V, 6.0 * _rand(g, M, V), 0.0)
    z = torch.where(_rand(g, M, V) < 0.02, -math.inf, z)  # tokens that a grammar forbids
    pick = _rand(g, 4, M)
    mixed = case["limits"] == "mixed"
    s = dict(logits=z.to(_type(case["logits"])), temperature=0.5 + _rand(g, M), uniform=_rand(g, M),
             top_k=None, top_p=None, min_p=None)
    if mixed:
        s["temperature"] = torch.where(pick[0] < 0.1, 0.0, s["temperature"])
    if case["limits"] != "none":
        k = (5 + 95 * _rand(g, M)).to(torch.int32)
        s["top_k"] = torch.where(pick[1] < 0.4, 0, k).to(torch.int32) if mixed else k
        p = 0.5 + 0.49 * _rand(g, M)
        s["top_p"] = torch.where(pick[2] < 0.4, 1.0, p) if mixed else p
    if mixed:
        s["min_p"] = torch.where(pick[3] < 0.6, 0.0, 0.1 * _rand(g, M))
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = dict(norm=_prepare_norm, linear8=_prepare_linear8, rope=_prepare_rope, sample=_prepare_sample)[case["op"]]
    return dict(make(case, g), op=case["op"], out=case.get("out"))


# ------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    h, r = s["x"].float(), s["residual"]
    if r is not None:
        h = h + r.float()
        r = h.to(r.dtype)
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["gamma"]
    if s["out"] == "bf16":
        return dict(y=y.to(torch.bfloat16), residual=r)
    top = y.abs().amax(dim=1)
    scales = top / torch.full_like(top, 127.0)            # (a Python divisor becomes a product)
    c = torch.where(scales[:, None] > 0, torch.round(y / scales[:, None]), 0.0).clamp(-127, 127)
    return dict(values=(c * scales[:, None]).to(torch.bfloat16), scales=scales, residual=r)


def _plain_linear8(s):
    y = (s["qx"].float() @ s["qw"].float().t()) * s["sx"][:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y if s["out"] == "fp32" else y.to(torch.bfloat16)


def _plain_turn(x, cos, sin, rot, interleaved):
    head = x[..., :rot].float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned.to(torch.bfloat16), x[..., rot:].to(torch.bfloat16)), dim=-1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
    s["q_out"].copy_(_plain_turn(s["q"], cos, sin, s["rot"], s["interleaved"]))
    s["k_out"].copy_(_plain_turn(s["k"], cos, sin, s["rot"], s["interleaved"]))
    return s["q_out"], s["k_out"]


def _plain_sample(s):
    z, t = s["logits"].double(), s["temperature"].double()[:, None]
    rows, vocab = z.shape
    top = z.amax(dim=1, keepdim=True)
    w = torch.exp((z - top) / torch.where(t > 0, t, 1.0))
    w = torch.round(w * 2.0 ** UNIT).to(torch.int64)
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    sw = torch.gather(w, 1, order)
    rank = torch.arange(vocab, device=DEV)
    stay = torch.where(t > 0, vocab, 1) > rank
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        stay = stay & (rank < torch.where(k > 0, k, vocab))
    if s["top_p"] is not None:
        sw = torch.where(stay, sw, 0)
        before = torch.cumsum(sw, dim=1) - sw
        p = s["top_p"].double()[:, None]
        least = p * sw.sum(dim=1, keepdim=True).double()
        stay = stay & ((before.double() < least) | (p >= 1) | (rank == 0))
    if s["min_p"] is not None:
        stay = stay & (sw.double() >= s["min_p"].double()[:, None] * 2.0 ** UNIT)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(stay, sw, 0))
    total = kept.sum(dim=1)
    at = torch.floor(total.double() * s["uniform"].double()).to(torch.int64)
    at = torch.minimum(at, total - 1)
    tokens = (torch.cumsum(kept, dim=1) <= at[:, None]).sum(dim=1)
    share = torch.gather(kept, 1, tokens[:, None])[:, 0].double() / total.double()
    return tokens.to(torch.int32), share.float()


def run(state):
    s, op = state, state["op"]
    if not own:
        return dict(norm=_plain_norm, linear8=_plain_linear8, rope=_plain_rope, sample=_plain_sample)[op](s)
    if op == "norm":
        if s["out"] == "bf16":
            y, residual = s["norm"](s["x"], s["residual"])
            return dict(y=y, residual=residual)
        rows8, residual = s["norm"].rows8(s["x"], s["residual"])
        values = torch.empty_like(rows8.codes, dtype=torch.bfloat16)
        torch.mul(rows8.codes, rows8.scales[:, None], out=values)   # what the codes stand for
        return dict(values=values, scales=rows8.scales, residual=residual)
    if op == "linear8":
        return s["linear"](s["rows8"], out_dtype=torch.float32 if s["out"] == "fp32" else torch.bfloat16)
    if op == "rope":
        return s["rope"](s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
    from bit_post_quantized_amd import decoder
    return decoder.sample(s["logits"], s["temperature"], s["uniform"], s["top_k"], s["top_p"], s["min_p"])


# ----------------------------------------------------------------------------- work and exact
def _size(name):
    return 4 if name == "fp32" else 2


def work(case):
    op, M = case["op"], case["rows"]
    if op == "norm":
        K = case["hidden"]
        stream = 0 if case["residual"] == "none" else 2 * _size(case["residual"])
        return dict(bytes=M * K * (_size(case["x"]) + stream + (2 if case["out"] == "bf16" else 1)) + 4 * K
                    + (0 if case["out"] == "bf16" else 4 * M), flops=6 * M * K)
    if op == "linear8":
        K, N = case["k"], case["n"]
        return dict(bytes=K * (M + N) + _size(case["out"]) * M * N + 4 * (M + N) + (2 * N if case["bias"] else 0),
                    flops=2 * M * N * K)
    if op == "rope":
        n = M * (case["heads"] + case["kv_heads"])
        return dict(bytes=n * case["dim"] * (_size(case["x"]) + 2) + 4 * M + 4 * case["rot"], flops=3 * n * case["rot"])
    return dict(bytes=M * (case["vocab"] * _size(case["logits"]) + 28), flops=20 * M * case["vocab"])


def _exact_sample(s):
    import numpy as np
    z, t, u = (s[x].double().cpu().numpy() for x in ("logits", "temperature", "uniform"))
    k, p, m = (None if s[x] is None else s[x].double().cpu().numpy() for x in ("top_k", "top_p", "min_p"))
    tokens, share = [], []
    for b in range(z.shape[0]):
        if t[b] <= 0:
            tokens.append(int(np.argmax(z[b])))
            share.append(1.0)
            continue
        w = np.rint(np.exp((z[b] - z[b].max()) / t[b]) * float(1 << UNIT)).astype(np.int64)
        live = np.flatnonzero(w)                          # (nothing else can be drawn)
        by = live[np.lexsort((live, -z[b][live]))]
        if k is not None and k[b] > 0:
            by = by[:int(k[b])]
        if p is not None and p[b] < 1:
            run_ = np.concatenate(([0], np.cumsum(w[by])))
            by = by[:max(1, int(np.searchsorted(run_[:-1], p[b] * float(run_[-1]), side="left")))]
        if m is not None:
            by = by[w[by] >= m[b] * float(1 << UNIT)]
        by = np.sort(by)
        run_ = np.cumsum(w[by])
        at = min(int(np.floor(float(run_[-1]) * u[b])), int(run_[-1]) - 1)
        j = int(np.searchsorted(run_, at, side="right"))
        tokens.append(int(by[j]))
        share.append(float(w[by[j]]) / float(run_[-1]))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(share, dtype=torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
        y = h * s["gamma"].double() / (h.square().sum(dim=1, keepdim=True) / h.shape[1] + s["eps"]).sqrt()
        r = None if s["residual"] is None else h
        if s["out"] == "bf16":
            return dict(y=y, residual=r)
        scales = y.abs().amax(dim=1) / 127.0
        y /= scales[:, None]
        return dict(values=y.round_().mul_(scales[:, None]), scales=scales, residual=r)
    if case["op"] == "linear8":
        y = torch.empty(case["rows"], case["n"], dtype=torch.float64, device=DEV)
        x = s["qx"].double()
        step = max(1, (1 << 28) // case["k"])
        for n0 in range(0, case["n"], step):
            part = slice(n0, min(case["n"], n0 + step))
            y[:, part] = torch.matmul(x, s["qw"][part].double().t())
        y *= s["sx"].double()[:, None] * s["sw"].double()[None, :]
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "rope":
        turn = torch.polar(torch.full_like(s["freqs"], s["scale"])[None, :].expand(case["rows"], -1).contiguous(),
                           s["positions"].double()[:, None] * s["freqs"][None, :])[:, None, :]
        rot, half = case["rot"], case["rot"] // 2
        got = []
        for x in (s["q"].double(), s["k"].double()):
            first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            got.append(y)
        return tuple(got)
    return _exact_sample(s)
