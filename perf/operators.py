"""The operators of a decoding step, as cases that can be timed and checked: a linear layer on
few rows with 4-bit weights and 16-bit activations, the block tables and slot maps of a paged
cache built from request lengths, the append to a cache held in 8 bits with a scale for each
block of tokens and head, and the attention that reads it.

``run`` computes a case in plain torch operations (``own`` false) or through the framework's
entry points (``own`` true); ``exact`` computes it in 64 bits from the definitions.

Definitions (bs tokens to a block, G = K / 64 groups, codes c in [-127, 127] stored as c + 128):

  linear     Y[m, n] = sum_k X^[m, k] q[n, k] s[k / 64, n] + sum_j (X^ L1)[m, j] L2[j, n]
             + bias[n],  X^ = fl32(X inv_lambda)
  plan       request b with ctx_b tokens cached and new_b to come needs
             ceil((ctx_b + new_b) / bs) - ceil(ctx_b / bs) more blocks; they come off the end of
             the free list in the requests' order. A request whose tokens do not fit its table
             row gets status 2 and one whose blocks the free list no longer holds status 1;
             either keeps its table and length, and its slots are -1.
  append     per block and head: s = max(s_old, fl32(amax / 127)) (s_old = 0 for a block whose
             first token is among the new ones), old codes rne(c fl32(s_old / s)) where s grew,
             new codes clamp(rne(fl32(x / s)), -127, 127); 0 where s = 0. Values read back are
             bf16(fl32(c s)).
  attention  out[i, h] = softmax_t(sm_scale q[i, h] . K[t, h']) V[t, h'], h' = h kv_heads / heads,
             over the tokens t < seq_len, and with ``causal`` t <= seq_len - new + i for row i of
             the request's new rows; 0 for a row with no token.
"""
import math

import torch

own = False

GROUP = 64
DEV = "cuda"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through a square projection with the low-rank branch and a bias
        dict(name="linear_1x4096x4096_r32", op="linear", rows=1, k=4096, n=4096, rank=32, bias=True, out="bf16"),
        # a small batch of decoding requests through an FFN up-projection
        dict(name="linear_8x4096x12288_r32", op="linear", rows=8, k=4096, n=12288, rank=32, bias=False, out="bf16"),
        # a batch, or several draft tokens of a few requests, through an FFN down-projection,
        # with an adapter joined to the branch, accumulated further in fp32
        dict(name="linear_24x12288x4096_r48_f32", op="linear", rows=24, k=12288, n=4096, rank=48, bias=True, out="fp32"),
        # one token through a vocabulary projection, weights only
        dict(name="linear_1x4096x131072", op="linear", rows=1, k=4096, n=131072, rank=0, bias=False, out="bf16"),
        # a handful of requests, one new token each: the smallest call of a serving step
        dict(name="plan_8_decode", op="plan", requests=8, max_ctx=4096, rows=8, block=16, short=False),
        # a large batch that mixes prompts and decoding, against a free list that runs out
        dict(name="plan_1000_mixed", op="plan", requests=1000, max_ctx=32768, rows=65536, block=64, short=True),
        # one new token for each of a batch of requests, blocks partly filled
        dict(name="append_64_decode", op="append", requests=64, max_ctx=8192, rows=64, block=16, heads=8, dim=128),
        # a few ragged prompts written to the cache
        dict(name="append_6_prompts", op="append", requests=6, max_ctx=100, rows=20000, block=64, heads=8, dim=128),
        # a single request decoding over the repository's cache shape
        dict(name="attention_1x10240_32h", op="attention", requests=1, max_ctx=10240, new=1, heads=32, kv_heads=32, dim=128, block=32, causal=False),
        # a batch of ragged requests decoding, four query heads to a cached head
        dict(name="attention_64x8192_gqa4", op="attention", requests=64, max_ctx=8192, new=1, heads=32, kv_heads=8, dim=128, block=16, causal=True),
        # a few draft tokens checked over a long context
        dict(name="attention_2x131071_draft", op="attention", requests=2, max_ctx=131071, new=5, heads=32, kv_heads=4, dim=128, block=64, causal=True),
        # prompts continued in chunks over what is cached already
        dict(name="attention_4x4096_chunk", op="attention", requests=4, max_ctx=4096, new=1000, heads=24, kv_heads=8, dim=64, block=16, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "plan", "append", "attention", "attention"))
    if op == "linear":
        return dict(op=op, rows=_log(rng, 1, 64), k=64 * _log(rng, 1, 192), n=_log(rng, 1, 24000),
                    rank=16 * rng.randint(0, 8), bias=rng.random() < 0.5,
                    out=rng.choice(("bf16", "bf16", "fp32")))
    if op == "plan":
        b = _log(rng, 1, 1000)
        return dict(op=op, requests=b, max_ctx=_log(rng, 1, 32768), rows=_log(rng, b, 65536),
                    block=rng.choice((16, 32, 64, 128)), short=rng.random() < 0.3)
    if op == "append":
        b = _log(rng, 1, 200)
        return dict(op=op, requests=b, max_ctx=_log(rng, 1, 4096), rows=_log(rng, b, 16000),
                    block=rng.choice((16, 32, 64, 128)), heads=rng.choice((1, 2, 4, 8, 12)),
                    dim=rng.choice((64, 128)))
    kv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 6, 8, 16))
    b = _log(rng, 1, 64)
    new = rng.choice((1, 1, 1, _log(rng, 2, 16), _log(rng, 17, 700)))
    # rows x context bounded, so that no draw costs more than the listed cases
    ctx = _log(rng, 1, max(2, min(131072, (1 << 19) // b // kv * 2, (1 << 23) // (b * new))))
    return dict(op=op, requests=b, max_ctx=ctx, new=new, heads=kv * group, kv_heads=kv,
                dim=rng.choice((64, 128)), block=rng.choice((16, 32, 64, 128)),
                causal=rng.random() < 0.7)


# ----------------------------------------------------------------------------------- inputs
def _lens(g, n, total_max, low=0.25):
    """n ragged lengths in [low * total_max, total_max], the first of them total_max."""
    x = (total_max * (low + (1.0 - low) * _rand(g, n))).to(torch.int32)
    x[0] = total_max
    return x


def _split(g, n, rows):
    """n ragged counts >= 1 that sum to rows or a few less (n <= rows); all 1 when n = rows."""
    if rows <= n:
        return torch.ones(n, dtype=torch.int32, device=DEV)
    w = _rand(g, n) ** 3 + 0.01
    x = 1 + torch.floor((rows - n) * w / w.sum() * 0.999).to(torch.int32)
    return x


def _blocks_of(lens, bs):
    return (lens + bs - 1) // bs


def _tables(g, lens, bs, width, num_blocks):
    """[n, width] block ids, -1 past each request's blocks, from a random order of the pool."""
    need = _blocks_of(lens, bs).to(torch.int64)
    start = torch.cumsum(need, 0) - need
    perm = torch.randperm(num_blocks, generator=g, device=DEV)
    j = torch.arange(width, device=DEV)[None, :]
    at = (start[:, None] + j).clamp(max=num_blocks - 1)
    return torch.where(j < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32)


def _codes(g, *shape):
    """Codes c + 128 of values whose block maximum maps to 127: near normal, std about 36."""
    c = torch.empty(*shape, device=DEV, dtype=torch.float32).normal_(0.0, 36.0, generator=g)
    return c.round_().clamp_(-127, 127).add_(128).to(torch.uint8)


def _prepare_linear(case, g):
    M, K, N, r = case["rows"], case["k"], case["n"], case["rank"]
    hot = _rand(g, K) < 0.01                     # outlier channels, moved into the weights
    x = _randn(g, M, K) * torch.where(hot, 20.0, 1.0)
    inv = torch.where(hot, 0.08, 0.9) * torch.exp(0.2 * _randn(g, K))
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // K)
    for n0 in range(0, N, step):                 # residual codes: near normal, group maximum at 7
        c = (_randn(g, min(step, N - n0), K) * 2.4).round_().clamp_(-8, 7).to(torch.int16) & 15
        wq[n0:n0 + step] = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)
    ws = ((0.4 + 0.1 * _rand(g, K // GROUP, N)) / math.sqrt(K)).to(torch.float16)
    s = dict(x=x.to(torch.bfloat16), inv_lambda=inv.float().contiguous(), wq=wq, w_scales=ws,
             l1p=(_randn(g, r, K) / math.sqrt(K)).to(torch.bfloat16),
             l2p=(_randn(g, N, r) / math.sqrt(max(r, 1))).to(torch.bfloat16),
             bias=_randn(g, N).to(torch.bfloat16) if case["bias"] else None)
    if own:
        from bit_post_quantized_amd import layer, serve
        s["linear"] = serve.DecodeLinear(layer.PackedWeights(
            K=K, N=N, rank=r, inv_lambda=s["inv_lambda"], L1p=s["l1p"], L2p=s["l2p"], wq=wq,
            w_scales=ws, bias=s["bias"]))
    return s


def _prepare_plan(case, g):
    B, bs, rows = case["requests"], case["block"], case["rows"]
    ctx = _lens(g, B, case["max_ctx"], low=0.0)
    new = _split(g, B, rows)
    width = (case["max_ctx"] + rows + bs - 1) // bs if rows <= 4 * B else case["max_ctx"] // bs + 1 + rows // (2 * bs)
    need = int((_blocks_of(ctx + new, bs) - _blocks_of(ctx, bs)).sum())
    held = int(_blocks_of(ctx, bs).sum())
    free = max(1, int(need * (0.7 if case["short"] else 1.2)))
    num = held + free + 8
    ids = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    blocks = _blocks_of(ctx, bs).to(torch.int64)
    j = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(blocks, 0) - blocks)[:, None] + j
    tables = torch.where(j < blocks[:, None], ids[at.clamp(max=num - 1)], -1).to(torch.int32)
    s = dict(ctx=ctx, new=new, tables=tables.contiguous(), free=ids[held:].contiguous(),
             free_count=torch.tensor([free], dtype=torch.int32, device=DEV), rows=rows, block=bs)
    if own:
        from bit_post_quantized_amd import serve
        s["planner"] = serve.BlockPlanner(s["tables"], s["free"], bs, rows)
    return s


def _prepare_append(case, g):
    B, bs, rows, H, D = case["requests"], case["block"], case["rows"], case["heads"], case["dim"]
    ctx, new = _lens(g, B, case["max_ctx"]), _split(g, B, rows)
    total = int(new.sum())
    first = ctx // bs                                    # first block that the new tokens touch
    touched = (_blocks_of(ctx + new, bs) - first).to(torch.int64)
    tb = int(touched.sum())
    num = tb + 16
    perm = torch.randperm(num, generator=g, device=DEV)
    base = torch.cumsum(touched, 0) - touched
    cu = torch.cumsum(new.to(torch.int64), 0)
    t = torch.arange(total, device=DEV)
    req = torch.searchsorted(cu, t, right=True)
    pos = ctx[req].to(torch.int64) + t - (cu - new)[req]
    slots = perm[base[req] + pos // bs - first[req]] * bs + pos % bs
    slots = torch.cat([slots, torch.full((rows - total,), -1, dtype=torch.int64, device=DEV)])
    # what is read back: every filled token of every touched block
    u = torch.arange(tb * bs, device=DEV)
    blk = u // bs
    breq = torch.searchsorted(torch.cumsum(touched, 0), blk, right=True)
    bpos = (first[breq].to(torch.int64) + blk - base[breq]) * bs + u % bs
    filled = bpos < (ctx + new)[breq]
    back = torch.full(((rows // bs + 2 * B) * bs,), -1, dtype=torch.int64, device=DEV)
    back[:tb * bs] = torch.where(filled, perm[blk] * bs + u % bs, -1)
    q = _randn(g, rows, (2 + 2) * H, D) * torch.exp(0.5 * _randn(g, 4 * H, 1))
    qkv = q.to(torch.bfloat16)                           # k and v are slices of a fused projection
    s = dict(k=qkv[:, 2 * H:3 * H], v=qkv[:, 3 * H:], slots=slots, back=back, block=bs,
             k_codes=_codes(g, num, H, bs, D), v_codes=_codes(g, num, H, D, bs),
             k_scale=0.03 * torch.exp(0.3 * _randn(g, num, H)),
             v_scale=0.03 * torch.exp(0.3 * _randn(g, num, H)),
             k_out=torch.zeros(back.numel(), H, D, dtype=torch.bfloat16, device=DEV),
             v_out=torch.zeros(back.numel(), H, D, dtype=torch.bfloat16, device=DEV))
    if own:
        from bit_post_quantized_amd import serve
        s["cache"] = serve.BlockCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s


def _rows_of(new, requests):
    """Ragged counts of new rows, new the largest, and the rows of the batch: with more than one
    to a request two rows stand behind the last sequence, as in a batch padded to a size."""
    n = [max(1, int(new * (0.3 + 0.7 * (i + 1) / requests))) for i in range(requests)]
    return n, sum(n) + (2 if new > 1 else 0)


def _prepare_attention(case, g):
    B, bs, H, D, new = case["requests"], case["block"], case["kv_heads"], case["dim"], case["new"]
    seq = _lens(g, B, case["max_ctx"])
    n, rows = _rows_of(new, B)
    n = torch.tensor(n, dtype=torch.int32, device=DEV)[torch.randperm(B, generator=g, device=DEV)]
    if B > 2:
        seq[1] = 0                                       # a padded place of the batch
    seq = torch.where(seq > 0, torch.maximum(seq, n), seq)
    width = (max(case["max_ctx"], new) + bs - 1) // bs
    num = int(_blocks_of(seq, bs).sum()) + 8
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(n, 0)
    s = dict(q=_randn(g, rows, case["heads"], D).to(torch.bfloat16), cu=cu, seq=seq,
             tables=_tables(g, seq, bs, width, num), new=new, causal=case["causal"],
             k_codes=_codes(g, num, H, bs, D), v_codes=_codes(g, num, H, D, bs),
             k_scale=torch.exp(0.25 * _randn(g, num, H)) / 30.0,
             v_scale=torch.exp(0.25 * _randn(g, num, H)) / 30.0, sm_scale=1.0 / math.sqrt(D),
             out=torch.zeros(rows, case["heads"], D, dtype=torch.bfloat16, device=DEV))
    if own:
        from bit_post_quantized_amd import serve
        s["cache"] = serve.BlockCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = dict(linear=_prepare_linear, plan=_prepare_plan, append=_prepare_append,
                attention=_prepare_attention)[case["op"]]
    return dict(make(case, g), op=case["op"], out_dtype=case.get("out"))


# ------------------------------------------------------------------------------ plain forms
def _plain_linear(s):
    xh = s["x"].float() * s["inv_lambda"]
    wq = s["wq"]
    q = torch.stack((wq & 15, wq >> 4), dim=-1).reshape(wq.shape[0], -1).to(torch.int8)
    q = torch.where(q >= 8, q - 16, q).float()
    w = (q.view(q.shape[0], -1, GROUP) * s["w_scales"].float().t()[:, :, None]).view_as(q)
    y = xh @ w.t() + (xh @ s["l1p"].float().t()) @ s["l2p"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y if s["out_dtype"] == "fp32" else y.to(torch.bfloat16)


def _plain_plan(s):
    ctx, new, tables, bs = s["ctx"], s["new"], s["tables"], s["block"]
    width, rows = tables.shape[1], s["rows"]
    have, end = _blocks_of(ctx, bs), _blocks_of(ctx + new, bs)
    narrow = end > width
    need = torch.where(narrow, 0, end - have)
    incl = torch.cumsum(need, 0)
    dry = (incl > s["free_count"]) & (need > 0)
    status = torch.where(narrow, 2, torch.where(dry, 1, 0)).to(torch.int32)
    ok = status == 0
    taken = torch.where(ok, need, 0)
    left = (s["free_count"] - taken.sum()).to(torch.int32)
    j = torch.arange(width, device=DEV)[None, :]
    fresh = ok[:, None] & (j >= have[:, None]) & (j < end[:, None])
    at = s["free_count"] - 1 - ((incl - need)[:, None] + j - have[:, None])
    tables = torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1).long()], tables)
    s["tables"].copy_(tables)
    cu = torch.zeros(ctx.numel() + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(rows, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    live = req < ctx.numel()
    req = req.clamp(max=ctx.numel() - 1)
    pos = torch.where(live, ctx[req] + t - cu[req], 0).to(torch.int32)
    block = tables[req, (pos // bs).clamp(max=width - 1).long()].long()
    slots = torch.where(live & ok[req], block * bs + pos % bs, -1)
    return dict(tables=s["tables"], cu=cu, seq=torch.where(ok, ctx + new, ctx).to(torch.int32),
                positions=pos, slots=slots, status=status, free_count=left)


def _plain_store(x, slots, codes, scale, bs, transposed):
    """The append of one of K and V; returns nothing, the cache is written in place."""
    num, H = scale.shape
    live = slots >= 0
    block = torch.where(live, slots // bs, num)          # rows without a slot go to a spare block
    off = torch.where(live, slots % bs, 0)
    amax = x.float().abs().amax(dim=-1)                  # [T, H]
    top = torch.zeros(num + 1, H, device=DEV).scatter_reduce(
        0, block[:, None].expand(-1, H), amax, "amax")[:num]
    start = torch.full((num + 1,), bs, dtype=torch.int64, device=DEV).scatter_reduce(
        0, block, off, "amin")[:num]
    old = torch.where((start == 0)[:, None], 0.0, scale)
    # a tensor as divisor: torch divides by a Python number with a product by its reciprocal
    s = torch.where((start == bs)[:, None], scale,
                    torch.maximum(old, top / torch.full_like(top, 127.0)))
    grew = (s > old) & (start < bs)[:, None]
    ratio = torch.where(s > 0, old / s, 0.0)
    c = codes.float() - 128.0
    codes.copy_(torch.where(grew[:, :, None, None], torch.round(c * ratio[:, :, None, None]) + 128.0,
                            codes.float()))
    scale.copy_(s)
    st = s[block.clamp(max=num - 1)]                     # [T, H]
    q = torch.where(st[:, :, None] > 0, torch.round(x.float() / st[:, :, None]), 0.0).clamp(-127, 127) + 128.0
    b, o = torch.where(live, block, 0), off
    h = torch.arange(H, device=DEV)
    tok = codes.transpose(2, 3) if transposed else codes  # a view: tokens before channels
    first = live.to(torch.uint8).argmax()                # rows without a slot write its value again
    pick = torch.where(live, torch.arange(live.numel(), device=DEV), first)
    tok[b[pick][:, None], h[None, :], o[pick][:, None]] = q[pick].to(torch.uint8)


def _plain_load(slots, codes, scale, bs, transposed, out):
    live = slots >= 0
    b, o = torch.where(live, slots // bs, 0), torch.where(live, slots % bs, 0)
    h = torch.arange(scale.shape[1], device=DEV)
    tok = codes.transpose(2, 3) if transposed else codes
    v = (tok[b[:, None], h[None, :], o[:, None]].float() - 128.0) * scale[b][:, :, None]
    return torch.where(live[:, None, None], v.to(torch.bfloat16), out)


def _plain_append(s):
    _plain_store(s["k"], s["slots"], s["k_codes"], s["k_scale"], s["block"], False)
    _plain_store(s["v"], s["slots"], s["v_codes"], s["v_scale"], s["block"], True)
    return (_plain_load(s["back"], s["k_codes"], s["k_scale"], s["block"], False, s["k_out"]),
            _plain_load(s["back"], s["v_codes"], s["v_scale"], s["block"], True, s["v_out"]))


def _plain_attention(s):
    q, cu, seq, tables, n = s["q"], s["cu"].long(), s["seq"].long(), s["tables"], s["new"]
    B, W = tables.shape
    _, KV, bs, D = s["k_codes"].shape
    g = q.shape[1] // KV
    L = W * bs
    t = tables.clamp(min=0).long()
    k = (s["k_codes"][t].float() - 128.0) * s["k_scale"][t][..., None, None]   # [B, W, KV, bs, D]
    k = k.permute(0, 2, 1, 3, 4).reshape(B * KV, L, D)
    i = torch.arange(n, device=DEV)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                         # [B, n]
    qp = q[row].float().view(B, n, KV, g, D).permute(0, 2, 1, 3, 4).reshape(B * KV, n * g, D)
    p = torch.bmm(qp, k.transpose(1, 2).contiguous()).view(B, KV, n, g, L) * s["sm_scale"]
    del k
    last = (seq - count)[:, None] + i if s["causal"] else (seq - 1)[:, None].expand(B, n)
    seen = torch.arange(L, device=DEV) <= last[:, :, None]                      # [B, n, L]
    seen = (seen & (torch.arange(L, device=DEV) < seq[:, None, None]))[:, None, :, None, :]
    p = torch.where(seen, p, -math.inf)
    top = p.amax(dim=-1, keepdim=True)
    p = torch.exp(p - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    v = (s["v_codes"][t].float() - 128.0) * s["v_scale"][t][..., None, None]   # [B, W, KV, D, bs]
    v = v.permute(0, 2, 1, 4, 3).reshape(B * KV, L, D)
    o = torch.bmm(p.view(B * KV, n * g, L), v).view(B, KV, n, g, D).permute(0, 2, 1, 3, 4)
    o = o.reshape(B * n, KV * g, D).to(torch.bfloat16)
    r = torch.arange(q.shape[0], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True).clamp(max=B - 1)
    at = (b * n + r - cu[b]).clamp(max=B * n - 1)
    return torch.where((r < cu[-1])[:, None, None], o[at], s["out"])


def run(state):
    op = state["op"]
    if own:
        if op == "linear":
            return state["linear"](state["x"], out_dtype=torch.float32 if state["out_dtype"] == "fp32" else torch.bfloat16)
        if op == "plan":
            p = state["planner"].plan(state["ctx"], state["new"], state["free_count"])
            return dict(tables=state["tables"], cu=p.cu_rows, seq=p.seq_lens, positions=p.positions,
                        slots=p.slots, status=p.status, free_count=p.free_count)
        if op == "append":
            state["cache"].append(state["k"], state["v"], state["slots"])
            return state["cache"].read(state["back"], state["k_out"], state["v_out"])
        return state["cache"].attention(state["q"], state["tables"], state["seq"], state["cu"],
                                        state["new"], causal=state["causal"],
                                        sm_scale=state["sm_scale"], out=state["out"])
    return dict(linear=_plain_linear, plan=_plain_plan, append=_plain_append,
                attention=_plain_attention)[op](state)


# ----------------------------------------------------------------------------- work and exact
def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N, r = case["rows"], case["k"], case["n"], case["rank"]
        out = 4 if case["out"] == "fp32" else 2
        return dict(bytes=N * K // 2 + 2 * (K // GROUP) * N + 2 * r * (K + N) + 2 * M * K + 4 * K
                    + out * M * N + (2 * N if case["bias"] else 0),
                    flops=2 * M * K * N + 2 * M * r * (K + N))
    if op == "plan":
        B, rows, bs = case["requests"], case["rows"], case["block"]
        # lengths in and out; per row a position and a slot; a table entry read or written per block
        return dict(bytes=6 * 4 * B + 12 * rows + 8 * (rows // bs + B), flops=8 * rows)
    if op == "append":
        rows, H, D, B, bs = case["rows"], case["heads"], case["dim"], case["requests"], case["block"]
        blocks = rows // bs + B
        # K and V: values in, codes out; then each filled token's codes in and values out
        return dict(bytes=2 * H * (D * rows * (2 + 1) + (rows + B * bs // 2) * D * (1 + 2) + 8 * blocks),
                    flops=2 * H * D * rows * 6)
    B, L, n, H, KV, D = (case[x] for x in ("requests", "max_ctx", "new", "heads", "kv_heads", "dim"))
    mean = L if B == 1 else L * 0.625
    rows = sum(_rows_of(n, B)[0])
    return dict(bytes=2 * B * mean * KV * (D + 4.0 / case["block"]) + 4 * rows * H * D,
                flops=4 * rows * H * D * max(1.0, mean - (rows / B / 2 if case["causal"] else 0)))


def _exact_plan(s):
    ctx, new, tables = s["ctx"].tolist(), s["new"].tolist(), s["tables"].tolist()
    free, left, bs, width = s["free"].tolist(), int(s["free_count"]), s["block"], s["tables"].shape[1]
    stack, dry = free[:left], False
    cu, seq, pos, slots, status = [0], [], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        need = -(-(c + n) // bs) - -(-c // bs)
        if -(-(c + n) // bs) > width:
            st = 2
        else:
            dry = dry or need > len(stack)
            st = 1 if need > 0 and dry else 0
        if st == 0:
            for j in range(-(-c // bs), -(-(c + n) // bs)):
                tables[b][j] = stack.pop()
        status.append(st)
        seq.append(c + n if st == 0 else c)
        cu.append(cu[-1] + n)
        for p in range(c, c + n):
            pos.append(p)
            slots.append(tables[b][p // bs] * bs + p % bs if st == 0 else -1)
    pad = s["rows"] - len(pos)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(tables=i32(tables), cu=i32(cu), seq=i32(seq), positions=i32(pos + [0] * pad),
                slots=torch.tensor(slots + [-1] * pad, dtype=torch.int64), status=i32(status),
                free_count=i32([len(stack)]))


def _fl32(x):
    return x.to(torch.float32).to(torch.float64)


def _exact_append(s, name):
    """Block by block in 64 bits; a quotient rounded to 32 bits and then to whole numbers, as the
    definition says (64 bits are enough for the first rounding to be the correct one)."""
    bs = s["block"]
    x = s[name].double().cpu()
    codes = s[name + "_codes"].cpu().double() - 128.0
    if name == "v":
        codes = codes.transpose(2, 3)
    codes = codes.contiguous()
    scale = s[name + "_scale"].double().cpu()
    slots = s["slots"].cpu()
    live = (slots >= 0).nonzero().flatten()
    blocks = (slots[live] // bs)
    for b in torch.unique(blocks).tolist():
        rows = live[blocks == b]
        off = slots[rows] % bs
        new = x[rows]                                                   # [n, H, D]
        old = torch.zeros_like(scale[b]) if int(off.min()) == 0 else scale[b].clone()
        top = torch.maximum(old, _fl32(new.abs().amax(dim=(0, 2)) / 127.0))
        safe = torch.where(top > 0, top, 1.0)
        ratio = _fl32(old / safe)
        moved = torch.round(_fl32(codes[b] * ratio[:, None, None]))
        codes[b] = torch.where((top > old)[:, None, None], moved, codes[b])
        q = torch.round(_fl32(new / safe[None, :, None])).clamp(-127, 127)
        codes[b][:, off] = torch.where(top[None, :, None] > 0, q, 0.0).transpose(0, 1)
        scale[b] = top
    back = s["back"].cpu()
    got = (back >= 0)
    b, o = back.clamp(min=0) // bs, back.clamp(min=0) % bs
    h = torch.arange(scale.shape[1])
    v = _fl32(codes[b[:, None], h[None, :], o[:, None]] * scale[b][:, :, None])
    return torch.where(got[:, None, None], v, 0.0)


def _exact_attention(s):
    q, cu, seq = s["q"].double(), s["cu"].tolist(), s["seq"].tolist()
    _, KV, bs, D = s["k_codes"].shape
    g = q.shape[1] // KV
    out = torch.zeros_like(q)
    for b, length in enumerate(seq):
        rows = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        ids = s["tables"][b, :-(-length // bs)].long()
        for h in range(KV):
            k = ((s["k_codes"][ids, h].double() - 128.0) * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:length]
            v = ((s["v_codes"][ids, h].double() - 128.0) * s["v_scale"][ids, h].double()[:, None, None])
            v = v.transpose(1, 2).reshape(-1, D)[:length]
            if length == 0:
                continue
            w = torch.matmul(q[rows, h * g:(h + 1) * g].reshape(n * g, D), k.t()).view(n, g, length) * s["sm_scale"]
            if s["causal"]:
                far = torch.arange(length, device=DEV)[None, :] > torch.arange(length - n, length, device=DEV)[:, None]
                w = w.masked_fill(far[:, None, :], -math.inf)
            w = torch.softmax(w, dim=-1)
            out[rows, h * g:(h + 1) * g] = torch.matmul(w.view(n * g, length), v).view(n, g, D)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        xh = _fl32(s["x"].double() * s["inv_lambda"].double())
        y = torch.matmul(torch.matmul(xh, s["l1p"].double().t()), s["l2p"].double().t())
        step = max(1, (1 << 28) // case["k"])
        for n0 in range(0, case["n"], step):
            part = slice(n0, min(case["n"], n0 + step))
            b = s["wq"][part].to(torch.int32)
            c = torch.empty(b.shape[0], case["k"], dtype=torch.float64, device=DEV)
            c[:, 0::2], c[:, 1::2] = ((b & 15) ^ 8) - 8, ((b >> 4) ^ 8) - 8
            c *= s["w_scales"][:, part].double().t().repeat_interleave(GROUP, dim=1)
            y[:, part] += torch.matmul(xh, c.t())
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "plan":
        return _exact_plan(s)
    if op == "append":
        return _exact_append(s, "k"), _exact_append(s, "v")
    return _exact_attention(s)
