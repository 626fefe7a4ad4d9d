"""Cases, inputs and plain forms of the block-scaled 8-bit KV cache and of block-sparse decode
attention.

Operators (the field "op" of a case):

write    tokens quantised into a paged 8-bit cache as they are written (E4M3 codes, one
         power-of-two scale per block of tokens and KV head)
read     a range of cached tokens of every sequence read back as bf16 rows
attend   decode attention of one query token per sequence over that cache
bounds   the key bounds of cache blocks (int8 lower and upper bound of every key dim)
sparse   decode attention over the blocks that a score on the bounds selects for each query

Layouts, with bs tokens per block and 128 dims per head: tables int32 [B][MB] (-1 where unused),
8-bit pools uint8 [NB][n_kv][bs/8][8][8][16] (token slot s, dim i at [s/8][i/16][s%8][i%16]) with
scales fp32 [NB][n_kv], bf16 pools [NB][n_kv][bs/8][16][8][8], bounds int8 [NB][n_kv][2][128] with
scales fp32 [NB][n_kv].  A tile is one (block, KV head), numbered block * n_kv + head.
"""
import math
import random

import torch

own = False

D = 128
E4M3_MAX = 448.0
CACHE_MIN_EXP = -100  # smallest exponent of a block's, a bound's or a query's scale


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's append for a full serving batch: latency alone
        dict(name="write_step64", op="write", batch=64, lo=1, hi=1, past=9000, n_kv=8, bs=16,
             lens=11),
        # ragged prompts and prompt chunks behind cached tokens, written at admission
        dict(name="write_prompts", op="write", batch=24, lo=1, hi=4500, past=700, n_kv=8, bs=32,
             lens=12),
        # a few short ranges read back: a chunk's own past for a prompt pass
        dict(name="read_chunks", op="read", batch=5, lo=90, hi=700, past=800, n_kv=8, bs=16,
             lens=13),
        # a batch's whole caches read back (moved to a bf16 cache, or checked)
        dict(name="read_batch16", op="read", batch=16, lo=8192, hi=8192, past=0, n_kv=8, bs=16,
             lens=14),
        # one short conversation
        dict(name="attend_ctx512", op="attend", batch=1, lo=512, hi=512, n_q=32, n_kv=8, bs=16,
             lens=15),
        # the serving batch that the benchmark quotes
        dict(name="attend_batch16_ctx8192", op="attend", batch=16, lo=8192, hi=8192, n_q=32,
             n_kv=8, bs=16, lens=16),
        # a large ragged batch with eight query heads to a KV head
        dict(name="attend_ragged64_g8", op="attend", batch=64, lo=128, hi=32768, n_q=64, n_kv=8,
             bs=32, lens=17),
        # one long document: the context split over all SMs
        dict(name="attend_ctx131072", op="attend", batch=1, lo=131072, hi=131072, n_q=32, n_kv=8,
             bs=16, lens=18),
        # the bounds of newly admitted prompts, bf16 cache
        dict(name="bounds_prompts", op="bounds", batch=20, lo=200, hi=8192, past=0, n_kv=8, bs=16,
             fp8=False, lens=19),
        # the bounds after one decode step, 8-bit cache
        dict(name="bounds_step48", op="bounds", batch=48, lo=1, hi=1, past=6000, n_kv=8, bs=32,
             fp8=True, lens=20),
        # a quarter of each context read, bf16 cache
        dict(name="sparse_batch16_ctx8192", op="sparse", batch=16, lo=8192, hi=8192, n_q=32,
             n_kv=8, bs=16, width=128, first=1, last=4, fp8=False, lens=21),
        # one long document, 8-bit cache, a 32nd of the context read
        dict(name="sparse_ctx131072", op="sparse", batch=1, lo=131072, hi=131072, n_q=32, n_kv=8,
             bs=16, width=256, first=2, last=8, fp8=True, lens=22),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "bounds", "sparse"])
    n_kv = rng.choice([1, 2, 4, 8, 8, 10])
    G = rng.choice([1, 2, 4, 4, 8])
    bs = rng.choice([16, 32])
    c = dict(op=op, n_kv=n_kv, bs=bs, lens=rng.randrange(1 << 20))
    if op in ("write", "read"):
        hi = _log_int(rng, 1, 6000)
        c.update(batch=min(_log_int(rng, 1, 96), max(1, 100000 // hi)), hi=hi,
                 lo=rng.randint(1, hi), past=_log_int(rng, 1, 5000))
    elif op == "bounds":
        hi = _log_int(rng, 1, 9000)
        c.update(batch=min(_log_int(rng, 1, 96), max(1, 130000 // hi)), hi=hi,
                 lo=rng.randint(1, hi), past=_log_int(rng, 1, 5000), fp8=rng.random() < 0.5)
    else:
        hi = _log_int(rng, 20, 60000)
        c.update(batch=min(_log_int(rng, 1, 128), max(1, 400000 // hi)), hi=hi,
                 lo=rng.randint(1, hi), n_q=n_kv * G)
        if op == "sparse":
            first, last = rng.randint(0, 3), rng.randint(1, 8)
            c.update(width=first + last + _log_int(rng, 1, 500), first=first, last=last,
                     fp8=rng.random() < 0.5)
    return c


def _lens(case):
    """Tokens of every sequence: written or read, or the context of attention."""
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _past(case):
    """Tokens of every sequence before the written, read or updated ones."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, case["past"]) for _ in range(case["batch"])]


def _blocks(tokens, bs):
    return (tokens + bs - 1) // bs


def work(case):
    lens, n_kv, bs, op = _lens(case), case["n_kv"], case["bs"], case["op"]
    n = sum(lens)
    if op in ("write", "read"):
        touched = sum(_blocks(p + t, bs) - p // bs for p, t in zip(_past(case), lens))
        return {"bytes": 2 * n * n_kv * D * 3 + 2 * touched * n_kv * 4 + 8 * len(lens),
                "flops": 2 * n * n_kv * D * 2}
    if op == "bounds":
        past = _past(case)
        touched = sum(_blocks(p + t, bs) - p // bs for p, t in zip(past, lens))
        tokens = sum(p + t - p // bs * bs for p, t in zip(past, lens))
        return {"bytes": tokens * n_kv * D * (1 if case["fp8"] else 2) + touched * n_kv * 260,
                "flops": tokens * n_kv * D * 2}
    n_q = case["n_q"]
    nblk = [_blocks(t, bs) for t in lens]
    if op == "attend":
        return {"bytes": n * n_kv * 2 * D + sum(nblk) * (n_kv * 8 + 4) + len(lens) * n_q * D * 4,
                "flops": 4 * n * n_q * D}
    W = case["width"]
    scored = sum(x for x in nblk if x > W)
    tokens = sum(t if x <= W else (W - 1) * bs + t - (x - 1) * bs for t, x in zip(lens, nblk))
    kept = sum(min(x, W) for x in nblk)
    return {"bytes": scored * n_kv * 260 + tokens * n_kv * 2 * D * (1 if case["fp8"] else 2)
            + kept * n_kv * (16 if case["fp8"] else 8) + len(lens) * n_q * D * 4,
            "flops": scored * n_q * 4 * D + 4 * tokens * n_q * D}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _randn_bf16(shape, gen, spread=None):
    """Normal values in bf16, drawn in pieces; `spread`: a factor for each of the last dim."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for i in range(0, flat.shape[0], step):
        x = torch.randn(flat[i:i + step].shape, generator=gen, device="cuda")
        flat[i:i + step] = x if spread is None else x * spread
    return out


def _random_codes(shape, gen):
    """E4M3 codes of values spread as quantised rows are: normal, the largest near 448."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        x = torch.randn(flat[i:i + step].numel(), generator=gen, device="cuda")
        x = x.mul_(110.0).clamp_(-E4M3_MAX, E4M3_MAX)
        flat[i:i + step] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _random_scales(shape, gen):
    """Powers of two about 1/128, most blocks alike and a few of small or large values."""
    e = torch.randn(shape, generator=gen, device="cuda").mul_(0.8).round_().clamp_(-4, 4)
    return torch.exp2(e - 7)


def _tables(nblk, spare, seed):
    """Tables over a random permutation of the pool's blocks, and the number of blocks."""
    total = sum(nblk)
    NB = total + max(1, total // 20) + spare
    perm = torch.randperm(NB, generator=torch.Generator().manual_seed(seed * 31 + 5))
    first = torch.tensor([0] + nblk).cumsum(0)
    j = torch.arange(max(nblk))
    at = (first[:-1, None] + j).clamp(max=NB - 1)
    t = torch.where(j < torch.tensor(nblk)[:, None], perm[at], torch.tensor(-1))
    return t.to(torch.int32).cuda(), NB


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _spoil(pool, tables, lens, bs, value):
    """Slots behind every context hold `value` (never to be read as a token)."""
    ctx = torch.tensor(lens)
    last = tables.cpu()[torch.arange(len(lens)), (ctx - 1) // bs]
    b, s = torch.nonzero(torch.arange(bs)[None, :] > ((ctx - 1) % bs)[:, None], as_tuple=True)
    if b.numel():
        pool[last[b].cuda().long(), :, (s // 8).cuda(), :, (s % 8).cuda()] = value


def prepare(case, seed):
    op, n_kv, bs, B = case["op"], case["n_kv"], case["bs"], case["batch"]
    g, lens = _gen(seed), _lens(case)
    s = {"op": op, "n_kv": n_kv, "bs": bs, "batch": B, "scale": D ** -0.5}
    if op in ("write", "read", "bounds"):
        past = _past(case)
        s["tables"], NB = _tables([_blocks(p + t, bs) for p, t in zip(past, lens)], 0, seed)
        s["positions"], s["most"] = _int32(past), max(lens)
        if op != "bounds":
            starts = [0]
            for t in lens:
                starts.append(starts[-1] + t)
            s["starts"], s["tokens"] = _int32(starts), starts[-1]
    else:
        s["tables"], NB = _tables([_blocks(t, bs) for t in lens], 0, seed)
    s["num_blocks"] = NB
    spread = torch.exp(0.4 * torch.randn(D, generator=g, device="cuda"))
    shape8 = (NB, n_kv, bs // 8, D // 16, 8, 16)
    if op == "write":
        s["k_new"] = _randn_bf16((s["tokens"], n_kv, D), g, spread)
        s["v_new"] = _randn_bf16((s["tokens"], n_kv, D), g)
    if op in ("write", "read", "attend") or case.get("fp8"):
        s["k"], s["v"] = _random_codes(shape8, g), _random_codes(shape8, g)
        s["k_scales"], s["v_scales"] = _random_scales((NB, n_kv), g), _random_scales((NB, n_kv), g)
    elif op in ("bounds", "sparse"):
        shape = (NB, n_kv, bs // 8, D // 8, 8, 8)
        s["k"] = _randn_bf16(shape, g)
        s["v"] = _randn_bf16(shape, g) if op == "sparse" else None
        s["k_scales"] = s["v_scales"] = None
    if op == "read":
        s["k_rows"] = torch.empty((s["tokens"], n_kv, D), dtype=torch.bfloat16, device="cuda")
        s["v_rows"] = torch.empty_like(s["k_rows"])
    if op == "bounds":
        ctx = [p + t for p, t in zip(past, lens)]
        s["ctx"] = _int32(ctx)
        _spoil(s["k"], s["tables"], ctx, bs, 0x7F if case["fp8"] else float("nan"))
        s["bounds"] = torch.randint(-127, 128, (NB, n_kv, 2, D), generator=g, device="cuda",
                                    dtype=torch.int8)
        s["bound_scales"] = _random_scales((NB, n_kv), g)
    if op in ("attend", "sparse"):
        n_q = case["n_q"]
        s["q"] = _randn_bf16((B, n_q, D), g, spread)
        s["ctx"] = _int32(lens)
        s["out"] = torch.empty_like(s["q"])
        fp8 = op == "attend" or case["fp8"]
        for pool in (s["k"], s["v"]):
            _spoil(pool, s["tables"], lens, bs, 0x7F if fp8 else float("nan"))
        # the scratch that a serving loop keeps: zero-filled once
        s["workspace"] = torch.zeros(8192 + 8 * B * n_kv + (B * n_kv + 2048) * (n_q // n_kv) * 560,
                                     dtype=torch.uint8, device="cuda")
    if op == "sparse":
        W = case["width"]
        s["width"], s["first"], s["last"] = W, case["first"], case["last"]
        lo = torch.randint(-120, 40, (NB, n_kv, D), generator=g, device="cuda")
        hi = torch.minimum(lo + torch.randint(10, 120, lo.shape, generator=g, device="cuda"),
                           torch.tensor(127, device="cuda"))
        s["bounds"] = torch.stack([lo, hi], 2).to(torch.int8)
        s["bound_scales"] = torch.exp2(
            torch.randint(-6, -3, (NB, n_kv), generator=g, device="cuda").float())
        s["tiles"] = torch.empty((B, n_kv, W), dtype=torch.int32, device="cuda")
        s["tile_tokens"] = torch.empty((B, n_kv), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _pow2_at_least(amax, top):
    """The smallest power of two p (2^-100 at least) with amax <= top * p."""
    m, e = torch.frexp(amax / top)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, CACHE_MIN_EXP).clamp(min=CACHE_MIN_EXP)
    return torch.exp2(e.float())


def _token_places(s):
    """Sequence, block and slot of every packed token."""
    n = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), n, right=True)
    p = s["positions"].long()[b] + n - s["starts"].long()[b]
    return s["tables"].long()[b, p // s["bs"]], p % s["bs"]


def _write_plain(s, new, codes, scales):
    bs, n_kv = s["bs"], s["n_kv"]
    blk, slot = _token_places(s)
    x = new.float()
    need = torch.zeros_like(scales).index_reduce_(0, blk, x.abs().amax(-1), "amax")
    need = _pow2_at_least(need, E4M3_MAX)
    # the block that a sequence's first new token falls into may hold earlier tokens
    p0 = s["positions"].long()
    some = s["starts"][1:] > s["starts"][:-1]
    b0 = s["tables"].long()[torch.arange(s["batch"], device="cuda"), p0 // bs]
    begun = torch.zeros_like(scales, dtype=torch.bool)
    begun[b0] = (some & (p0 % bs > 0))[:, None]
    written = torch.zeros_like(begun)
    written[blk] = True
    grown = torch.where(begun, torch.maximum(scales, need), need)
    grown = torch.where(written, grown, scales)
    old = codes[b0].view(torch.float8_e4m3fn).float()
    kept = (old * (scales[b0] / grown[b0])[:, :, None, None, None, None]).to(torch.float8_e4m3fn)
    at = torch.arange(bs, device="cuda").view(bs // 8, 1, 8, 1)
    early = (at < (p0 % bs)[:, None, None, None, None]) & some[:, None, None, None, None]
    codes[b0] = torch.where(early[:, None], kept.view(torch.uint8), codes[b0])
    y = (x / grown[blk][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[blk, :, slot // 8, :, slot % 8, :] = y.view(-1, n_kv, D // 16, 16)
    scales.copy_(grown)


def _read_plain(s, codes, scales):
    blk, slot = _token_places(s)
    x = codes[blk, :, slot // 8, :, slot % 8, :].view(torch.float8_e4m3fn).float()
    return (x.flatten(2) * scales[blk][:, :, None]).to(torch.bfloat16)


def _tile_rows(pool, scales, tiles):
    """fp32 token rows [..., tiles * bs, 128] of the given tiles (-1: tile 0, to be masked)."""
    t = tiles.clamp(min=0).long()
    x = pool.flatten(0, 1)[t]
    if scales is None:
        x = x.float()
    else:
        x = x.view(torch.float8_e4m3fn).float()
    x = x.transpose(-2, -3).flatten(-2)  # [..., tile, bs/8, 8, 128]
    x = x.flatten(-3, -2)
    if scales is not None:
        x = x * scales.flatten()[t][..., None, None]
    return x.flatten(-3, -2)


def _attend_plain(s, tiles, tokens):
    """Softmax attention of every query head over its KV head's tiles, [B][n_kv][tiles]."""
    k = _tile_rows(s["k"], s["k_scales"], tiles)
    there = torch.arange(k.shape[2], device="cuda") < tokens[:, :, None]
    q = s["q"].float().view(s["batch"], s["n_kv"], -1, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    x = x.masked_fill(~there[:, :, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _tile_rows(s["v"], s["v_scales"], tiles)
    v = v.masked_fill_(~there[..., None], 0.0)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.to(torch.bfloat16).view(s["q"].shape)


def _all_tiles(s):
    head = torch.arange(s["n_kv"], device="cuda")
    t = s["tables"][:, None, :] * s["n_kv"] + head[:, None]
    return torch.where(s["tables"][:, None, :] < 0, -1, t)


def _bounds_plain(s):
    bs, p0 = s["bs"], s["positions"].long()
    first = p0 // bs
    j = first[:, None] + torch.arange((s["most"] + bs - 2) // bs + 1, device="cuda")
    b, i = torch.nonzero(j * bs < s["ctx"][:, None], as_tuple=True)
    j = j[b, i]
    blk = s["tables"].long()[b, j]
    tiles = blk[:, None] * s["n_kv"] + torch.arange(s["n_kv"], device="cuda")
    x = _tile_rows(s["k"], s["k_scales"], tiles[..., None])  # [blocks][n_kv][bs][128]
    there = torch.arange(bs, device="cuda") < (s["ctx"][b] - j * bs)[:, None]
    there = there[:, None, :, None]
    lo = x.masked_fill(~there, float("inf")).amin(2)
    hi = x.masked_fill(~there, float("-inf")).amax(2)
    p = _pow2_at_least(torch.maximum(lo.abs(), hi.abs()).amax(-1), 127.0)
    both = torch.stack([torch.floor(lo / p[..., None]), torch.ceil(hi / p[..., None])], 2)
    s["bounds"][blk] = both.to(torch.int8)
    s["bound_scales"][blk] = p


def _select_plain(s):
    """Tiles [B][n_kv][W] and tokens [B][n_kv] of the selected blocks.  The scores are exact
    (whole numbers below 2^24 times powers of two), so ties are real and go to the lowest."""
    bs, n_kv, W = s["bs"], s["n_kv"], s["width"]
    nblk = (s["ctx"].long() + bs - 1) // bs
    blk = s["tables"].long().clamp(min=0)
    j = torch.arange(blk.shape[1], device="cuda")
    q = s["q"].float().view(s["batch"], n_kv, -1, D)
    f = _pow2_at_least(q.abs().amax(-1, keepdim=True), 127.0)
    q = torch.round(q / f)
    bounds = s["bounds"][blk].float().permute(0, 2, 3, 4, 1)  # [B][n_kv][2][128][J]
    x = torch.matmul(q.clamp(min=0), bounds[:, :, 1]) + torch.matmul(q.clamp(max=0),
                                                                     bounds[:, :, 0])
    x = (x * f).amax(2) * s["bound_scales"][blk].transpose(1, 2)
    kept = (j < s["first"]) | (j >= (nblk - s["last"])[:, None])
    x = x.masked_fill(kept[:, None], float("inf"))
    x = x.masked_fill((j >= nblk[:, None])[:, None], float("-inf"))
    top = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :W]
    top = torch.sort(torch.where(top < nblk[:, None, None], top, 1 << 30), dim=-1).values
    head = torch.arange(n_kv, device="cuda")[:, None]
    tile = blk.gather(1, top.clamp(max=blk.shape[1] - 1).flatten(1)).view(top.shape) * n_kv + head
    tiles = torch.full((s["batch"], n_kv, W), -1, dtype=torch.int32, device="cuda")
    tiles[..., :top.shape[-1]] = torch.where(top < (1 << 30), tile, -1)
    tail = s["ctx"].long() - (nblk - 1) * bs
    tokens = ((nblk.clamp(max=W) - 1) * bs + tail)[:, None].expand(-1, n_kv)
    return tiles, tokens.to(torch.int32).contiguous()


def run(s):
    op = s["op"]
    if own:
        import paged_gqa_decode_kv_gb300 as pgd

        if op == "write":
            pgd.kv_append_fp8b(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scales"],
                               s["v_scales"], s["tables"], s["positions"],
                               token_starts=s["starts"], max_tokens=s["most"])
        elif op == "read":
            pgd.kv_read_fp8b(s["k_rows"], s["v_rows"], s["k"], s["v"], s["k_scales"],
                             s["v_scales"], s["tables"], s["positions"],
                             token_starts=s["starts"], max_tokens=s["most"])
        elif op == "attend":
            pgd.paged_decode_attention_fp8b(s["out"], s["q"], s["k"], s["v"], s["k_scales"],
                                            s["v_scales"], s["tables"], s["ctx"], s["scale"],
                                            workspace=s["workspace"])
        elif op == "bounds":
            pgd.block_bounds(s["bounds"], s["bound_scales"], s["k"], s["tables"], s["ctx"],
                             positions=s["positions"], max_tokens=s["most"],
                             k_scales=s["k_scales"])
        else:
            pgd.sparse_decode_attention(s["out"], s["q"], s["k"], s["v"], s["bounds"],
                                        s["bound_scales"], s["tables"], s["ctx"], s["tiles"],
                                        s["tile_tokens"], s["first"], s["last"], s["scale"],
                                        k_scales=s["k_scales"], v_scales=s["v_scales"],
                                        workspace=s["workspace"])
    elif op == "write":
        _write_plain(s, s["k_new"], s["k"], s["k_scales"])
        _write_plain(s, s["v_new"], s["v"], s["v_scales"])
    elif op == "read":
        s["k_rows"].copy_(_read_plain(s, s["k"], s["k_scales"]))
        s["v_rows"].copy_(_read_plain(s, s["v"], s["v_scales"]))
    elif op == "attend":
        tokens = s["ctx"][:, None].expand(-1, s["n_kv"])
        s["out"].copy_(_attend_plain(s, _all_tiles(s), tokens))
    elif op == "bounds":
        _bounds_plain(s)
    else:
        tiles, tokens = _select_plain(s)
        s["tiles"].copy_(tiles)
        s["tile_tokens"].copy_(tokens)
        s["out"].copy_(_attend_plain(s, tiles, tokens))
    if op == "write":
        return {"k": s["k"].view(torch.float8_e4m3fn), "k_scales": s["k_scales"],
                "v": s["v"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"]}
    if op == "read":
        return {"k": s["k_rows"], "v": s["v_rows"]}
    if op == "attend":
        return {"out": s["out"]}
    if op == "bounds":
        return {"bounds": s["bounds"], "scales": s["bound_scales"]}
    return {"out": s["out"], "tiles": s["tiles"], "tokens": s["tile_tokens"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3_values():
    """The value of every E4M3 code, from its bits: sign, four of exponent (bias 7), three."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if (c & 127) == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _to_e4m3(x):
    """The nearest E4M3 value, ties to even, at most 448 in size."""
    a = x.abs().clamp(min=1e-300)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3)
    up = torch.exp2((torch.floor(torch.log2(a)) + 1).clamp(min=-6.0) - 3)
    step = torch.where(a >= step * 16, up, step)  # where log2 rounded down over a power of two
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _rows64(pool, scales, table, ctx, bs, head):
    """Rows [ctx][128] of one sequence and KV head, in 64 bits."""
    n = _blocks(ctx, bs)
    x = pool[table[:n].long(), head]
    if scales is None:
        x = x.double()
    else:
        x = _e4m3_values()[x.long()] * scales[table[:n].long(), head].double().view(-1, 1, 1, 1, 1)
    return x.permute(0, 1, 3, 2, 4).reshape(n * bs, D)[:ctx]


def _least_pow2(amax, top):
    e = CACHE_MIN_EXP
    if amax > 0:
        e = max(e, math.ceil(math.log2(amax / top) - 1e-9))
        while amax > top * 2.0 ** e:
            e += 1
        while e > CACHE_MIN_EXP and amax <= top * 2.0 ** (e - 1):
            e -= 1
    return 2.0 ** e


def _exact_write(s, case, new, codes, scales):
    bs, values, sc = s["bs"], _e4m3_values(), scales.double()
    rows = values[codes.long()].permute(0, 1, 2, 4, 3, 5).reshape(*codes.shape[:2], bs, D)
    start = 0
    for b, (p, t) in enumerate(zip(_past(case), _lens(case))):
        x = new[start:start + t].double()
        start += t
        for j in range(p // bs, _blocks(p + t, bs)):
            blk = int(s["tables"][b, j])
            lo, hi = max(p, j * bs), min(p + t, (j + 1) * bs)
            y, slot = x[lo - p:hi - p], lo - j * bs
            tops = y.abs().amax((0, 2)).tolist()
            olds = sc[blk].tolist()
            p2 = [max(_least_pow2(a, E4M3_MAX), o if slot else 0.0) for a, o in zip(tops, olds)]
            p2 = torch.tensor(p2, dtype=torch.float64, device="cuda")
            if slot:
                rows[blk, :, :slot] = _to_e4m3(rows[blk, :, :slot] * (sc[blk] / p2)[:, None, None])
            rows[blk, :, slot:slot + hi - lo] = _to_e4m3(y.transpose(0, 1) / p2[:, None, None])
            sc[blk] = p2
    rows = rows.view(*codes.shape[:3], 8, D // 16, 16).permute(0, 1, 2, 4, 3, 5)
    return rows.contiguous(), sc


def exact(case, seed):
    s, op, bs, n_kv = prepare(case, seed), case["op"], case["bs"], case["n_kv"]
    lens = _lens(case)
    if op == "write":
        if sum(_blocks(t, bs) + 1 for t in lens) > 6000:
            return None  # one block after another: too long
        k, ks = _exact_write(s, case, s["k_new"], s["k"], s["k_scales"])
        v, vs = _exact_write(s, case, s["v_new"], s["v"], s["v_scales"])
        return {"k": k, "k_scales": ks, "v": v, "v_scales": vs}
    if op == "read":
        got = {}
        for name in ("k", "v"):
            got[name] = torch.empty((s["tokens"], n_kv, D), dtype=torch.float64, device="cuda")
            start = 0
            for b, (p, t) in enumerate(zip(_past(case), lens)):
                for h in range(n_kv):
                    rows = _rows64(s[name], s[name + "_scales"], s["tables"][b], p + t, bs, h)
                    got[name][start:start + t, h] = rows[p:]
                start += t
        return got
    if op == "bounds":
        scales = s["bound_scales"].double()
        for b, (p, t) in enumerate(zip(_past(case), lens)):
            at = s["tables"][b, p // bs:_blocks(p + t, bs)].long()
            for h in range(n_kv):
                x = _rows64(s["k"], s["k_scales"], s["tables"][b], p + t, bs, h)[p // bs * bs:]
                x = torch.nn.functional.pad(x.abs().amax(1), (0, len(at) * bs - len(x)))
                x = x.view(len(at), bs).amax(1)
                e = torch.ceil(torch.log2(x / 127.0) - 1e-9)
                e = torch.where(x > 127.0 * torch.exp2(e), e + 1, e)
                scales[at, h] = torch.exp2(e.clamp(min=CACHE_MIN_EXP))
        return {"bounds": None, "scales": scales}
    n_q = case["n_q"]
    G, out = n_q // n_kv, torch.empty((case["batch"], n_q, D), dtype=torch.float64, device="cuda")
    for b, t in enumerate(lens):
        n = _blocks(t, bs)
        for h in range(n_kv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            k = _rows64(s["k"], s["k_scales"], s["tables"][b], t, bs, h)
            v = _rows64(s["v"], s["v_scales"], s["tables"][b], t, bs, h)
            if op == "sparse" and n > s["width"]:
                at = s["tables"][b, :n].long()
                lo, hi = s["bounds"][at, h].double().unbind(1)
                x = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
                for r in q:
                    f = _least_pow2(float(r.abs().max()), 127.0)
                    r = torch.round(r / f)
                    dot = torch.where(r > 0, r * hi, r * lo).sum(1)
                    x = torch.maximum(x, dot * f)
                x = x * s["bound_scales"][at, h].double()
                x[:s["first"]] = math.inf
                x[n - s["last"]:] = math.inf
                chosen = torch.argsort(x, descending=True, stable=True)[:s["width"]].sort().values
                at = (chosen[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
                at = at[at < t]
                k, v = k[at], v[at]
            p = torch.softmax(q @ k.T * s["scale"], -1)
            out[b, h * G:(h + 1) * G] = p @ v
    return {"out": out} if op == "attend" else {"out": out, "tiles": None, "tokens": None}
