"""Cases, inputs and plain forms of the 4-bit KV cache and its attention, of rotary positions, and of
block tables grown and cut on the GPU.

Operators (the field "op" of a case):

tables   every request grows by its new tokens (blocks taken from a pool, the lowest free ids in
         row order; positions, token starts and slots of the new tokens), then is cut back to where
         it was, as after a verification that rejects them or an admission called off
rope     rotary positions on packed rows: rows to rows ("rows"), or q to rows and K, V into a paged
         bf16 cache ("append")
write    tokens quantised into a paged 4-bit cache (E2M1 codes, one E4M3 scale per token, head and
         16 dims), and the range that was written read back as bf16 rows
read     a range of cached tokens of every sequence read back as bf16 rows
attend   decode attention of one query token per sequence over the 4-bit cache

Layouts, with bs tokens per block and 128 dims per head: tables int32 [B][MB] (-1 where unused);
bf16 pools [NB][n_kv][bs/8][16][8][8] (slot s, dim i at [s/8][i/8][s%8][i%8]); 4-bit pools uint8
[NB][n_kv][bs/16][1152]: per 16 tokens 1024 bytes of codes, 128 of scales.  K: the codes of token t
at t * 64, two dims a byte (the even one low), its scale of dims 16 g .. at 1024 + t * 8 + g.  V: dim
i of token t at (i/64) * 512 + (i%8) * 64 + (t/4) * 16 + (i/8%8) * 2 + (t%4)/2, the even token low,
and the scale at 1024 + (t/4) * 32 + g * 4 + t%4.  A value is E2M1 * E4M3 * (the call's scale).
Block pools: refs int32 [NB], and free_bits int32 [NB/32 rounded up], bit id % 32 of word id / 32.
"""
import math
import random

import torch

own = False

D = 128
GROUP = 1152  # bytes of 16 tokens of a 4-bit tile
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one verification step of a full serving batch: a few drafted tokens each, latency alone
        dict(name="tables_step64", op="tables", batch=64, lo=1, hi=4, past=9000, bs=16, spare=30000,
             lens=11),
        # admission of many ragged prompts from a large, fragmented pool
        dict(name="tables_prompts", op="tables", batch=256, lo=1, hi=4500, past=700, bs=16,
             spare=200000, lens=12),
        # one decode step of a serving batch, rotated and appended
        dict(name="rope_step64", op="rope", mode="append", batch=64, lo=1, hi=1, past=9000, n_q=32,
             n_kv=8, d=128, first=0, rotary=128, pairs="half", bs=16, lens=13),
        # ragged prompts, q and k within one projection's output, half of each head rotated
        dict(name="rope_prompts", op="rope", mode="rows", batch=20, lo=200, hi=4500, past=1000000,
             n_q=32, n_kv=8, d=128, first=0, rotary=64, pairs="interleaved", bs=16, lens=14),
        # one decode step's append for a full serving batch: latency alone
        dict(name="write_step64", op="write", batch=64, lo=1, hi=1, past=9000, n_kv=8, bs=16,
             lens=15),
        # ragged prompts and prompt chunks behind cached tokens, written at admission
        dict(name="write_prompts", op="write", batch=24, lo=1, hi=4500, past=700, n_kv=8, bs=32,
             lens=16),
        # a few short ranges read back: a chunk's own past for a prompt pass
        dict(name="read_chunks", op="read", batch=5, lo=90, hi=700, past=800, n_kv=8, bs=16,
             lens=17),
        # a batch's whole caches read back (moved to a bf16 cache, or checked)
        dict(name="read_batch16", op="read", batch=16, lo=8192, hi=8192, past=0, n_kv=8, bs=16,
             lens=18),
        # one short conversation
        dict(name="attend_ctx512", op="attend", batch=1, lo=512, hi=512, n_q=32, n_kv=8, bs=16,
             lens=19),
        # the serving batch that the benchmark quotes
        dict(name="attend_batch16_ctx8192", op="attend", batch=16, lo=8192, hi=8192, n_q=32,
             n_kv=8, bs=16, lens=20),
        # a large ragged batch with eight query heads to a KV head
        dict(name="attend_ragged64_g8", op="attend", batch=64, lo=128, hi=32768, n_q=64, n_kv=8,
             bs=32, lens=21),
        # one long document: the context split over all SMs
        dict(name="attend_ctx131072", op="attend", batch=1, lo=131072, hi=131072, n_q=32, n_kv=8,
             bs=16, lens=22),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "write", "read", "attend", "attend"])
    n_kv = rng.choice([1, 2, 4, 8, 8, 10])
    G = rng.choice([1, 2, 4, 4, 8])
    bs = rng.choice([16, 32])
    c = dict(op=op, bs=bs, lens=rng.randrange(1 << 20))
    if op == "tables":
        hi = _log_int(rng, 1, 6000)
        c.update(batch=min(_log_int(rng, 1, 512), max(1, 550000 // hi)), hi=hi,
                 lo=rng.randint(0, hi), past=_log_int(rng, 1, 5000), spare=_log_int(rng, 1, 200000))
    elif op == "rope":
        hi = _log_int(rng, 1, 5000)
        mode = rng.choice(["rows", "append"])
        d, first, rotary = D, 0, rng.choice([16, 32, 64, 96, 128])
        if mode == "rows" and rng.random() < 0.5:
            d, first, rotary = rng.choice([(64, 0, 64), (576, 512, 64), (192, 128, 64),
                                           (256, 0, 64), (80, 0, 32)])
            if d == 576:
                n_kv, G = 1, rng.choice([16, 64, 128])
        cost = n_kv * (G + 1) * d
        c.update(mode=mode, batch=min(_log_int(rng, 1, 96), max(1, 200000000 // (hi * cost))),
                 hi=min(hi, 200000000 // cost), past=_log_int(rng, 1, 1000000), n_q=n_kv * G,
                 n_kv=n_kv, d=d, first=first, rotary=rotary,
                 pairs=rng.choice(["half", "interleaved"]))
        c.update(lo=rng.randint(1, c["hi"]))
    elif op in ("write", "read"):
        hi = _log_int(rng, 1, 6000)
        c.update(batch=min(_log_int(rng, 1, 96), max(1, 100000 // hi)), hi=hi, n_kv=n_kv,
                 lo=rng.randint(1, hi), past=_log_int(rng, 1, 5000))
    else:
        hi = _log_int(rng, 1, 60000)
        c.update(batch=min(_log_int(rng, 1, 128), max(1, 400000 // hi)), hi=hi, n_kv=n_kv,
                 lo=rng.randint(1, hi), n_q=n_kv * G)
    return c


def _lens(case):
    """Tokens of every sequence: new, written or read, or the context of attention."""
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _past(case):
    """Tokens of every sequence before the new, written or read ones."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, case["past"]) for _ in range(case["batch"])]


def _blocks(tokens, bs):
    return (tokens + bs - 1) // bs


def work(case):
    lens, bs, op = _lens(case), case["bs"], case["op"]
    n = sum(lens)
    if op == "tables":
        past = _past(case)
        taken = sum(_blocks(p + t, bs) - _blocks(p, bs) for p, t in zip(past, lens))
        held = sum(_blocks(p, bs) for p in past)
        # the pool's bits, a slot and a position per token, an entry and a count per block, twice
        return {"bytes": (held + taken + case["spare"]) // 8 + 12 * n + 16 * taken + 32 * len(lens),
                "flops": 2 * n}
    n_kv = case["n_kv"]
    if op == "rope":
        rows = case["n_q"] * 4 * case["d"] + n_kv * 4 * case["d"]
        if case["mode"] == "append":
            rows += n_kv * 4 * D + 8
        return {"bytes": n * (rows + 4), "flops": n * (case["n_q"] + n_kv) * case["rotary"] * 3}
    if op in ("write", "read"):
        touched = sum(_blocks(p + t, bs) - p // bs for p, t in zip(_past(case), lens))
        passes = 2 if op == "write" else 1
        return {"bytes": passes * 2 * n * n_kv * (2 * D + 72) + 4 * touched + 8 * len(lens),
                "flops": passes * 2 * n * n_kv * D * 2}
    n_q = case["n_q"]
    return {"bytes": n * n_kv * 144 + 4 * sum(_blocks(t, bs) for t in lens)
            + len(lens) * n_q * D * 4, "flops": 4 * n * n_q * D}


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


def _random_pool4(NB, n_kv, bs, gen):
    """A 4-bit pool as quantised rows fill it: normal values of which a group's largest is about
    6, and scales about 0.37 times a row's spread."""
    z = torch.randn(65536, 2, generator=gen, device="cuda").mul_(2.7)
    mag = torch.bucketize(z.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],
                                                device="cuda"))
    nib = mag + 8 * (z < 0)
    pair = (nib[:, 0] + 16 * nib[:, 1]).to(torch.uint8)
    out = torch.empty(NB * n_kv * (bs // 16), GROUP, dtype=torch.uint8, device="cuda")
    step = 1 << 16
    for i in range(0, out.shape[0], step):
        n = out[i:i + step].shape[0]
        at = torch.randint(0, 65536, (n, 1024), generator=gen, device="cuda", dtype=torch.int32)
        out[i:i + step, :1024] = pair[at.long()]
        x = torch.randn(n, 128, generator=gen, device="cuda").mul_(0.3).exp_().mul_(0.37)
        out[i:i + step, 1024:] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out.view(NB, n_kv, bs // 16, GROUP)


def _tables(nblk, spare, seed, width=0):
    """Tables over a random permutation of the pool's blocks, and the number of blocks."""
    total = sum(nblk)
    NB = total + max(1, total // 20) + spare
    perm = torch.randperm(NB, generator=torch.Generator().manual_seed(seed * 31 + 5))
    first = torch.tensor([0] + nblk).cumsum(0)
    j = torch.arange(max(max(nblk), width, 1))
    at = (first[:-1, None] + j).clamp(max=NB - 1)
    t = torch.where(j < torch.tensor(nblk)[:, None], perm[at], torch.tensor(-1))
    return t.to(torch.int32).cuda(), NB


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _scale_places(is_v, slot):
    """Places in a group's 1152 bytes of the eight scales of slots [n]: [n][8]."""
    g = torch.arange(8, device="cuda")
    t = (slot % 16)[:, None]
    return 1024 + (t // 4 * 32 + g * 4 + t % 4 if is_v else t * 8 + g)


def _spoil(pool, is_v, tables, lens, bs):
    """Slots behind every context hold NaN scales (never to be read as a token)."""
    ctx = torch.tensor(lens)
    last = tables.cpu()[torch.arange(len(lens)), (ctx - 1) // bs]
    b, s = torch.nonzero(torch.arange(bs)[None, :] > ((ctx - 1) % bs)[:, None], as_tuple=True)
    if b.numel():
        blk, s = last[b].cuda().long()[:, None], s.cuda()
        pool[blk, :, (s // 16)[:, None], _scale_places(is_v, s)] = 0x7F


def _frequencies(case):
    """Radians a position of every rotated pair: 10000^(-2 i / r), the slow half of them slowed
    further for a context four times as long."""
    r = case["rotary"]
    f = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    return [x if 2 * i < r // 2 else x / 4 for i, x in enumerate(f)]


def _starts(lens):
    starts = [0]
    for t in lens:
        starts.append(starts[-1] + t)
    return starts


def prepare(case, seed):
    op, bs, B = case["op"], case["bs"], case["batch"]
    g, lens = _gen(seed), _lens(case)
    s = {"op": op, "bs": bs, "batch": B, "scale": D ** -0.5}
    if op == "tables":
        past = _past(case)
        nblk = [_blocks(p, bs) for p in past]
        most = max(_blocks(p + t, bs) for p, t in zip(past, lens))
        # as many free blocks again as the requests take, at least, all over the pool
        want = sum(_blocks(p + t, bs) for p, t in zip(past, lens)) - sum(nblk)
        s["tables"], NB = _tables(nblk, case["spare"] + 2 * want, seed, most)
        s["num_blocks"] = NB
        used = torch.rand(NB, generator=g, device="cuda") < 0.4  # other requests' blocks
        held = torch.zeros(NB, dtype=torch.int32, device="cuda")
        held.index_add_(0, s["tables"][s["tables"] >= 0].long(),
                        torch.ones(sum(nblk), dtype=torch.int32, device="cuda"))
        s["refs"] = torch.where(held > 0, held, used.to(torch.int32))
        s["free_bits"] = _pack_bits(s["refs"] == 0)
        s["ctx"], s["keep"], s["new"] = _int32(past), _int32(past), _int32(lens)
        s["positions"], s["starts"] = _int32([0] * B), _int32([0] * (B + 1))
        s["copy_src"], s["copy_dst"], s["result"] = _int32([0] * B), _int32([0] * B), _int32([0] * 4)
        room = max(1, sum(lens) + sum(lens) // 8)  # a padded batch
        s["slots"] = torch.zeros(room, dtype=torch.int64, device="cuda")
        s["token_positions"] = torch.zeros(room, dtype=torch.int32, device="cuda")
        return s
    n_kv = s["n_kv"] = case["n_kv"]
    spread = torch.exp(0.4 * torch.randn(case.get("d", D), generator=g, device="cuda"))
    if op == "rope":
        n_q, d, T, past = case["n_q"], case["d"], sum(lens), _past(case)
        s.update(mode=case["mode"], first=case["first"], rotary=case["rotary"],
                 interleaved=case["pairs"] == "interleaved", tokens=T)
        s["inv_freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) for f in _frequencies(case)]
        turns = [x - (1 << 64) if x >= 1 << 63 else x for x in turns]
        s["frequencies"] = torch.tensor(turns, dtype=torch.int64, device="cuda")
        pos = torch.cat([torch.arange(p, p + t) for p, t in zip(past, lens)])
        s["positions"] = pos.to(torch.int32).cuda()
        s["factor"] = 0.1 * math.log(4.0) + 1.0
        # the output of one projection: q, k and v heads side by side
        qkv = _randn_bf16((T, n_q + 2 * n_kv, d), g, spread)
        s["q"], s["k"], s["v"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        s["q_out"] = torch.empty((T, n_q, d), dtype=torch.bfloat16, device="cuda")
        if case["mode"] == "rows":
            s["k_out"] = torch.empty((T, n_kv, d), dtype=torch.bfloat16, device="cuda")
        else:
            NB = _blocks(T, bs) + 3
            s["k_cache"] = torch.zeros((NB, n_kv, bs // 8, D // 8, 8, 8), dtype=torch.bfloat16,
                                       device="cuda")
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            perm = torch.randperm(NB * bs, generator=g, device="cuda")
            s["slots"] = perm[:T].contiguous()
        return s
    if op in ("write", "read"):
        past = _past(case)
        s["tables"], NB = _tables([_blocks(p + t, bs) for p, t in zip(past, lens)], 0, seed)
        s["positions"], s["most"] = _int32(past), max(lens)
        s["starts"], s["tokens"] = _int32(_starts(lens)), sum(lens)
    else:
        s["tables"], NB = _tables([_blocks(t, bs) for t in lens], 0, seed)
    s["num_blocks"] = NB
    s["k"], s["v"] = _random_pool4(NB, n_kv, bs, g), _random_pool4(NB, n_kv, bs, g)
    s["k_scale"], s["v_scale"] = 0.5, 2.0  # a layer's calibrated scales
    if op in ("write", "read"):
        s["k_rows"] = torch.empty((s["tokens"], n_kv, D), dtype=torch.bfloat16, device="cuda")
        s["v_rows"] = torch.empty_like(s["k_rows"])
    if op == "write":
        s["k_new"] = _randn_bf16((s["tokens"], n_kv, D), g, spread)
        s["v_new"] = _randn_bf16((s["tokens"], n_kv, D), g)
    if op == "attend":
        n_q = case["n_q"]
        s["q"] = _randn_bf16((B, n_q, D), g, spread)
        s["ctx"] = _int32(lens)
        s["out"] = torch.empty_like(s["q"])
        _spoil(s["k"], False, s["tables"], lens, bs)
        _spoil(s["v"], True, s["tables"], lens, bs)
        # the scratch that a serving loop keeps: zero-filled once
        s["workspace"] = torch.zeros((1 << 19) + (B * n_kv + 2048) * (n_q // n_kv) * 560,
                                     dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _pack_bits(free):
    """Truth values [n] as bits of int32 words."""
    f = torch.nn.functional.pad(free.long(), (0, -free.numel() % 32)).view(-1, 32)
    w = (f << torch.arange(32, device="cuda")).sum(1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _grow_plain(s):
    bs, B = s["bs"], s["batch"]
    old, new = s["ctx"].long(), s["new"].long()
    s["positions"].copy_(s["ctx"])
    s["slots"].fill_(-1)
    s["token_positions"].zero_()
    s["starts"].zero_()
    s["copy_src"].fill_(-1)
    s["copy_dst"].fill_(-1)
    row = torch.arange(B, device="cuda")
    nblk = (old + bs - 1) // bs
    last = s["tables"].long()[row, ((old - 1) // bs).clamp(min=0)]
    copied = (old % bs > 0) & (new > 0) & (s["refs"][last.clamp(min=0)] > 1)
    need = (old + new + bs - 1) // bs - nblk + copied
    free = torch.nonzero(s["refs"] == 0).flatten()
    total = int(need.sum())
    if total > free.numel():
        s["result"].copy_(_int32([1, 0, total - free.numel(), 0]))
        return
    r = torch.repeat_interleave(row, need)
    i = torch.arange(total, device="cuda") - (need.cumsum(0) - need)[r]
    j = nblk[r] - copied[r].long() + i
    ids = free[:total].to(torch.int32)
    off = need.cumsum(0) - need
    s["copy_src"].copy_(torch.where(copied, last, -1))
    dst = ids[off.clamp(max=max(total - 1, 0))] if total else torch.full_like(last, -1)
    s["copy_dst"].copy_(torch.where(copied, dst, -1))
    s["tables"][r, j] = ids
    s["refs"][ids.long()] = 1
    s["refs"].index_add_(0, last.clamp(min=0), -copied.to(torch.int32))
    s["free_bits"].copy_(_pack_bits(s["refs"] == 0))
    n = int(new.sum())
    s["starts"][1:] = new.cumsum(0)
    b = torch.repeat_interleave(row, new)
    p = old[b] + torch.arange(n, device="cuda") - s["starts"].long()[b]
    s["slots"][:n] = s["tables"].long()[b, p // bs] * bs + p % bs
    s["token_positions"][:n] = p.to(torch.int32)
    s["ctx"].add_(s["new"])
    s["result"].copy_(_int32([0, total, 0, n]))


def _trim_plain(s):
    bs = s["bs"]
    j = torch.arange(s["tables"].shape[1], device="cuda")
    old, keep = s["ctx"].long(), torch.minimum(s["ctx"], s["keep"]).long()
    gone = (j >= ((keep + bs - 1) // bs)[:, None]) & (j < ((old + bs - 1) // bs)[:, None])
    ids = s["tables"][gone].long()
    s["refs"].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    s["free_bits"].copy_(_pack_bits(s["refs"] == 0))
    s["tables"].masked_fill_(gone, -1)
    s["ctx"].copy_(keep)


def _rotate_plain(s, x, cos, sin):
    """Rows [T][heads][d] with their rotary dims turned, in 32 bits, rounded once."""
    r, first = s["rotary"], s["first"]
    y = x.float()
    part = y[..., first:first + r]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
    u, w = a * cos - b * sin, b * cos + a * sin
    both = torch.stack([u, w], -1).flatten(-2) if s["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([y[..., :first], both, y[..., first + r:]], -1).to(torch.bfloat16)


def _rope_plain(s):
    # angles in 64 bits: 32 lose a far position's place in the circle
    a = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (torch.cos(a) * s["factor"]).float()[:, None]
    sin = (torch.sin(a) * s["factor"]).float()[:, None]
    s["q_out"].copy_(_rotate_plain(s, s["q"], cos, sin))
    k = _rotate_plain(s, s["k"], cos, sin)
    if s["mode"] == "rows":
        s["k_out"].copy_(k)
        return
    blk, slot = s["slots"] // s["bs"], s["slots"] % s["bs"]
    s["k_cache"][blk, :, slot // 8, :, slot % 8] = k.view(-1, s["n_kv"], D // 8, 8)
    s["v_cache"][blk, :, slot // 8, :, slot % 8] = s["v"].reshape(-1, s["n_kv"], D // 8, 8)


def _codes(groups, is_v):
    """Codes 0 .. 15 [...][16 tokens][128 dims] of groups [...][1152]."""
    c = groups[..., :1024]
    c = torch.stack([c & 15, c >> 4], -1)
    if not is_v:
        return c.reshape(*c.shape[:-2], 16, D)
    # plane, dim % 8, tokens / 4, dim / 16 % 4, dim / 8 % 2, token / 2 % 2, token % 2
    c = c.reshape(*c.shape[:-2], 2, 8, 4, 4, 2, 2, 2)
    n = c.dim() - 7
    c = c.permute(*range(n), n + 2, n + 5, n + 6, n, n + 3, n + 4, n + 1)
    return c.reshape(*c.shape[:n], 16, D)


def _pack_codes(c, is_v):
    """The other way: [...][16][128] to [...][1024] bytes."""
    n = c.dim() - 2
    if is_v:
        # tokens / 4, token / 2 % 2, token % 2, plane, dim / 16 % 4, dim / 8 % 2, dim % 8
        c = c.reshape(*c.shape[:-2], 4, 2, 2, 2, 4, 2, 8)
        c = c.permute(*range(n), n + 3, n + 6, n, n + 4, n + 5, n + 1, n + 2)
    c = c.reshape(*c.shape[:n], 1024, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _group_scales(groups, is_v):
    """Scale bytes [...][16 tokens][8] of groups [...][1152]."""
    x = groups[..., 1024:]
    if is_v:
        return x.reshape(*x.shape[:-1], 4, 8, 4).transpose(-1, -2).reshape(*x.shape[:-1], 16, 8)
    return x.reshape(*x.shape[:-1], 16, 8)


def _pack_scales(x, is_v):
    if is_v:
        x = x.reshape(*x.shape[:-2], 4, 4, 8).transpose(-1, -2)
    return x.reshape(*x.shape[:x.dim() - (3 if is_v else 2)], 128)


def _values(groups, is_v, scale):
    """fp32 rows [...][16][128] of groups [...][1152]."""
    c = _codes(groups, is_v)
    low = torch.tensor(E2M1, device="cuda")[(c & 7).int()]
    x = torch.where(c >= 8, -low, low)
    f = _group_scales(groups, is_v).contiguous().view(torch.float8_e4m3fn).float() * scale
    return x * f.repeat_interleave(16, -1)


def _token_places(s):
    """Block and slot of every packed token."""
    n = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), n, right=True)
    p = s["positions"].long()[b] + n - s["starts"].long()[b]
    return s["tables"].long()[b, p // s["bs"]], p % s["bs"]


def _write_plain(s, new, pool, is_v, scale):
    n_kv = s["n_kv"]
    blk, slot = _token_places(s)
    x = new.float().view(-1, n_kv, 8, 16)
    f = (x.abs().amax(-1) / 6 / scale).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = (x / (f.float() * scale)[..., None]).clamp(-6, 6)
    y = torch.where((f.float() == 0)[..., None], 0.0, y)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step  # ties to the even code
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    codes = (mag | (torch.signbit(x).to(torch.uint8) << 3)).view(-1, n_kv, D)
    codes = torch.where((f.float() == 0).repeat_interleave(16, -1), 0, codes)
    # the 16-token groups that hold new tokens, changed where they do and packed again
    group, at = torch.unique(blk * (s["bs"] // 16) + slot // 16, return_inverse=True)
    flat = pool.transpose(1, 2)  # [NB][groups of a tile][n_kv][1152]
    gb, gi = group // (s["bs"] // 16), group % (s["bs"] // 16)
    old = flat[gb, gi]
    all_codes, all_scales = _codes(old, is_v), _group_scales(old, is_v).clone()
    all_codes = all_codes.clone()
    all_codes[at, :, slot % 16] = codes
    all_scales[at, :, slot % 16] = f.view(torch.uint8)
    flat[gb, gi] = torch.cat([_pack_codes(all_codes, is_v), _pack_scales(all_scales, is_v)], -1)


def _read_plain(s, pool, is_v, scale):
    blk, slot = _token_places(s)
    group, at = torch.unique(blk * (s["bs"] // 16) + slot // 16, return_inverse=True)
    x = _values(pool.transpose(1, 2)[group // (s["bs"] // 16), group % (s["bs"] // 16)], is_v,
                scale)
    return x[at, :, slot % 16].to(torch.bfloat16)


def _attend_plain(s):
    """Softmax attention of every query head over its KV head's tokens."""
    blk = s["tables"].long().clamp(min=0)
    k = _values(s["k"][blk], False, s["k_scale"])  # [B][MB][n_kv][bs/16][16][128]
    k = k.transpose(1, 2).flatten(2, 4)
    there = torch.arange(k.shape[2], device="cuda") < s["ctx"][:, None]
    q = s["q"].float().view(s["batch"], s["n_kv"], -1, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    x = x.masked_fill(~there[:, None, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _values(s["v"][blk], True, s["v_scale"]).transpose(1, 2).flatten(2, 4)
    v = v.masked_fill_(~there[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.to(torch.bfloat16).view(s["q"].shape)


def run(s):
    op = s["op"]
    if own:
        import paged_gqa_decode_kv_gb300 as pgd

        if op == "tables":
            pgd.grow_tables(s["tables"], s["ctx"], s["new"], s["refs"], s["free_bits"], s["bs"],
                            s["positions"], s["starts"], s["slots"], s["token_positions"],
                            s["copy_src"], s["copy_dst"], s["result"])
            pgd.trim_tables(s["tables"], s["ctx"], s["keep"], s["refs"], s["free_bits"], s["bs"])
        elif op == "rope" and s["mode"] == "rows":
            pgd.rope(s["q_out"], s["k_out"], s["q"], s["k"], s["positions"], s["frequencies"],
                     interleaved=s["interleaved"], first=s["first"], factor=s["factor"])
        elif op == "rope":
            pgd.rope_append(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                            s["slots"], s["positions"], s["frequencies"],
                            interleaved=s["interleaved"], first=s["first"], factor=s["factor"])
        elif op == "attend":
            pgd.paged_decode_attention_fp4(s["out"], s["q"], s["k"], s["v"], s["tables"], s["ctx"],
                                           s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                           workspace=s["workspace"])
        else:
            if op == "write":
                pgd.kv_append_fp4(s["k_new"], s["v_new"], s["k"], s["v"], s["tables"],
                                  s["positions"], token_starts=s["starts"], max_tokens=s["most"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
            pgd.kv_read_fp4(s["k_rows"], s["v_rows"], s["k"], s["v"], s["tables"], s["positions"],
                            token_starts=s["starts"], max_tokens=s["most"], k_scale=s["k_scale"],
                            v_scale=s["v_scale"])
    elif op == "tables":
        _grow_plain(s)
        _trim_plain(s)
    elif op == "rope":
        _rope_plain(s)
    elif op == "attend":
        s["out"].copy_(_attend_plain(s))
    else:
        if op == "write":
            _write_plain(s, s["k_new"], s["k"], False, s["k_scale"])
            _write_plain(s, s["v_new"], s["v"], True, s["v_scale"])
        s["k_rows"].copy_(_read_plain(s, s["k"], False, s["k_scale"]))
        s["v_rows"].copy_(_read_plain(s, s["v"], True, s["v_scale"]))
    if op == "tables":
        return {n: s[n] for n in ("tables", "ctx", "refs", "free_bits", "positions", "starts",
                                  "slots", "token_positions", "copy_src", "copy_dst", "result")}
    if op == "rope" and s["mode"] == "rows":
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "rope":
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attend":
        return {"out": s["out"]}
    return {"k": s["k_rows"], "v": s["v_rows"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3_values():
    """The value of every E4M3 code, from its bits: sign, four of exponent (bias 7), three."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if (c & 127) == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _nearest(x, values):
    """The nearest of `values` (ascending, from zero, as their codes count) to each x >= 0, a tie
    to the even code, the last where x is beyond it."""
    hi = torch.searchsorted(values, x).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = values[hi] - x, x - values[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (x > values[-1]), hi, lo)


def _rows64(pool, is_v, table, ctx, bs, head, scale):
    """Rows [ctx][128] of one sequence and KV head, in 64 bits, by the layout's byte places."""
    t = torch.arange(ctx, device="cuda")
    i = torch.arange(D, device="cuda")
    base = ((table.long()[t // bs] * pool.shape[1] + head) * (bs // 16) + t % bs // 16) * GROUP
    u = (t % 16)[:, None]
    if is_v:
        byte = i // 64 * 512 + i % 8 * 64 + u // 4 * 16 + i // 8 % 8 * 2 + u % 4 // 2
        high, at = u % 2 == 1, 1024 + u // 4 * 32 + i // 16 * 4 + u % 4
    else:
        byte = u * 64 + i // 2
        high, at = (i % 2 == 1).expand(ctx, D), 1024 + u * 8 + i // 16
    flat = pool.view(-1)
    code = flat[base[:, None] + byte].long()
    code = torch.where(high, code >> 4, code & 15)
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")[code]
    return v * _e4m3_values()[flat[base[:, None] + at].long()] * scale


def _quantised64(new, scale):
    """What the 4-bit cache holds of rows [n][n_kv][128], in 64 bits."""
    x = new.double().view(-1, new.shape[1], 8, 16)
    e4m3 = _e4m3_values()[:127]
    f = e4m3[_nearest((x.abs().amax(-1) / (6 * scale)), e4m3)] * scale
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    y = x.abs() / torch.where(f > 0, f, 1.0)[..., None]
    y = torch.where((f > 0)[..., None], grid[_nearest(y, grid)], 0.0)
    return (torch.sign(x) * y * f[..., None]).view(-1, new.shape[1], D)


def _exact_tables(case, s):
    """The walk over requests, one after another, on the host."""
    bs, B = case["bs"], case["batch"]
    refs = s["refs"].tolist()
    free = [i for i, r in enumerate(refs) if r == 0]
    tables, at, n = s["tables"].tolist(), 0, 0
    slots, places = [-1] * len(s["slots"]), [0] * len(s["slots"])
    past, lens = _past(case), _lens(case)
    for b in range(B):
        for p in range(past[b], past[b] + lens[b]):
            if p % bs == 0:
                tables[b][p // bs] = free[at]
                at += 1
            slots[n], places[n] = tables[b][p // bs] * bs + p % bs, p
            n += 1
    return {"tables": s["tables"], "ctx": s["ctx"], "refs": s["refs"], "free_bits": s["free_bits"],
            "positions": _int32(past), "starts": _int32(_starts(lens)),
            "slots": torch.tensor(slots), "token_positions": _int32(places),
            "copy_src": _int32([-1] * B), "copy_dst": _int32([-1] * B),
            "result": _int32([0, at, 0, n])}


def _exact_rope(case, s):
    r, first, T = case["rotary"], case["first"], s["tokens"]
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full((T, r // 2), s["factor"], dtype=torch.float64, device="cuda"),
                    s["positions"].double()[:, None] * f)
    got = []
    for x in (s["q"], s["k"]):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[1]):
            y[:, h] = x[:, h].double()
            i = torch.arange(r // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + r // 2)
            w = torch.complex(y[:, h, first + a], y[:, h, first + b]) * z
            y[:, h, first + a], y[:, h, first + b] = w.real, w.imag
        got.append(y)
    if case["mode"] == "rows":
        return {"q": got[0], "k": got[1]}
    pools = []
    for x, name in ((got[1], "k_cache"), (s["v"].double(), "v_cache")):
        pool = s[name].double()
        rows = pool.permute(0, 2, 4, 1, 3, 5).reshape(-1, s["n_kv"], D)  # slot after slot
        rows[s["slots"]] = x
        rows = rows.view(pool.shape[0], pool.shape[2], 8, s["n_kv"], D // 8, 8)
        pools.append(rows.permute(0, 3, 1, 4, 2, 5).contiguous())
    return {"q": got[0], "k_cache": pools[0], "v_cache": pools[1]}


def exact(case, seed):
    s, op, bs = prepare(case, seed), case["op"], case["bs"]
    if op == "tables":
        return _exact_tables(case, s)
    if op == "rope":
        return _exact_rope(case, s)
    n_kv, lens = case["n_kv"], _lens(case)
    if op == "write":
        return {"k": _quantised64(s["k_new"], s["k_scale"]),
                "v": _quantised64(s["v_new"], s["v_scale"])}
    if op == "read":
        got = {}
        for name in ("k", "v"):
            got[name] = torch.empty((s["tokens"], n_kv, D), dtype=torch.float64, device="cuda")
            start = 0
            for b, (p, t) in enumerate(zip(_past(case), lens)):
                for h in range(n_kv):
                    rows = _rows64(s[name], name == "v", s["tables"][b], p + t, bs, h,
                                   s[name + "_scale"])
                    got[name][start:start + t, h] = rows[p:]
                start += t
        return got
    n_q = case["n_q"]
    G, out = n_q // n_kv, torch.empty((case["batch"], n_q, D), dtype=torch.float64, device="cuda")
    for b, t in enumerate(lens):
        for h in range(n_kv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            k = _rows64(s["k"], False, s["tables"][b], t, bs, h, s["k_scale"])
            v = _rows64(s["v"], True, s["tables"][b], t, bs, h, s["v_scale"])
            p = torch.softmax(q @ k.T * s["scale"], -1)
            out[b, h * G:(h + 1) * G] = p @ v
    return {"out": out}
