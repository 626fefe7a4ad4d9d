"""The block-scaled 8-bit cache and block-sparse decode attention on the GPU, against the plain
64-bit forms of block_scaled.py.  Codes, scales, bounds and selections are compared bit for bit
(their definitions are exact); attention outputs within the bound that block_scaled.close
derives."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native, inputs

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _starts(lens):
    return [0] + np.cumsum(lens).tolist()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(n, n_kv, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, n_kv, 128, generator=g) * std).to(torch.bfloat16)


def _same_pools(c, k, v, ks, vs):
    assert torch.equal(bsc.untile8(k.cpu()), c.k) and torch.equal(bsc.untile8(v.cpu()), c.v)
    assert torch.equal(ks.cpu(), c.k_scales) and torch.equal(vs.cpu(), c.v_scales)


# --------------------------------------------------------------------------- write, read back
# (cached tokens, new tokens) per sequence
RANGES = [
    [(0, 1)], [(5, 1), (16, 1), (31, 1), (0, 1)], [(0, 16), (0, 17), (7, 40), (40, 0), (3, 1)],
    [(15, 1), (15, 2), (15, 17), (15, 18)], [(100, 300), (0, 0), (1, 33)], [(0, 0)],
]


@pytest.mark.parametrize("ranges", RANGES, ids=str)
@pytest.mark.parametrize("n_kv,bs,more", [(1, 16, 0), (3, 32, 0), (8, 16, 0), (2, 16, 1 << 17),
                                          (4, 32, 1 << 17)])
def test_append_ranges(ranges, n_kv, bs, more):
    """`more`: max_tokens far above the ranges (warps then take runs of blocks)."""
    past, lens = [p for p, _ in ranges], [n for _, n in ranges]
    c = bsc.make_cache(past, n_kv, bs, seed=sum(lens) + bs, room=max(lens) + 1)
    st = _starts(lens)
    # a wide spread of sizes: some blocks grow, some do not; a row of zeros
    kn, vn = _rows(st[-1], n_kv, 3, 4.0), _rows(st[-1], n_kv, 4, 0.05)
    if st[-1] > 3:
        kn[2] = 0
        vn[-1] *= 1000
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, _i32(past),
                       token_starts=_i32(st), max_tokens=max(lens) + more)
    bsc.append(c, kn, vn, past, st)
    _same_pools(c, k, v, ks, vs)


def test_any_max_tokens():
    """max_tokens is a bound: the largest number does."""
    c = bsc.make_cache([20, 3], 2, 16, seed=5, room=30)
    kn, vn = _rows(31, 2, 1), _rows(31, 2, 2)
    k, v, ks, vs, tables, lens = c.cuda()
    st, most = [0, 30, 31], (1 << 31) - 1
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, lens, token_starts=_i32(st),
                       max_tokens=most)
    bsc.append(c, kn, vn, [20, 3], st)
    _same_pools(c, k, v, ks, vs)
    out = [torch.zeros_like(kn, device="cuda") for _ in range(2)]
    pgd.kv_read_fp8b(*out, k, v, ks, vs, tables, lens, token_starts=_i32(st), max_tokens=most)
    assert np.array_equal(bsc.f64(out[0][:30]), c.rows("k", 0, 50)[20:])
    bounds, scales = _empty_bounds(c)
    want, ws = _want_bounds(c, bounds.cpu(), scales.cpu(), [(0, j, 50) for j in range(4)] +
                            [(1, 0, 4)])
    pgd.block_bounds(bounds, scales, k, tables, _i32([50, 4]), max_tokens=most, k_scales=ks)
    assert torch.equal(bounds.cpu(), want) and torch.equal(scales.cpu(), ws)


def test_append_one_token_each_without_starts():
    past = [0, 4, 15, 16, 33]
    c = bsc.make_cache(past, 4, 16, seed=9, room=1)
    kn, vn = _rows(5, 4, 5), _rows(5, 4, 6, 30.0)
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, _i32(past))
    bsc.append(c, kn, vn, past, list(range(6)))
    _same_pools(c, k, v, ks, vs)


def test_append_extreme_rows():
    """Zeros, the largest and smallest bf16 values, subnormals, infinities and NaN; a block of
    zeros begun before that grows."""
    c = bsc.make_cache([0, 0, 3], 2, 16, seed=2, room=40)
    blk = int(c.tables[2, 0])
    c.k[blk, :, :3] = 0
    c.k_scales[blk] = 2.0 ** -100
    kn = _rows(20, 2, 7)
    kn[0] = 0
    kn[1, 0, 5], kn[1, 1, 5] = 3.38e38, -3.38e38
    kn[2] = torch.linspace(-1e-38, 1e-38, 128).to(torch.bfloat16)
    kn[9, 0, :2] = torch.tensor([float("inf"), -float("inf")])
    kn[9, 1, 7] = float("nan")
    st = [0, 9, 17, 20]
    vn = -kn.flip(0).contiguous()
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, _i32([0, 0, 3]),
                       token_starts=_i32(st), max_tokens=16)
    bsc.append(c, kn, vn, [0, 0, 3], st)
    got, want = bsc.untile8(k.cpu()), c.k
    nan = torch.from_numpy(np.isnan(bsc.VALUES[want.numpy()]))
    assert torch.equal(torch.from_numpy(np.isnan(bsc.VALUES[got.numpy()])), nan)
    assert torch.equal(got[~nan], want[~nan])
    assert torch.equal(ks.cpu(), c.k_scales) and torch.equal(vs.cpu(), c.v_scales)


def test_append_keeps_scales_that_are_no_powers_of_two():
    """A cache filled by the caller with scales of its own: blocks that need no larger scale keep
    theirs, the new rows divided by it."""
    c = bsc.make_cache([3, 9], 2, 16, seed=3, room=4)
    c.k_scales.mul_(1.37)
    c.v_scales.mul_(100.3)
    kn, vn = _rows(4, 2, 8, 2.0), _rows(4, 2, 9, 0.5)
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_append_fp8b(kn.view(2, 2, 2, 128).cuda(), vn.view(2, 2, 2, 128).cuda(), k, v, ks, vs,
                       tables, _i32([3, 9]))
    # fp32 quotients, as the definition has them: the plain form in 32 bits
    for new, codes, sc in ((kn, c.k, c.k_scales), (vn, c.v, c.v_scales)):
        for b, p in enumerate([3, 9]):
            blk, x = int(c.tables[b, 0]), new[2 * b:2 * b + 2].float()
            for g in range(2):
                old = sc[blk, g].clone()
                s = max(float(old), bsc.least_pow2(float(x[:, g].abs().max()), 448.0))
                s = torch.tensor(s, dtype=torch.float32)
                if s != old:
                    e = torch.from_numpy(bsc.VALUES[codes[blk, g, :p].numpy()]).float() * (old / s)
                    codes[blk, g, :p] = torch.from_numpy(bsc.e4m3_codes(e.numpy()))
                codes[blk, g, p:p + 2] = torch.from_numpy(bsc.e4m3_codes((x[:, g] / s).numpy()))
                sc[blk, g] = s
    _same_pools(c, k, v, ks, vs)


@pytest.mark.parametrize("ranges", RANGES, ids=str)
@pytest.mark.parametrize("n_kv,bs,more", [(1, 16, 0), (3, 32, 0), (8, 16, 0), (2, 16, 1 << 17)])
def test_read_ranges(ranges, n_kv, bs, more):
    """Every row bit for bit; rows that belong to no sequence stay as they were."""
    past, lens = [p for p, _ in ranges], [n for _, n in ranges]
    c = bsc.make_cache([p + n for p, n in ranges], n_kv, bs, seed=bs)
    st = _starts(lens)
    out = [torch.full((st[-1] + 3, n_kv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
           for _ in range(2)]
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_read_fp8b(*out, k, v, ks, vs, tables, _i32(past), token_starts=_i32(st),
                     max_tokens=max(lens) + more)
    for which, got in zip("kv", out):
        want = np.full((st[-1] + 3, n_kv, 128), 7.0)
        for b, (p, n) in enumerate(ranges):
            want[st[b]:st[b + 1]] = c.rows(which, b, p + n)[p:]
        assert np.array_equal(bsc.f64(got), want)


def test_read_back_of_what_was_written():
    """Each value is within half a step of E4M3 at its block's scale: 2^-4 of itself, or 2^-10 of
    the scale below E4M3's smallest normal."""
    lens = [700, 1, 90]
    c = bsc.make_cache([0, 0, 0], 4, 32, room=700)
    kn, vn = _rows(791, 4, 1), _rows(791, 4, 2, 100.0)
    k, v, ks, vs, tables, _ = c.cuda()
    st = _i32(_starts(lens))
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, _i32([0, 0, 0]),
                       token_starts=st, max_tokens=700)
    ko, vo = torch.empty_like(kn, device="cuda"), torch.empty_like(vn, device="cuda")
    pgd.kv_read_fp8b(ko, vo, k, v, ks, vs, tables, _i32([0, 0, 0]), token_starts=st,
                     max_tokens=700)
    for x, y, s in ((kn, ko, ks), (vn, vo, vs)):
        err = (y.cpu().double() - x.double()).abs()
        assert (err <= torch.maximum(x.double().abs() * 2 ** -4, s.max().cpu() * 2.0 ** -10)).all()


@pytest.mark.parametrize("call", ["append", "read"])
def test_bad_ranges_are_flagged_and_skipped(call):
    """Positions outside the table, starts out of order, beyond the rows or over max_tokens apart
    and bad block ids: flagged; the other sequences are served."""
    c = bsc.make_cache([4, 4, 4, 4], 2, 16, room=12)
    k, v, ks, vs, tables, _ = c.cuda()
    rows = [_rows(12, 2, 1).cuda(), _rows(12, 2, 2).cuda()]
    fn = pgd.kv_append_fp8b if call == "append" else pgd.kv_read_fp8b
    for pos, st, most, bad_id, bad in [
            ([4, -1, 4, 4], [0, 3, 6, 9, 12], 3, False, 1),
            ([4, 30, 4, 4], [0, 3, 6, 9, 12], 3, False, 1),
            ([4, 4, 4, 4], [0, 3, 2, 2, 5], 3, False, 1),
            ([4, 4, 4, 4], [0, 3, 6, 9, 13], 4, False, 3),
            ([4, 4, 4, 4], [0, 3, 12, 12, 12], 3, False, 1),
            ([4, 4, 4, 4], [0, 3, 6, 9, 12], 3, True, 1)]:
        t = tables.clone()
        if bad_id:
            t[1, 0] = 1 << 20
        before = [x.clone() for x in (k, v, ks, vs, *rows)]
        fn(*rows, k, v, ks, vs, t, _i32(pos), token_starts=_i32(st), max_tokens=most)
        assert pgd.device_errors(clear=True) == (_native.DEVERR_BAD_BLOCK_ID if bad_id
                                                 else _native.DEVERR_BAD_POSITION)
        blk, first = int(tables[bad, 0]), int(tables[0, 0])
        if call == "append":
            assert torch.equal(k[blk], before[0][blk]) and torch.equal(vs[blk], before[3][blk])
            assert not torch.equal(v[first], before[1][first])
        else:  # (slots 4 .. hold the spoiled NaN)
            assert torch.isnan(rows[0][0:3]).all()
            mine = slice(st[1], min(st[2], 12)) if bad == 1 else slice(st[3], 12)
            others = set(range(0, 3)) | (set(range(st[3], st[4])) if bad == 1 else set())
            for i in range(mine.start, mine.stop):
                if i not in others:
                    assert torch.equal(rows[0][i], before[4][i])
        for x, y in zip((k, v, ks, vs, *rows), before):
            x.copy_(y)


# ------------------------------------------------------------------------------- attention
SMALL = [
    # (n_q, n_kv, bs, contexts)
    (4, 4, 16, [1]), (8, 4, 16, [16, 17, 1]), (16, 4, 16, [33, 200, 513]),
    (16, 2, 32, [31, 32, 33, 700]), (32, 4, 32, [64, 1, 95]), (32, 8, 16, [512]),
    (64, 8, 32, [129, 1000, 32]), (8, 1, 16, [300, 5]), (2, 1, 16, [47]), (40, 40, 16, [90, 250]),
    (4, 4, 32, [127, 128, 129]), (8, 1, 32, [4000, 3]), (10, 10, 16, [2100]),
]


@pytest.mark.parametrize("case", SMALL, ids=str)
@pytest.mark.parametrize("num_splits", [0, 1, 3, 64])
def test_attention(case, num_splits):
    n_q, n_kv, bs, ctx = case
    c = bsc.make_cache(ctx, n_kv, bs, seed=n_q + bs)
    q = bsc.make_query(len(ctx), n_q)
    k, v, ks, vs, tables, lens = c.cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE,
                                          num_splits=num_splits)
    bsc.close(got, *bsc.paged(c, q, SCALE), label=str(case))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 32])
def test_attention_ragged(G, bs):
    ctx = torch.randint(1, 1500, (23,), generator=torch.Generator().manual_seed(G + bs)).tolist()
    c = bsc.make_cache(ctx, 3, bs, seed=G)
    q = bsc.make_query(23, 3 * G)
    k, v, ks, vs, tables, lens = c.cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE)
    bsc.close(got, *bsc.paged(c, q, SCALE))


@pytest.mark.parametrize("limit", [1024, 600, 0])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n_kv, bs, ctx", [
    (4, 16, [2048, 1, 129]), (3, 32, [1025, 2033, 16]), (12, 16, [1023]), (13, 16, [1900]),
    (16, 32, [1200]), (1, 16, [2049, 700]), (2, 32, [1999, 1300]),
])
def test_attention_at_the_limits_of_short_contexts(n_kv, bs, ctx, G, limit):
    """Sizes on both sides of every bound of the kernel for short contexts, and of each of its
    two cluster sizes, at any limit."""
    c = bsc.make_cache(ctx, n_kv, bs, seed=n_kv + G)
    q = bsc.make_query(len(ctx), n_kv * G)
    k, v, ks, vs, tables, lens = c.cuda()
    before = pgd.set_short_context_tokens(limit)
    try:
        got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE)
    finally:
        pgd.set_short_context_tokens(before)
    bsc.close(got, *bsc.paged(c, q, SCALE))


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_attention_scores_grow_along_the_context(G, num_splits):
    """The K scales of later blocks 8 and then 32 times as large: the running maximum moves far
    and often."""
    ctx = [1500, 1300, 1700]
    c = bsc.make_cache(ctx, 2, 16, seed=60 + G)
    for b in range(3):
        for j in range(32, -(-ctx[b] // 16)):
            c.k_scales[int(c.tables[b, j])] *= 32.0 if j >= 64 else 8.0
    q = bsc.make_query(3, 2 * G)
    q[:, ::3] = 0
    k, v, ks, vs, tables, lens = c.cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE,
                                          num_splits=num_splits)
    bsc.close(got, *bsc.paged(c, q, SCALE))


@pytest.mark.parametrize("G", [1, 4, 8])
def test_attention_value_scales_far_apart(G):
    """V scales over 40 binades, the heavy weights on blocks of small values (a first token that
    takes most of the weight and holds next to nothing), blocks of zeros with the least scale."""
    ctx = [1000, 260, 40]
    c = bsc.make_cache(ctx, 2, 16, seed=70 + G)
    g = torch.Generator().manual_seed(8)
    c.v_scales.copy_(torch.exp2(torch.randint(-30, 11, c.v_scales.shape, generator=g).float()))
    for b in range(3):
        blk = int(c.tables[b, 0])
        c.v_scales[blk] = 2.0 ** -20
        c.k_scales[blk] *= 16
    zero = int(c.tables[0, 9])
    c.v[zero] = 0
    c.v_scales[zero] = 2.0 ** -100
    q = bsc.make_query(3, 2 * G)
    k, v, ks, vs, tables, lens = c.cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE)
    bsc.close(got, *bsc.paged(c, q, SCALE))


def test_attention_one_heavy_token_among_many_light_ones():
    """One token holds half the weight, the rest shares the other half among 60000 (each 2^-16 of
    it): the light ones must not be lost."""
    n = 60000
    c = bsc.make_cache([n], 1, 16, scale_spread=0)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    q[:, :, 0] = 8.0
    c.k_scales.fill_(1.0)
    c.k[..., 0] = 0
    # the heavy token's score is 8 * 15 * scale = ln(60000) + 0.03 above the others'
    c.k[int(c.tables[0, 0]), 0, 5, 0] = int(bsc.e4m3_codes([15.0])[0])
    scale = float(np.log(n) / (8 * 15.0))
    k, v, ks, vs, tables, lens = c.cuda()
    # values all of one sign, so that what is lost would show
    c.v = torch.where(torch.from_numpy(np.isnan(bsc.VALUES[c.v.numpy()])), c.v, c.v & 0x7F)
    v = bsc.tile8(c.v).cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, scale)
    bsc.close(got, *bsc.paged(c, q, scale))


def test_attention_query_of_many_binades():
    ctx = [700, 300]
    for G in (1, 8):
        c = bsc.make_cache(ctx, 2, 32, seed=90 + G)
        g = torch.Generator().manual_seed(5)
        mag = torch.randint(-12, 13, (2, 2 * G, 128), generator=g).float()
        q = torch.randn(2, 2 * G, 128, generator=g) * torch.exp2(mag) / 512.0
        q[:, 0] = torch.randn(2, 128, generator=g) * 2.0 ** -100
        q = q.to(torch.bfloat16)
        k, v, ks, vs, tables, lens = c.cuda()
        got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE)
        bsc.close(got, *bsc.paged(c, q, SCALE))


@pytest.mark.parametrize("num_splits", [0, 2])
def test_append_attention(num_splits):
    past = [0, 15, 16, 699, 2047]
    c = bsc.make_cache(past, 8, 16, seed=4, room=1)
    kn, vn = _rows(5, 8, 1, 3.0), _rows(5, 8, 2, 3.0)
    q = bsc.make_query(5, 32)
    k, v, ks, vs, tables, _ = c.cuda()
    ctx = [p + 1 for p in past]
    got = pgd.append_decode_attention_fp8b(None, q.cuda(), kn.cuda(), vn.cuda(), k, v, ks, vs,
                                           tables, _i32(ctx), SCALE, num_splits=num_splits)
    bsc.append(c, kn, vn, past, list(range(6)))
    _same_pools(c, k, v, ks, vs)
    c.ctx = ctx
    bsc.close(got, *bsc.paged(c, q, SCALE))


def test_attention_flags_contexts_and_ids():
    c = bsc.make_cache([40, 40, 40, 40], 2, 16)
    q = bsc.make_query(4, 8).cuda()
    k, v, ks, vs, tables, _ = c.cuda()
    want, mag = bsc.paged(c, q.cpu(), SCALE)
    tables[2, 1] = -5
    got = pgd.paged_decode_attention_fp8b(None, q, k, v, ks, vs, tables, _i32([40, 0, 40, 40]),
                                          SCALE)
    assert pgd.device_errors(clear=True) == (_native.DEVERR_BAD_CONTEXT |
                                             _native.DEVERR_BAD_BLOCK_ID)
    keep = [0, 3]
    bsc.close(got[keep], want[keep], mag[keep])
    pgd.paged_decode_attention_fp8b(None, q, k, v, ks, vs, c.tables.cuda(),
                                    _i32([40, 65, 40, 40]), SCALE)
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_CONTEXT


@pytest.mark.parametrize("num_splits", [0, 3])
@pytest.mark.parametrize("bs", [16, 32])
def test_attention_timeout_then_normal_call(num_splits, bs):
    """The kernel's timeout exit, made to happen by a wait limit of 1 ns: the call returns and
    reports it, and the next one on the same workspace is right."""
    ctx = [3000, 17, 900, 2048, 1, 5000, 64, 333, 1200, 4096, 700, 16]
    c = bsc.make_cache(ctx, 2, bs, seed=31)
    q = bsc.make_query(12, 8)
    k, v, ks, vs, tables, lens = c.cuda()
    ws = pgd.make_block_workspace(12, 8, 2, num_splits)
    call = lambda: pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens,
                                                   SCALE, num_splits=num_splits, workspace=ws)
    try:
        pgd.set_wait_limit_ns(1)
        call()
        torch.cuda.synchronize()
        assert pgd.device_errors(clear=True) & _native.DEVERR_TIMEOUT
    finally:
        pgd.set_wait_limit_ns(0)
    bsc.close(call(), *bsc.paged(c, q, SCALE))


# ------------------------------------------------------------------- bounds and selection
def _empty_bounds(c, fill=-77):
    NB = c.k.shape[0]
    return (torch.full((NB, c.n_kv, 2, 128), fill, dtype=torch.int8, device="cuda"),
            torch.full((NB, c.n_kv), -1.0, device="cuda"))


def _want_bounds(c, got, gs, blocks):
    """The plain bounds of the given (b, j, n) blocks in copies of the tensors before the call."""
    for b, j, n in blocks:
        for g in range(c.n_kv):
            lo, hi, s = bsc.bounds(c, b, j, g, n)
            blk = int(c.tables[b, j])
            got[blk, g, 0], got[blk, g, 1] = torch.from_numpy(lo), torch.from_numpy(hi)
            gs[blk, g] = s
    return got, gs


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,bs", [(1, 32), (5, 16)])
@pytest.mark.parametrize("first,most", [(None, None), ([0, 0, 31, 16, 200, 33], 315),
                                        ([0, 0, 31, 16, 200, 33], 1 << 17)],
                         ids=["all", "from", "from_runs"])
def test_bounds(fp8, n_kv, bs, first, most):
    ctx = [1, 16, 33, 17, 515, 33]
    c = bsc.make_cache(ctx, n_kv, bs, fp8=fp8, seed=bs + n_kv, scale_spread=6)
    if not fp8:  # zeros, tiny and huge keys
        c.k[int(c.tables[1, 0])] = 0
        c.k[int(c.tables[4, 1])] *= 1e-30
        c.k[int(c.tables[4, 2])] *= 1e36
    k, _, ks, _, tables, lens = c.cuda()
    got, gs = _empty_bounds(c)
    want, ws = _want_bounds(c, got.cpu(), gs.cpu(), [
        (b, j, n) for b, n in enumerate(ctx) for j in range(0 if first is None or first[b] == n
                                                            else first[b] // bs, -(-n // bs))
        if first is None or first[b] < n])
    pgd.block_bounds(got, gs, k, tables, lens, positions=None if first is None else _i32(first),
                     max_tokens=most, k_scales=ks)
    assert torch.equal(got.cpu(), want) and torch.equal(gs.cpu(), ws)


def test_bounds_flags():
    c = bsc.make_cache([40, 40, 40], 2, 16, fp8=False)
    k, _, _, _, tables, _ = c.cuda()
    for ctx, pos, most, flags in [([40, 65, 40], None, None, _native.DEVERR_BAD_CONTEXT),
                                  ([40, -1, 40], None, None, _native.DEVERR_BAD_CONTEXT),
                                  ([40, 40, 40], [0, -1, 0], 64, _native.DEVERR_BAD_POSITION),
                                  ([40, 40, 40], [0, 41, 0], 64, _native.DEVERR_BAD_POSITION),
                                  ([40, 40, 40], [20, 19, 20], 20, _native.DEVERR_BAD_POSITION)]:
        got, gs = _empty_bounds(c)
        pgd.block_bounds(got, gs, k, tables, _i32(ctx), max_tokens=most,
                         positions=None if pos is None else _i32(pos))
        assert pgd.device_errors(clear=True) == flags
        assert (got[tables[1, :3].long()] == -77).all()
        assert (gs[tables[2, 2].long()] > 0).all()


def _select_inputs(ctx, n_kv, G, bs, seed, ties=False):
    c = bsc.make_cache(ctx, n_kv, bs, fp8=False, seed=seed)
    g = torch.Generator().manual_seed(seed)
    NB = c.k.shape[0]
    lo = torch.randint(-127, 60, (NB, n_kv, 128), generator=g)
    hi = torch.minimum(lo + torch.randint(0, 150, lo.shape, generator=g), torch.tensor(127))
    if ties:  # blocks alike in threes
        lo, hi = lo[torch.arange(NB) // 3 * 3 % 4], hi[torch.arange(NB) // 3 * 3 % 4]
    bounds = torch.stack([lo, hi], 2).to(torch.int8)
    e = torch.zeros(NB, n_kv) if ties else torch.randint(-3, 2, (NB, n_kv), generator=g).float()
    return c, bounds, torch.exp2(e), bsc.make_query(len(ctx), n_kv * G, seed=seed)


def _chosen(c, q, bounds, scales, W, first, last):
    G = q.shape[1] // c.n_kv
    got = []
    for b, n in enumerate(c.ctx):
        at = c.tables[b, :-(-n // c.bs)].long()
        got.append([bsc.select(q[b, g * G:(g + 1) * G], bsc.f64(bounds[at, g, 0]),
                               bsc.f64(bounds[at, g, 1]), bsc.f64(scales[at, g]), W, first, last)
                    for g in range(c.n_kv)])
    return got


def _want_tiles(c, chosen, W):
    tiles = torch.full((len(c.ctx), c.n_kv, W), -1, dtype=torch.int32)
    tokens = torch.zeros(len(c.ctx), c.n_kv, dtype=torch.int32)
    for b, n in enumerate(c.ctx):
        for g, js in enumerate(chosen[b]):
            tiles[b, g, :len(js)] = c.tables[b, js] * c.n_kv + g
            tokens[b, g] = (len(js) - 1) * c.bs + n - (-(-n // c.bs) - 1) * c.bs
    return tiles, tokens


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("W,first,last", [(1, 0, 1), (5, 1, 2), (7, 3, 4), (40, 0, 1), (64, 2, 8)])
@pytest.mark.parametrize("ties", [False, True])
def test_select(G, W, first, last, ties):
    ctx = [1, 16, 17, 640, 641, 1023, 80, 5000]
    c, bounds, scales, q = _select_inputs(ctx, 2, G, 16, seed=W + G, ties=ties)
    tiles = torch.full((len(ctx), 2, W), 99, dtype=torch.int32, device="cuda")
    tokens = torch.full((len(ctx), 2), 99, dtype=torch.int32, device="cuda")
    pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(),
                      _i32(ctx), first, last, 16)
    want, wn = _want_tiles(c, _chosen(c, q, bounds, scales, W, first, last), W)
    assert torch.equal(tokens.cpu(), wn) and torch.equal(tiles.cpu(), want)


@pytest.mark.parametrize("n", [131072, 131072 - 15, 300000])
def test_select_of_a_long_context(n):
    c, bounds, scales, q = _select_inputs([n, 77], 1, 4, 16, seed=3)
    tiles = torch.empty(2, 1, 300, dtype=torch.int32, device="cuda")
    tokens = torch.empty(2, 1, dtype=torch.int32, device="cuda")
    pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(),
                      _i32([n, 77]), 2, 5, 16)
    want, wn = _want_tiles(c, _chosen(c, q, bounds, scales, 300, 2, 5), 300)
    assert torch.equal(tokens.cpu(), wn) and torch.equal(tiles.cpu(), want)


@pytest.mark.parametrize("n_kv", [1, 2, 4, 8])
@pytest.mark.parametrize("W, first, last, ties", [(7, 2, 5, False), (37, 0, 1, True),
                                                 (400, 260, 100, True), (2000, 1, 1, False)])
def test_select_in_clusters_of_every_size(n_kv, W, first, last, ties):
    """A wide table (16, 12, 8 and 4 CTAs a head) and contexts that leave slices empty, that end
    in the first one and that are selected whole; forced blocks over several slices."""
    ctx = [40000, 300, 640, 16 * 401]
    c, bounds, scales, q = _select_inputs(ctx, n_kv, 2, 16, seed=W + n_kv, ties=ties)
    tiles = torch.full((4, n_kv, W), 99, dtype=torch.int32, device="cuda")
    tokens = torch.full((4, n_kv), 99, dtype=torch.int32, device="cuda")
    want, wn = _want_tiles(c, _chosen(c, q, bounds, scales, W, first, last), W)
    args = (q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(), _i32(ctx), first, last, 16)
    for _ in range(3):
        pgd.select_blocks(tiles, tokens, *args)
        assert torch.equal(tokens.cpu(), wn) and torch.equal(tiles.cpu(), want)


def test_select_zero_and_extreme_queries():
    """A zero query (every score 0: the first blocks), queries of tiny and of huge values."""
    ctx = [900, 900, 900]
    c, bounds, scales, q = _select_inputs(ctx, 1, 2, 16, seed=6)
    q[0] = 0
    q[1] = (q[1].double() * 2.0 ** -110).to(torch.bfloat16)
    q[2] = (q[2].double() * 2.0 ** 80).to(torch.bfloat16)
    tiles = torch.empty(3, 1, 20, dtype=torch.int32, device="cuda")
    tokens = torch.empty(3, 1, dtype=torch.int32, device="cuda")
    pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(),
                      _i32(ctx), 0, 1, 16)
    want, _ = _want_tiles(c, _chosen(c, q, bounds, scales, 20, 0, 1), 20)
    assert torch.equal(tiles.cpu(), want)
    assert torch.equal(tiles[0, 0].cpu(), c.tables[0, [*range(19), 56]])


def test_select_flags():
    c, bounds, scales, q = _select_inputs([300, 300], 2, 2, 16, seed=7)
    tiles = torch.empty(2, 2, 4, dtype=torch.int32, device="cuda")
    tokens = torch.empty(2, 2, dtype=torch.int32, device="cuda")
    for bad in (0, -3, 20 * 16 + 1):
        pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(),
                          _i32([300, bad]), 0, 1, 16)
        assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_CONTEXT
        assert (tokens[1] == 0).all() and (tiles[1] == -1).all() and (tiles[0] >= 0).all()


# ---------------------------------------------------------------- attention over selections
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,n_kv,bs", [(1, 3, 16), (4, 8, 16), (8, 2, 32), (2, 4, 32)])
@pytest.mark.parametrize("W", [6, 80])
def test_sparse_attention(fp8, G, n_kv, bs, W):
    ctx = [1, 40, 333, 2500, 700]
    c = bsc.make_cache(ctx, n_kv, bs, fp8=fp8, seed=W + G)
    q = bsc.make_query(5, n_kv * G)
    k, v, ks, vs, tables, lens = c.cuda()
    bounds, scales = _empty_bounds(c)
    pgd.block_bounds(bounds, scales, k, tables, lens, k_scales=ks)
    tiles = torch.empty(5, n_kv, W, dtype=torch.int32, device="cuda")
    tokens = torch.empty(5, n_kv, dtype=torch.int32, device="cuda")
    got = pgd.sparse_decode_attention(None, q.cuda(), k, v, bounds, scales, tables, lens, tiles,
                                      tokens, 1, 2, SCALE, k_scales=ks, v_scales=vs)
    chosen = _chosen(c, q, bounds.cpu(), scales.cpu(), W, 1, 2)
    want, wn = _want_tiles(c, chosen, W)
    assert torch.equal(tiles.cpu(), want) and torch.equal(tokens.cpu(), wn)
    ref = bsc.selected(c, q, chosen, SCALE)
    bsc.close(got, *ref)
    # the two calls, and a workspace of the documented size
    ws = pgd.make_block_workspace(5, n_kv * G, n_kv)
    again = pgd.selected_decode_attention(None, q.cuda(), k, v, tiles, tokens, SCALE, k_scales=ks,
                                          v_scales=vs, workspace=ws)
    assert torch.equal(again, got)
    parts = pgd.selected_decode_attention(None, q.cuda(), k, v, tiles, tokens, SCALE, k_scales=ks,
                                          v_scales=vs, num_splits=2)
    bsc.close(parts, *ref)


def test_selected_attention_over_the_callers_tiles():
    """Tiles of the caller's own: another order, the same tile twice."""
    c = bsc.make_cache([500, 500], 2, 16, seed=8)
    q = bsc.make_query(2, 8)
    chosen = [[[9, 3, 3, 20], [0, 1, 2, 30]], [[5, 4, 3, 7], [30, 30, 30, 30]]]
    tiles = torch.tensor([[[int(c.tables[b, j]) * 2 + g for j in chosen[b][g]] for g in range(2)]
                          for b in range(2)], dtype=torch.int32, device="cuda")
    tokens = torch.full((2, 2), 64, dtype=torch.int32, device="cuda")
    k, v, ks, vs, _, _ = c.cuda()
    got = pgd.selected_decode_attention(None, q.cuda(), k, v, tiles, tokens, SCALE, k_scales=ks,
                                        v_scales=vs)
    bsc.close(got, *bsc.selected(c, q, chosen, SCALE))


def test_selected_attention_flags_tiles_and_tokens():
    c = bsc.make_cache([500, 500], 2, 16, seed=8)
    q = bsc.make_query(2, 8).cuda()
    k, v, ks, vs, _, _ = c.cuda()
    tiles = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    tiles[0, 0, 1] = k.shape[0] * 2
    pgd.selected_decode_attention(None, q, k, v, tiles, _i32([[64, 64], [64, 64]]), SCALE,
                                  k_scales=ks, v_scales=vs)
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_BLOCK_ID
    tiles.zero_()
    for n in (0, 65, -1):
        pgd.selected_decode_attention(None, q, k, v, tiles, _i32([[64, 64], [64, n]]), SCALE,
                                      k_scales=ks, v_scales=vs)
        assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_CONTEXT


# ------------------------------------------------------------------------ together, as used
def _serving_state(n_kv=4, G=4, bs=16, W=10):
    """Prompts written, their bounds made: what a serving loop holds before its first step."""
    lens = [333, 20, 150]
    c = bsc.make_cache([0, 0, 0], n_kv, bs, room=400, seed=11)
    kn, vn = _rows(sum(lens), n_kv, 21), _rows(sum(lens), n_kv, 22)
    st = _starts(lens)
    k, v, ks, vs, tables, _ = c.cuda()
    pgd.kv_append_fp8b(kn.cuda(), vn.cuda(), k, v, ks, vs, tables, _i32([0, 0, 0]),
                       token_starts=_i32(st), max_tokens=max(lens))
    bsc.append(c, kn, vn, [0, 0, 0], st)
    bounds, scales = _empty_bounds(c)
    pgd.block_bounds(bounds, scales, k, tables, _i32(lens), k_scales=ks)
    s = dict(c=c, lens=lens, k=k, v=v, ks=ks, vs=vs, tables=tables, bounds=bounds, scales=scales,
             q=torch.zeros(3, n_kv * G, 128, dtype=torch.bfloat16, device="cuda"),
             kn=torch.zeros(3, n_kv, 128, dtype=torch.bfloat16, device="cuda"),
             vn=torch.zeros(3, n_kv, 128, dtype=torch.bfloat16, device="cuda"),
             ctx=_i32(lens), pos=_i32(lens), W=W,
             out=torch.zeros(3, n_kv * G, 128, dtype=torch.bfloat16, device="cuda"),
             tiles=torch.zeros(3, n_kv, W, dtype=torch.int32, device="cuda"),
             tokens=torch.zeros(3, n_kv, dtype=torch.int32, device="cuda"),
             ws=pgd.make_block_workspace(3, n_kv * G, n_kv))
    return s


def _serving_step(s):
    """One decode step of one layer: positions from lengths, append, bounds, sparse attention."""
    s["pos"].copy_(s["ctx"])
    s["ctx"].add_(1)
    pgd.kv_append_fp8b(s["kn"], s["vn"], s["k"], s["v"], s["ks"], s["vs"], s["tables"], s["pos"])
    pgd.block_bounds(s["bounds"], s["scales"], s["k"], s["tables"], s["ctx"], positions=s["pos"],
                     max_tokens=1, k_scales=s["ks"])
    pgd.sparse_decode_attention(s["out"], s["q"], s["k"], s["v"], s["bounds"], s["scales"],
                                s["tables"], s["ctx"], s["tiles"], s["tokens"], 1, 2, SCALE,
                                k_scales=s["ks"], v_scales=s["vs"], workspace=s["ws"])


@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(graph):
    """Prompts, then 20 decode steps (across block borders), called or replayed from one graph:
    every step's cache, selection and output against the plain forms."""
    s = _serving_state()
    c, n_kv = s["c"], 4
    if graph:
        before = [s[n].clone() for n in ("ctx", "k", "v", "ks", "vs", "bounds", "scales")]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _serving_step(s)
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            _serving_step(s)
        for n, x in zip(("ctx", "k", "v", "ks", "vs", "bounds", "scales"), before):
            s[n].copy_(x)
    for i in range(20):
        q, kn, vn = bsc.make_query(3, 16, seed=100 + i), _rows(3, 4, 200 + i), _rows(3, 4, 300 + i)
        s["q"].copy_(q), s["kn"].copy_(kn), s["vn"].copy_(vn)
        captured.replay() if graph else _serving_step(s)
        bsc.append(c, kn, vn, [n + i for n in s["lens"]], [0, 1, 2, 3])
        c.ctx = [n + i + 1 for n in s["lens"]]
        if i in (0, 3, 11, 12, 19):
            _same_pools(c, s["k"], s["v"], s["ks"], s["vs"])
            want, ws = _want_bounds(c, s["bounds"].cpu(), s["scales"].cpu(),
                                    [(b, j, n) for b, n in enumerate(c.ctx)
                                     for j in range(-(-n // 16))])
            assert torch.equal(s["bounds"].cpu(), want) and torch.equal(s["scales"].cpu(), ws)
            chosen = _chosen(c, q, want, ws, 10, 1, 2)
            tiles, tokens = _want_tiles(c, chosen, 10)
            assert torch.equal(s["tiles"].cpu(), tiles) and torch.equal(s["tokens"].cpu(), tokens)
            bsc.close(s["out"], *bsc.selected(c, q, chosen, SCALE), label="step %d" % i)


def test_prepared_calls():
    s = _serving_state()
    q = bsc.make_query(3, 16).cuda()
    want = pgd.paged_decode_attention_fp8b(None, q, s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                           s["ctx"], SCALE)
    call = pgd.prepare("paged_decode_attention_fp8b", None, q, s["k"], s["v"], s["ks"], s["vs"],
                       s["tables"], s["ctx"], SCALE)
    assert torch.equal(call(), want) and torch.equal(call(), want)
    args = (q, s["k"], s["v"], s["bounds"], s["scales"], s["tables"], s["ctx"], s["tiles"],
            s["tokens"], 1, 2, SCALE)
    want = pgd.sparse_decode_attention(None, *args, k_scales=s["ks"], v_scales=s["vs"])
    call = pgd.prepare("sparse_decode_attention", None, *args, k_scales=s["ks"], v_scales=s["vs"])
    assert torch.equal(call(), want)
    rows = _rows(3, 4, 1).cuda()
    ctx = s["ctx"] + 1
    call = pgd.prepare("append_decode_attention_fp8b", None, q, rows, rows, s["k"], s["v"],
                       s["ks"], s["vs"], s["tables"], ctx, SCALE)
    got = call().clone()
    assert torch.equal(got, pgd.paged_decode_attention_fp8b(
        None, q, s["k"], s["v"], s["ks"], s["vs"], s["tables"], ctx, SCALE))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace and outputs, give what they give alone."""
    s = _serving_state()
    q = [bsc.make_query(3, 16, seed=i).cuda() for i in range(2)]
    ref = [pgd.paged_decode_attention_fp8b(None, x, s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                           s["ctx"], SCALE, num_splits=3) for x in q]
    ws = [pgd.make_block_workspace(3, 16, 4, 3) for _ in q]
    out = [torch.zeros_like(x) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, o, st in zip(q, ws, out, streams):
            pgd.paged_decode_attention_fp8b(o, x, s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                            s["ctx"], SCALE, num_splits=3, workspace=w, stream=st)
    torch.cuda.synchronize()
    for o, r in zip(out, ref):
        assert torch.equal(o, r)


def test_one_workspace_for_calls_of_different_sizes():
    """Two captured graphs and eager calls of other sizes share a workspace, every call split so
    that partial states lie in it: each gives what it gives with one of its own."""
    cases = []
    for i, (ctx, n_kv, G, bs, fp8) in enumerate([([900, 40], 2, 4, 16, True),
                                                 ([700] * 9, 8, 8, 32, True),
                                                 ([1500, 33, 64], 5, 1, 16, False)]):
        c = bsc.make_cache(ctx, n_kv, bs, fp8=fp8, seed=i)
        q = bsc.make_query(len(ctx), n_kv * G, seed=i).cuda()
        k, v, ks, vs, tables, lens = c.cuda()
        W = 20
        tiles = torch.zeros(len(ctx), n_kv, W, dtype=torch.int32, device="cuda")
        tiles += torch.arange(W, device="cuda", dtype=torch.int32)
        tokens = torch.full((len(ctx), n_kv), W * bs, dtype=torch.int32, device="cuda")
        k.copy_(torch.where(torch.isnan(k), 0, k) if not fp8 else torch.where(k == 0x7F, 0, k))
        v.copy_(torch.where(torch.isnan(v), 0, v) if not fp8 else torch.where(v == 0x7F, 0, v))

        def call(ws, q=q, k=k, v=v, ks=ks, vs=vs, tiles=tiles, tokens=tokens, tables=tables,
                 lens=lens, fp8=fp8):
            a = pgd.selected_decode_attention(None, q, k, v, tiles, tokens, SCALE, k_scales=ks,
                                              v_scales=vs, num_splits=5, workspace=ws)
            if not fp8:
                return a, a
            return a, pgd.paged_decode_attention_fp8b(None, q, k, v, ks, vs, tables, lens, SCALE,
                                                      num_splits=3, workspace=ws)

        cases.append((call, call(None)))
    ws = pgd.make_block_workspace(9, 64, 8, 5)
    graphs = []
    for call, _ in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call(ws)
        graphs.append((g, got))
    for _ in range(3):
        for (g, got), (_, want) in zip(graphs, cases):
            g.replay()
            again = cases[2][0](ws)
            torch.cuda.synchronize()
            for x, y in zip(got + again, want + cases[2][1]):
                assert torch.equal(x, y)


def test_binding_refuses_shapes_and_devices():
    s = _serving_state()
    q = bsc.make_query(3, 16).cuda()
    at = (s["ks"], s["vs"], s["tables"], s["ctx"], SCALE)
    with pytest.raises(ValueError, match="k_scales"):
        pgd.paged_decode_attention_fp8b(None, q, s["k"], s["v"], s["ks"][1:], *at[1:])
    with pytest.raises(ValueError, match="block_tables"):
        pgd.paged_decode_attention_fp8b(None, q[:2], s["k"], s["v"], *at)
    with pytest.raises(ValueError, match="v_cache"):
        pgd.paged_decode_attention_fp8b(None, q, s["k"], s["v"][1:], *at)
    with pytest.raises(ValueError, match="contiguous"):
        pgd.paged_decode_attention_fp8b(None, q.transpose(0, 1), s["k"], s["v"], *at)
    with pytest.raises(ValueError, match="max_tokens"):
        pgd.kv_append_fp8b(s["kn"], s["vn"], s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                           s["pos"], token_starts=_i32([0, 1, 2, 3]))
    with pytest.raises(ValueError, match="rows for"):
        pgd.kv_append_fp8b(s["kn"][:2], s["vn"][:2], s["k"], s["v"], s["ks"], s["vs"],
                           s["tables"], s["pos"])
    with pytest.raises(ValueError, match="tile_tokens"):
        pgd.select_blocks(s["tiles"], s["tokens"][:2], q, s["bounds"], s["scales"], s["tables"],
                          s["ctx"], 1, 2, 16)
    with pytest.raises(pgd.PGDError) as e:
        pgd.select_blocks(s["tiles"], s["tokens"], q, s["bounds"], s["scales"], s["tables"],
                          s["ctx"], 9, 2, 16)
    assert e.value.status == _native.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["single_ctx512", "batch16_ctx8192", "ragged64_g8",
                                  "single_ctx131072"])
def test_workload_full_size(name):
    """The workloads of the benchmark, a sample of rows checked: a row is one (sequence, head)."""
    w = inputs.WORKLOADS[name]
    ctx = inputs.context_lengths(w)
    g = torch.Generator(device="cuda").manual_seed(5)
    nblk = [-(-n // w.block_size) for n in ctx]
    NB, MB = sum(nblk), max(nblk)
    perm = torch.randperm(NB, generator=torch.Generator().manual_seed(6)).to(torch.int32)
    tables = torch.full((w.batch, MB), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
    shape = (NB, w.n_kv, w.block_size // 8, 8, 8, 16)
    pools = []
    for _ in range(2):
        pool = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for i in range(0, NB, 4096):
            x = torch.randn(pool[i:i + 4096].shape, generator=g, device="cuda") * 110
            pool[i:i + 4096] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pools.append(pool)
    scales = [torch.exp2(torch.randint(-8, -5, (NB, w.n_kv), generator=g, device="cuda").float())
              for _ in range(2)]
    q = torch.randn(w.batch, w.n_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    got = pgd.paged_decode_attention_fp8b(None, q, *pools, *scales, tables.cuda(), _i32(ctx),
                                          w.scale)
    pick = torch.Generator().manual_seed(7)
    for _ in range(6):
        b = int(torch.randint(w.batch, (1,), generator=pick))
        h = int(torch.randint(w.n_kv, (1,), generator=pick))
        ids = tables[b, :nblk[b]].long().cuda()
        rows = []
        for pool, sc in zip(pools, scales):
            x = torch.from_numpy(bsc.VALUES).cuda()[pool[ids, h].long()]
            x = x * sc[ids, h].double().view(-1, 1, 1, 1, 1)
            rows.append(x.permute(0, 1, 3, 2, 4).reshape(-1, 1, 128)[:ctx[b]].cpu().numpy())
        G = w.n_q // w.n_kv
        hs = slice(h * G, (h + 1) * G)
        bsc.close(got[b, hs], *bsc.attention(q[b, hs].cpu(), *rows, w.scale),
                  label="%s b=%d h=%d" % (name, b, h))
