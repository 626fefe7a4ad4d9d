"""The calls on the block-scaled cache and on selections at the ends of the sizes they take."""
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [65535, 65536, 131071])
@pytest.mark.parametrize("first", [False, True])
def test_bounds_of_more_sequences_than_a_grid_has_rows(B, first):
    """One token a sequence, but for every seventh, which has none: its block keeps its bounds."""
    g = torch.Generator(device="cuda").manual_seed(B)
    k = torch.randn(B, 1, 2, 16, 8, 8, generator=g, device="cuda").to(torch.bfloat16)
    tables = torch.randperm(B, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    ctx = (torch.arange(B, device="cuda") % 7 > 0).to(torch.int32)
    bounds = torch.full((B, 1, 2, 128), -77, dtype=torch.int8, device="cuda")
    scales = torch.full((B, 1), -1.0, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda") if first else None
    pgd.block_bounds(bounds, scales, k, tables, ctx, positions=pos, max_tokens=1)
    has = torch.zeros(B, dtype=torch.bool, device="cuda")
    has[tables[:, 0].long()] = ctx > 0
    x = k[:, 0, 0, :, 0].reshape(B, 128).double()  # slot 0 of every block
    m, e = torch.frexp(x.abs().amax(1))  # m in [1/2, 1); 127 * 2^n = (127/128) * 2^(n + 7)
    e = torch.where(m <= 127 / 128, e - 7, e - 6).double()
    s = torch.where(has, torch.exp2(e), torch.tensor(-1.0, device="cuda").double())
    y = x / torch.exp2(e)[:, None]
    want = torch.stack([torch.floor(y), torch.ceil(y)], 1)
    want = torch.where(has[:, None, None], want, torch.tensor(-77.0, device="cuda").double())
    assert torch.equal(scales[:, 0].double(), s)
    assert torch.equal(bounds[:, 0].double(), want)


def test_attention_at_the_end_of_the_cost_space():
    """B * n_kv * (MB + 24) = 2^31 - 2, every context full: the cuts of the work are computed next to
    the largest 32-bit number.  The tables repeat 64 blocks, so a softmax over those with their
    multiplicities is the reference."""
    B, n_kv, MB, NB = 2046, 21, 49957, 64
    assert B * n_kv * (MB + 24) == 2 ** 31 - 2
    c = bsc.make_cache([NB * 16], n_kv, 16, seed=4, spoil=False)
    k, v, ks, vs, tables, _ = c.cuda()
    row = tables[0, :NB][torch.arange(MB, device="cuda") % NB]
    q = bsc.make_query(B, n_kv).cuda()
    got = pgd.paged_decode_attention_fp8b(None, q, k, v, ks, vs, row.repeat(B, 1),
                                          _i32([MB * 16]).repeat(B), SCALE)
    times = torch.full((NB,), MB // NB, dtype=torch.float64)
    times[:MB % NB] += 1
    times = times.repeat_interleave(16).cuda()  # of every token
    kd, vd = (torch.from_numpy(c.rows(x, 0, NB * 16)).cuda() for x in "kv")
    s = torch.einsum("bhd,thd->bht", q.double(), kd) * SCALE
    w = torch.exp(s - s.amax(-1, keepdim=True)) * times
    w /= w.sum(-1, keepdim=True)
    want, mag = (torch.einsum("bht,thd->bhd", w, x) for x in (vd, vd.abs()))
    bsc.close(got, want.cpu().numpy(), mag.cpu().numpy())


@pytest.mark.parametrize("call", ["append", "read"])
def test_ranges_whose_items_pass_32_bits(call):
    """max_tokens as long as a table of 2^20 blocks, 1100 heads: 2.3e9 (block, head, K or V) items of
    one sequence, of which three tokens' exist.  (The write takes blocks in fours: a quarter.)"""
    n_kv, MB = 1100, 1 << 20
    c = bsc.make_cache([18], n_kv, 16, seed=7, spoil=False)
    k, v, ks, vs, tables, _ = c.cuda()
    table = torch.full((1, MB), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = tables[0, :2]
    g = torch.Generator().manual_seed(2)
    rows = [torch.randn(3, n_kv, 128, generator=g).to(torch.bfloat16) for _ in range(2)]
    up = [x.cuda() for x in rows]
    fn = pgd.kv_append_fp8b if call == "append" else pgd.kv_read_fp8b
    fn(*up, k, v, ks, vs, table, _i32([15]), token_starts=_i32([0, 3]), max_tokens=16 * MB)
    if call == "append":
        bsc.append(c, *rows, [15], [0, 3])
        assert torch.equal(bsc.untile8(k.cpu()), c.k) and torch.equal(bsc.untile8(v.cpu()), c.v)
        assert torch.equal(ks.cpu(), c.k_scales) and torch.equal(vs.cpu(), c.v_scales)
    else:
        for which, got in zip("kv", up):
            assert (bsc.f64(got) == c.rows(which, 0, 18)[15:]).all()


@pytest.mark.parametrize("B", [1, 40])
def test_select_from_the_widest_table(B):
    """49152 blocks a sequence, every context full, in one cluster and in more than fit side by
    side."""
    MB, W = 49152, 700
    g = torch.Generator().manual_seed(B)
    lo = torch.randint(-127, 60, (MB, 1, 128), generator=g)
    hi = torch.minimum(lo + torch.randint(0, 150, lo.shape, generator=g), torch.tensor(127))
    bounds = torch.stack([lo, hi], 2).to(torch.int8)
    scales = torch.exp2(torch.randint(-3, 2, (MB, 1), generator=g).float())
    tables = torch.stack([torch.randperm(MB, generator=g) for _ in range(B)]).to(torch.int32)
    q = bsc.make_query(B, 4, seed=B)
    tiles = torch.empty(B, 1, W, dtype=torch.int32, device="cuda")
    tokens = torch.empty(B, 1, dtype=torch.int32, device="cuda")
    pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), tables.cuda(),
                      _i32([MB * 16 - 3]).repeat(B), 2, 5, 16)
    assert (tokens == W * 16 - 3).all()
    for b in range(0, B, 13):
        at = tables[b].long()
        js = bsc.select(q[b], bsc.f64(bounds[at, 0, 0]), bsc.f64(bounds[at, 0, 1]),
                        bsc.f64(scales[at, 0]), W, 2, 5)
        assert torch.equal(tiles[b, 0].cpu(), tables[b, js])


@pytest.mark.parametrize("fp8", [True, False])
def test_pools_past_32_bits_of_bytes(fp8):
    """The last blocks of pools of more than 2^32 bytes: every call gives what it gives on the same
    blocks at the start of small pools."""
    n_kv, G, bs, far = 8, 4, 16, 280000
    lens = [900, 70]
    c = bsc.make_cache(lens, n_kv, bs, fp8=fp8, seed=9, room=20)
    k, v, ks, vs, tables, ctx = c.cuda()
    small = k.shape[0]
    big = [torch.empty((far + small, *k.shape[1:]), dtype=k.dtype, device="cuda") for _ in "kv"]
    assert big[0].nbytes > 1 << 32
    big[0][far:], big[1][far:] = k, v
    big_scales = [None, None]
    if fp8:
        big_scales = [torch.ones(far + small, n_kv, device="cuda") for _ in "kv"]
        big_scales[0][far:], big_scales[1][far:] = ks, vs
    q = bsc.make_query(2, n_kv * G).cuda()
    rows = [torch.randn(2, 9, n_kv, 128, generator=torch.Generator().manual_seed(i)).to(
        torch.bfloat16).cuda() for i in range(2)]
    got = []
    moved = torch.where(tables < 0, tables, tables + far)
    for pools, scales, t, at in [((k, v), (ks, vs), tables, 0), (big, big_scales, moved, far)]:
        kw = dict(k_scales=scales[0], v_scales=scales[1])
        new = ctx.clone()
        res = []
        if fp8:
            pgd.kv_append_fp8b(*rows, *pools, *scales, t, ctx)
            new += 9
            back = [torch.empty_like(x) for x in rows]
            pgd.kv_read_fp8b(*back, *pools, *scales, t, ctx)
            res += back + [pgd.paged_decode_attention_fp8b(None, q, *pools, *scales, t, new, SCALE,
                                                           num_splits=n) for n in (0, 2)]
        NB = pools[0].shape[0]
        bounds = torch.zeros(NB, n_kv, 2, 128, dtype=torch.int8, device="cuda")
        bound_scales = torch.ones(NB, n_kv, device="cuda")
        pgd.block_bounds(bounds, bound_scales, pools[0], t, new, k_scales=scales[0])
        tiles = torch.empty(2, n_kv, 12, dtype=torch.int32, device="cuda")
        tokens = torch.empty(2, n_kv, dtype=torch.int32, device="cuda")
        res.append(pgd.sparse_decode_attention(None, q, *pools, bounds, bound_scales, t, new, tiles,
                                               tokens, 1, 2, SCALE, **kw))
        res += [bounds[at:at + small], bound_scales[at:at + small], tokens,
                torch.where(tiles < 0, tiles, tiles - at * n_kv)]
        got.append(res)
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_calls_of_no_sequences():
    """B = 0 through the binding."""
    c = bsc.make_cache([20], 2, 16, seed=9)
    k, v, ks, vs, tables, ctx = c.cuda()
    none, q = ctx[:0], bsc.make_query(1, 8).cuda()[:0]
    rows = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pgd.kv_append_fp8b(rows, rows, k, v, ks, vs, tables[:0], none)
    pgd.kv_read_fp8b(rows, rows, k, v, ks, vs, tables[:0], none, token_starts=ctx * 0, max_tokens=4)
    out = pgd.paged_decode_attention_fp8b(None, q, k, v, ks, vs, tables[:0], none, SCALE)
    assert out.shape == q.shape
    bounds = torch.zeros(k.shape[0], 2, 2, 128, dtype=torch.int8, device="cuda")
    scales = torch.ones(k.shape[0], 2, device="cuda")
    pgd.block_bounds(bounds, scales, k, tables[:0], none, k_scales=ks)
    tiles = torch.empty(0, 2, 4, dtype=torch.int32, device="cuda")
    tokens = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    pgd.sparse_decode_attention(None, q, k, v, bounds, scales, tables[:0], none, tiles, tokens, 1, 2,
                                SCALE, k_scales=ks, v_scales=vs)


def test_a_shared_block_copied_before_an_append():
    """Two sequences that share their last, begun block: the second takes a copy of its tiles, scales
    and bounds and appends large rows; the first keeps its values, both attend to their own."""
    c = bsc.make_cache([40, 40], 2, 16, seed=12, room=8)
    shared, own = int(c.tables[0, 2]), int(c.tables[1, 2])
    c.tables[1, :2] = c.tables[0, :2]
    k, v, ks, vs, tables, _ = c.cuda()
    bounds = torch.zeros(k.shape[0], 2, 2, 128, dtype=torch.int8, device="cuda")
    bound_scales = torch.ones(k.shape[0], 2, device="cuda")
    pgd.block_bounds(bounds, bound_scales, k, tables[:1], _i32([40]), k_scales=ks)
    for x in (k, v, ks, vs, bounds, bound_scales):
        x[own] = x[shared]
    for x in (c.k, c.v, c.k_scales, c.v_scales):
        x[own] = x[shared]
    before = [x[shared].clone() for x in (k, v, ks, vs, bounds, bound_scales)]
    g = torch.Generator().manual_seed(3)
    rows = [(torch.randn(2, 2, 128, generator=g) * 50).to(torch.bfloat16) for _ in range(2)]
    q = bsc.make_query(2, 8)
    # (the first sequence appends nothing)
    pgd.kv_append_fp8b(*(x.cuda() for x in rows), k, v, ks, vs, tables, _i32([40, 40]),
                       token_starts=_i32([0, 0, 2]), max_tokens=2)
    pgd.block_bounds(bounds, bound_scales, k, tables, _i32([40, 42]), positions=_i32([40, 40]),
                     max_tokens=2, k_scales=ks)
    bsc.append(c, *rows, [40, 40], [0, 0, 2])
    c.ctx = [40, 42]
    for x, y in zip((k, v, ks, vs, bounds, bound_scales), before):
        assert torch.equal(x[shared], y)
    assert torch.equal(bsc.untile8(k.cpu()), c.k) and torch.equal(vs.cpu(), c.v_scales)
    for g_ in range(2):
        lo, hi, s = bsc.bounds(c, 1, 2, g_, 42)
        assert (bounds[own, g_].cpu().numpy() == [lo, hi]).all()
        assert float(bound_scales[own, g_]) == s
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, _i32([40, 42]), SCALE)
    bsc.close(got, *bsc.paged(c, q, SCALE))
