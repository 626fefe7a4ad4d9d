"""The 4-bit cache on the GPU: write, read-back and attention against their 64-bit forms."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
BAD_ID, BAD_CTX, BAD_POS = (_native.DEVERR_BAD_BLOCK_ID, _native.DEVERR_BAD_CONTEXT,
                            _native.DEVERR_BAD_POSITION)


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(n, n_kv, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, n_kv, 128, generator=g) * std
    return (x * torch.exp(torch.randn(n, n_kv, 1, generator=g))).to(torch.bfloat16)


def _same(c, k, v, label=""):
    """Pools hold what the plain cache holds, every byte (a zero's sign apart)."""
    for i, p in enumerate((k, v)):
        codes, scales = fp4.unpack(p.cpu().numpy(), i == 1)
        assert (scales == c.scales[i]).all(), label
        nan = np.repeat(scales & 0x7F, 16, -1) == 0x7F  # (their codes say nothing)
        assert ((codes == c.codes[i]) | ((codes | c.codes[i]) == 8) | nan).all(), label


# ----------------------------------------------------------------- write, read
RANGES = [  # (n_kv, bs, positions, tokens)
    (1, 16, [0], [1]),
    (2, 16, [0, 15, 16, 31], [16, 1, 17, 2]),
    (8, 32, [3, 30, 0, 64], [70, 5, 0, 32]),
    (3, 32, [100, 0, 17], [1, 200, 15]),
    (10, 16, [7, 129, 40], [1, 1, 1]),
]


@pytest.mark.parametrize("case", RANGES, ids=str)
@pytest.mark.parametrize("S", [(1.0, 1.0), (0.5, 4.0), (2.0 ** -32, 2.0 ** 32)], ids=str)
def test_append_and_read(case, S):
    n_kv, bs, pos, n = case
    c = fp4.Cache([p + t for p, t in zip(pos, n)], n_kv, bs, seed=3, S=S)
    k, v, tables, _ = c.cuda()
    starts = [0] + np.cumsum(n).tolist()
    new = [_rows(starts[-1], n_kv, 5 + i, std=S[i]) for i in range(2)]
    if starts[-1] > 3:
        new[0][1, 0, 5], new[1][2, -1, 100] = 0.0, -0.0
        new[0][0, 0, 16:32] = 0
    pgd.kv_append_fp4(new[0].cuda(), new[1].cuda(), k, v, tables, _i32(pos),
                      token_starts=_i32(starts), max_tokens=max(n), k_scale=S[0], v_scale=S[1])
    c.append(*new, pos, starts)
    _same(c, k, v)
    room = 3  # rows that belong to no sequence
    out = [torch.full((starts[-1] + room, n_kv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
           for _ in range(2)]
    pgd.kv_read_fp4(*out, k, v, tables, _i32(pos), token_starts=_i32(starts), max_tokens=max(n),
                    k_scale=S[0], v_scale=S[1])
    for i, got in enumerate(out):
        want = np.concatenate([c.rows(i, b, p + t, p) for b, (p, t) in enumerate(zip(pos, n))])
        assert (bsc.f64(got)[:starts[-1]] == want).all()
        assert (got[starts[-1]:] == 7.0).all()


@pytest.mark.parametrize("bs", [16, 32])
def test_append_without_starts(bs):
    c = fp4.Cache([40, 9, 70], 2, bs, seed=4, room=9)
    k, v, tables, _ = c.cuda()
    for T in (1, 6):
        pos = c.ctx
        new = [_rows(3 * T, 2, 8 + T + i) for i in range(2)]
        shaped = [x.view(3, T, 2, 128).cuda() if T > 1 else x.cuda() for x in new]
        pgd.kv_append_fp4(*shaped, k, v, tables, _i32(pos), **fp4.scales_kw(c))
        c.append(*new, pos, [0, T, 2 * T, 3 * T])
        c.ctx = [p + T for p in pos]
        _same(c, k, v, str(T))
    out = [torch.empty(3, 7, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = [p - 7 for p in c.ctx]
    pgd.kv_read_fp4(*out, k, v, tables, _i32(at), **fp4.scales_kw(c))
    for i, got in enumerate(out):
        assert (bsc.f64(got) == np.stack([c.rows(i, b, p + 7, p) for b, p in enumerate(at)])).all()


def test_every_quotient_next_to_a_tie():
    """Values at, just above and just below every quotient where a code changes, for every
    significand of a scale: 16 dims whose first sets the scale."""
    rows = []
    for m in range(8):                      # scale (1 + m / 8)
        s = 1 + m / 8
        top = torch.tensor(6 * s, dtype=torch.bfloat16)
        for tie in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            x = torch.tensor([tie * s], dtype=torch.bfloat16)
            assert float(x) == tie * s
            bits = x.view(torch.int16)
            near = torch.cat([bits - 2, bits - 1, bits, bits + 1, bits + 2]).view(torch.bfloat16)
            rows.append(torch.cat([top[None], near, -near, torch.zeros(5, dtype=torch.bfloat16)]))
    x = torch.stack(rows).view(-1, 1, 128)  # [7][1][8 groups]
    n = len(x)
    for S in (1.0, 2.0 ** -7):
        c = fp4.Cache([n], 1, 16, seed=1, S=(S, S))
        k, v, tables, _ = c.cuda()
        new = (x.float() * S).to(torch.bfloat16)
        pgd.kv_append_fp4(new.cuda(), new.cuda(), k, v, tables, _i32([0]),
                          token_starts=_i32([0, n]), max_tokens=n, k_scale=S, v_scale=S)
        c.append(new, new, [0], [0, n])
        _same(c, k, v)


def test_scales_next_to_a_tie():
    """Largest values at and next to 6 times the quotients where a scale changes, subnormal and
    saturating scales among them."""
    got = []
    for e in (-9, -8, -7, -6, 0, 5, 8):
        for m in range(16):
            t = 6 * (1 + m / 16 + 1 / 32) * 2.0 ** e
            x = torch.tensor([t], dtype=torch.bfloat16).view(torch.int16)
            got += [x + d for d in (-1, 0, 1)]
    got += [torch.tensor([y], dtype=torch.bfloat16).view(torch.int16)
            for y in (0.0, 1e-38, 0.005, 0.0117, 2688.0, 2700.0, 1e5, 3e38, float("inf"))]
    top = torch.cat(got).view(torch.bfloat16)
    top = top[:len(top) // 8 * 8]
    x = torch.zeros(len(top), 16, dtype=torch.bfloat16)
    x[:, 3], x[:, 7], x[:, 11] = -top, top / 3, top / 7
    x = x.view(-1, 1, 128)
    n = len(x)
    c = fp4.Cache([n], 1, 32, seed=1, S=(1.0, 1.0))
    k, v, tables, _ = c.cuda()
    pgd.kv_append_fp4(x.cuda(), x.cuda(), k, v, tables, _i32([0]), token_starts=_i32([0, n]),
                      max_tokens=n)
    c.append(x, x, [0], [0, n])
    _same(c, k, v)


def test_values_that_are_not_finite():
    x = _rows(20, 2, 3)
    x[3, 0, 17], x[4, 1, 127], x[5, 0, 0] = float("nan"), float("inf"), -float("inf")
    x[6, 1, 40], x[6, 1, 41] = float("nan"), float("inf")
    c = fp4.Cache([20], 2, 16, S=(1.0, 1.0))
    k, v, tables, _ = c.cuda()
    pgd.kv_append_fp4(x.cuda(), x.cuda(), k, v, tables, _i32([0]), token_starts=_i32([0, 20]),
                      max_tokens=20)
    c.append(x, x, [0], [0, 20])
    _same(c, k, v)
    out = [torch.empty(20, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pgd.kv_read_fp4(*out, k, v, tables, _i32([0]), token_starts=_i32([0, 20]), max_tokens=20)
    for i, got in enumerate(out):
        assert np.array_equal(bsc.f64(got), c.rows(i, 0, 20), equal_nan=True)


def test_append_token_by_token_is_append_at_once():
    n, n_kv = 75, 3
    new = [_rows(n, n_kv, 11 + i).cuda() for i in range(2)]
    pools = []
    for step in (n, 1, 7):
        c = fp4.Cache([n], n_kv, 32, seed=6)
        k, v, tables, _ = c.cuda()
        for p in range(0, n, step):
            m = min(step, n - p)
            pgd.kv_append_fp4(new[0][p:p + m], new[1][p:p + m], k, v, tables, _i32([p]),
                              token_starts=_i32([0, m]), max_tokens=step, **fp4.scales_kw(c))
        pools.append((k, v))
    for k, v in pools[1:]:
        assert torch.equal(k, pools[0][0]) and torch.equal(v, pools[0][1])


def test_bad_ranges_write_nothing_and_are_flagged():
    c = fp4.Cache([40, 40, 40], 2, 16, seed=2, room=24)
    k, v, tables, _ = c.cuda()
    new = [_rows(12, 2, 20 + i).cuda() for i in range(2)]
    kw = dict(max_tokens=4, **fp4.scales_kw(c))

    def run(pos, starts, t=tables):
        pgd.kv_append_fp4(*new, k, v, t, _i32(pos), token_starts=_i32(starts), **kw)

    for pos, starts in [([-1, -1, -1], [0, 4, 8, 12]), ([61, 62, 63], [0, 4, 8, 12]),
                        ([0, 0, 0], [-1, -1, -1, -5]), ([0, 0, 0], [13, 14, 15, 16]),
                        ([0, 0, 0], [12, 8, 4, 0]), ([0, 0, 0], [0, 5, 10, 15])]:
        run(pos, starts)
        assert pgd.device_errors(clear=True) == BAD_POS, (pos, starts)
        _same(c, k, v, str((pos, starts)))
    for bad in (-1, c.NB, 2 ** 31 - 1):
        t = tables.clone()
        t[:, 2] = bad
        run([40, 40, 40], [0, 4, 8, 12], t)
        assert pgd.device_errors(clear=True) == BAD_ID
        _same(c, k, v, str(bad))


# ------------------------------------------------------------------ attention
CASES = [  # (n_q, n_kv, bs, contexts)
    (4, 4, 16, [1]), (16, 4, 16, [33, 200, 513]), (16, 2, 32, [31, 32, 33, 700]),
    (64, 8, 32, [129, 1000, 32]), (8, 1, 16, [300, 5]), (8, 1, 32, [4000, 3]),
    (2, 2, 16, [9000]), (12, 3, 16, [1400, 77, 512, 16, 640, 1, 129]),
    (20, 10, 32, [17] * 40 + [400, 90]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_attention(case, num_splits):
    n_q, n_kv, bs, ctx = case
    c = fp4.Cache(ctx, n_kv, bs, seed=n_q + bs)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(len(ctx), n_q)
    ws = pgd.make_fp4_workspace(len(ctx), n_q, n_kv, num_splits)
    got = [pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, lens, SCALE,
                                          num_splits=num_splits, workspace=ws, **fp4.scales_kw(c))
           for _ in range(3)]
    want, tol = fp4.bounds_of(c, q, SCALE)
    err = np.abs(bsc.f64(got[0]) - want) / tol
    assert np.isfinite(err).all() and err.max() <= 1, err.max()
    assert all(torch.equal(x, got[0]) for x in got[1:])
    assert not ws.view(torch.int32)[:65536].any()  # (the counters)


def _over_few_blocks(ctx, n_kv, bs, blocks=64, seed=3):
    """A cache whose sequences read the same few blocks, each from a place of its own, over and over."""
    c = fp4.Cache([blocks * bs], n_kv, bs, seed=seed)
    r = np.random.default_rng(seed)
    MB = -(-max(ctx) // bs)
    held = c.tables[0, :blocks]
    c.tables = np.stack([held[(np.arange(MB) + r.integers(blocks)) % blocks] for _ in ctx])
    c.ctx = list(ctx)
    return c


PATHS = [  # (n_q, n_kv, bs, sequences, shortest, longest context)
    # clusters of 16, of 8, of 4
    (8, 1, 16, 1, 1025, 1025), (18, 9, 32, 1, 8192, 8192), (3, 3, 16, 3, 1, 2000),
    (2, 2, 32, 19, 1, 40), (16, 2, 16, 19, 1, 900), (8, 1, 32, 30, 1, 5000),
    (8, 8, 16, 1, 1024, 1024), (20, 5, 16, 4, 129, 129),
    (3, 3, 32, 13, 385, 500), (48, 6, 16, 19, 1, 600), (8, 2, 32, 40, 1, 1500),
    # whole units of 4, 8 and 16 warps
    (40, 10, 16, 4, 30, 384), (24, 6, 16, 20, 1, 380), (4, 2, 16, 700, 1, 90), (32, 8, 32, 90, 1, 384),
    (8, 8, 16, 80, 1, 30),
    (1, 1, 32, 2048, 1, 70), (8, 8, 32, 40, 1, 4000),
    (8, 8, 16, 30, 1, 2000), (16, 2, 32, 100, 1, 700), (4, 1, 16, 300, 1, 500),
    (16, 8, 16, 15, 1500, 2700), (19, 19, 32, 8, 2500, 2600),
    # parts through the workspace: few sequences, up to 128, more; 16 warps; three waves
    (24, 6, 16, 12, 1, 4000), (8, 2, 16, 33, 1, 8300), (4, 1, 32, 128, 1, 5000),
    (4, 1, 16, 129, 1, 5000), (4, 2, 16, 700, 1, 4200), (1, 1, 32, 2048, 1, 4200),
    (8, 1, 16, 1, 98000, 98000), (8, 4, 32, 2, 30000, 40000),
    (32, 4, 16, 20, 20000, 46000), (10, 10, 32, 31, 20000, 21000), (8, 8, 16, 128, 1, 20000),
    (8, 8, 16, 24, 15000, 40000),
    (4, 4, 16, 60, 1, 3500),
    # clusters of 16 CTAs of 16 warps, and few units through the workspace
    (8, 1, 16, 1, 20000, 20000), (4, 2, 32, 2, 1, 30000), (16, 4, 16, 1, 32768, 32768),
    (8, 1, 16, 1, 60000, 60000), (2, 2, 32, 2, 100, 90000), (6, 6, 16, 1, 9000, 9000),
]


@pytest.mark.parametrize("case", PATHS, ids=str)
def test_attention_of_every_size(case):
    n_q, n_kv, bs, B, lo, hi = case
    ctx = np.random.default_rng(n_q + B).integers(lo, hi + 1, B)
    ctx[B // 2] = hi
    ctx[B // 3] = lo if B > 1 else hi
    c = _over_few_blocks(ctx.tolist(), n_kv, bs)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(B, n_q)
    ws = pgd.make_fp4_workspace(B, n_q, n_kv)
    out = [torch.full((B, n_q, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for x in out[:2]:
        pgd.paged_decode_attention_fp4(x, q.cuda(), k, v, tables, lens, SCALE, workspace=ws,
                                       **fp4.scales_kw(c))
    assert torch.equal(*out[:2])
    assert not ws.view(torch.int32)[:65536].any()  # (the counters)
    pgd.paged_decode_attention_fp4(out[2], q.cuda(), k, v, tables, lens, SCALE, num_splits=1,
                                   **fp4.scales_kw(c))
    some = {0, B // 3, B // 2, B - 1} | set(range(0, B, max(1, B // (20 if hi < 3000 else 6))))
    for b in sorted(some):
        n = int(ctx[b])
        want, tol = fp4.bound(bsc.f64(q[b]), c.rows(0, b, n), c.rows(1, b, n), SCALE)
        for x in (out[0], out[2]):
            err = np.abs(bsc.f64(x[b]) - want) / tol
            assert np.isfinite(err).all() and err.max() <= 1, (b, n, err.max())


@pytest.mark.parametrize("ctx", [[5, 3000], [700, 40, 1]], ids=str)
def test_a_table_much_wider_than_its_contexts(ctx):
    """Also contexts beside a table of more entries, none of which is read (they hold no ids)."""
    for G in (1, 4, 8):
        c = fp4.Cache(ctx, 2, 16, seed=4 + G)
        k, v, tables, lens = c.cuda()
        wide = torch.full((len(ctx), 9000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        wide[:, :tables.shape[1]] = torch.where(tables < 0, wide[:, :tables.shape[1]], tables)
        q = bsc.make_query(len(ctx), 2 * G)
        want, tol = fp4.bounds_of(c, q, SCALE)
        for t in (wide, wide[:, :tables.shape[1]].contiguous()):
            for splits in (0, 2, 300):
                got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, t, lens, SCALE,
                                                     num_splits=splits, **fp4.scales_kw(c))
                assert (np.abs(bsc.f64(got) - want) <= tol).all()


@pytest.mark.parametrize("ctx,MB", [([33, 200], 13), ([1500, 33], 94), ([33, 700, 200], 1200)], ids=str)
@pytest.mark.parametrize("what", ["k", "v", "q"])
def test_nan_stays_with_its_head_and_dims(ctx, MB, what):
    """A NaN scale of the last token of head 1 (alone in its step), or a NaN or infinity of a query,
    reaches what the formula says and no more."""
    G, n_kv = 2, 3
    c = fp4.Cache(ctx, n_kv, 16, seed=6)
    q = bsc.make_query(len(ctx), G * n_kv)
    b = ctx.index(33)
    hit = np.zeros((len(ctx), G * n_kv, 128), bool)
    if what == "q":
        q[b, 1, 9], q[b, 4, 77] = float("nan"), float("inf")
        hit[b, 1] = hit[b, 4] = True
    else:
        i = "kv".index(what)
        c.scales[i][c.tables[b, 2], 1, 0, 3] = 0x7F
        if what == "k":
            hit[b, 2:4] = True
        else:
            hit[b, 2:4, 48:64] = True
    k, v, tables, lens = c.cuda()
    t = torch.full((len(ctx), MB), -1, dtype=torch.int32, device="cuda")
    t[:, :tables.shape[1]] = tables
    with np.errstate(invalid="ignore"):
        want, tol = fp4.bounds_of(c, q, SCALE)
    for splits in (0, 1, 2):
        x = bsc.f64(pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, t, lens, SCALE,
                                                   num_splits=splits, **fp4.scales_kw(c)))
        assert np.isnan(x[hit]).all()
        assert (np.abs(x - want) <= tol)[~hit].all()


@pytest.mark.parametrize("MB", [60, 900])
def test_captured_and_on_two_streams(MB):
    """Captured calls of two shapes on two streams at once, replayed over new contents and lengths."""
    sides = []
    for n_kv, ctx in [(1, [400, 900]), (6, [30, 800, 1, 64, 950, 333, 17])]:
        c = fp4.Cache(ctx, n_kv, 16, seed=n_kv)
        k, v, tables, lens = c.cuda()
        t = torch.full((len(ctx), MB), -1, dtype=torch.int32, device="cuda")
        t[:, :tables.shape[1]] = tables
        q = bsc.make_query(len(ctx), 4 * n_kv)
        stream = torch.cuda.Stream()
        qd, out = q.cuda(), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
        ws = pgd.make_fp4_workspace(len(ctx), 4 * n_kv, n_kv)
        call = lambda a=(out, qd, k, v, t, lens, SCALE), w=ws, kw=fp4.scales_kw(c): (  # noqa: E731
            pgd.paged_decode_attention_fp4(*a, workspace=w, **kw))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            call()
            graph = torch.cuda.CUDAGraph()
            stream.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                call()
                call()
        sides.append((c, q, qd, lens, out, stream, graph))
    for turn in range(3):
        for c, q, qd, lens, out, stream, graph in sides:
            out.fill_(3.0)
            if turn:
                q.copy_(bsc.make_query(*q.shape[:2], std=0.5 * turn))
                qd.copy_(q)
                c.ctx = [max(1, n - 5) for n in c.ctx]
                lens.copy_(torch.tensor(c.ctx, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for *_, stream, graph in sides:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for c, q, qd, lens, out, stream, graph in sides:
            want, tol = fp4.bounds_of(c, q, SCALE)
            assert (np.abs(bsc.f64(out) - want) <= tol).all()


@pytest.mark.parametrize("n_kv,ctx", [(1, [1100]), (8, [900, 1]), (5, [500] * 20), (8, [40, 7] * 40)],
                         ids=str)
def test_append_then_attend_of_every_size(n_kv, ctx):
    c = fp4.Cache(ctx, n_kv, 16, seed=n_kv)
    k, v, tables, lens = c.cuda()
    B = len(ctx)
    new = [_rows(B, n_kv, 40 + i) for i in range(2)]
    q = bsc.make_query(B, 2 * n_kv)
    got = pgd.append_decode_attention_fp4(None, q.cuda(), new[0].cuda(), new[1].cuda(), k, v, tables,
                                          lens, SCALE, **fp4.scales_kw(c))
    c.append(*new, [n - 1 for n in ctx], list(range(B + 1)))
    _same(c, k, v)
    want, tol = fp4.bounds_of(c, q, SCALE)
    assert (np.abs(bsc.f64(got) - want) <= tol).all()


@pytest.mark.parametrize("std", [1e-30, 2.0 ** -60, 40.0])
def test_queries_of_any_size(std):
    """Scores next to zero, and scores whose softmax is one token's."""
    c = fp4.Cache([700, 45], 2, 16, seed=9)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(2, 8, std=std)
    q[0, 1] = 0
    got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, lens, SCALE,
                                         **fp4.scales_kw(c))
    want, tol = fp4.bounds_of(c, q, SCALE)
    assert (np.abs(bsc.f64(got) - want) <= tol).all()


def test_outputs_that_cancel():
    """Each sequence two heavy tokens whose values are opposite: what is left is the error of the
    weights, and the light tokens."""
    r = np.random.default_rng(4)
    c = fp4.Cache([32, 64, 40], 2, 16, seed=5, S=(1.0, 1.0))
    q = bsc.make_query(3, 2, std=0.25)
    for b, n in enumerate(c.ctx):
        for h in range(2):
            x = bsc.f64(q[b, h])
            heavy = r.choice(n, 2, replace=False)
            for t in range(n):
                blk, s = c.tables[b, t // 16], t % 16
                row = np.sign(x) * (3.0 if t in heavy else -3.0)
                c.codes[0][blk, h, s], c.scales[0][blk, h, s] = [
                    y[0] for y in fp4.quantise(row[None], 1.0)]
            one = r.standard_normal((1, 128)) * 50
            for t, sign in zip(heavy, (1, -1)):
                blk, s = c.tables[b, t // 16], t % 16
                cc, ss = fp4.quantise(sign * one, 1.0)
                c.codes[1][blk, h, s], c.scales[1][blk, h, s] = cc[0], ss[0]
    k, v, tables, lens = c.cuda()
    want, tol = fp4.bounds_of(c, q, SCALE)
    for splits in (0, 1, 2):
        got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, lens, SCALE,
                                             num_splits=splits)
        assert (np.abs(bsc.f64(got) - want) <= tol).all()


def test_rising_scores_move_the_reference():
    """Scores that rise by 3 powers of two a token, to 2^600 times the first weight: every step
    moves the reference, weights before it vanish."""
    n = 200
    c = fp4.Cache([n], 1, 16, seed=8, S=(1.0, 1.0))
    q = torch.ones(1, 4, 128, dtype=torch.bfloat16)
    q[0, 1], q[0, 2], q[0, 3] = -1, 0.5, 0.001
    for t in range(n):
        blk, s = c.tables[0, t // 16], t % 16
        x = np.full((1, 128), 3 * np.log(2) * t / 128 / SCALE)
        cc, ss = fp4.quantise(bsc.f64(torch.from_numpy(x).to(torch.bfloat16)), 1.0)
        c.codes[0][blk, 0, s], c.scales[0][blk, 0, s] = cc[0], ss[0]
    k, v, tables, lens = c.cuda()
    want, tol = fp4.bounds_of(c, q, SCALE)
    for splits in (0, 1, 5):
        got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, lens, SCALE,
                                             k_scale=1.0, v_scale=1.0, num_splits=splits)
        # (V was quantised with the scale 1 too)
        assert (np.abs(bsc.f64(got) - want) <= tol).all()


@pytest.mark.parametrize("G", [1, 4, 8])
def test_append_then_attend(G):
    ctx = [1, 16, 17, 300, 700]
    c = fp4.Cache(ctx, 2, 16, seed=7 + G)
    k, v, tables, lens = c.cuda()
    new = [_rows(5, 2, 30 + i) for i in range(2)]
    q = bsc.make_query(5, 2 * G)
    kw = fp4.scales_kw(c)
    k2, v2 = k.clone(), v.clone()
    one = pgd.append_decode_attention_fp4(None, q.cuda(), new[0].cuda(), new[1].cuda(), k, v,
                                          tables, lens, SCALE, **kw)
    pgd.kv_append_fp4(new[0].cuda(), new[1].cuda(), k2, v2, tables, lens - 1, **kw)
    two = pgd.paged_decode_attention_fp4(None, q.cuda(), k2, v2, tables, lens, SCALE, **kw)
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(one, two)
    c.append(*new, [n - 1 for n in ctx], list(range(6)))
    _same(c, k, v)
    want, tol = fp4.bounds_of(c, q, SCALE)
    assert (np.abs(bsc.f64(one) - want) <= tol).all()


def test_bad_ids_and_contexts_are_flagged_and_leave_other_sequences_right():
    c = fp4.Cache([100, 90, 200], 2, 16, seed=3)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(3, 8)
    want, tol = fp4.bounds_of(c, q, SCALE)
    for bad in (-1, c.NB, -2 ** 31):
        t = tables.clone()
        t[1, 3] = bad
        got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, t, lens, SCALE,
                                             **fp4.scales_kw(c))
        assert pgd.device_errors(clear=True) == BAD_ID
        assert (np.abs(bsc.f64(got) - want) <= tol)[[0, 2]].all()
    for bad in (0, -5, tables.shape[1] * 16 + 1, 2 ** 31 - 1):
        n = lens.clone()
        n[1] = bad
        got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, n, SCALE,
                                             **fp4.scales_kw(c))
        assert pgd.device_errors(clear=True) == BAD_CTX
        assert (np.abs(bsc.f64(got) - want) <= tol)[[0, 2]].all()
    n = torch.zeros_like(lens)
    pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, tables, n, SCALE, **fp4.scales_kw(c))
    assert pgd.device_errors(clear=True) == BAD_CTX


def test_one_workspace_for_calls_of_all_sizes():
    """Calls in turn on one workspace, the largest's; a block-scaled call of another cache between."""
    ws = None
    got = {}
    for turn in range(2):
        for n_q, n_kv, ctx in [(32, 4, [3000, 5, 900]), (4, 4, [2000]), (64, 8, [600] * 9)]:
            c = fp4.Cache(ctx, n_kv, 16, seed=n_q)
            k, v, tables, lens = c.cuda()
            q = bsc.make_query(len(ctx), n_q).cuda()
            if ws is None:
                n = max(pgd.fp4_workspace_size(9, 64, 8), pgd.block_workspace_size(9, 64, 8))
                ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
            x = pgd.paged_decode_attention_fp4(None, q, k, v, tables, lens, SCALE, workspace=ws,
                                               **fp4.scales_kw(c))
            want, tol = fp4.bounds_of(c, q.cpu(), SCALE)
            assert (np.abs(bsc.f64(x) - want) <= tol).all()
            assert torch.equal(x, got.setdefault(n_q, x))
            b = bsc.make_cache([900, 31], 2, 16, seed=3)
            bk, bv, bks, bvs, bt, bl = b.cuda()
            bq = bsc.make_query(2, 8)
            y = pgd.paged_decode_attention_fp8b(None, bq.cuda(), bk, bv, bks, bvs, bt, bl, SCALE,
                                                num_splits=3, workspace=ws)
            bsc.close(y, *bsc.paged(b, bq, SCALE), p_err=2.0 ** -11)


def test_copy_blocks():
    c = fp4.Cache([64, 64], 3, 16, seed=5)
    k, v, tables, _ = c.cuda()
    src = tables[0, :3].clone()
    dst = tables[1, :3].clone()
    src[1] = dst[1] = -1
    k2, v2 = k.clone(), v.clone()
    for i in (0, 2):
        k2[dst[i].long()], v2[dst[i].long()] = k2[src[i].long()], v2[src[i].long()]
    pgd.copy_blocks(k, v, src, dst)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    dst[0] = -1
    pgd.copy_blocks(k, v, src, dst)
    assert pgd.device_errors(clear=True) == BAD_ID
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_pools_past_32_bits_of_bytes():
    far, n_kv, bs = 520000, 8, 16
    c = fp4.Cache([900, 70], n_kv, bs, seed=9, room=20)
    k, v, tables, lens = c.cuda()
    big = [torch.empty((far + c.NB, *k.shape[1:]), dtype=torch.uint8, device="cuda") for _ in "kv"]
    assert big[0].nbytes > 1 << 32
    big[0][far:], big[1][far:] = k, v
    moved = torch.where(tables < 0, tables, tables + far)
    q = bsc.make_query(2, 32).cuda()
    new = [_rows(2 * 9, n_kv, i).view(2, 9, n_kv, 128).cuda() for i in range(2)]
    got = []
    for pools, t, at in [((k, v), tables, 0), (big, moved, far)]:
        pgd.kv_append_fp4(*new, *pools, t, lens, **fp4.scales_kw(c))
        rows = [torch.empty_like(x) for x in new]
        pgd.kv_read_fp4(*rows, *pools, t, lens, **fp4.scales_kw(c))
        out = pgd.paged_decode_attention_fp4(None, q, *pools, t, lens + 9, SCALE,
                                             **fp4.scales_kw(c))
        got.append([out, *rows, *[p[at:at + c.NB] for p in pools]])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_contexts_at_the_end_of_the_line():
    """B * n_kv * MB * bs just below 2^35, every context full, over tables that repeat 64 blocks."""
    B, n_kv, MB = 63, 4, (1 << 22) + 1
    assert B * n_kv * (MB * 32 // 32) < 1 << 30 and MB * 32 < 2 ** 31
    B = (1 << 30) // (n_kv * MB)
    c = fp4.Cache([64 * 32], n_kv, 32, seed=4)
    k, v, tables, _ = c.cuda()
    row = tables[0, :64][torch.arange(MB, device="cuda") % 64]
    q = bsc.make_query(B, n_kv)
    got = pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, row.repeat(B, 1),
                                         _i32([MB * 32]).repeat(B), SCALE, **fp4.scales_kw(c))
    w = np.full(64 * 32, float(MB // 64))
    w[:32 * (MB % 64)] += 1
    kd, vd = c.rows(0, 0, 2048), c.rows(1, 0, 2048)
    x = bsc.f64(got)
    for b in range(0, B, 9):
        for h in range(n_kv):
            s = kd[:, h] @ bsc.f64(q[b, h]) * SCALE
            p = np.exp(s - s.max()) * w
            p /= p.sum()
            # a warp's share of the line is 2^35 / 2432 tokens, 2^20 products of 16 whose sums may
            # each be cut by 2^-23: an eighth at most
            mag = p @ np.abs(vd[:, h])
            tol = (2.0 ** -8) * np.abs(p @ vd[:, h]) + 2.0 ** -3 * mag
            assert (np.abs(x[b, h] - p @ vd[:, h]) <= tol).all()


def test_empty_calls():
    c = fp4.Cache([20], 2, 16)
    k, v, tables, lens = c.cuda()
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    new = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    none = tables[:0]
    assert pgd.paged_decode_attention_fp4(None, q, k, v, none, lens[:0], SCALE).shape == q.shape
    pgd.kv_append_fp4(new, new, k, v, none, lens[:0])
    pgd.kv_read_fp4(new, new, k, v, tables, lens, token_starts=_i32([0, 0]), max_tokens=5)
    _same(c, k, v)


def test_binding_refuses_tensors_that_do_not_fit():
    c = fp4.Cache([20, 9, 4], 2, 16)
    k, v, t, lens = c.cuda()
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    for args, err in [((x, x[:2], k, v, t, lens), ValueError), ((x, x, k[..., :1100], v, t, lens),
                                                               ValueError),
                      ((x, x, k.float(), v, t, lens), TypeError),
                      ((x[:, :1], x[:, :1], k, v, t, lens), ValueError),
                      ((x, x, k, v[1:], t, lens), ValueError),
                      ((x, x, k, v, t, lens.long()), TypeError),
                      ((x, x, k, v, t, lens[:2]), ValueError),
                      ((x, x, k, v.cpu(), t, lens), ValueError),
                      ((x.transpose(0, 1).contiguous().transpose(0, 1), x, k, v, t, lens),
                       ValueError)]:
        for fn in (pgd.kv_append_fp4, pgd.kv_read_fp4):
            with pytest.raises(err):
                fn(*args)
    for args, err in [((q, q[:, :4], k, v, t, lens), ValueError), ((q, q, k, v[1:], t, lens),
                                                                  ValueError),
                      ((q, q, k, v, t[:2], lens), ValueError), ((q, q.float(), k, v, t, lens),
                                                                TypeError),
                      ((q, q, k, v, t.long(), lens), TypeError)]:
        with pytest.raises(err):
            pgd.paged_decode_attention_fp4(*args, SCALE)
    with pytest.raises(ValueError, match="max_tokens"):
        pgd.kv_append_fp4(x, x, k, v, t, lens, token_starts=_i32([0, 1, 2, 3]))
    with pytest.raises(pgd.PGDError):
        pgd.kv_append_fp4(x, x, k, v, t, lens, k_scale=3.0)
    with pytest.raises(pgd.PGDError):
        pgd.paged_decode_attention_fp4(None, q, k, v, t, lens, SCALE,
                                       workspace=torch.zeros(4096, dtype=torch.uint8,
                                                             device="cuda"))
    _same(c, k, v)
