"""Block selection with scores at the ends of the range and beyond it."""
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
GUARD = 0x5A5A5A5A


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _case(ctx, n_kv, G, seed):
    """Tables, bounds and scales as a cache of the given contexts has them, and a query."""
    c = bsc.make_cache(ctx, n_kv, 16, fp8=False, seed=seed)
    g = torch.Generator().manual_seed(seed)
    lo = torch.randint(-127, 60, (c.k.shape[0], n_kv, 128), generator=g)
    hi = torch.minimum(lo + torch.randint(0, 150, lo.shape, generator=g), torch.tensor(127))
    scales = torch.exp2(torch.randint(-3, 2, lo.shape[:2], generator=g).float())
    return c, torch.stack([lo, hi], 2).to(torch.int8), scales, bsc.make_query(len(ctx), n_kv * G,
                                                                              seed=seed)


def _select(c, q, bounds, scales, W, first, last):
    """Tiles and tokens of a selection whose outputs lie between guard words."""
    B, n = len(c.ctx), len(c.ctx) * c.n_kv * W
    room = torch.full((n + 512,), GUARD, dtype=torch.int32, device="cuda")
    tiles = room[256:256 + n].view(B, c.n_kv, W)
    tokens = torch.full((B, c.n_kv), -7, dtype=torch.int32, device="cuda")
    pgd.select_blocks(tiles, tokens, q.cuda(), bounds.cuda(), scales.cuda(), c.tables.cuda(),
                      torch.tensor(c.ctx, dtype=torch.int32, device="cuda"), first, last, 16)
    torch.cuda.synchronize()
    assert (room[:256] == GUARD).all() and (room[256 + n:] == GUARD).all()
    return tiles.cpu(), tokens.cpu()


def _check_form(c, tiles, tokens, W, first, last):
    """W different blocks of each context, in its order, the forced ones among them."""
    for b, n in enumerate(c.ctx):
        nblk = -(-n // 16)
        place = {int(t): j for j, t in enumerate(c.tables[b, :nblk])}
        for g in range(c.n_kv):
            t = tiles[b, g]
            assert (t % c.n_kv == g).all()
            js = [place[int(x)] for x in t // c.n_kv]
            assert js == sorted(set(js)) and len(js) == W
            assert js[:first] == list(range(first))
            assert js[W - last:] == list(range(nblk - last, nblk))
            assert int(tokens[b, g]) == (W - 1) * 16 + n - (nblk - 1) * 16


@pytest.mark.parametrize("G", [1, 2, 8])
@pytest.mark.parametrize("ctx", [[1600, 1000], [8192, 5000], [40000, 9000]], ids=str)
@pytest.mark.parametrize("W,first,last", [(20, 0, 1), (62, 2, 8)])
def test_scores_of_queries_that_are_not_finite(ctx, G, W, first, last):
    """One, some and all elements of a query infinite: many scores at the ends of the range beside
    ordinary ones of the other sign.  A selection has its form and stays within its output."""
    c, bounds, scales, q = _case(ctx, 2, G, seed=W + G)
    for k, value in [(1, float("inf")), (40, float("-inf")), (128, float("inf")),
                     (3, float("nan")), (128, 3.3e38)]:
        x = q.clone()
        x[0, :, :k] = value
        x[1, 0, ::max(1, 128 // k)] = value
        tiles, tokens = _select(c, x, bounds, scales, W, first, last)
        _check_form(c, tiles, tokens, W, first, last)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38])
@pytest.mark.parametrize("ctx", [[1600, 1000], [40000, 9000]], ids=str)
def test_scores_of_bounds_that_were_never_made(ctx, value):
    """Scales of blocks that hold whatever their memory held."""
    c, bounds, scales, q = _case(ctx, 2, 2, seed=3)
    g = torch.Generator().manual_seed(4)
    for share in (0.02, 0.4, 1.0):
        s = torch.where(torch.rand(scales.shape, generator=g) < share, torch.tensor(value), scales)
        tiles, tokens = _select(c, q, bounds, s, 30, 1, 2)
        _check_form(c, tiles, tokens, 30, 1, 2)


def _want(c, q, bounds, scales, W, first, last):
    G = q.shape[1] // c.n_kv
    tiles = torch.empty(len(c.ctx), c.n_kv, W, dtype=torch.int32)
    for b, n in enumerate(c.ctx):
        at = c.tables[b, :-(-n // 16)].long()
        for g in range(c.n_kv):
            js = bsc.select(q[b, g * G:(g + 1) * G], bsc.f64(bounds[at, g, 0]),
                            bsc.f64(bounds[at, g, 1]), bsc.f64(scales[at, g]), W, first, last)
            tiles[b, g] = c.tables[b, js] * c.n_kv + g
    return tiles


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("q_exp", [-100, 0, 106, 114, 122])
@pytest.mark.parametrize("s_exp", [-90, 0, 100])
def test_scores_of_any_magnitude(G, q_exp, s_exp):
    """Finite queries and keys from 2^-100 to 2^122, whose scores leave fp32's range at either end;
    the heads of a KV head 2^0 to 2^-7 of the largest: the selection of the 64-bit definition."""
    c, bounds, scales, q = _case([1600, 5000], 2, G, seed=G)
    by_head = torch.arange(2 * G, dtype=torch.float64) % G
    q = (q.double() * torch.exp2(q_exp - by_head)[:, None]).to(torch.bfloat16)
    scales = scales * 2.0 ** s_exp
    tiles, tokens = _select(c, q, bounds, scales, 40, 1, 2)
    assert torch.equal(tiles, _want(c, q, bounds, scales, 40, 1, 2))
    _check_form(c, tiles, tokens, 40, 1, 2)


def test_a_score_that_is_no_number_is_the_lowest():
    c, bounds, scales, q = _case([1600], 1, 2, seed=8)
    scales[c.tables[0, 10:60].long()] = float("nan")
    tiles, tokens = _select(c, q, bounds, scales, 49, 0, 1)
    left = [j for j in range(100) if not 10 <= j < 60]
    assert set(tiles[0, 0].tolist()) <= {int(c.tables[0, j]) for j in left}
    tiles, _ = _select(c, q, bounds, scales, 55, 0, 1)
    assert tiles[0, 0].tolist() == [int(c.tables[0, j]) for j in [*range(15), *range(60, 100)]]


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("ctx", [[1600, 900], [20000, 5000]], ids=str)
def test_scores_that_are_zero_in_many_ways(ctx, G):
    """Blocks of zero bounds, and small bounds that meet few query elements: sums that cancel to 0,
    which tie with those that are 0 throughout."""
    c, bounds, scales, q = _case(ctx, 2, G, seed=20 + G)
    g = torch.Generator().manual_seed(G)
    lo = torch.randint(-1, 2, bounds[:, :, 0].shape, generator=g)
    hi = torch.maximum(lo, torch.randint(-1, 2, lo.shape, generator=g))
    bounds = torch.stack([lo, hi], 2).to(torch.int8)
    bounds[torch.rand(bounds.shape[0], generator=g) < 0.3] = 0
    few = torch.zeros_like(q)
    few[..., 5], few[..., 70], few[..., 71] = 1.0, -1.0, 0.5
    tiles, tokens = _select(c, few, bounds, scales, 40, 1, 2)
    assert torch.equal(tiles, _want(c, few, bounds, scales, 40, 1, 2))
    _check_form(c, tiles, tokens, 40, 1, 2)


def test_heads_far_apart():
    """Eight heads 2^3 apart, the largest with no positive score anywhere: the others decide."""
    c, bounds, scales, q = _case([1600, 5000], 2, 8, seed=33)
    q = (q.double() * torch.exp2(-3.0 * (torch.arange(16) % 8).double())[:, None]).to(torch.bfloat16)
    q[:, ::8] = q[:, ::8].abs()
    bounds = torch.minimum(bounds, torch.tensor(0, dtype=torch.int8))
    tiles, _ = _select(c, q, bounds, scales, 40, 1, 2)
    assert torch.equal(tiles, _want(c, q, bounds, scales, 40, 1, 2))
