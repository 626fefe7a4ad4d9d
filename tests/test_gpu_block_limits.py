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
