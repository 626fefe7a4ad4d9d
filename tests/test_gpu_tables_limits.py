"""Block tables at the ends of the sizes that the calls take."""
import pytest
import torch

import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _outputs(B, N):
    """Of grow_tables, in the order of its arguments."""
    return [_i32([9] * B), _i32([9] * (B + 1)), torch.full((N,), 9, device="cuda"), _i32([9] * N),
            _i32([9] * B), _i32([9] * B), _i32([9] * 4)]


@pytest.mark.parametrize("cut", [1, 5, 8, 9, 256, 511, 512, 513, 700])
def test_a_row_of_the_most_blocks(cut):
    """A row of 2^31 - 1 blocks of one token, grown to its last place and cut: places behind the row's
    end are past 2^31."""
    MB, NB = 2 ** 31 - 1, 800
    tables = torch.full((1, MB), -1, dtype=torch.int32, device="cuda")
    ctx = _i32([MB - cut])
    refs, bits = pgd.make_block_pool(NB)
    all_free = bits.clone()
    out = _outputs(1, 900)
    pgd.grow_tables(tables, ctx, _i32([cut]), refs, bits, 1, *out)
    ids = list(range(cut))
    assert out[6].tolist() == [0, cut, 0, cut] and ctx.tolist() == [MB]
    assert tables[0, MB - cut:].tolist() == ids and refs.tolist() == [1] * cut + [0] * (NB - cut)
    assert out[2].tolist() == ids + [-1] * (900 - cut)
    assert out[3].tolist() == list(range(MB - cut, MB)) + [0] * (900 - cut)
    pgd.trim_tables(tables, ctx, _i32([MB - cut]), refs, bits, 1)
    assert ctx.tolist() == [MB - cut]
    assert not refs.any() and torch.equal(bits, all_free)
    assert int(tables.max()) == -1 == int(tables.min())


@pytest.mark.parametrize("rows", [2, 3, 4, 31, 700])
@pytest.mark.parametrize("N", [16, 9000])  # one CTA, a cluster
@pytest.mark.parametrize("free", [True, False])
def test_sums_of_new_tokens_past_32_bits(rows, N, free):
    """Rows that each fit their table and together make 2^31 tokens and more: refused as too many, whether
    blocks are there or not, and nothing changes."""
    bs, NB = 2 ** 30, 1000
    tables = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    ctx = _i32([0] * rows)
    refs, bits = pgd.make_block_pool(NB)
    if not free:
        refs.fill_(1)
        bits.zero_()
    before = [x.clone() for x in (tables, ctx, refs, bits)]
    out = _outputs(rows, N)
    pgd.grow_tables(tables, ctx, _i32([bs] * rows), refs, bits, bs, *out)
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_POSITION
    assert out[6].tolist() == [2, 0, 0, 0]
    for a, b in zip(before, (tables, ctx, refs, bits)):
        assert torch.equal(a, b)
    assert not out[0].any() and not out[1].any() and (out[2] == -1).all() and not out[3].any()
    assert (out[4] == -1).all()


@pytest.mark.parametrize("free", [2, 3])
def test_the_last_owner_of_a_shared_block_copies_too(free):
    """Three rows of one partly filled block, a token more each: the host allocator, which asks at each
    row's turn, makes two copies; grow_tables makes three, or reports the block that it misses."""
    bs, MB, NB = 16, 2, 1 + free
    host = pgd.BlockAllocator(NB)
    rows = [[-1] * MB for _ in range(3)]
    for pos in range(5):
        host.append_slot(rows[0], pos, bs)
    for b in (1, 2):
        host.fork(rows[0], 5, bs, rows[b])
    shared = rows[0][0]
    refs, bits = pgd.make_block_pool(NB)
    tables = _i32([[0, -1]] * 3)
    refs[0] = 3
    bits[0] &= ~1
    ctx, out = _i32([5] * 3), _outputs(3, 4)
    before = [x.clone() for x in (tables, ctx, refs, bits)]
    copies = [host.append_slot(row, 5, bs) for row in rows]
    assert [src for src, _ in copies] == [shared, shared, -1] and host.num_free == free - 2
    pgd.grow_tables(tables, ctx, _i32([1] * 3), refs, bits, bs, *out)
    if free == 2:
        assert out[6].tolist() == [1, 0, 1, 0]
        for a, b in zip(before, (tables, ctx, refs, bits)):
            assert torch.equal(a, b)
    else:
        assert out[6].tolist() == [0, 3, 0, 3] and out[4].tolist() == [0] * 3
        assert out[5].tolist() == [1, 2, 3] and tables[:, 0].tolist() == [1, 2, 3]
        assert refs.tolist() == [0, 1, 1, 1] and int(bits) == 1 and ctx.tolist() == [6] * 3
