"""Block tables at the ends of the sizes that the calls take."""
import pytest
import torch

import paged_gqa_decode_kv_gb300 as pgd

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
