"""Decode attention over a block-scaled cache whose V scales lie far apart: blocks of zeros, which
take the least scale, beside blocks of ordinary and of large values."""
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


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("zeros", ["stages", "blocks", "first", "last"])
@pytest.mark.parametrize("exponent", [-7, 30, 60, 100])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_blocks_of_zeros_beside_large_values(G, bs, zeros, exponent, num_splits):
    """Half of the blocks (or the first or last half of a context) hold zeros with the scale 2^-100
    and about half of the weight; the others' scales are 2^exponent."""
    ctx = [2200, 700]
    c = bsc.make_cache(ctx, 2, bs, seed=G)
    c.v_scales.fill_(2.0 ** exponent)
    for b, n in enumerate(ctx):
        nblk = -(-n // bs)
        for j in range(nblk):
            if {"stages": j * bs // 128 % 2 == 0, "blocks": j % 2 == 0, "first": 2 * j < nblk,
                    "last": 2 * j >= nblk}[zeros]:
                blk = int(c.tables[b, j])
                c.v[blk] = torch.where(c.v[blk] == bsc.NAN_CODE, c.v[blk], 0)
                c.v_scales[blk] = 2.0 ** -100
    q = bsc.make_query(2, 2 * G)
    k, v, ks, vs, tables, lens = c.cuda()
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE,
                                          num_splits=num_splits)
    bsc.close(got, *bsc.paged(c, q, SCALE))
