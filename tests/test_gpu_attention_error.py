"""Decode attention over the block-scaled cache within the bound that attention_error.py derives from
the stated arithmetic, on outputs that cancel and on ordinary ones."""
import pytest
import torch

import attention_error as ae
import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _attend(c, q, num_splits, short):
    """On the tensor cores, or (short) by the fp32 kernel of an automatic call's short contexts."""
    k, v, ks, vs, tables, lens = c.cuda()
    before = pgd.set_short_context_tokens(1024 if short else 0)
    try:
        return pgd.paged_decode_attention_fp8b(None, q.cuda(), k, v, ks, vs, tables, lens, SCALE,
                                               num_splits=num_splits)
    finally:
        pgd.set_short_context_tokens(before)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("num_splits", [0, 1, 2])
def test_outputs_that_cancel(G, bs, num_splits):
    c, q = ae.cancelling_cache(24, 4, G, bs, 5, SCALE)
    ae.check(_attend(c, q, num_splits, False), *ae.bounds_of(c, q, SCALE, False))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 32])
def test_short_outputs_that_cancel(G, bs):
    c, q = ae.cancelling_cache(6, 4, G, bs, 6, SCALE)  # (24 heads: the fp32 kernel's for every G)
    ae.check(_attend(c, q, 0, True), *ae.bounds_of(c, q, SCALE, True))


@pytest.mark.parametrize("case", [
    (4, 4, 16, [1]), (16, 4, 16, [33, 200, 513]), (16, 2, 32, [31, 32, 33, 700]),
    (64, 8, 32, [129, 1000, 32]), (8, 1, 16, [300, 5]), (8, 1, 32, [4000, 3]),
    (2, 2, 16, [9000]), (12, 3, 16, [1400, 77, 512, 16, 640, 1, 129]),
], ids=str)
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_ordinary_outputs(case, num_splits):
    n_q, n_kv, bs, ctx = case
    c = bsc.make_cache(ctx, n_kv, bs, seed=n_q + bs)
    q = bsc.make_query(len(ctx), n_q)
    ae.check(_attend(c, q, num_splits, False), *ae.bounds_of(c, q, SCALE, False))


@pytest.mark.parametrize("case", [
    (4, 4, 16, [1]), (16, 4, 16, [33, 200, 513]), (16, 2, 32, [31, 32, 33, 700]),
    (8, 1, 16, [300, 5]), (8, 8, 16, [2000]), (64, 8, 32, [129, 1000, 32])], ids=str)
def test_ordinary_short_outputs(case):
    n_q, n_kv, bs, ctx = case
    c = bsc.make_cache(ctx, n_kv, bs, seed=n_q + bs)
    q = bsc.make_query(len(ctx), n_q)
    ae.check(_attend(c, q, 0, True), *ae.bounds_of(c, q, SCALE, True))


@pytest.mark.parametrize("G", [1, 4, 8])
def test_selected_outputs_that_cancel(G):
    """Attention over given tiles, both of every sequence's blocks."""
    c, q = ae.cancelling_cache(24, 4, G, 16, 7, SCALE)
    k, v, ks, vs, tables, lens = c.cuda()
    head = torch.arange(4, device="cuda", dtype=torch.int32)
    tiles = (tables[:, None, :2] * 4 + head[:, None]).contiguous()
    tokens = lens[:, None].expand(-1, 4).contiguous()
    got = pgd.selected_decode_attention(None, q.cuda(), k, v, tiles, tokens, SCALE, k_scales=ks,
                                        v_scales=vs, num_splits=1)
    ae.check(got, *ae.bounds_of(c, q, SCALE, False))
