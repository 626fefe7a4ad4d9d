"""The timeout exit of the 4-bit attention's clusters, made to happen on purpose: a CTA that waits for its
peers' states longer than the limit (here 1 ns) reports it, waits for what is on its way and leaves; the
next call is right."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def _limit_restored():
    pgd.device_errors(clear=True)
    yield
    pgd.set_wait_limit_ns(0)
    assert pgd.device_errors(clear=True) == 0


@pytest.mark.parametrize("n_q,n_kv,bs,ctx", [
    (32, 8, 16, [2000]), (4, 4, 32, [5000, 33]),        # 16 CTAs of 4 warps
    (8, 2, 16, [30000, 100]), (6, 6, 32, [9000]),       # 16 of 16
    (32, 8, 16, [512]), (8, 8, 32, [900, 1, 700]),      # 8
    (16, 16, 16, [500, 130, 400]), (64, 8, 32, [700] * 10),  # 4
], ids=str)
def test_timeout_then_normal_call(n_q, n_kv, bs, ctx):
    c = fp4.Cache(ctx, n_kv, bs, seed=n_q)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(len(ctx), n_q)
    call = lambda: pgd.paged_decode_attention_fp4(  # noqa: E731
        None, q.cuda(), k, v, tables, lens, SCALE, **fp4.scales_kw(c))
    pgd.set_wait_limit_ns(1)
    seen = 0
    for _ in range(5):
        call()
        torch.cuda.synchronize()
        seen |= pgd.device_errors(clear=True)
    assert seen == _native.DEVERR_TIMEOUT
    for limit in (0, 2 * 10 ** 9, 500 * 10 ** 3):  # (500 us: not met)
        pgd.set_wait_limit_ns(limit)
        got = call()
        assert pgd.device_errors(clear=True) == 0
        want, tol = fp4.bounds_of(c, q, SCALE)
        assert (np.abs(bsc.f64(got) - want) <= tol).all()
