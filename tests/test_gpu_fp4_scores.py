"""The 4-bit attention where scores are large: a score's size takes nothing from what its distance to the
largest score says."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
SCALE = 2.0 ** -3
CTX = [700, 33, 1200, 260]
SIZES = [10, 18, 21, 23, 24, 26, 27, 28, 30, 36, 60, 100]


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _cache(keys, seed):
    """keys: [sequence][tokens][128], the same for both KV heads."""
    c = fp4.Cache(CTX, 2, 16, seed=seed, S=(1.0, 1.0))
    for b, n in enumerate(CTX):
        codes, scales = fp4.quantise(keys[b], 1.0)
        p = np.arange(n)
        blk = c.tables[b, p // 16]
        for h in range(2):
            c.codes[0][blk, h, p % 16], c.scales[0][blk, h, p % 16] = codes, scales
    return c


def _outputs(c, q):
    k, v, tables, lens = c.cuda()
    wide = torch.full((len(CTX), 800), -1, dtype=torch.int32, device="cuda")
    wide[:, :tables.shape[1]] = tables
    for t in (tables, wide):
        for splits in (0, 1, 3):
            yield bsc.f64(pgd.paged_decode_attention_fp4(None, q.cuda(), k, v, t, lens, SCALE,
                                                         num_splits=splits))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", SIZES)
def test_one_token_has_all_the_weight(size, sign):
    """Scores of about 2^size times 1 to 4 (or -1 to -4) and one half as large again as any other (or half
    as small): the output is its value, rounded to bf16 (2^-8) behind a division and a few roundings."""
    r = np.random.default_rng(size)
    at = [n * (i + 1) // (len(CTX) + 1) for i, n in enumerate(CTX)]
    keys = []
    for n, t in zip(CTX, at):
        x = r.choice([1.0, 1.5, 2.0, 3.0, 4.0], n)
        x[t] = 6.0 if sign > 0 else 0.5
        keys.append(np.repeat(x[:, None], 128, 1))
    c = _cache(keys, size)
    q = torch.full((len(CTX), 8, 128), sign * 2.0 ** (size - 4), dtype=torch.bfloat16)
    q[:, ::3] *= 1.25
    for got in _outputs(c, q):
        for b, t in enumerate(at):
            v = np.repeat(c.rows(1, b, CTX[b])[t], 4, 0)
            assert (np.abs(got[b] - v) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(v)).all(), (b, t)


@pytest.mark.parametrize("size", SIZES)
def test_outputs_stay_between_the_values(size):
    """Scores that differ by little and by much: a mean of values is never outside them."""
    r = np.random.default_rng(size)
    keys = []
    for n in CTX:
        x = np.repeat(r.choice([4.0, 6.0], (n, 1), p=[0.3, 0.7]), 128, 1)
        x[:, 16:32] = r.choice([0.0, 0.5, 1.0, 2.0, 3.0, -1.0], (n, 16))
        keys.append(x)
    c = _cache(keys, size)
    q = torch.randn(len(CTX), 8, 128, generator=torch.Generator().manual_seed(size)).to(torch.bfloat16)
    q[:, :, 40] = 2.0 ** (size + 1)
    q[:, 1::2, 40] *= -1
    for got in _outputs(c, q):
        for b, n in enumerate(CTX):
            v = np.repeat(c.rows(1, b, n), 4, 1)
            room = (2.0 ** -8 + 2.0 ** -10) * np.abs(v).max(0)
            assert (got[b] <= v.max(0) + room).all() and (got[b] >= v.min(0) - room).all(), b
