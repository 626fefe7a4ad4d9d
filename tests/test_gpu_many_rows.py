"""Batches of more rows than the attention kernel has threads (the work is cut by a scan in which a
thread then takes several), up to the largest, with contexts that are refused among them."""
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native, inputs

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
D = 128


def _pools(NB, n_kv, bs, fp8, g):
    """(pools and scales as the calls take them, K and V of every tile in 64 bits
    [NB * n_kv][bs][128])."""
    pools, scales, values = [], [], []
    for _ in range(2):
        x = torch.randn(NB, n_kv, bs, D, generator=g)
        if fp8:
            codes = (x * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
            s = torch.exp2(torch.randint(-9, -4, (NB, n_kv), generator=g).float())
            pools.append(bsc.tile8(codes.view(torch.uint8)).cuda())
            scales.append(s.cuda())
            x = codes.double() * s.double()[:, :, None, None]
        else:
            x = x.to(torch.bfloat16)
            pools.append(inputs.tile_pool(x).cuda())
            scales.append(None)
        values.append(x.double().cuda().flatten(0, 1))
    return (*pools, *scales), values


def _attention(q, values, tiles, tokens):
    """q [U][G][128], tiles [U][W], tokens [U] -> (outputs, weighted means of |v|), [U][G][128], row
    by row over its tokens; rows whose tokens are out of range are left 0."""
    k, v = values
    U, G = q.shape[:2]
    bs = k.shape[1]
    out = torch.zeros(U, G, D, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for u in range(U):
        n = int(tokens[u])
        if not 1 <= n <= tiles.shape[1] * bs:
            continue
        at = tiles[u, :-(-n // bs)].long()
        ku, vu = k[at].flatten(0, 1)[:n], v[at].flatten(0, 1)[:n]
        w = torch.softmax(q[u].double() @ ku.T * SCALE, -1)
        out[u], mag[u] = w @ vu, w @ vu.abs()
    return out, mag


def _check(got, want, mag, good):
    bsc.close(got[good], want[good].cpu().numpy(), mag[good].cpu().numpy())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_splits", [0, 1])
@pytest.mark.parametrize("B,n_kv,G", [(171, 3, 1), (128, 10, 4), (256, 8, 8), (2048, 1, 2)])
def test_selected_attention_of_many_rows(B, n_kv, G, num_splits, fp8):
    g = torch.Generator().manual_seed(B + G)
    NB, bs, W, U = 64, 16, 6, B * n_kv
    pools, values = _pools(NB, n_kv, bs, fp8, g)
    tiles = torch.randint(0, NB, (B, n_kv, W), generator=g) * n_kv + torch.arange(n_kv)[:, None]
    tokens = torch.randint(1, W * bs + 1, (U,), generator=g)
    bad = torch.tensor([0, U // 2, U - 1])
    tokens[bad] = torch.tensor([0, W * bs + 1, -3])
    q = bsc.make_query(B, n_kv * G, seed=G)
    out = torch.full((B, n_kv * G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    pgd.device_errors(clear=True)
    pgd.selected_decode_attention(out, q.cuda(), pools[0], pools[1], tiles.to(torch.int32).cuda(),
                                  tokens.to(torch.int32).view(B, n_kv).cuda(), SCALE,
                                  k_scales=pools[2], v_scales=pools[3], num_splits=num_splits)
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_CONTEXT
    want, mag = _attention(q.cuda().view(U, G, D), values, tiles.view(U, W).cuda(), tokens)
    good = torch.ones(U, dtype=torch.bool)
    good[bad] = False
    _check(out.view(U, G, D), want, mag, good.cuda())


@pytest.mark.parametrize("B,n_kv,G,bs", [(513, 1, 4, 16), (1100, 2, 1, 32), (2048, 1, 8, 16)])
@pytest.mark.parametrize("num_splits", [0, 1, 2])
def test_paged_attention_of_many_sequences(B, n_kv, G, bs, num_splits):
    """Mostly short contexts beside a few long ones, the first and the last sequence refused."""
    g = torch.Generator().manual_seed(B)
    NB, MB = 96, 1200 // bs
    pools, values = _pools(NB, n_kv, bs, True, g)
    ctx = torch.randint(1, 60, (B,), generator=g)
    ctx[torch.randint(0, B, (9,), generator=g)] = torch.randint(600, MB * bs, (9,), generator=g)
    ctx[0], ctx[B - 1] = 0, MB * bs + 1
    tables = torch.randint(0, NB, (B, MB), generator=g)
    q = bsc.make_query(B, n_kv * G, seed=G)
    pgd.device_errors(clear=True)
    got = pgd.paged_decode_attention_fp8b(None, q.cuda(), *pools, tables.to(torch.int32).cuda(),
                                          ctx.to(torch.int32).cuda(), SCALE, num_splits=num_splits)
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_CONTEXT
    tiles = (tables[:, None] * n_kv + torch.arange(n_kv)[:, None]).view(B * n_kv, MB)
    tokens = ctx[:, None].expand(-1, n_kv).flatten()
    want, mag = _attention(q.cuda().view(B * n_kv, G, D), values, tiles.cuda(), tokens)
    good = ((tokens >= 1) & (tokens <= MB * bs)).cuda()
    _check(got.view(B * n_kv, G, D), want, mag, good)
