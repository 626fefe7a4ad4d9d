"""Rotary positions on the GPU against their 64-bit form: rows to rows, and into the paged cache."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _randn(*shape, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def _positions(T, seed=1):
    """Small ones, far ones and the ends of int32."""
    r = np.random.default_rng(seed)
    p = np.concatenate([r.integers(0, 9000, T), r.integers(-2 ** 31, 2 ** 31, T)])
    p[:2] = 0, 1
    p[-2:] = 2 ** 31 - 1, -2 ** 31
    return r.permutation(p)[:T] if T > 4 else p[-T:]


def _close(got, want, tol):
    err = np.abs(bsc.f64(got) - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


HEADS = [  # (d, first, rotary)
    (128, 0, 128), (128, 0, 64), (128, 64, 64), (128, 8, 16), (128, 16, 96), (64, 0, 64),
    (576, 512, 64), (80, 0, 32), (16, 0, 16), (192, 128, 64), (2048, 0, 2048), (2048, 1000, 32)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 5, 130])
def test_rows(heads, interleaved, T):
    d, first, rotary = heads
    n_q, n_kv = (5, 1) if d < 2048 else (2, 1)
    q, k = _randn(T, n_q, d, seed=T), _randn(T, n_kv, d, seed=T + 1)
    pos = _positions(T, T)
    freq = pgd.rope_frequencies(rotary, 10000.0)
    got = pgd.rope(None, None, q.cuda(), k.cuda(),
                   torch.from_numpy(pos).to(torch.int32).cuda(), freq, interleaved=interleaved,
                   first=first, factor=1.25)
    for x, y in zip((q, k), got):
        _close(y, *fp4.turned(bsc.f64(x), pos, freq.tolist(), first, interleaved, 1.25))


@pytest.mark.parametrize("T", [1023, 1024, 1025, 1030])
@pytest.mark.parametrize("d,rotary", [(128, 128), (80, 48)])
def test_rows_of_many_tokens(T, d, rotary):
    q, k = _randn(T, 3, d), _randn(T, 2, d, seed=2)
    pos = _positions(T)
    freq = pgd.rope_frequencies(rotary, 500000.0)
    got = pgd.rope(None, None, q.cuda(), k.cuda(), torch.from_numpy(pos).to(torch.int32).cuda(),
                   freq)
    for x, y in zip((q, k), got):
        _close(y, *fp4.turned(bsc.f64(x), pos, freq.tolist(), 0, False, 1.0))


@pytest.mark.parametrize("T", [7, 1500])
@pytest.mark.parametrize("interleaved", [False, True])
def test_views_of_one_projection_and_in_place(T, interleaved):
    """q and k within one tensor's rows, to other rows and to themselves; heads-first storage too.
    What lies beside them stays as it was."""
    qkv = _randn(T, 6 + 2 + 2, 128, seed=T)
    pos = _positions(T)
    p = torch.from_numpy(pos).to(torch.int32).cuda()
    freq = pgd.rope_frequencies(64)
    kw = dict(interleaved=interleaved, first=32)
    want = fp4.turned(bsc.f64(qkv), pos, freq.tolist(), 32, interleaved, 1.0)
    x = qkv.cuda()
    a, b = pgd.rope(None, None, x[:, :6], x[:, 6:8], p, freq, **kw)
    _close(a, want[0][:, :6], want[1][:, :6])
    _close(b, want[0][:, 6:8], want[1][:, 6:8])
    assert torch.equal(x.cpu(), qkv)
    y = x.clone()
    pgd.rope(y[:, :6], y[:, 6:8], y[:, :6], y[:, 6:8], p, freq, **kw)
    assert torch.equal(y[:, :6], a) and torch.equal(y[:, 6:8], b)
    assert torch.equal(y[:, 8:].cpu(), qkv[:, 8:])
    z = x.transpose(0, 1).contiguous().transpose(0, 1)  # heads first
    wide = torch.full((T, 9, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    pgd.rope(wide[:, 1:7], wide[:, 7:], z[:, :6], z[:, 6:8], p, freq, **kw)
    assert torch.equal(wide[:, 1:7], a) and torch.equal(wide[:, 7:], b) and (wide[:, 0] == 3).all()


def test_q_alone_and_k_alone():
    q = _randn(9, 4, 128).cuda()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    f = pgd.rope_frequencies(128)
    a, none = pgd.rope(None, None, q, None, pos, f)
    b, c = pgd.rope(None, None, q[:, :0], q, pos, f)
    assert none is None and b.shape == (9, 0, 128) and torch.equal(a, c)
    e = pgd.rope(None, None, q[:0], q[:0], pos[:0], f)
    assert e[0].shape == (0, 4, 128)


def test_special_values_stay_in_their_pairs():
    x = _randn(1, 1, 128)
    x[0, 0, 3], x[0, 0, 70] = float("nan"), float("inf")
    f = pgd.rope_frequencies(64)
    got, _ = pgd.rope(None, None, x.cuda(), None, torch.ones(1, dtype=torch.int32, device="cuda"), f)
    got = got.cpu()[0, 0]
    bad = ~torch.isfinite(got)
    assert bad.nonzero().flatten().tolist() == [3, 35, 70]  # (70 is copied)
    assert got[70] == float("inf")


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("T", [1, 64, 1100])
@pytest.mark.parametrize("rotary,first,interleaved", [(128, 0, False), (64, 0, True), (32, 96, False)])
def test_append(bs, T, rotary, first, interleaved):
    n_q, n_kv, NB = 8, 2, T // bs + 4
    r = np.random.default_rng(T)
    qkv = _randn(T, n_q + 2 * n_kv, 128, seed=T).cuda()
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    pos = torch.from_numpy(_positions(T, 3)).to(torch.int32).cuda()
    slots = torch.from_numpy(r.permutation(NB * bs)[:T]).cuda()
    left_out = torch.from_numpy(r.random(T) < 0.2).cuda() if T > 1 else torch.zeros(
        1, dtype=torch.bool, device="cuda")
    slots[left_out] = -1
    f = pgd.rope_frequencies(rotary)
    kw = dict(interleaved=interleaved, first=first, factor=0.75)
    qw, kw_rows = pgd.rope(None, None, q, k, pos, f, **kw)
    pools = [torch.randn(NB, n_kv, bs // 8, 16, 8, 8, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    want = [inputs.untile_pool(p).clone() for p in pools]  # [NB][n_kv][bs][128]
    q_out = torch.full((T, n_q, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    got = pgd.rope_append(q_out, q, k, v, *pools, slots, pos, f, **kw)
    assert got is q_out
    at = slots[~left_out]
    for w, rows in zip(want, (kw_rows, v)):
        w[at // bs, :, at % bs] = rows[~left_out]
    for p, w in zip(pools, want):
        assert torch.equal(inputs.untile_pool(p), w)
    assert torch.equal(q_out[~left_out], qw[~left_out]) and (q_out[left_out] == 5).all()


def test_append_is_rope_and_kv_append():
    """A decode step by positions and tables."""
    lens = [5, 100, 33, 64]
    pb = inputs.make_batch(4, 8, 2, 16, [n + 1 for n in lens], device="cuda", seed=3)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (_randn(4, n, 128, seed=n + i).cuda() for i, n in enumerate((8, 2, 2)))
    f = pgd.rope_frequencies(128, 500000.0, "ramp_wavelength", 8.0, 8192.0, 1.0, 4.0)
    k2, v2 = pb.k_cache.clone(), pb.v_cache.clone()
    qr, kr = pgd.rope(None, None, q, k, pos, f)
    pgd.kv_append(kr, v, k2, v2, pb.block_tables, pos)
    blk = pb.block_tables.gather(1, (pos.long() // 16)[:, None])[:, 0].long()
    got = pgd.rope_append(None, q, k, v, pb.k_cache, pb.v_cache, blk * 16 + pos % 16, pos, f)
    assert torch.equal(got, qr)
    for a, b in ((pb.k_cache, k2), (pb.v_cache, v2)):  # (as bits: unused slots hold NaN)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scattered", [False, True])
def test_many_tokens_are_few_at_a_time(interleaved, scattered):
    """Calls that give a thread a share of many tokens' heads, against the same tokens 50 at a time;
    padding among them."""
    T, n_q, n_kv, bs = 9600, 62, 5, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(T, n_q + 2 * n_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([n_q, n_kv, n_kv], 1)
    places = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, device="cuda").to(torch.int32)
    freq = pgd.rope_frequencies(96, 5000.0)
    NB = T // bs + 2
    slots = (torch.randperm(NB * bs, generator=g, device="cuda")[:T] if scattered else
             torch.arange(T, device="cuda") + 5)
    slots[::7] = -1
    got = []
    for step in (T, 50):
        q_out, k_out = (torch.full((T, n, 128), 3.0, dtype=torch.bfloat16, device="cuda")
                        for n in (n_q, n_kv))
        q_app = torch.full_like(q_out, 3.0)
        kc, vc = (torch.zeros(NB, n_kv, bs // 8, 16, 8, 8, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        for i in range(0, T, step):
            at = slice(i, i + step)
            pgd.rope(q_out[at], k_out[at], q[at], k[at], places[at], freq, interleaved, first=16)
            pgd.rope_append(q_app[at], q[at], k[at], v[at], kc, vc, slots[at], places[at], freq,
                            interleaved, first=16)
        got.append((q_out, k_out, q_app, kc, vc))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    left_out = slots < 0
    assert (got[0][2][left_out] == 3.0).all()
    assert torch.equal(got[0][2][~left_out], got[0][0][~left_out])


def test_append_flags_slots_past_the_pool():
    k_cache = torch.zeros(3, 2, 2, 16, 8, 8, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    x = _randn(4, 2, 128).cuda()
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.tensor([48, 2 ** 62, -2 ** 63, 47], device="cuda")
    out = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pgd.rope_append(out, x, x, x, k_cache, v_cache, slots, pos, pgd.rope_frequencies(128))
    assert pgd.device_errors(clear=True) == _native.DEVERR_BAD_POSITION
    rows = inputs.untile_pool(k_cache)
    assert torch.equal(rows[2, :, 15], x[3]) and rows.abs().sum() == x[3].abs().sum()
    assert torch.equal(out[3], x[3]) and not out[:3].any()


def test_append_into_a_pool_past_32_bits_of_bytes():
    NB, bs = 600000, 16
    k_cache = torch.empty(NB, 2, bs // 8, 16, 8, 8, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.empty_like(k_cache)
    assert k_cache.nbytes > 1 << 32
    x = _randn(3, 2, 128).cuda()
    slots = torch.tensor([NB * bs - 1, NB * bs // 2 + 3, 0], device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    pgd.rope_append(None, x, x, -x, k_cache, v_cache, slots, pos, pgd.rope_frequencies(128))
    for t, s in enumerate(slots.tolist()):
        blk, at = s // bs, s % bs
        assert torch.equal(k_cache[blk, :, at // 8, :, at % 8].reshape(2, 128), x[t])
        assert torch.equal(v_cache[blk, :, at // 8, :, at % 8].reshape(2, 128), -x[t])


def test_binding_refuses_tensors_that_do_not_fit():
    q, k = _randn(3, 8, 128).cuda(), _randn(3, 2, 128).cuda()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = pgd.rope_frequencies(64)
    for a in [(q, k, q, k.float(), pos, f), (q, k, q, k, pos.long(), f), (q, k, q, k, pos, f.int())]:
        with pytest.raises(TypeError):
            pgd.rope(*a)
    for a in [(q, k, q, k[:2], pos, f), (q, None, q, k[..., :64], pos, f), (q, k, q, k, pos[:2], f),
              (q, k, q, None, pos, f), (q, k[:, :1], q, k, pos, f),
              (q, k, q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, f),
              (q[:, :1].expand(3, 8, 128), k, q, k, pos, f), (q[:1].expand(3, 8, 128), k, q, k, pos, f),
              (q, k, q, k.cpu(), pos, f)]:
        with pytest.raises(ValueError):
            pgd.rope(*a)
    for rotary, first in [(24, 0), (64, 4), (64, 72), (0, 0)]:
        with pytest.raises(pgd.PGDError):
            pgd.rope(q, k, q, k, pos, torch.zeros(rotary // 2, dtype=torch.int64, device="cuda"),
                     first=first)
    odd = torch.zeros(3 * 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 8, 128)
    with pytest.raises(pgd.PGDError):
        pgd.rope(None, None, odd, None, pos, f)
    kc = torch.zeros(3, 2, 2, 16, 8, 8, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    for a in [(q, q, k, k[:, :1], kc, kc, slots, pos, f), (q, q, k, k, kc, kc[1:], slots, pos, f),
              (q, q, k, k, kc, kc, slots[:2], pos, f), (q, q[..., :64], k, k, kc, kc, slots, pos, f)]:
        with pytest.raises(ValueError):
            pgd.rope_append(*a)
    with pytest.raises(TypeError):
        pgd.rope_append(q, q, k, k, kc, kc, slots.int(), pos, f)
