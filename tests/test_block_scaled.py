"""The block-scaled cache and block-sparse attention without a GPU: the plain forms that the GPU
tests compare with, and every refusal that the host makes before it touches a device."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native


@pytest.fixture(scope="module")
def L():
    from paged_gqa_decode_kv_gb300 import build
    build.build()
    return pgd.lib()


# ------------------------------------------------------------------------------- plain forms
def test_codes_agree_with_the_tensor_type():
    """Every code's value, and the rounding of values in and beyond the range, ties included."""
    c = torch.arange(256, dtype=torch.uint8)
    v = c.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(bsc.VALUES))
    assert np.array_equal(v[~np.isnan(v)], bsc.VALUES[~np.isnan(v)])
    pos = bsc.VALUES[:127]
    x = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, pos * 0.999, np.linspace(-448, 448, 9999)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(bsc.e4m3_codes(x.astype(np.float32)), want)
    assert bsc.e4m3_codes([1e9, -np.inf, np.nan]).tolist() == [0x7E, 0xFE, 0x7F]


@pytest.mark.parametrize("top", [448.0, 127.0])
def test_least_power_of_two(top):
    for a in [0.0, 1e-40, 2.0 ** -90, 1.0, top, top * (1 + 2.0 ** -7), top / 2, 3e38]:
        p = bsc.least_pow2(a, top)
        assert a <= top * p and (p == 2.0 ** -100 or a > top * p / 2)


def test_append_grows_a_scale_and_keeps_earlier_values():
    """A block begun with small values and grown by a large one: the earlier values stay within
    half a step of the new scale."""
    c = bsc.make_cache([5], 1, 16, room=11, spoil=False)
    before = c.rows("k", 0, 5)
    new = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    new[0, 0, 3] = 100.0
    bsc.append(c, new, new, [5], [0, 1])
    s = float(c.k_scales[int(c.tables[0, 0]), 0])
    assert s == 0.25
    step = np.maximum(np.abs(before) * 2.0 ** -4, s * 2.0 ** -10)
    assert (np.abs(c.rows("k", 0, 5) - before) <= step).all()
    assert c.rows("k", 0, 6)[5, 0, 3] == 96.0  # 400, between 384 and 416: to the even 384


def test_selection_bounds_every_left_out_key():
    """No key of a block that is left out has a larger product with a rounded query (times its
    step) than the least selected score."""
    c = bsc.make_cache([400], 1, 16, seed=4)
    q = bsc.make_query(1, 2, seed=5)[0]
    lo, hi, s = map(np.array, zip(*[bsc.bounds(c, 0, j, 0, 400) for j in range(25)]))
    chosen = bsc.select(q, lo, hi, s, 6, 0, 1)
    assert len(chosen) == 6 and chosen[-1] == 24
    k = c.rows("k", 0, 400)[:, 0]
    best = np.full(400, -np.inf)
    score = np.full(25, -np.inf)
    for x in q.double().numpy():
        f = bsc.least_pow2(float(np.abs(x).max()), 127.0)
        r = np.rint(x / f)
        best = np.maximum(best, k @ r * f)
        score = np.maximum(score, (np.maximum(r, 0) * hi + np.minimum(r, 0) * lo).sum(1) * f * s)
    least = min(score[j] for j in chosen if j != 24)
    for j in range(25):
        if j not in chosen:
            assert best[16 * j:16 * j + 16].max() <= least


# ---------------------------------------------------------------------------------- refusals
def P(x):
    return None if x is None else ctypes.c_void_p(x)


def _range(L, name, **kw):
    a = dict(k=16, v=16, kc=16, vc=16, ks=16, vs=16, t=16, p=16, st=16, B=2, T=4, N=8, n_kv=2,
             d=128, bs=16, MB=4, NB=8)
    a.update(kw)
    return getattr(L, name)(*[P(a[n]) for n in ("k", "v", "kc", "vc", "ks", "vs", "t", "p", "st")],
                            *[a[n] for n in ("B", "T", "N", "n_kv", "d", "bs", "MB", "NB")], None)


RANGE_REFUSALS = [
    (dict(d=64), _native.ERR_UNSUPPORTED), (dict(bs=64), _native.ERR_UNSUPPORTED),
    (dict(B=-1), _native.ERR_INVALID_ARG), (dict(T=-1), _native.ERR_INVALID_ARG),
    (dict(N=-1), _native.ERR_INVALID_ARG), (dict(st=None, N=7), _native.ERR_INVALID_ARG),
    (dict(n_kv=0), _native.ERR_INVALID_ARG), (dict(NB=1 << 30, n_kv=4), _native.ERR_INVALID_ARG),
    (dict(B=1 << 20, T=1 << 20, MB=1 << 20), _native.ERR_INVALID_ARG),
    (dict(k=None), _native.ERR_INVALID_ARG), (dict(v=24), _native.ERR_INVALID_ARG),
    (dict(kc=8), _native.ERR_INVALID_ARG), (dict(vc=None), _native.ERR_INVALID_ARG),
    (dict(ks=None), _native.ERR_INVALID_ARG), (dict(vs=18), _native.ERR_INVALID_ARG),
    (dict(t=None), _native.ERR_INVALID_ARG), (dict(p=None), _native.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("name", ["pgd_kv_append_fp8b", "pgd_kv_read_fp8b"])
@pytest.mark.parametrize("kw,status", RANGE_REFUSALS, ids=lambda x: str(x))
def test_range_calls_refuse(L, name, kw, status):
    assert _range(L, name, **kw) == status
    assert L.pgd_last_error_detail()


@pytest.mark.parametrize("name", ["pgd_kv_append_fp8b", "pgd_kv_read_fp8b"])
@pytest.mark.parametrize("kw", [dict(B=0, N=0), dict(T=0, N=0), dict(N=0)], ids=str)
def test_range_calls_of_nothing(L, name, kw):
    assert _range(L, name, **kw) == _native.OK


def _attend(L, append=False, **kw):
    a = dict(out=16, q=16, kn=16, vn=16, k=16, v=16, ks=16, vs=16, t=16, c=16, B=2, n_q=8, n_kv=2,
             d=128, bs=16, MB=4, NB=8, scale=0.1, splits=0, ws=None, wsb=0)
    a.update(kw)
    names = ["out", "q"] + (["kn", "vn"] if append else []) + ["k", "v", "ks", "vs", "t", "c"]
    fn = L.pgd_append_decode_attention_fp8b if append else L.pgd_paged_decode_attention_fp8b
    return fn(*[P(a[n]) for n in names],
              *[a[n] for n in ("B", "n_q", "n_kv", "d", "bs", "MB", "NB", "scale", "splits")],
              P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(d=64), _native.ERR_UNSUPPORTED), (dict(bs=8), _native.ERR_UNSUPPORTED),
    (dict(n_q=6), _native.ERR_UNSUPPORTED), (dict(n_q=7), _native.ERR_INVALID_ARG),
    (dict(B=2049), _native.ERR_UNSUPPORTED), (dict(scale=0.0), _native.ERR_INVALID_ARG),
    (dict(scale=float("nan")), _native.ERR_INVALID_ARG), (dict(q=None), _native.ERR_INVALID_ARG),
    (dict(k=24), _native.ERR_INVALID_ARG), (dict(splits=-1), _native.ERR_INVALID_ARG),
    (dict(ks=None), _native.ERR_INVALID_ARG), (dict(vs=2), _native.ERR_INVALID_ARG),
    (dict(B=2048, n_kv=8, MB=(1 << 17) - 23), _native.ERR_UNSUPPORTED),
    (dict(B=2048, n_kv=40, n_q=40), _native.ERR_UNSUPPORTED),
    (dict(ws=None), _native.ERR_WORKSPACE), (dict(ws=256, wsb=16), _native.ERR_WORKSPACE),
    (dict(ws=264, wsb=1 << 30), _native.ERR_WORKSPACE),
], ids=lambda x: str(x))
def test_attention_refuses(L, append, kw, status):
    assert _attend(L, append, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kn=None), _native.ERR_INVALID_ARG), (dict(vn=8), _native.ERR_INVALID_ARG)], ids=str)
def test_append_attention_refuses_its_rows(L, kw, status):
    assert _attend(L, True, **kw) == status


def test_workspace_size(L):
    """Grows with the batch from one counter region for all sizes; 0 where no call would do."""
    size = pgd.block_workspace_size
    assert 65536 * 4 < size(1, 8, 8) <= size(4, 32, 8) <= size(64, 32, 8)
    assert size(64, 32, 8, 4) - size(64, 32, 8, 2) == 2 * 64 * 8 * 4 * (128 + 2) * 4
    assert size(2048, 2048 * 40, 40) == size(3, 7, 2) == size(2, 8, 2, d=64) == 0


def test_attention_of_nothing(L):
    assert _attend(L, B=0) == _attend(L, True, B=0) == _native.OK


def _bounds(L, **kw):
    a = dict(b=16, s=16, k=16, ks=None, t=16, p=None, c=16, B=2, T=64, n_kv=2, d=128, bs=16, MB=4,
             NB=8)
    a.update(kw)
    return L.pgd_block_bounds(*[P(a[n]) for n in ("b", "s", "k", "ks", "t", "p", "c")],
                              *[a[n] for n in ("B", "T", "n_kv", "d", "bs", "MB", "NB")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=256), _native.ERR_UNSUPPORTED), (dict(bs=24), _native.ERR_UNSUPPORTED),
    (dict(T=-1), _native.ERR_INVALID_ARG), (dict(b=None), _native.ERR_INVALID_ARG),
    (dict(b=8), _native.ERR_INVALID_ARG), (dict(s=None), _native.ERR_INVALID_ARG),
    (dict(k=None), _native.ERR_INVALID_ARG), (dict(ks=6), _native.ERR_INVALID_ARG),
    (dict(t=None), _native.ERR_INVALID_ARG), (dict(c=None), _native.ERR_INVALID_ARG),
], ids=lambda x: str(x))
def test_bounds_refuse(L, kw, status):
    assert _bounds(L, **kw) == status


def test_bounds_of_nothing(L):
    assert _bounds(L, B=0) == _bounds(L, T=0) == _native.OK


def _select(L, **kw):
    a = dict(ti=16, tt=16, q=16, b=16, s=16, t=16, c=16, B=2, n_q=8, n_kv=2, d=128, bs=16, MB=40,
             NB=8, W=9, first=1, last=2)
    a.update(kw)
    return L.pgd_select_blocks(*[P(a[n]) for n in ("ti", "tt", "q", "b", "s", "t", "c")],
                               *[a[n] for n in ("B", "n_q", "n_kv", "d", "bs", "MB", "NB", "W",
                                                "first", "last")], None)


SELECT_REFUSALS = [
    (dict(d=64), _native.ERR_UNSUPPORTED), (dict(bs=64), _native.ERR_UNSUPPORTED),
    (dict(n_q=32), _native.ERR_UNSUPPORTED), (dict(n_q=9), _native.ERR_INVALID_ARG),
    (dict(W=0), _native.ERR_INVALID_ARG), (dict(first=-1), _native.ERR_INVALID_ARG),
    (dict(last=0), _native.ERR_INVALID_ARG), (dict(first=5, last=5), _native.ERR_INVALID_ARG),
    (dict(MB=49153), _native.ERR_UNSUPPORTED), (dict(B=1025), _native.ERR_UNSUPPORTED),
    (dict(NB=1 << 30, n_kv=4), _native.ERR_INVALID_ARG), (dict(q=None), _native.ERR_INVALID_ARG),
    (dict(b=24), _native.ERR_INVALID_ARG), (dict(s=None), _native.ERR_INVALID_ARG),
    (dict(ti=None), _native.ERR_INVALID_ARG), (dict(tt=2), _native.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", SELECT_REFUSALS, ids=lambda x: str(x))
def test_select_refuses(L, kw, status):
    assert _select(L, **kw) == status


def _selected(L, sparse=False, **kw):
    a = dict(out=16, q=16, k=16, v=16, ks=None, vs=None, b=16, s=16, t=16, c=16, ti=16, tt=16, B=2,
             n_q=8, n_kv=2, d=128, bs=16, MB=40, NB=8, W=9, first=1, last=2, scale=0.1, splits=0,
             ws=None, wsb=0)
    a.update(kw)
    names = ["out", "q", "k", "v", "ks", "vs"] + (["b", "s", "t", "c"] if sparse else [])
    ints = ["B", "n_q", "n_kv", "d", "bs"] + (["MB"] if sparse else []) + ["NB", "W"] + (
        ["first", "last"] if sparse else [])
    fn = L.pgd_sparse_decode_attention if sparse else L.pgd_selected_decode_attention
    return fn(*[P(a[n]) for n in names + ["ti", "tt"]], *[a[n] for n in ints], a["scale"],
              a["splits"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(d=64), _native.ERR_UNSUPPORTED), (dict(n_q=6), _native.ERR_UNSUPPORTED),
    (dict(B=1025), _native.ERR_UNSUPPORTED), (dict(W=0), _native.ERR_INVALID_ARG),
    (dict(NB=1 << 30, n_kv=4), _native.ERR_INVALID_ARG), (dict(scale=-1.0), _native.ERR_INVALID_ARG),
    (dict(out=None), _native.ERR_INVALID_ARG), (dict(k=8), _native.ERR_INVALID_ARG),
    (dict(ti=None), _native.ERR_INVALID_ARG), (dict(ks=16), _native.ERR_INVALID_ARG),
    (dict(vs=16), _native.ERR_INVALID_ARG), (dict(ks=6, vs=16), _native.ERR_INVALID_ARG),
    (dict(ws=None), _native.ERR_WORKSPACE),
], ids=lambda x: str(x))
def test_selected_attention_refuses(L, sparse, kw, status):
    assert _selected(L, sparse, **kw) == status


def test_sparse_attention_refuses_its_selection(L):
    for kw, status in SELECT_REFUSALS:
        assert _selected(L, True, **kw) == status, kw


def test_selection_of_nothing(L):
    assert _select(L, B=0) == _selected(L, B=0) == _selected(L, True, B=0) == _native.OK


def test_binding_refuses_before_the_library():
    """Types, shapes and places, on host tensors."""
    u8, bf, i32 = torch.uint8, torch.bfloat16, torch.int32
    kc = torch.zeros(4, 2, 2, 8, 8, 16, dtype=u8)
    rows = torch.zeros(3, 2, 128, dtype=bf)
    sc = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.kv_append_fp8b(rows, rows, kc, kc, sc, sc, torch.zeros(3, 2, dtype=i32),
                           torch.zeros(3, dtype=i32))
    with pytest.raises(TypeError, match="k rows"):
        pgd.kv_read_fp8b(rows.float(), rows, kc, kc, sc, sc, torch.zeros(3, 2, dtype=i32),
                         torch.zeros(3, dtype=i32))
    with pytest.raises(ValueError, match="contiguous"):
        pgd.kv_append_fp8b(rows.transpose(0, 1), rows, kc, kc, sc, sc,
                           torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32))
    with pytest.raises(TypeError, match="k_cache"):
        pgd.paged_decode_attention_fp8b(None, rows, kc.float(), kc, sc, sc, None, None, 1.0)
    with pytest.raises(ValueError, match="both scales"):
        pgd.selected_decode_attention(None, rows, kc, kc, None, None, 1.0, k_scales=sc)
    with pytest.raises(TypeError, match="bounds"):
        pgd.select_blocks(None, None, rows, kc, sc, None, None, 0, 1, 16)
    with pytest.raises(ValueError, match="no prepared form"):
        pgd.prepare("kv_read_fp8b")
