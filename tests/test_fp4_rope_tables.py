"""The 4-bit cache, rotary positions and block tables on the CPU: the plain forms that the GPU tests
compare with, the frequencies, and the calls that are refused before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def L():
    return _native.lib()


# ------------------------------------------------------------------ plain forms
@pytest.mark.parametrize("is_v", [False, True])
def test_layout_places_every_nibble_and_scale_once(is_v):
    byte, high, sc = fp4._places(is_v)
    assert sorted(zip(byte.ravel().tolist(), high.ravel().tolist())) == [
        (b, h) for b in range(1024) for h in (False, True)]
    assert sorted(sc[:, ::16].ravel().tolist()) == list(range(1024, 1152))
    r = np.random.default_rng(0)
    c, s = r.integers(0, 16, (3, 2, 32, 128)), r.integers(0, 256, (3, 2, 32, 8))
    c2, s2 = fp4.unpack(fp4.pack(c, s, is_v), is_v)
    assert (c2 == c).all() and (s2 == s).all()


def test_quantise_takes_the_nearest_code():
    x = bsc.f64(torch.randn(200, 128, generator=torch.Generator().manual_seed(1)).bfloat16())
    c, s = fp4.quantise(x, 0.5)
    f = np.repeat(bsc.VALUES[s], 16, -1) * 0.5
    best = np.abs(np.abs(x)[..., None] - fp4.E2M1 * f[..., None]).min(-1)
    assert np.allclose(np.abs(np.abs(x) - np.abs(fp4.values(c, s, 0.5))), best, rtol=0, atol=1e-15)
    m = np.abs(x).reshape(200, 8, 16).max(-1) / 3.0
    assert (np.abs(bsc.VALUES[s] - m) <= 2.0 ** -4 * np.maximum(m, 2.0 ** -6)).all()


def test_quantise_special_values():
    x = np.zeros((1, 128))
    x[0, 16:18] = 1e30, -np.inf   # an infinity and what saturates beside it
    x[0, 32] = np.nan
    x[0, 48] = 1e-20              # next to nothing: a scale of 0
    c, s = fp4.quantise(x, 1.0)
    v = fp4.values(c, s, 1.0)
    assert v[0, 0] == 0 and v[0, 16] == 2688 and v[0, 17] == -2688 and v[0, 48] == 0
    assert np.isnan(v[0, 32:48]).all() and not np.isnan(v[0, 48:]).any()


# ------------------------------------------------------------------ frequencies
def _radians(t):
    return [int(x) / 2.0 ** 64 * 2 * math.pi for x in t.tolist()]


@pytest.mark.parametrize("rotary,base", [(128, 10000.0), (64, 500000.0), (16, 1e6), (2, 10000.0)])
def test_plain_and_linear_frequencies(rotary, base):
    f = [base ** (-2 * i / rotary) for i in range(rotary // 2)]
    assert _radians(pgd.rope_frequencies(rotary, base, device="cpu")) == pytest.approx(f, rel=1e-14)
    got = pgd.rope_frequencies(rotary, base, "linear", factor=8.0, device="cpu")
    assert _radians(got) == pytest.approx([x / 8 for x in f], rel=1e-14)


def test_base_scaling_keeps_the_fastest_and_divides_the_slowest():
    got = _radians(pgd.rope_frequencies(128, 10000.0, "base", factor=4.0, device="cpu"))
    assert got[0] == pytest.approx(1.0, rel=1e-14)
    assert got[-1] == pytest.approx(10000.0 ** (-126 / 128) / 4, rel=1e-12)


def test_ramp_by_dim():
    n, base, ctx, factor = 128, 10000.0, 4096, 16.0
    got = _radians(pgd.rope_frequencies(n, base, "ramp_dim", factor, ctx, 1.0, 32.0, device="cpu"))

    def pair(turns):
        return n * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    assert 0 < lo < hi < 64
    for i in range(64):
        f = base ** (-2 * i / n)
        part = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert got[i] == pytest.approx(f * (1 - part) + f / factor * part, rel=1e-12)
    assert got[0] == pytest.approx(1.0) and got[63] == pytest.approx(base ** (-126 / 128) / 16)


def test_ramp_by_wavelength():
    n, base, ctx, factor = 128, 500000.0, 8192, 8.0
    got = _radians(pgd.rope_frequencies(n, base, "ramp_wavelength", factor, ctx, 1.0, 4.0,
                                        device="cpu"))
    kinds = set()
    for i in range(64):
        f = base ** (-2 * i / n)
        length = 2 * math.pi / f
        if length < ctx / 4.0:
            want, kind = f, "kept"
        elif length > ctx / 1.0:
            want, kind = f / factor, "slowed"
        else:
            smooth, kind = (ctx / length - 1.0) / 3.0, "between"
            want = (1 - smooth) * f / factor + smooth * f
        kinds.add(kind)
        assert got[i] == pytest.approx(want, rel=1e-12)
    assert kinds == {"kept", "slowed", "between"}


@pytest.mark.parametrize("kw", [
    dict(rotary=0), dict(rotary=7), dict(rotary=-2), dict(base=1.0), dict(base=float("nan")),
    dict(factor=0.5, scaling="linear"), dict(scaling="base", rotary=2),
    dict(scaling="ramp_dim"), dict(scaling="ramp_dim", original_context=4096.0, slow_turns=4.0,
                                   fast_turns=4.0),
    dict(scaling="ramp_wavelength", original_context=float("inf"))], ids=str)
def test_frequencies_refused(kw):
    with pytest.raises(pgd.PGDError) as e:
        pgd.rope_frequencies(**{"rotary": 64, "device": "cpu", **kw})
    assert e.value.status == INVALID
    with pytest.raises(ValueError):
        pgd.rope_frequencies(64, scaling="other", device="cpu")


# ------------------------------------------------------------------ refusals
P = 1 << 20  # an address that is never read: these calls end on the host


def _range(L, fn="pgd_kv_append_fp4", **kw):
    a = dict(k=P, v=P, kc=P, vc=P, tables=P, pos=P, starts=None, B=2, T=3, N=6, n_kv=2, d=128,
             bs=16, MB=4, NB=9, ks=1.0, vs=1.0, st=None)
    a.update(kw)
    return getattr(L, fn)(*a.values())


@pytest.mark.parametrize("fn", ["pgd_kv_append_fp4", "pgd_kv_read_fp4"])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(vc=None), INVALID), (dict(tables=None), INVALID),
    (dict(pos=None), INVALID), (dict(v=P + 2), INVALID), (dict(kc=P + 8), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(N=5), INVALID),
    (dict(starts=P, N=-1), INVALID), (dict(n_kv=0), INVALID), (dict(NB=0), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(bs=64), UNSUPPORTED),
    (dict(MB=1 << 28), INVALID), (dict(ks=0.0), INVALID), (dict(ks=3.0), INVALID),
    (dict(vs=-1.0), INVALID), (dict(vs=float("nan")), INVALID), (dict(ks=2.0 ** 33), INVALID),
    (dict(vs=float("inf")), INVALID),
    (dict(B=1 << 20, T=1 << 12, N=0, n_kv=16, starts=P, MB=1 << 12),
     INVALID)], ids=str)
def test_ranges_refused(L, fn, kw, status):
    assert _range(L, fn, **kw) == status
    assert L.pgd_last_error_detail()


@pytest.mark.parametrize("kw", [dict(B=0, N=0), dict(T=0, N=0), dict(N=0, starts=P)], ids=str)
def test_ranges_of_nothing(L, kw):
    assert _range(L, **kw) == 0


def _attend(L, append=False, **kw):
    a = dict(out=P, q=P, kn=P, vn=P, kc=P, vc=P, tables=P, ctx=P, B=2, n_q=8, n_kv=2, d=128, bs=16,
             MB=4, NB=9, scale=0.1, ks=1.0, vs=1.0, splits=0, ws=P, wb=1 << 30, st=None)
    a.update(kw)
    if not append:
        del a["kn"], a["vn"]
    fn = L.pgd_append_decode_attention_fp4 if append else L.pgd_paged_decode_attention_fp4
    return fn(*a.values())


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=P + 4), INVALID), (dict(kc=None), INVALID),
    (dict(ctx=None), INVALID), (dict(B=-1), INVALID), (dict(B=2049), UNSUPPORTED),
    (dict(n_q=6, n_kv=4), INVALID), (dict(n_q=32, n_kv=2), UNSUPPORTED),
    (dict(n_q=6, n_kv=2), UNSUPPORTED), (dict(d=64), UNSUPPORTED), (dict(bs=24), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(splits=-1), INVALID),
    (dict(scale=1e38, ks=2.0 ** 32), INVALID),
    (dict(ks=1.5), INVALID), (dict(vs=0.0), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=P + 16), WORKSPACE), (dict(wb=1000), WORKSPACE),
    (dict(B=2048, n_q=64, n_kv=64), UNSUPPORTED),
    (dict(B=2048, n_kv=8, MB=1 << 20), INVALID), (dict(B=1000, n_kv=8, MB=1 << 21), UNSUPPORTED)],
    ids=str)
def test_attention_refused(L, append, kw, status):
    assert _attend(L, append, **kw) == status


@pytest.mark.parametrize("kw", [dict(kn=None), dict(vn=None), dict(kn=P + 8)], ids=str)
def test_append_attention_refused(L, kw):
    assert _attend(L, True, **kw) == INVALID
    assert _attend(L, True, B=0) == 0


def test_workspace_sizes():
    assert pgd.fp4_workspace_size(4, 32, 8) > 0
    assert pgd.fp4_workspace_size(4, 32, 8, 100) > pgd.fp4_workspace_size(4, 32, 8, 1)
    assert pgd.fp4_workspace_size(4, 30, 8) == 0 and pgd.fp4_workspace_size(4, 32, 8, -1) == 0
    assert pgd.fp4_workspace_size(2048, 64, 64) == 0


def _rope(L, **kw):
    a = dict(qo=P, ko=P, q=P, k=P, pos=P, f=P, T=4, n_q=8, n_kv=2, d=128, first=0, rotary=64,
             inter=0, factor=1.0, strides=None, st=None)
    a.update(kw)
    return L.pgd_rope(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(q=None), INVALID),
    (dict(k=P + 2), INVALID), (dict(pos=None), INVALID), (dict(f=None), INVALID),
    (dict(f=P + 4), INVALID), (dict(T=-1), INVALID), (dict(n_q=-1), INVALID),
    (dict(n_kv=-1), INVALID), (dict(n_q=70000), INVALID), (dict(d=72), UNSUPPORTED),
    (dict(n_q=65532, n_kv=2), INVALID),
    (dict(d=0), UNSUPPORTED), (dict(d=4096), UNSUPPORTED), (dict(rotary=24), UNSUPPORTED),
    (dict(rotary=0), UNSUPPORTED), (dict(rotary=144), UNSUPPORTED), (dict(first=4), UNSUPPORTED),
    (dict(first=-8), UNSUPPORTED), (dict(first=72), UNSUPPORTED),
    (dict(factor=float("nan")), INVALID)], ids=str)
def test_rope_refused(L, kw, status):
    assert _rope(L, **kw) == status


def test_rope_strides_refused(L):
    for bad in range(8):
        s = [1024, 128, 256, 128, 1024, 128, 256, 128]
        for x in (4, -128):
            t = list(s)
            t[bad] = x
            assert _rope(L, strides=(ctypes.c_int64 * 8)(*t)) == INVALID
    assert _rope(L, T=0) == 0 and _rope(L, n_q=0, n_kv=0) == 0


def _rope_append(L, **kw):
    a = dict(qo=P, q=P, k=P, v=P, kc=P, vc=P, slots=P, pos=P, f=P, T=4, n_q=8, n_kv=2, d=128, bs=16,
             NB=9, first=0, rotary=64, inter=0, factor=1.0, strides=None, st=None)
    a.update(kw)
    return L.pgd_rope_append(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(qo=None), INVALID), (dict(v=None), INVALID), (dict(k=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=P + 8), INVALID), (dict(slots=None), INVALID),
    (dict(slots=P + 4), INVALID), (dict(n_kv=0), INVALID), (dict(n_q=-1), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(NB=0), INVALID),
    (dict(rotary=136), UNSUPPORTED), (dict(T=-1), INVALID)], ids=str)
def test_rope_append_refused(L, kw, status):
    assert _rope_append(L, **kw) == status


def _grow(L, **kw):
    a = dict(tables=P, ctx=P, new=P, refs=P, bits=P, pos=P, starts=P, slots=P, tp=P, src=P, dst=P,
             result=P, B=4, N=9, bs=16, MB=4, NB=9, st=None)
    a.update(kw)
    return L.pgd_grow_tables(*a.values())


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), INVALID) for n in (
    "tables", "ctx", "new", "refs", "bits", "pos", "starts", "slots", "tp", "src", "dst", "result")]
    + [(dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(bs=0), INVALID), (dict(MB=0), INVALID),
       (dict(NB=0), INVALID), (dict(MB=1 << 28), INVALID), (dict(B=16385), UNSUPPORTED),
       (dict(slots=P + 4), INVALID)], ids=str)
def test_grow_refused(L, kw, status):
    assert _grow(L, **kw) == status


@pytest.mark.parametrize("kw", [dict([(n, None)]) for n in ("tables", "ctx", "keep", "refs", "bits")]
                         + [dict(B=-1), dict(bs=0), dict(MB=0), dict(NB=-1), dict(MB=1 << 28)],
                         ids=str)
def test_trim_refused(L, kw):
    a = dict(tables=P, ctx=P, keep=P, refs=P, bits=P, B=4, bs=16, MB=4, NB=9, st=None)
    assert L.pgd_trim_tables(*{**a, **kw}.values()) == INVALID
    assert L.pgd_trim_tables(*{**a, "B": 0}.values()) == 0


def test_copy_blocks_fp4_refused(L):
    a = dict(k=P, v=P, src=P, dst=P, n=2, n_kv=2, d=128, bs=16, NB=9, st=None)
    for kw in (dict(k=None), dict(src=None), dict(v=P + 4), dict(n=-1), dict(NB=0),
               dict(n_kv=1 << 21)):
        assert L.pgd_copy_blocks_fp4(*{**a, **kw}.values()) == INVALID
    assert L.pgd_copy_blocks_fp4(*{**a, "d": 64}.values()) == UNSUPPORTED
    assert L.pgd_copy_blocks_fp4(*{**a, "n": 0}.values()) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    """On the CPU, so that a call that is not refused for its shape is for its device."""
    bf, i32 = torch.bfloat16, torch.int32
    pool = torch.zeros(9, 2, 1, 1152, dtype=torch.uint8)
    t, ctx = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32)
    q, rows = torch.zeros(3, 8, 128, dtype=bf), torch.zeros(3, 2, 128, dtype=bf)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for args, err in [((rows.float(), rows, pool, pool, t, ctx), TypeError),
                      ((rows, rows, pool, pool, t, ctx), ValueError)]:
        for fn in (pgd.kv_append_fp4, pgd.kv_read_fp4):
            with pytest.raises(err):
                fn(*args)
    for args in [(q, q[:, :4], pool, pool, t, ctx), (q, q, pool, pool[:8], t, ctx),
                 (q, q, pool, pool, t[:2], ctx), (q, q, pool, pool, t, ctx)]:
        with pytest.raises(ValueError):
            pgd.paged_decode_attention_fp4(*args, 0.1, workspace=ws)
    with pytest.raises(TypeError):
        pgd.append_decode_attention_fp4(q, q, None, rows, pool, pool, t, ctx, 0.1, workspace=ws)
    f, pos = torch.zeros(32, dtype=torch.int64), torch.zeros(3, dtype=i32)
    k = torch.zeros(3, 2, 128, dtype=bf)
    with pytest.raises(TypeError):
        pgd.rope(q, k, q.float(), k, pos, f)
    for a in [(q[..., ::2], k, q[..., ::2], k, pos, f), (q, k, q, k, pos, f)]:
        with pytest.raises(ValueError):
            pgd.rope(*a)
    with pytest.raises(ValueError):
        pgd.trim_tables(t, ctx, ctx, pos, torch.zeros(2, dtype=i32), 16)
    with pytest.raises(ValueError):
        pgd.make_block_pool(0)


def test_make_block_pool():
    for n in (1, 31, 32, 33, 100):
        refs, bits = pgd.make_block_pool(n, device="cpu")
        t = fp4.Tables([], [], refs.tolist(), 16)
        assert bits.tolist() == t.bits() and len(refs) == n
