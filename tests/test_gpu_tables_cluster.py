"""Tables grown by the cluster kernel while its CTAs start at different times: the GPU's SMs are busy with
other calls, and calls follow one another without a pause on two streams."""
import numpy as np
import pytest
import torch

import fp4
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
B, MB, NB, BS, N = 40, 30, 5000, 16, 9000


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _fresh():
    ctx = _i32([0] * B)
    tables = _i32([[-1] * MB] * B)
    out = [_i32([9] * B), _i32([9] * (B + 1)), torch.full((N,), 9, device="cuda"), _i32([9] * N),
           _i32([9] * B), _i32([9] * B), _i32([9] * 4)]
    return tables, ctx, out


def test_every_call_among_busy_sms_has_one_outcome():
    """Growth by exactly the pool's free blocks: a CTA that missed a count would find too few."""
    r = np.random.default_rng(1)
    new = [int(x) for x in r.integers(40, 380, B)]
    need = sum(-(-x // BS) for x in new)
    refs0 = np.ones(NB, int)
    refs0[r.permutation(NB)[:need]] = 0
    host = fp4.Tables([[-1] * MB] * B, [0] * B, refs0, BS)
    want_bits = host.bits()
    want = host.grow(new, N)
    assert want["result"] == [0, need, 0, sum(new)] and N > 8192
    add, refs_at, bits_at = _i32(new), _i32(refs0), _i32(want_bits)
    rows = torch.randn(4000, 40, 128, device="cuda").to(torch.bfloat16)
    at, freq = _i32(list(range(4000))), pgd.rope_frequencies(128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sides = [(_fresh(), refs_at.clone(), bits_at.clone()) for _ in streams]
    wrong = torch.zeros(2, dtype=torch.int64, device="cuda")
    want_tables, want_slots = _i32(host.tables), torch.tensor(want["slots"], device="cuda")
    noise = [torch.empty_like(rows) for _ in streams]
    torch.cuda.synchronize()
    for turn in range(60):
        for i, st in enumerate(streams):
            (tables, ctx, out), refs, bits = sides[i]
            with torch.cuda.stream(st):
                tables.fill_(-1)
                ctx.zero_()
                refs.copy_(refs_at)
                bits.copy_(bits_at)
                pgd.rope(noise[i], None, rows, None, at, freq)
                pgd.grow_tables(tables, ctx, add, refs, bits, BS, *out)
                bad = (tables != want_tables).any() | (out[2] != want_slots).any()
                bad |= (ctx != add).any() | (bits != 0).any() | (refs < 1).any() | (out[6][0] != 0)
                wrong[i] += bad
    torch.cuda.synchronize()
    assert wrong.tolist() == [0, 0]
    for (tables, ctx, out), refs, bits in sides:
        assert out[6].tolist() == want["result"] and refs.tolist() == host.refs
