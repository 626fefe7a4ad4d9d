"""Block tables grown and cut on the GPU, against one request after another on the host."""
import numpy as np
import pytest
import torch

import fp4
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import _native

pytestmark = pytest.mark.gpu
BAD_ID, BAD_CTX, BAD_POS = (_native.DEVERR_BAD_BLOCK_ID, _native.DEVERR_BAD_CONTEXT,
                            _native.DEVERR_BAD_POSITION)


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Device:
    """The state on the GPU beside the host's, compared after every call."""

    def __init__(self, host, MB, N):
        self.host, self.B, self.N = host, len(host.ctx), N
        self.tables = _i32(host.tables).view(self.B, MB)
        self.ctx, self.refs, self.bits = _i32(host.ctx), _i32(host.refs), _i32(host.bits())
        B = self.B
        self.out = dict(positions=_i32([9] * B), token_starts=_i32([9] * (B + 1)),
                        slots=torch.full((N,), 9, device="cuda"), token_positions=_i32([9] * N),
                        copy_src=_i32([9] * B), copy_dst=_i32([9] * B), result=_i32([9] * 4))

    def grow(self, new, flags=0):
        want = self.host.grow(new, self.N)
        pgd.grow_tables(self.tables, self.ctx, _i32(new), self.refs, self.bits, self.host.bs,
                        *self.out.values())
        assert pgd.device_errors(clear=True) == flags
        for name, x in want.items():
            assert self.out[name].tolist() == x, name
        self.same()
        return want

    def trim(self, keep, flags=0):
        self.host.trim(keep)
        pgd.trim_tables(self.tables, self.ctx, _i32(keep), self.refs, self.bits, self.host.bs)
        assert pgd.device_errors(clear=True) == flags
        self.same()

    def same(self):
        assert self.tables.tolist() == self.host.tables
        assert self.ctx.tolist() == self.host.ctx
        assert self.refs.tolist() == self.host.refs
        assert self.bits.tolist() == self.host.bits()


def _state(B, MB, NB, bs, seed=0, most=None, used=0.3):
    """Requests of random lengths over random blocks, other blocks in use elsewhere."""
    r = np.random.default_rng(seed)
    most = MB * bs if most is None else most
    ctx = r.integers(0, most + 1, B)
    nblk = -(-ctx // bs)
    ids = r.permutation(NB)
    assert nblk.sum() <= NB
    tables = np.full((B, MB), -1)
    refs = np.zeros(NB, int)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = ids[at:at + n]
        refs[ids[at:at + n]] = 1
        at += n
    rest = ids[at:]
    refs[rest[r.random(len(rest)) < used]] = 1
    return fp4.Tables(tables, ctx, refs, bs), r


@pytest.mark.parametrize("B,MB,NB,bs,N", [
    (1, 4, 9, 16, 64), (7, 10, 101, 16, 600), (64, 40, 3000, 32, 9000), (300, 6, 2000, 16, 300),
    (1025, 5, 7001, 16, 8192), (2500, 3, 9000, 16, 8193), (5, 900, 40000, 16, 60000),
    (3, 50, 300, 1, 150), (4, 9, 64, 128, 4000)])
def test_random_steps(B, MB, NB, bs, N):
    host, r = _state(B, MB, NB, bs, seed=B, most=MB * bs // 2)
    dev = Device(host, MB, N)
    dev.same()
    for step in range(6):
        room = [MB * bs - n for n in host.ctx]
        most = max(1, min(N // B, max(room)))
        new = [int(min(x, r.integers(0, most + 1))) for x in room]
        if step == 2:
            new = [min(1, x) for x in room]
        dev.grow(new)
        keep = [int(r.integers(0, n + 3)) if r.random() < 0.5 else n for n in host.ctx]
        if step % 2:
            keep = [0 if r.random() < 0.3 else k for k in keep]
        dev.trim(keep)


def test_shared_blocks_are_copied_on_growth_and_freed_at_the_last_reference():
    bs, MB, NB = 16, 6, 40
    host, _ = _state(5, MB, NB, bs, seed=3, most=0, used=0.2)
    dev = Device(host, MB, 64)
    dev.grow([20, 32, 0, 5, 0])

    def share(src, dst, n):  # row dst takes row src's first n tokens
        for j in range(-(-n // bs)):
            host.tables[dst][j] = host.tables[src][j]
            host.refs[host.tables[src][j]] += 1
        host.ctx[dst] = n
        dev.tables[dst], dev.ctx[dst] = _i32(host.tables[dst]), n
        dev.refs.copy_(_i32(host.refs))

    share(0, 2, 20)
    share(1, 4, 32)  # whole blocks: nothing to copy
    dev.same()
    got = dev.grow([0, 1, 1, 1, 1])
    assert got["copy_src"][2] >= 0 and got["copy_src"].count(-1) == 4
    dev.trim([20, 33, 21, 6, 33])
    share(3, 2, 6)   # (row 2's own blocks stay with it in the pool: they are leaked on purpose)
    share(3, 4, 6)
    got = dev.grow([0, 0, 1, 2, 3])  # three rows of one block: three copies
    src = got["copy_src"]
    assert src[2] == src[3] == src[4] >= 0 and len(set(got["copy_dst"][2:])) == 3
    assert host.refs[src[2]] == 0
    dev.trim([0, 0, 0, 0, 0])
    dev.grow([16, 16, 16, 16, 0])


@pytest.mark.parametrize("N", [5000, 9000])
def test_many_shared_blocks(N):
    """300 rows, every third sharing all blocks of the row before, the last partly filled or not;
    with few tokens and with many (the other kernel)."""
    B, MB, NB, bs = 300, 9, 4000, 16
    host, r = _state(B, MB, NB, bs, seed=9, most=90)
    for b in range(2, B, 3):
        old = -(-host.ctx[b] // bs)
        for j in range(old):
            host.refs[host.tables[b][j]] -= 1
        host.ctx[b] = host.ctx[b - 1]
        host.tables[b] = list(host.tables[b - 1])
        for j in range(-(-host.ctx[b] // bs)):
            host.refs[host.tables[b][j]] += 1
    dev = Device(host, MB, N)
    for step in range(4):
        got = dev.grow([int(x) for x in r.integers(0, 1 + min(16, N // B), B)])
        assert got["result"][0] == 0
        assert sum(x >= 0 for x in got["copy_src"]) > (20 if step == 0 else -1)
        dev.trim([int(max(0, n - x)) for n, x in zip(host.ctx, r.integers(-2, 20, B))])
    dev.trim([0] * B)


def test_too_few_blocks_or_too_many_tokens_change_nothing():
    host, _ = _state(4, 8, 30, 16, seed=1, most=30, used=1.0)  # no block free
    dev = Device(host, 8, 90)
    got = dev.grow([20, 3, 40, 0])
    assert got["result"][0] == 1 and got["result"][2] > 0
    got = dev.grow([90, 1, 0, 0], flags=BAD_POS)
    assert got["result"][0] == 2
    got = dev.grow([0, 0, 0, 0])
    assert got["result"] == [0, 0, 0, 0]


def test_exactly_the_free_blocks():
    host, _ = _state(3, 20, 50, 16, seed=5, most=30, used=0.0)
    dev = Device(host, 20, 1000)
    free = host.refs.count(0)
    give = [0, 0, 0]
    for b in range(3):
        room = 20 - -(-host.ctx[b] // 16)
        n = min(room, free)
        free -= n
        give[b] = -(-host.ctx[b] // 16) * 16 + 16 * n - host.ctx[b]
    assert free == 0 or all(g + n == 320 for g, n in zip(give, host.ctx))
    got = dev.grow(give)
    assert got["result"][0] == 0
    dev.trim([1, 2, 3])


def test_bad_rows_get_nothing_and_are_flagged():
    host, _ = _state(6, 4, 60, 16, seed=2, most=20)
    dev = Device(host, 4, 100)
    for b, n in ((0, -1), (3, 65), (4, -2 ** 31)):
        host.ctx[b] = n
    dev.ctx.copy_(_i32(host.ctx))
    dev.grow([1, 2, -3, 1, 5, 7], flags=BAD_CTX)
    dev.grow([1, 2 ** 31 - 1, 0, 2 ** 31 - 1, 5, 7], flags=BAD_CTX)
    dev.trim([0, -1, 2, 0, 0, 1], flags=BAD_CTX)
    host.ctx[0], host.ctx[3], host.ctx[4] = 0, 0, 0
    dev.ctx.copy_(_i32(host.ctx))
    b = next(b for b in range(6) if host.ctx[b] % 16)
    good = host.tables[b][host.ctx[b] // 16]
    for bad in (-1, 60, 2 ** 31 - 1, -2 ** 31):
        host.tables[b][host.ctx[b] // 16] = bad
        dev.tables.copy_(_i32(host.tables))
        dev.grow([1 if i == b else 0 for i in range(6)], flags=BAD_ID)
    host.tables[b][host.ctx[b] // 16] = good
    dev.tables.copy_(_i32(host.tables))
    dev.grow([1 if i == b else 0 for i in range(6)])


def test_trim_of_bad_and_unheld_blocks():
    host, _ = _state(2, 4, 20, 16, seed=2, most=0, used=0.0)
    dev = Device(host, 4, 100)
    dev.grow([60, 40])
    host.tables[0][2] = 99
    unheld = next(i for i, r in enumerate(host.refs) if r == 0)
    host.tables[1][1] = unheld
    dev.tables.copy_(_i32(host.tables))
    dev.trim([0, 0], flags=BAD_ID)


@pytest.mark.parametrize("n", [8, 9, 40, 511, 513, 1200])
def test_trim_of_many_blocks(n):
    """n blocks of a row and as many that two rows share, a bad id and one without references among
    them; cut in two goes, the rest afterwards."""
    host, _ = _state(3, 1300, 6000, 16, seed=n, most=0, used=0.3)
    dev = Device(host, 1300, 50000)
    dev.grow([16 * n, 16 * n, 0])
    host.tables[2][:n], host.ctx[2] = host.tables[1][:n], 16 * n
    for i in host.tables[1][:n]:
        host.refs[i] += 1
    host.tables[0][n - 3] = 6000
    unheld = next(i for i, r in enumerate(host.refs) if r == 0)
    host.tables[0][n // 2] = unheld
    dev.tables.copy_(_i32(host.tables))
    dev.ctx.copy_(_i32(host.ctx))
    dev.refs.copy_(_i32(host.refs))
    dev.trim([5, 16 * n - 40, 3], flags=BAD_ID)
    dev.trim([0, 17, 0])
    dev.grow([100, 0, 16 * n])
    dev.trim([0, 0, 0])


@pytest.mark.parametrize("N", [0, 5, 9000])
def test_no_rows(N):
    host = fp4.Tables([], [], [0] * 40, 16)
    dev = Device(host, 3, N)
    dev.grow([])
    dev.trim([])


@pytest.mark.parametrize("NB", [1, 31, 32, 33, 32768, 32769, 200001])
def test_pools_of_any_size(NB):
    """All blocks but the last ones in use; bits past the pool, set by mistake, do not count."""
    refs = [1] * NB
    for i in {NB - 1, NB // 2, 0}:
        refs[i] = 0
    host = fp4.Tables([[-1, -1, -1]], [0], refs, 16)
    dev = Device(host, 3, 64)
    dev.grow([16 * min(3, refs.count(0))])
    host = fp4.Tables([[-1, -1, -1]], [0], [1] * NB, 16)
    dev = Device(host, 3, 64)
    if NB % 32:
        dev.bits[-1] |= 1 << 30 if NB % 32 <= 30 else -2 ** 31
        want = host.grow([16], 64)
        pgd.grow_tables(dev.tables, dev.ctx, _i32([16]), dev.refs, dev.bits, 16, *dev.out.values())
        assert dev.out["result"].tolist() == want["result"] == [1, 0, 1, 0]


def test_most_rows():
    B = 16384
    host, r = _state(B, 2, 40000, 16, seed=7, most=20, used=0.0)
    dev = Device(host, 2, 20000)
    dev.grow([int(x) for x in r.integers(0, 2, B)])
    dev.trim([int(x) for x in r.integers(0, 20, B)])


def test_binding_refuses_tensors_that_do_not_fit():
    host, _ = _state(3, 4, 40, 16)
    dev = Device(host, 4, 50)
    args = [dev.tables, dev.ctx, _i32([1, 1, 1]), dev.refs, dev.bits, 16, *dev.out.values()]
    for i, x in enumerate(args):
        if i == 5:
            continue
        for wrong, err in [(x.float(), TypeError), (x.cpu(), ValueError)]:
            bad = list(args)
            bad[i] = wrong
            with pytest.raises(err):
                pgd.grow_tables(*bad)
        if i not in (0, 3, 8):  # (those give the sizes)
            bad = list(args)
            bad[i] = torch.cat([x, x])
            with pytest.raises(ValueError):
                pgd.grow_tables(*bad)
    with pytest.raises(pgd.PGDError):
        pgd.grow_tables(*args[:5], 0, *args[6:])
    with pytest.raises(ValueError):
        pgd.trim_tables(dev.tables, dev.ctx, _i32([1]), dev.refs, dev.bits, 16)
    dev.same()
