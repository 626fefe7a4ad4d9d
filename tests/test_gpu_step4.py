"""Steps of a serving loop on the device alone: tables grown, positions turned, tokens cached in four
bits (and in bf16), attention, rejected tokens cut off; run, captured and replayed, on other streams."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu
SCALE, S = 128 ** -0.5, (0.5, 1.0)
N_Q, N_KV, BS, B, MB, NB = 8, 2, 16, 4, 12, 60


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


class Loop:
    """The buffers that a serving loop keeps, for up to N new tokens a step."""

    def __init__(self, N):
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tables, self.ctx, self.new, self.keep = i32(B, MB).fill_(-1), i32(B), i32(B), i32(B)
        self.refs, self.bits = pgd.make_block_pool(NB)
        self.out = [i32(B), i32(B + 1), torch.zeros(N, dtype=torch.int64, device="cuda"), i32(N),
                    i32(B), i32(B), i32(4)]
        self.k4, self.v4 = (torch.zeros(pgd.pool_shape4(NB, N_KV, BS), dtype=torch.uint8,
                                        device="cuda") for _ in range(2))
        self.k16, self.v16 = (torch.zeros(NB, N_KV, BS // 8, 16, 8, 8, dtype=torch.bfloat16,
                                          device="cuda") for _ in range(2))
        self.qkv = torch.zeros(N, N_Q + 2 * N_KV, 128, dtype=torch.bfloat16, device="cuda")
        self.q_rows = torch.zeros(N, N_Q, 128, dtype=torch.bfloat16, device="cuda")
        self.q_rows16 = torch.zeros_like(self.q_rows)
        self.k_rows = torch.zeros(N, N_KV, 128, dtype=torch.bfloat16, device="cuda")
        self.v_rows = torch.zeros_like(self.k_rows)
        self.o4, self.o16 = (torch.zeros(B, N_Q, 128, dtype=torch.bfloat16, device="cuda")
                             for _ in range(2))
        self.freq = pgd.rope_frequencies(128, 10000.0, "linear", 4.0)
        self.ws4 = pgd.make_fp4_workspace(B, N_Q, N_KV)
        self.ws16 = pgd.make_workspace(B, N_Q, N_KV)
        self.N = N

    def step(self):
        """Every request's new tokens cached; the last of each attends."""
        pos, starts, slots, places, src, dst, _ = self.out
        pgd.grow_tables(self.tables, self.ctx, self.new, self.refs, self.bits, BS, *self.out)
        pgd.copy_blocks(self.k4, self.v4, src, dst)
        pgd.copy_blocks(self.k16, self.v16, src, dst)
        q, k, v = self.qkv.split([N_Q, N_KV, N_KV], 1)
        pgd.rope(self.q_rows, self.k_rows, q, k, places, self.freq)
        self.v_rows.copy_(v)
        pgd.kv_append_fp4(self.k_rows, self.v_rows, self.k4, self.v4, self.tables, pos,
                          token_starts=starts, max_tokens=self.N, k_scale=S[0], v_scale=S[1])
        pgd.rope_append(self.q_rows16, q, k, v, self.k16, self.v16, slots, places, self.freq)
        last = (starts[1:].long() - 1).clamp(min=0)
        pgd.paged_decode_attention_fp4(self.o4, self.q_rows[last], self.k4, self.v4, self.tables,
                                       self.ctx, SCALE, k_scale=S[0], v_scale=S[1],
                                       workspace=self.ws4)
        pgd.paged_decode_attention(self.o16, self.q_rows16[last], self.k16, self.v16, self.tables,
                                   self.ctx, SCALE, workspace=self.ws16)
        pgd.trim_tables(self.tables, self.ctx, self.keep, self.refs, self.bits, BS)


class Host:
    """The same step by step: every request's turned keys and values, in 64 bits."""

    def __init__(self):
        self.k, self.v = [[] for _ in range(B)], [[] for _ in range(B)]

    def step(self, loop, new, keep, qkv):
        freq, n = loop.freq.tolist(), 0
        want4, tol4, want16 = [], [], []
        for b in range(B):
            for t in range(new[b]):
                row = bsc.f64(qkv[n:n + 1])
                p = [len(self.k[b])]
                y, _ = fp4.turned(row[:, :N_Q + N_KV], p, freq, 0, False, 1.0)
                # (what the kernel's rounding made of them, which may differ by a bit)
                self.k[b].append((y[0, N_Q:], bsc.f64(loop.k_rows[n])))
                self.v[b].append(bsc.f64(qkv[n, N_Q + N_KV:]))
                assert np.abs(self.k[b][-1][0] - self.k[b][-1][1]).max() <= 2.0 ** -6
                q = bsc.f64(loop.q_rows[n])
                assert np.abs(q - y[0, :N_Q]).max() <= 2.0 ** -6
                n += 1
            kk, vv = np.stack([x for _, x in self.k[b]]), np.stack(self.v[b])
            c = [fp4.values(*fp4.quantise(x, s), s) for x, s in ((kk, S[0]), (vv, S[1]))]
            w, t4 = fp4.bound(q, *c, SCALE)
            want4.append(w)
            tol4.append(t4)
            want16.append(bsc.attention(torch.from_numpy(q), kk, vv, SCALE)[0])
            del self.k[b][keep[b]:], self.v[b][keep[b]:]
        err = np.abs(bsc.f64(loop.o4) - np.stack(want4))
        assert (err <= np.stack(tol4)).all()
        assert np.abs(bsc.f64(loop.o16) - np.stack(want16)).max() <= 2e-2


PLAN = [  # (new tokens, tokens kept): prompts, steps, verifications with rejected tokens
    ([20, 1, 33, 7], [20, 1, 33, 7]), ([1, 1, 1, 1], [21, 2, 34, 8]), ([4, 4, 4, 4], [22, 6, 35, 9]),
    ([3, 40, 2, 1], [25, 40, 36, 10]), ([1, 1, 1, 1], [26, 41, 37, 11]), ([9, 2, 12, 60],
                                                                          [30, 43, 49, 71])]


def _feed(loop, new, keep, seed):
    qkv = torch.randn(loop.N, N_Q + 2 * N_KV, 128, generator=torch.Generator().manual_seed(seed)).to(
        torch.bfloat16)
    loop.qkv.copy_(qkv)
    loop.new.copy_(torch.tensor(new, dtype=torch.int32))
    loop.keep.copy_(torch.tensor(keep, dtype=torch.int32))
    return qkv


def test_steps():
    loop, host = Loop(96), Host()
    for i, (new, keep) in enumerate(PLAN):
        qkv = _feed(loop, new, keep, i)
        loop.step()
        torch.cuda.synchronize()
        assert loop.out[-1].tolist()[0] == 0
        host.step(loop, new, keep, qkv)
    assert loop.ctx.tolist() == PLAN[-1][1]


def test_captured_steps():
    """One graph, replayed for steps of other lengths, prompts among them."""
    loop, host = Loop(96), Host()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # (what the first calls set up is not captured)
        warm = Loop(96)
        _feed(warm, *PLAN[0], 0)
        warm.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loop.step()
    assert not loop.ctx.any()
    for i, (new, keep) in enumerate(PLAN):
        qkv = _feed(loop, new, keep, 10 + i)
        g.replay()
        torch.cuda.synchronize()
        host.step(loop, new, keep, qkv)


def test_two_loops_on_two_streams():
    loops = [Loop(96) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, (new, keep) in enumerate(PLAN):
        qkv = _feed(loops[2], new, keep, i)
        torch.cuda.synchronize()
        for loop, st in zip(loops, streams):
            with torch.cuda.stream(st):
                loop.qkv.copy_(loops[2].qkv)
                loop.new.copy_(loops[2].new)
                loop.keep.copy_(loops[2].keep)
                loop.step()
        torch.cuda.synchronize()
        loops[2].step()
        torch.cuda.synchronize()
        for loop in loops[:2]:
            for a, b in [(loop.o4, loops[2].o4), (loop.o16, loops[2].o16), (loop.k4, loops[2].k4),
                         (loop.tables, loops[2].tables), (loop.refs, loops[2].refs)]:
                assert torch.equal(a, b)
        del qkv


def test_out_of_blocks_leaves_the_caches_alone():
    loop = Loop(96)
    _feed(loop, [20, 1, 33, 7], [20, 1, 33, 7], 1)
    loop.step()
    torch.cuda.synchronize()
    loop.bits.zero_()  # no block is free any more
    loop.refs.clamp_(min=1)
    before = [x.clone() for x in (loop.k4, loop.v4, loop.k16, loop.v16, loop.tables, loop.ctx)]
    _feed(loop, [40, 1, 1, 1], [99, 99, 99, 99], 2)
    loop.step()
    torch.cuda.synchronize()
    assert loop.out[-1].tolist() == [1, 0, 2, 0]  # (20 + 40 tokens: two blocks more)
    for a, b in zip(before, (loop.k4, loop.v4, loop.k16, loop.v16, loop.tables, loop.ctx)):
        assert torch.equal(a, b)


def test_calls_on_another_stream_make_their_buffers_there():
    c = fp4.Cache([900, 40, 1300], 2, 16, seed=3)
    k, v, tables, lens = c.cuda()
    q = bsc.make_query(3, 8).cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    want = pgd.paged_decode_attention_fp4(None, q, k, v, tables, lens, SCALE, num_splits=3,
                                          **fp4.scales_kw(c))
    junk = [torch.ones(want.numel() * 200, dtype=torch.uint8, device="cuda") for _ in range(3)]
    del junk
    for _ in range(5):
        got = pgd.paged_decode_attention_fp4(None, q, k, v, tables, lens, SCALE, num_splits=3,
                                             stream=st, **fp4.scales_kw(c))
        st.synchronize()
        assert torch.equal(got, want)
    call = pgd.prepare("paged_decode_attention_fp4", None, q, k, v, tables, lens, SCALE,
                       num_splits=3, **fp4.scales_kw(c))
    new = [torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    for _ in range(2):
        assert torch.equal(call(), want)
    both = pgd.prepare("append_decode_attention_fp4", None, q, *new, k, v, tables, lens, SCALE,
                       **fp4.scales_kw(c))
    a = both().clone()
    assert torch.equal(a, pgd.paged_decode_attention_fp4(None, q, k, v, tables, lens, SCALE,
                                                         **fp4.scales_kw(c)))
    f = pgd.rope_frequencies(128)
    x, y = pgd.rope(None, None, q, new[0], lens, f, stream=st)
    z = pgd.rope(None, None, q, new[0], lens, f)
    torch.cuda.synchronize()
    assert torch.equal(x, z[0]) and torch.equal(y, z[1])
