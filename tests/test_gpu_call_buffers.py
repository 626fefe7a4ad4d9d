"""Buffers that a call of the binding makes itself (its workspace, its output): how long they live
and on which stream they are made.  Every call is split so that partial states and their counters lie
in the workspace, and equals the same call on buffers of the caller's, bit for bit."""
import pytest
import torch

import block_scaled as bsc
import paged_gqa_decode_kv_gb300 as pgd
from paged_gqa_decode_kv_gb300 import inputs

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
LENS = [900, 40, 1300]
SPLITS = 3


@pytest.fixture(autouse=True)
def _clean_errors():
    pgd.device_errors(clear=True)
    yield
    assert pgd.device_errors(clear=True) == 0


def _paged(fp8=False, append=False):
    pb = inputs.make_batch(3, 8, 2, 16, LENS, seed=5, table_seed=6, device="cuda", append=append,
                           kv_format="fp8" if fp8 else "bf16")
    new = (pb.k_new, pb.v_new) if append else ()
    return (pb.q, *new, pb.k_cache, pb.v_cache, pb.block_tables, pb.context_lens, pb.scale)


def _verify():
    vb = inputs.make_verify_batch(3, 8, 2, 16, LENS, 4, seed=5, table_seed=6, device="cuda")
    pb = vb.paged
    return (vb.q, vb.k_new, vb.v_new, pb.k_cache, pb.v_cache, pb.block_tables, pb.context_lens,
            pb.scale)


def _mla(append=False):
    mb = inputs.make_mla_batch(3, 16, 16, LENS, seed=5, table_seed=6, device="cuda", append=append)
    return (mb.q, *((mb.c_new,) if append else ()), mb.cache, mb.block_tables, mb.context_lens,
            mb.scale)


def _blocks(append=False):
    c = bsc.make_cache(LENS, 2, 16, seed=3)
    k, v, ks, vs, tables, lens = c.cuda()
    q = bsc.make_query(3, 8).cuda()
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(3, 2, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    return (q, *(new if append else ()), k, v, ks, vs, tables, lens, SCALE)


def _selection(fp8):
    c = bsc.make_cache(LENS, 2, 16, fp8=fp8, seed=3)
    k, v, ks, vs, tables, lens = c.cuda()
    bounds = torch.zeros(k.shape[0], 2, 2, 128, dtype=torch.int8, device="cuda")
    scales = torch.ones(k.shape[0], 2, device="cuda")
    pgd.block_bounds(bounds, scales, k, tables, lens, k_scales=ks)
    tiles = torch.zeros(3, 2, 30, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    q = bsc.make_query(3, 8).cuda()
    return (q, k, v, bounds, scales, tables, lens, tiles, tokens, 1, 2, SCALE), dict(k_scales=ks,
                                                                                    v_scales=vs)


def _selected(fp8):
    args, kw = _selection(fp8)
    pgd.select_blocks(*args[7:9], args[0], *args[3:7], 1, 2, 16)
    return (*args[:3], *args[7:9], SCALE), kw


def _size(of):
    return {"paged": lambda: pgd.workspace_size(3, 8, 2, SPLITS),
            "verify": lambda: pgd.verify_workspace_size(3, 4, 8, 2, SPLITS),
            "mla": lambda: pgd.mla_workspace_size(3, 16, SPLITS),
            "blocks": lambda: pgd.block_workspace_size(3, 8, 2, SPLITS)}[of]()


# call: (its arguments behind the output, the kind of its workspace, whether it can be prepared)
CALLS = {
    "paged_decode_attention": (lambda: (_paged(), {}), "paged", True),
    "paged_decode_attention_fp8": (lambda: (_paged(True), {}), "paged", True),
    "append_decode_attention": (lambda: (_paged(append=True), {}), "paged", True),
    "append_decode_attention_fp8": (lambda: (_paged(True, True), {}), "paged", True),
    "append_verify_attention": (lambda: (_verify(), {}), "verify", True),
    "paged_decode_attention_fp8b": (lambda: (_blocks(), {}), "blocks", True),
    "append_decode_attention_fp8b": (lambda: (_blocks(True), {}), "blocks", True),
    "sparse_decode_attention": (lambda: _selection(True), "blocks", True),
    "sparse_decode_attention, bf16": (lambda: _selection(False), "blocks", True),
    "selected_decode_attention": (lambda: _selected(True), "blocks", False),
    "paged_verify_attention": (lambda: ((_verify()[0], *_paged()[1:]), {}), "verify", False),
    "mla_decode_attention": (lambda: (_mla(), {}), "mla", False),
    "mla_append_decode_attention": (lambda: (_mla(True), {}), "mla", False),
}
PREPARED = [name for name, c in CALLS.items() if c[2]]


def _setup(name):
    """(the call, its arguments, its keywords, what it gives on buffers of the caller's, bytes of
    its workspace)"""
    make, of, _ = CALLS[name]
    args, kw = make()
    kw = dict(kw, num_splits=SPLITS)
    fn = getattr(pgd, name.split(",")[0])
    n = _size(of)
    want = fn(None, *args, workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"), **kw)
    torch.cuda.synchronize()
    return fn, args, kw, want.clone(), n


def _ones(n, count=4):
    """Memory that an allocation of n bytes may be given next."""
    return [torch.ones(n, dtype=torch.uint8, device="cuda") for _ in range(count)]


@pytest.mark.parametrize("name", PREPARED)
def test_a_prepared_call_keeps_what_it_made(name):
    """The workspace and the output of a prepared call are its own for as long as it lives: later
    allocations of their sizes are other memory, which the call does not write."""
    fn, args, kw, want, n = _setup(name)
    call = pgd.prepare(name.split(",")[0], None, *args, **kw)
    later = _ones(n) + _ones(want.numel() * 2)
    for _ in range(3):
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert all(bool((x == 1).all()) for x in later)


def _busy(stream):
    """A few milliseconds of copies on a stream."""
    with torch.cuda.stream(stream):
        a = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
        b = torch.empty_like(a)
        for _ in range(24):
            b.copy_(a)


@pytest.mark.parametrize("slow", ["current", "given"])
@pytest.mark.parametrize("name", CALLS)
def test_buffers_made_for_a_call_on_another_stream(name, slow):
    """While the current stream is busy, and while the given one is: the fill of the counters comes
    before the call, and what the call has given back is not handed out before it is done."""
    fn, args, kw, want, n = _setup(name)
    side = torch.cuda.Stream()
    del _ones(n, 6)[:]  # what the allocator gives out next is not zero
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream() if slow == "current" else side)
    got = fn(None, *args, stream=side, **kw)
    later = _ones(n) + _ones(want.numel() * 2)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((x == 1).all()) for x in later)


def test_a_prepared_call_on_another_stream():
    fn, args, kw, want, n = _setup("paged_decode_attention_fp8b")
    side = torch.cuda.Stream()
    del _ones(n, 6)[:]
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    call = pgd.prepare("paged_decode_attention_fp8b", None, *args, stream=side, **kw)
    got = call()
    later = _ones(n)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(call(), want)
    assert all(bool((x == 1).all()) for x in later)


@pytest.mark.parametrize("name", ["paged_decode_attention", "sparse_decode_attention"])
def test_a_stream_given_by_its_handle(name):
    """Any object with a cuda_stream will do, as it does where the caller gives the buffers."""
    fn, args, kw, want, n = _setup(name)

    class Handle:
        cuda_stream = torch.cuda.Stream().cuda_stream

    got = fn(None, *args, stream=Handle(), **kw)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
