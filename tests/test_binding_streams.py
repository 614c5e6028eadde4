"""What the binding allocates for a call on a stream of the caller's own. No GPU is needed: streams and the library
are stood in for, and the allocations are watched as torch makes them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import routed_long_context_b200 as m
from routed_long_context_b200 import api

D = 128
ALLOCATIONS = ("empty", "new_empty", "empty_like", "zeros", "new_zeros", "zeros_like", "fill_", "zero_", "full")


class Stream:
    def __init__(self, cuda_stream, index=0):
        self.cuda_stream, self.device_index = cuda_stream, index


class Watch(TorchDispatchMode):
    """Where each allocation or fill happened: the current stream of that moment."""

    def __init__(self, world):
        super().__init__()
        self.world, self.seen = world, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        name = func.overloadpacket.__name__
        if name in ALLOCATIONS:
            self.seen.append((name, self.world.current))
        return func(*args, **(kwargs or {}))


class World:
    """Streams as torch would show them, and the records of what is kept for which."""

    def __init__(self, monkeypatch):
        self.usual, self.side = Stream(7), Stream(9)
        self.current, self.kept, self.launched = self.usual, [], []

        monkeypatch.setattr(torch.cuda, "set_stream", lambda s: setattr(self, "current", s))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.current.cuda_stream)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.kept.append((t, s)))
        monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)

    def stub(self, monkeypatch, name):
        monkeypatch.setattr(api.lib, name, lambda *a: self.launched.append((name, a)) or 0)

    def kept_for(self, t):
        return [s for x, s in self.kept if x is t]


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _cache(monkeypatch):
    kv = m.PagedKV(torch.empty((3, 2, 2, 16, D), dtype=torch.float8_e4m3fn), torch.ones((3, 2, 2)),
                   torch.zeros((1, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                   torch.zeros((3, 2, 2, D), dtype=torch.bfloat16))
    monkeypatch.setattr(m.PagedKV, "_check", lambda *a: None)
    return kv


def _paged_calls(kv):
    q, off = torch.zeros((2, 4, D), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    k, cs = torch.zeros((2, 2, D), dtype=torch.bfloat16), torch.zeros((4, D // 2, 2))
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    return {
        "append": ("msa_paged_append", lambda **s: m.msa_paged_append(kv, k, k, off, 2, cs, q=q, **s)),
        "select": ("msa_page_select", lambda **s: m.msa_page_select(kv, q, off, 2, 3, **s)),
        "select, scratch given": ("msa_page_select", lambda **s: m.msa_page_select(kv, q, off, 2, 3, ws=ws, **s)),
        "attend": ("msa_paged_attn", lambda **s: m.msa_paged_attn(kv, q, off, 2, want_lse=True, **s)),
        "attend, scratch given": ("msa_paged_attn", lambda **s: m.msa_paged_attn(kv, q, off, 2, want_lse=True, ws=ws, **s)),
    }


@pytest.mark.parametrize("which", ["append", "select", "select, scratch given", "attend", "attend, scratch given"])
def test_what_a_paged_call_allocates_belongs_to_its_stream(monkeypatch, world, which):
    """Memory of the current stream may still be in use by what is queued there: results and scratch come from the
    call's own stream, and the results are kept until the current stream is done with them."""
    kv = _cache(monkeypatch)
    name, call = _paged_calls(kv)[which]
    world.stub(monkeypatch, name)
    with Watch(world) as w:
        got = call(stream=world.side)
    assert w.seen and all(s is world.side for _, s in w.seen), w.seen
    assert [a[-1] for _, a in world.launched] == [world.side.cuda_stream] and world.current is world.usual
    for t in got if isinstance(got, tuple) else (got,):
        assert world.usual in world.kept_for(t)


@pytest.mark.parametrize("which", ["append", "select", "attend"])
def test_a_paged_call_without_a_stream_stays_on_the_current_one(monkeypatch, world, which):
    kv = _cache(monkeypatch)
    name, call = _paged_calls(kv)[which]
    world.stub(monkeypatch, name)
    with Watch(world) as w:
        call()
    assert all(s is world.usual for _, s in w.seen) and not world.kept
    assert world.launched[0][1][-1] == world.usual.cuda_stream


def test_a_stream_of_another_device_is_refused(monkeypatch, world):
    kv = _cache(monkeypatch)
    for name, call in _paged_calls(kv).values():
        world.stub(monkeypatch, name)
        with pytest.raises(ValueError, match="device"):
            call(stream=Stream(11, index=1))
    assert not world.launched


def _older_calls():
    bf, i32, i64, f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    x, off = torch.zeros((6, 2, D), dtype=bf), torch.tensor([0, 3, 6])
    off2 = torch.tensor([0, 1, 2])
    chunks, cs, doc = torch.zeros((2, 2, D), dtype=bf), torch.zeros((8, D // 2, 2)), torch.zeros(2, dtype=i32)
    bank, qr = torch.zeros((2, 2, 2, D), dtype=bf), torch.zeros((1, 3, 2, D), dtype=bf)
    q, loc = torch.zeros((1, 3, 4, D), dtype=bf), torch.zeros((1, 4, 2, D), dtype=bf)
    mem, ln = torch.zeros((1, 2, 2, 2, D), dtype=bf), torch.zeros(1, dtype=i32)
    sc, idx = torch.zeros((1, 2)), torch.zeros((1, 1), dtype=i32)
    fq, dmem = torch.zeros((1, 3, 4)), torch.zeros((1, 2, 2, 2, D))
    return {
        "msa_chunk_doc_map": lambda **s: m.chunk_doc_map(off, 6, **s),
        "msa_pool_chunks": lambda **s: m.msa_pool_chunks(x, x, x, off, off2, doc, 3, cos_sin=cs, **s),
        "msa_pack_tokens": lambda **s: m.msa_pack_tokens(x, x, off, cs, **s),
        "msa_route_scores": lambda **s: m.msa_route_scores(chunks, doc, 2, qr, want_chunk_scores=True, **s),
        "msa_topk_docs": lambda **s: m.msa_topk_docs(sc, 1, **s),
        "msa_topk_docs_noalloc": lambda **s: m.msa_topk_docs_noalloc(sc, 1, **s),
        "msa_topk_merge": lambda **s: m.msa_topk_merge(sc[None], idx.expand(1, 2)[None].contiguous(), [0, 2], 1, **s),
        "msa_gather_kv": lambda **s: m.msa_gather_kv(bank, off2, idx, 2, device="cpu", **{"copy_" + n: v for n, v in s.items()}),
        "msa_gather_kv_device": lambda **s: m.msa_gather_kv_device(bank, off2, idx, 2, **s),
        "msa_sparse_attn": lambda **s: m.msa_sparse_attn(q, mem, ln, loc, loc, 4, 1, **s),
        "msa_sparse_attn_split": lambda **s: m.msa_sparse_attn_split(q, mem, ln, loc, loc, 4, 1, **s),
        "msa_sparse_attn_backward": lambda **s: m.msa_sparse_attn_backward(q, mem, ln, loc, loc, 4, 1, q, q, fq, **s),
        "msa_gather_kv_backward": lambda **s: m.msa_gather_kv_backward(dmem, off2, idx, 2, **s),
        "msa_pool_chunks_backward": lambda **s: m.msa_pool_chunks_backward(
            torch.zeros((2, 2, 2, D)), torch.zeros((2, 2, D)), off, off2, doc, 3, 6, kr=x, cos_sin=cs, **s),
        "msa_router_aux_loss": lambda **s: m.msa_router_aux_loss(sc, idx.to(i64), 0.1, **s),
        "msa_route_backward": lambda **s: m.msa_route_backward(chunks, off2, qr, sc, **s),
    }


def _made(w):
    return [s for _, s in w.seen]


@pytest.mark.parametrize("name", list(_older_calls()))
def test_what_a_call_allocates_or_fills_belongs_to_its_stream(monkeypatch, world, name):
    call = _older_calls()[name]
    world.stub(monkeypatch, name)
    with Watch(world) as w:
        call()                                     # the inputs' own conversions may allocate too: not on this list
    assert all(s is world.usual for s in _made(w)) and not world.kept
    with Watch(world) as w:
        got = call(stream=world.side)
    assert world.side in _made(w)
    # what the call made after it began: everything from the first allocation on the side stream
    assert all(s is world.side for s in _made(w)[_made(w).index(world.side):])
    handles = [a[-1] for _, a in world.launched]
    assert handles == [world.usual.cuda_stream, world.side.cuda_stream]
    for t in got if isinstance(got, tuple) else (got,):
        assert world.usual in world.kept_for(t)


def test_a_stream_may_be_given_by_place(monkeypatch, world):
    world.stub(monkeypatch, "msa_topk_docs")
    sc = torch.zeros((1, 2))
    with Watch(world) as w:
        m.msa_topk_docs(sc, 1, None, None, None, world.side)
    assert _made(w) and all(s is world.side for s in _made(w))
    given = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 1))
    world.kept.clear()
    got = m.msa_topk_docs(sc, 1, idx=given[0], score=given[1], stream=world.side)
    assert got[0] is given[0] and not world.kept       # the caller's own tensors are the caller's


def test_where_nothing_is_allocated_the_current_stream_stays(monkeypatch, world):
    """The call goes to the stream by its handle alone, and nothing is kept for anyone."""
    kv = _cache(monkeypatch)
    for name in ("msa_paged_append", "msa_page_select", "msa_paged_attn", "msa_topk_docs", "msa_route_scores", "msa_sparse_attn"):
        world.stub(monkeypatch, name)
    monkeypatch.setattr(torch.cuda, "set_stream", None)
    q, off = torch.zeros((2, 4, D), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    k, cs, ws = torch.zeros((2, 2, D), dtype=torch.bfloat16), torch.zeros((4, D // 2, 2)), torch.zeros(1 << 20, dtype=torch.uint8)
    sel, lse, sc = torch.zeros((2, 2, 3), dtype=torch.int32), torch.zeros((2, 4)), torch.zeros((1, 2))
    idx, doc = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    qr, q4, loc = torch.zeros((1, 3, 2, D)), q[None], torch.zeros((1, 2, 2, D), dtype=torch.bfloat16)
    mem = torch.zeros((1, 2, 2, 2, D), dtype=torch.bfloat16)
    s = {"stream": world.side}
    with Watch(world) as w:
        m.msa_paged_append(kv, k, k, off, 2, cs, **s)
        m.msa_paged_append(kv, k, k, off, 2, cs, q=q, q_rot=q, **s)
        m.msa_page_select(kv, q, off, 2, 3, sel=sel, ws=ws, **s)
        m.msa_paged_attn(kv, q, off, 2, out=q, ws=ws, **s)
        m.msa_paged_attn(kv, q, off, 2, out=q, lse=lse, want_lse=True, ws=ws, **s)
        m.msa_topk_docs(sc, 1, idx, sc[:, :1], ws, world.side)
        m.msa_route_scores(qr[0], doc, 2, qr, doc_scores=sc, ws=ws, **s)
        m.msa_sparse_attn(q4, mem, doc, loc, loc, 2, 0, out=q4, **s)
    assert not w.seen and not world.kept
    assert [a[-1] for _, a in world.launched] == [world.side.cuda_stream] * 8


def test_the_current_stream_given_by_name_is_no_switch(monkeypatch, world):
    kv = _cache(monkeypatch)
    monkeypatch.setattr(torch.cuda, "set_stream", None)
    for name, call in _paged_calls(kv).values():
        world.stub(monkeypatch, name)
        call(stream=world.usual)
    assert not world.kept and all(a[-1] == world.usual.cuda_stream for _, a in world.launched)


def test_chunk_scores_that_are_wanted_belong_to_the_stream_too(monkeypatch, world):
    world.stub(monkeypatch, "msa_route_scores")
    qr, sc = torch.zeros((1, 3, 2, D)), torch.zeros((1, 2))
    args = qr[0], torch.zeros(2, dtype=torch.int32), 2, qr
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with Watch(world) as w:
        got = m.msa_route_scores(*args, doc_scores=sc, want_chunk_scores=True, ws=ws, stream=world.side)
    assert _made(w) == [world.side] and got[0] is sc
    assert world.kept_for(got[1]) == [world.usual] and not world.kept_for(sc)
    assert world.launched[0][1][-1] == world.side.cuda_stream and world.current is world.usual
