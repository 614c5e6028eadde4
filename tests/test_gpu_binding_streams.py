"""Calls on a stream of the caller's own while the current stream still has work queued: neither may overwrite what
the other uses."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
NAP = 20_000_000            # cycles: some 10 ms


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def _leave_queued(sizes):
    """Memory of these sizes that the current stream has freed but not yet written for the last time."""
    torch.cuda._sleep(NAP)
    for junk in [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]:
        junk.fill_(0xFF)


def _paged(m, new):
    g = torch.Generator(device="cuda").manual_seed(new)
    hkv, hq, page, n_seq = 2, 8, 32, 2
    kv = m.PagedKV.empty(80, n_seq, 40, hkv, page)
    kv.pages.copy_((torch.randn(kv.pages.shape, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn))
    kv.scales.fill_(2.0 ** -6)
    keys = kv.pages[:, 0].float() * 2.0 ** -6
    kv.bounds.copy_(torch.stack((keys.amin(2), keys.amax(2)), 2))
    kv.page_table.copy_(torch.randperm(80, generator=g, device="cuda").view(2, 40))
    kv.seq_len.copy_(torch.tensor([1100, 900]))
    off = torch.tensor([0, new, 2 * new], device="cuda")
    cs = m.rope_table(2000, D)
    k, v = (torch.randn((2 * new, hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((2 * new, hq, D), generator=g, device="cuda").bfloat16()

    def step(q=q, **s):
        """Append, pick, attend over the picked pages and over all."""
        qr = m.msa_paged_append(kv, k, v, off, new, cs, q=q, **s)
        sel = m.msa_page_select(kv, qr, off, new, 6, **s)
        return qr, sel, *m.msa_paged_attn(kv, qr, off, new, sel=sel, want_lse=True, **s), *m.msa_paged_attn(
            kv, qr, off, new, want_lse=True, **s)

    sizes = [m.page_select_workspace_size(2 * new, hkv, 40), m.paged_attn_workspace_size(2 * new, 2, new, hq, hkv, 40, page),
             m.paged_attn_workspace_size(2 * new, 2, new, hq, hkv, 40, page, 6)]
    return q, step, sizes


@pytest.mark.parametrize("new", [1, 80])
def test_a_backlog_on_the_current_stream_does_not_reach_a_paged_call(m, new):
    q, step, sizes = _paged(m, new)
    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        _leave_queued([x.nbytes for x in want] + sizes)
        got = step(stream=side)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert m.device_status() == 0


@pytest.mark.parametrize("new", [1, 80])
def test_results_of_a_paged_call_outlive_what_the_current_stream_reads(m, new):
    """Results dropped while the current stream has yet to read them are not handed to the side stream's next call."""
    q, step, _ = _paged(m, new)
    want = [x.clone() for x in step()]
    other = q.flip(0).contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(NAP)
        kept = [x.clone() for x in got]
        del got
        step(other, stream=side)
        torch.cuda.synchronize()
        for x, y in zip(kept, want):
            assert torch.equal(x, y)
    assert m.device_status() == 0


def test_a_backlog_on_the_current_stream_does_not_reach_an_older_call(m):
    """Selection (results and scratch), the fetch (rows that the call zeroes before it fills them) and attention."""
    g = torch.Generator(device="cuda").manual_seed(3)
    C, k, hkv = 4000, 8, 2
    scores = torch.randn((4, C), generator=g, device="cuda")
    bank = torch.randn((C, 2, hkv, D), generator=g, device="cuda").bfloat16().cpu().pin_memory()
    off = torch.arange(C + 1, device="cuda")
    q = torch.randn((4, 16, 8, D), generator=g, device="cuda").bfloat16()
    loc = torch.randn((4, 16, hkv, D), generator=g, device="cuda").bfloat16()

    def step(**s):
        idx, top = m.msa_topk_docs(scores, k, **s)
        mem, n = m.msa_gather_kv_device(bank, off, idx, k, **s)
        return idx, top, mem, n, m.msa_sparse_attn(q, mem, n, loc, loc, 16, 0, **s), m.msa_sparse_attn_split(
            q, mem, n, loc, loc, 16, 0, **s)

    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    sizes = [x.nbytes for x in want] + [m.topk_workspace_size(4, C, k), m.sparse_attn_split_workspace_size(4, 16, 8, hkv, k, 16)]
    side = torch.cuda.Stream()
    for _ in range(3):
        _leave_queued(sizes)
        got = step(stream=side)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert m.device_status() == 0
