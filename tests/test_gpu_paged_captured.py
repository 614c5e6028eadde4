"""Paged attention of many rows in CUDA graphs: lengths, table, queries and pages move on between replays."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.mark.parametrize("new,n_seq", [(20, 3), (200, 2), (40, 600)])      # 128 rows, 256 rows, two launches
@pytest.mark.parametrize("own_scratch", [False, True])
def test_a_captured_round_of_many_rows_replays(m, new, n_seq, own_scratch):
    """A table of this size takes the calls to the kernel for many rows (as they would go eagerly: the eager call is
    compared). Two graphs whose calls allocate for themselves, or two calls that share the caller's scratch."""
    hkv, hq, page, room = 2, 8, 64, 4096
    g = torch.Generator().manual_seed(new)
    n_pages = 400
    kv = m.PagedKV.empty(n_pages, n_seq, room, hkv, page)
    kv.page_table[:, :40] = torch.randint(0, n_pages - 200, (n_seq, 40), generator=g).int().cuda()   # pages to read are shared
    kv.pages.copy_((torch.randn(kv.pages.shape, generator=g) * 60).to(torch.float8_e4m3fn))
    kv.scales.fill_(2.0 ** -6)
    per = [max(1, new - 7 * (i % 5)) for i in range(n_seq)] if n_seq < 10 else [new if i % 300 == 5 else i % 2 for i in range(n_seq)]
    off = torch.tensor([0, *torch.tensor(per).cumsum(0).tolist()], device="cuda")
    n_tok = int(off[-1])
    q = torch.empty((n_tok, hq, D), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    lses = [torch.empty((n_tok, hq), device="cuda") for _ in range(2)]
    need = m.paged_attn_workspace_size(n_tok, n_seq, new, hq, hkv, room, page)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if own_scratch else None
    lens = torch.tensor([max(n, 900 + 31 * (i % 7)) for i, n in enumerate(per)], dtype=torch.int32)

    def refill(i):
        torch.manual_seed(i)
        q.copy_(torch.randn(q.shape))
        kv.seq_len.copy_(lens + i * 173)
        kv.page_table[:, :40] = kv.page_table[:, :40].flip(1)

    def call(j):
        m.msa_paged_attn(kv, q, off, new, out=outs[j], lse=lses[j], ws=ws)

    refill(0)
    call(0)
    torch.cuda.synchronize()
    assert m.device_status() == 0
    graphs = []
    for j in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(j)
            call(j)
        graphs.append(graph)
    for i in range(1, 6):
        refill(i)
        for x in outs + lses:
            x.fill_(7.0)
        for graph in graphs:
            graph.replay()
        out, lse = m.msa_paged_attn(kv, q, off, new, want_lse=True)
        for j in range(2):
            assert torch.equal(outs[j], out) and torch.equal(lses[j], lse), (i, j)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert m.device_status() == 0
