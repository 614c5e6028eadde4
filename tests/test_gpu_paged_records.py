"""Sequences that contradict themselves are recorded by every call on a paged cache, also where no new token, and no
page of the packed layout, leads to them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def _world(m, n_seq, lens, off, hkv=1, hq=2, page=16, max_pages=20):
    kv = m.PagedKV.empty(64, n_seq, max_pages, hkv, page)
    kv.pages.view(torch.uint8).fill_(0x38)
    kv.page_table.copy_(torch.arange(n_seq * max_pages).view(n_seq, max_pages) % 64)
    kv.seq_len.copy_(torch.tensor(lens))
    off = torch.tensor(off, device="cuda")
    n_tok = int(off.max())
    q = torch.ones((n_tok, hq, D), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((n_tok, hkv, D), dtype=torch.bfloat16, device="cuda")
    cs = m.rope_table(max_pages * page, D)
    sel = torch.zeros((n_tok, hkv, 2), dtype=torch.int32, device="cuda")

    def calls(new):
        return {"append": lambda: m.msa_paged_append(kv, k, k, off, new, cs, q=q),
                "select": lambda: m.msa_page_select(kv, q, off, new, 2),
                "list": lambda: m.msa_paged_attn(kv, q, off, new, sel=sel),
                "attend": lambda: m.msa_paged_attn(kv, q, off, new)}
    return kv, calls


@pytest.mark.parametrize("call", ["append", "select", "list", "attend"])
def test_offsets_that_decrease(m, call):
    """The second sequence's end lies before its start; rows 50 .. 99 then belong to two others."""
    _, calls = _world(m, 3, [100, 0, 100], [0, 100, 50, 150])
    calls(100)[call]()
    assert m.device_status() == 3


@pytest.mark.parametrize("call", ["append", "select", "list", "attend"])
@pytest.mark.parametrize("n_seq", [3, 700])
@pytest.mark.parametrize("bad", [-1, 20 * 16 + 1])
def test_a_length_that_cannot_be_of_a_sequence_without_new_tokens(m, call, n_seq, bad):
    for where in (1, n_seq - 1):
        lens, off = [5] * n_seq, [0, 5] + [5] * (n_seq - 1)
        kv, calls = _world(m, n_seq, lens, off)
        for new in (5, 300):
            calls(new)[call]()
            assert m.device_status() == 0
            kv.seq_len[where] = bad
            calls(new)[call]()
            assert m.device_status() == 3
            kv.seq_len[where] = 5
