"""Paged attention over lists and page selection, what the host sees of them: a page list without entries is refused (it
is not the same as no list), scratch is bounded. No GPU is needed."""
import pytest
import torch

import routed_long_context_b200 as m
from routed_long_context_b200 import api

D = 128


@pytest.mark.parametrize("shape", [(2, 2, 0), (2, 0), (0,), ()])
def test_an_empty_page_list_is_refused(monkeypatch, shape):
    kv = m.PagedKV(torch.empty((3, 2, 2, 16, D), dtype=torch.float8_e4m3fn), torch.ones((3, 2, 2)),
                   torch.zeros((1, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    monkeypatch.setattr(m.PagedKV, "_check", lambda *a: None)
    monkeypatch.setattr(m.PagedKV, "_stream", lambda *a: 0)
    launched = []
    monkeypatch.setattr(api.lib, "msa_paged_attn", lambda *a: launched.append(a) or 0)
    q, off = torch.zeros((2, 4, D), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="sel"):
        m.msa_paged_attn(kv, q, off, 2, sel=torch.zeros(shape, dtype=torch.int32))
    assert not launched
    m.msa_paged_attn(kv, q, off, 2, sel=torch.zeros((2, 2, 1), dtype=torch.int32))
    assert launched[0][7] and launched[0][8] == 1


@pytest.mark.parametrize("n_tok,hkv,max_pages", [(65536, 8, 1025), (16384, 8, 12501), (1 << 20, 8, 16385), (4096, 1, 1 << 20)])
def test_the_scratch_of_a_long_selection_is_bounded(n_tok, hkv, max_pages):
    assert m.page_select_workspace_size(n_tok, hkv, max_pages) <= 256 << 20


@pytest.mark.parametrize("n_tok,hkv,max_pages", [(1, 1, 1), (1, 8, 1025), (64, 8, 6251), (7, 3, 129), (1, 64, 1 << 20)])
def test_the_scratch_of_a_selection_holds_a_row_of_scores_a_token(n_tok, hkv, max_pages):
    """8 bytes a page, and a maximum of 128 pages' bounds beside them."""
    least = n_tok * hkv * (8 * max_pages + 4 * -(-max_pages // 128))
    assert least <= m.page_select_workspace_size(n_tok, hkv, max_pages) <= least + 512


def test_the_testing_hook_of_attention_refuses_what_is_no_setting():
    assert api.lib.msa_paged_inject_stall(-1) == 1 and api.lib.msa_paged_inject_stall(1001) == 1
    assert api.lib.msa_paged_inject_stall(0) == 0
