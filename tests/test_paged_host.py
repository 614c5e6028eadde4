"""The paged cache's entry points refuse bad arguments on the host, before any launch. No GPU is needed."""
import ctypes

import pytest
import torch

import routed_long_context_b200 as m
from routed_long_context_b200 import _lib

lib = _lib.lib
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def _kv(**over):
    a = dict(pages=256, scales=256, bounds=256, page_table=256, seq_len=256, n_pages=10, n_seq=2, max_pages=4, page=32,
             hkv=2, d=128)
    a.update(over)
    return _lib.PagedKVArgs(*(a[n] for n, _ in _lib.PagedKVArgs._fields_))


def _append(kv, k=256, v=256, q=256, dt=1, n_tok=3, hq=8, off=256, max_new=2, pos=0, cs=256, max_pos=9, q_rot=256):
    return lib.msa_paged_append(ctypes.byref(kv), k, v, q, dt, n_tok, hq, off, max_new, pos, cs, max_pos, q_rot, None)


def _attn(kv, q=256, dt=1, n_tok=3, hq=8, off=256, max_new=2, sel=None, k=0, out=256, lse=None, ws=256, nb=1 << 40):
    return lib.msa_paged_attn(ctypes.byref(kv), q, dt, n_tok, hq, off, max_new, sel, k, 0.1, out, lse, ws, nb, None)


def _select(kv, q=256, dt=1, n_tok=3, hq=8, off=256, max_new=2, k=2, recent=1, sel=256, ws=256, nb=1 << 40):
    return lib.msa_page_select(ctypes.byref(kv), q, dt, n_tok, hq, off, max_new, k, recent, sel, ws, nb, None)


@pytest.mark.parametrize("over,want", [
    (dict(pages=None), INVALID), (dict(scales=None), INVALID), (dict(page_table=None), INVALID),
    (dict(seq_len=None), INVALID), (dict(pages=264), INVALID), (dict(bounds=264), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_seq=0), INVALID), (dict(max_pages=0), INVALID), (dict(hkv=0), INVALID), (dict(d=64), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(max_pages=1 << 27), INVALID),
    (dict(n_pages=1 << 40), INVALID)])
def test_every_call_refuses_a_bad_cache(over, want):
    kv = _kv(**over)
    assert _append(kv) == want and _attn(kv) == want and _select(kv) == want
    assert lib.msa_paged_append(None, 256, 256, None, 1, 1, 0, 256, 1, 0, 256, 9, None, None) == INVALID


@pytest.mark.parametrize("over,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cs=None), INVALID), (dict(off=None), INVALID),
    (dict(q_rot=None), INVALID), (dict(hq=7), INVALID), (dict(hq=0), INVALID), (dict(dt=5), INVALID),
    (dict(n_tok=-1), INVALID), (dict(max_new=-1), INVALID), (dict(pos=-1), INVALID), (dict(max_pos=0), INVALID),
    (dict(k=260), INVALID), (dict(q=264), INVALID), (dict(n_tok=1 << 31), INVALID)])
def test_append_refuses(over, want):
    assert _append(_kv(), **over) == want and lib.msa_last_error()


@pytest.mark.parametrize("over,want", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(off=None), INVALID),
    (dict(dt=0), UNSUPPORTED), (dict(dt=9), INVALID), (dict(hq=7), INVALID), (dict(hq=6), UNSUPPORTED),
    (dict(hq=32), UNSUPPORTED), (dict(sel=256, k=0), INVALID), (dict(out=264), INVALID), (dict(nb=16), WORKSPACE),
    (dict(n_tok=-1), INVALID)])
def test_attention_refuses(over, want):
    assert _attn(_kv(), **over) == want and lib.msa_last_error()


@pytest.mark.parametrize("over,want", [
    (dict(q=None), INVALID), (dict(sel=None), INVALID), (dict(ws=None), INVALID), (dict(off=None), INVALID),
    (dict(dt=0), UNSUPPORTED), (dict(hq=7), INVALID), (dict(hq=6), UNSUPPORTED), (dict(k=0), INVALID),
    (dict(recent=0), INVALID), (dict(recent=3), INVALID), (dict(nb=16), WORKSPACE)])
def test_selection_refuses(over, want):
    assert _select(_kv(), **over) == want and lib.msa_last_error()
    assert _select(_kv(bounds=None)) == INVALID


def test_nothing_to_do_is_no_launch():
    assert _append(_kv(), n_tok=0) == 0 and _attn(_kv(), n_tok=0) == 0 and _select(_kv(), n_tok=0) == 0
    assert _append(_kv(), max_new=0) == 0 and _attn(_kv(), max_new=0) == 0 and _select(_kv(), max_new=0) == 0


def test_generic_workspace_queries_agree():
    n = ctypes.c_size_t(0)
    cfg = _lib.PagedAttnWsCfg(3, 2, 2, 8, 2, 4, 32, 0)
    assert lib.msa_workspace_size(_lib.MSA_OP_PAGED_ATTN, ctypes.byref(cfg), ctypes.byref(n)) == 0
    assert n.value == m.paged_attn_workspace_size(3, 2, 2, 8, 2, 4, 32)
    cfg = _lib.PageSelectWsCfg(3, 2, 4)
    assert lib.msa_workspace_size(_lib.MSA_OP_PAGE_SELECT, ctypes.byref(cfg), ctypes.byref(n)) == 0
    assert n.value == m.page_select_workspace_size(3, 2, 4)
    assert lib.msa_paged_attn_workspace_size(3, 0, 2, 8, 2, 4, 32, 0, ctypes.byref(n)) == INVALID
    assert lib.msa_page_select_workspace_size(-1, 2, 4, ctypes.byref(n)) == INVALID


def test_the_binding_checks_shapes_and_devices():
    f8, f32, i32 = torch.float8_e4m3fn, torch.float32, torch.int32
    pages, scales = torch.empty((3, 2, 2, 16, 128), dtype=f8), torch.ones((3, 2, 2))
    table, lens = torch.zeros((2, 2), dtype=i32), torch.zeros(2, dtype=i32)
    kv = m.PagedKV(pages, scales, table, lens)
    with pytest.raises(ValueError, match="scales"):
        m.PagedKV(pages, scales[:2], table, lens)
    with pytest.raises(ValueError, match="pages"):
        m.PagedKV(pages.view(torch.uint8), scales, table, lens)
    with pytest.raises(ValueError, match="seq_len"):
        m.PagedKV(pages, scales, table, lens.long())
    with pytest.raises(ValueError, match="bounds"):
        m.PagedKV(pages, scales, table, lens, torch.zeros((3, 2, 2, 128), dtype=f32))
    with pytest.raises(ValueError, match="contiguous"):
        m.PagedKV(pages, scales, torch.zeros((2, 4), dtype=i32)[:, ::2], lens)
    q, off = torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    if not torch.cuda.is_available():
        with pytest.raises(ValueError, match="current CUDA device"):
            m.msa_paged_attn(kv, q, off, 1)
        with pytest.raises(ValueError, match="current CUDA device"):
            m.msa_page_select(kv, q, off, 1, 1)
        with pytest.raises(ValueError, match="current CUDA device"):
            m.msa_paged_append(kv, q[:, :2].contiguous(), q[:, :2].contiguous(), off, 1, torch.zeros((4, 64, 2)))
