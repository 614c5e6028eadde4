"""Page selection where the 32-bit scores do not decide: queries and bounds that are not finite, more pages than
candidates are kept for, near-ties."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_cache as C

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def _cache(m, lo, hi, page=16):
    """One sequence of len(lo) full pages with these bounds [pages, hkv, d], in shuffled places; keys do not matter."""
    n, hkv, _ = lo.shape
    kv = m.PagedKV.empty(n + 3, 1, n, hkv, page)
    ids = torch.from_numpy(np.random.default_rng(n).permutation(n + 3)[:n].astype(np.int32))
    kv.page_table.copy_(ids[None])
    kv.seq_len.fill_(n * page)
    kv.bounds[ids.long().cuda()] = torch.stack((lo, hi), 2).cuda().bfloat16()
    return kv


def _near_ties(seed, n, hkv=1):
    """Bounds of which one element is large, so that the sums of the small ones are lost in 32 bits."""
    x = torch.rand((n, hkv, D), generator=torch.Generator().manual_seed(seed)) * 0.1
    x[..., 0] = 2.0 ** 20
    x = x.bfloat16().float()
    return -x, x


def _want(lo, hi, q, k, recent):
    """The definition over the heads of q [G, d] (finite ones)."""
    return C.pick(C.page_scores(q, lo.double().numpy(), hi.double().numpy()), k, recent)


@pytest.mark.parametrize("k", [20, 300])
@pytest.mark.parametrize("where", [1, 2])
def test_a_query_head_that_is_nan_does_not_blur_the_others(m, where, k):
    """Its sum counts for nothing, and what the sums of the other heads may be off by is still allowed for."""
    lo, hi = _near_ties(1, 700)
    kv = _cache(m, lo, hi)
    q = torch.zeros((1, 4, D))
    q[0, 0] = 1.0
    q[0, where, 7] = math.nan
    off = torch.tensor([0, 1], device="cuda")
    sel = m.msa_page_select(kv, q.bfloat16().cuda(), off, 1, k).cpu().numpy()
    assert m.device_status() == 0
    np.testing.assert_array_equal(sel[0, 0], _want(lo[:, 0], hi[:, 0], np.ones((1, D)), k, 1))


@pytest.mark.parametrize("place", [0, 1, 127, 128, 500])
def test_a_page_whose_bounds_are_nan_does_not_blur_the_others(m, place):
    lo, hi = _near_ties(2, 700)
    nan_lo, nan_hi = lo.clone(), hi.clone()
    nan_lo[place], nan_hi[place] = math.nan, math.nan
    # the largest bounds of the other pages come before and after it
    kv = _cache(m, nan_lo, nan_hi)
    off = torch.tensor([0, 1], device="cuda")
    sel = m.msa_page_select(kv, torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda"), off, 1, 20).cpu().numpy()
    assert m.device_status() == 0
    s = C.page_scores(np.ones((1, D)), lo[:, 0].double().numpy(), hi[:, 0].double().numpy())
    s[place] = -np.inf
    np.testing.assert_array_equal(sel[0, 0], C.pick(s, 20, 1))


def _ordinary(seed, n, hkv):
    g = torch.Generator().manual_seed(seed)
    a, b = torch.randn((2, n, hkv, D), generator=g).bfloat16().float()
    return torch.minimum(a, b), torch.maximum(a, b)


@pytest.mark.parametrize("n", [18, 33, 65, 255, 257, 300, 511, 513, 1000, 1025, 2047, 2081])
@pytest.mark.parametrize("k", [1, 17, 63, 250])
def test_any_number_of_pages(m, n, k):
    """Warps whose lanes have unlike numbers of pages, and single lanes with one."""
    lo, hi = _ordinary(n + k, n, 2)
    kv = _cache(m, lo, hi)
    q = torch.randn((1, 4, D), generator=torch.Generator().manual_seed(k)).bfloat16()
    off = torch.tensor([0, 1], device="cuda")
    recent = min(2, k)
    sel = m.msa_page_select(kv, q.cuda(), off, 1, k, recent).cpu().numpy()
    assert m.device_status() == 0
    for g in range(2):
        np.testing.assert_array_equal(sel[0, g], _want(lo[:, g], hi[:, g], q[0, 2 * g:2 * g + 2].double().numpy(), k, recent))


@pytest.mark.parametrize("room", [40000, 60000])
@pytest.mark.parametrize("first", [0, 5])
def test_a_selection_that_goes_through_its_tokens_in_slices(m, room, first):
    """A table with room for long contexts: the scratch holds fewer tokens than the call has. The slices end within
    sequences; the same call with a tight table takes all tokens at once."""
    hkv, G, page, news, lens = 8, 2, 16, [150, 0, 90, 33], [1700, 40, 2600, 33]
    n_tok = first + sum(news) + 4
    rows = n_tok * hkv * 8
    assert m.page_select_workspace_size(n_tok, hkv, room) < rows * room and rows * 200 < 1 << 27
    g = torch.Generator().manual_seed(room)
    tight = m.PagedKV.empty(300, 4, 200, hkv, page)
    a, b = torch.randn((2, 300, hkv, D), generator=g)
    tight.bounds.copy_(torch.stack((torch.minimum(a, b), torch.maximum(a, b)), 2))
    tight.page_table.copy_(torch.stack([torch.randperm(300, generator=g)[:200] for _ in range(4)]))
    tight.seq_len.copy_(torch.tensor(lens))
    table = torch.zeros((4, room), dtype=torch.int32, device="cuda")
    table[:, :200] = tight.page_table
    wide = m.PagedKV(tight.pages, tight.scales, table, tight.seq_len, tight.bounds)
    off = torch.tensor(np.concatenate([[0], np.cumsum(news)]) + first, device="cuda")
    q = torch.randn((n_tok, hkv * G, D), generator=g).bfloat16().cuda()
    sels = []
    for kv in (tight, wide):
        sel = torch.full((n_tok, hkv, 7), 77, dtype=torch.int32, device="cuda")
        m.msa_page_select(kv, q, off, max(news), 7, 2, sel=sel)
        sels.append(sel)
    assert m.device_status() == 0
    assert torch.equal(*sels)
    assert (sels[0][:first] == 77).all() and (sels[0][-4:] == 77).all() and (sels[0][first:-4] < 77 * 3).all()
    qs, bounds = q.double().cpu().numpy(), tight.bounds.double().cpu().numpy()
    at = first
    for s, n in enumerate(news):
        for i in range(0, n, 29):
            ids = tight.page_table[s, :(lens[s] - n + i) // page + 1].long().cpu().numpy()
            for h in (0, hkv - 1):
                sc = C.page_scores(qs[at + i, h * G:h * G + G], bounds[ids, h, 0], bounds[ids, h, 1])
                np.testing.assert_array_equal(sels[0][at + i, h].cpu().numpy(), C.pick(sc, 7, 2))
        at += n


def test_guards_beside_the_scratch_of_slices(m):
    hkv, room, n_tok = 8, 40000, 150
    kv = m.PagedKV.empty(40, 1, room, hkv, 16)
    kv.page_table[0, :40] = torch.arange(40, device="cuda")
    kv.seq_len.fill_(640)
    need = m.page_select_workspace_size(n_tok, hkv, room)
    assert need < n_tok * hkv * room * 8
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    q = torch.randn((n_tok, hkv, D), device="cuda").bfloat16()
    m.msa_page_select(kv, q, torch.tensor([0, n_tok], device="cuda"), n_tok, 3, ws=buf[256:256 + need])
    assert m.device_status() == 0
    assert (buf[:256] == 0x5A).all() and (buf[256 + need:] == 0x5A).all()


@pytest.mark.parametrize("n", [1000, 3001])
@pytest.mark.parametrize("k", [257, 300, 901])
def test_more_pages_picked_than_candidates_are_kept_for(m, n, k):
    lo, hi = _ordinary(n * 3 + k, n, 2)
    kv = _cache(m, lo, hi)
    new = 3
    q = torch.randn((new, 8, D), generator=torch.Generator().manual_seed(n)).bfloat16()
    off = torch.tensor([0, new], device="cuda")
    sel = m.msa_page_select(kv, q.cuda(), off, new, k, 4).cpu().numpy()
    assert m.device_status() == 0
    for i in range(new):
        for g in range(2):
            np.testing.assert_array_equal(
                sel[i, g], _want(lo[:, g], hi[:, g], q[i, 4 * g:4 * g + 4].double().numpy(), k, 4))


@pytest.mark.parametrize("above,k", [(0, 20), (100, 120), (100, 139), (280, 281), (280, 300), (280, 319)])
@pytest.mark.parametrize("near", [40, 250, 257])
def test_near_ties_at_the_border_alone(m, above, k, near):
    """Pages far above and far below, and some at the border that 32-bit sums cannot tell apart."""
    n = 1500
    lo, hi = _near_ties(above + near, n)
    kind = torch.from_numpy(np.random.default_rng(near).permutation(n))
    hi[kind < above, 0, 0] = 2.0 ** 21
    hi[kind >= above + near, 0, 0] = 2.0 ** 19
    kv = _cache(m, lo, hi)
    off = torch.tensor([0, 1], device="cuda")
    sel = m.msa_page_select(kv, torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda"), off, 1, k).cpu().numpy()
    assert m.device_status() == 0
    np.testing.assert_array_equal(sel[0, 0], _want(lo[:, 0], hi[:, 0], np.ones((1, D)), k, 1))
