"""Failure detection of paged attention on the GPU without a fault: a testing hook makes the loaders of a launch bring
nothing from some tile on; the other warps' bounded waits run out, the kernel records a timeout and leaves, and the
context keeps working."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


# new tokens a sequence, pages of the table, listed pages: row blocks of 8 rows, the same over lists, row blocks of 128, of 256
@pytest.mark.parametrize("new,room,k", [(1, 300, 0), (1, 300, 120), (20, 4096, 0), (100, 4096, 0)])
@pytest.mark.parametrize("on", [1, 2])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(m, new, room, k, on):
    from routed_long_context_b200 import _lib

    g = torch.Generator(device="cuda").manual_seed(new)
    hkv, hq, page, n_seq, pages = 8, 32, 64, 2, 290
    kv = m.PagedKV.empty(pages, n_seq, room, hkv, page)
    kv.pages.copy_((torch.randn(kv.pages.shape, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn))
    kv.scales.fill_(2.0 ** -6)
    for s in range(n_seq):
        kv.page_table[s, :pages] = torch.randperm(pages, generator=g, device="cuda").int()
    kv.seq_len.copy_(torch.tensor([pages * page, pages * page - 700]))
    off = torch.tensor([0, new, 2 * new], device="cuda")
    q = torch.randn((2 * new, hq, D), generator=g, device="cuda").bfloat16()
    sel = torch.arange(k, device="cuda").int().repeat(2 * new, hkv, 1) if k else None
    ws = torch.zeros(m.paged_attn_workspace_size(2 * new, n_seq, new, hq, hkv, room, page, k), dtype=torch.uint8, device="cuda")
    call = lambda: m.msa_paged_attn(kv, q, off, new, sel=sel, want_lse=True, ws=ws)  # noqa: E731
    want = call()
    assert m.device_status() == 0
    _lib.check(_lib.lib.msa_paged_inject_stall(on), "inject")
    try:
        t0 = time.time()
        call()
        code = m.device_status()                   # synchronises: the launch returns after its bounded waits
        waited = time.time() - t0
    finally:
        _lib.check(_lib.lib.msa_paged_inject_stall(0), "inject")
    assert code == 2, code                         # MSA_DEV_WAIT_TIMEOUT
    assert 1.0 < waited < 30.0, waited
    for _ in range(2):
        got = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert m.device_status() == 0
