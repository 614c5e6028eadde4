"""Paged attention where a block adds up very many key tiles: pages that a table names again and again stand for the
long context, and the reference counts each key as often as it is seen. 64 bits, on the GPU.

Tolerances: as in test_gpu_paged.py, 2^-8 of the output and of the weighted magnitudes for the two roundings to bf16, the
logits' own errors, and 2^-11 for the sums: at most 4,096 steps of the tensor cores in a row, each cut off at 2^-23."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def _cache(m, n_pages, n_seq, room, hkv, page, g, positive=False):
    kv = m.PagedKV.empty(n_pages, n_seq, room, hkv, page, bounds=False)
    x = torch.randn(kv.pages.shape, generator=g, device="cuda") * 60
    if positive:
        x[:, 1].abs_()
    kv.pages.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn))
    kv.scales.fill_(2.0 ** -6)
    return kv


def _check(kv, s, head, q, out, lse, first_seen, scale):
    """q, out [n, G, D], lse [n, G] of the tokens that see first_seen, first_seen + 1, ... keys of sequence s."""
    n, page = q.shape[0], kv.page
    stored = kv.pages.view(torch.uint8)[:, :, head].view(torch.float8_e4m3fn).double() * 2.0 ** -6
    k, v = stored[:, 0].reshape(-1, D), stored[:, 1].reshape(-1, D)
    mult = torch.zeros((n, kv.pages.shape[0], page), dtype=torch.float64, device="cuda")
    for i in range(n):
        full, rest = divmod(first_seen + i, page)
        mult[i] += torch.bincount(kv.page_table[s, :full], minlength=mult.shape[1])[:, None]
        if rest:
            mult[i, kv.page_table[s, full].long(), :rest] += 1
    mult = mult.reshape(n, 1, -1)
    q = q.double()
    z = torch.einsum("ngd,kd->ngk", q, k) * scale + torch.log(mult)
    p = torch.softmax(z, -1)
    ref, a, l = p @ v, p @ v.abs(), torch.logsumexp(z, -1)
    delta = abs(scale) * 2.0 ** -17 * (q.abs().amax(-1, keepdim=True) * k.abs().sum(-1) + torch.einsum("ngd,kd->ngk", q.abs(), k.abs()))
    delta = torch.where(mult > 0, delta, 0.0).amax(-1)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11 + torch.expm1(2 * delta))[..., None] * a
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - l).abs() <= delta + 2.0 ** -20 * (l.abs() + 40)).all()


@pytest.mark.parametrize("new,G", [(1, 4), (40, 1), (40, 4)])           # few rows, row blocks of 128, of 256
def test_the_longest_context_that_a_table_can_name(m, new, G):
    """2^31 - 256 keys, one page over and over, values of one sign: a sum that is cut off step by step falls short."""
    page, L = 128, 2 ** 31 - 256
    g = torch.Generator(device="cuda").manual_seed(new + G)
    kv = _cache(m, 1, 1, L // page, 1, page, g, positive=True)
    kv.page_table.zero_()
    kv.seq_len.fill_(L)
    q = torch.randn((new, G, D), generator=g, device="cuda").bfloat16()
    out, lse = m.msa_paged_attn(kv, q, torch.tensor([0, new], device="cuda"), new, want_lse=True)
    assert m.device_status() == 0
    _check(kv, 0, 0, q, out, lse, L - new + 1, 1 / math.sqrt(D))


@pytest.mark.parametrize("new,n_seq,least", [(20, 100, 150_000), (50, 60, 150_000), (20, 149, 65_000), (50, 149, 65_000), (3, 9, 400_000)])
@pytest.mark.parametrize("scale", [1 / math.sqrt(D), 0.6])
def test_shares_of_many_tiles(m, new, n_seq, least, scale):
    """Whole segments and parts of them, of up to 2,300 tiles a block, with lengths on and off the borders of tiles and runs;
    the sharper softmax moves the maximum from run to run."""
    page, G, n_pages = 64, 4, 200
    g = torch.Generator(device="cuda").manual_seed(new + n_seq)
    lens = (least + torch.randint(0, least, (n_seq,), generator=g, device="cuda")).tolist()
    lens[0], lens[1], lens[2] = 2 * 65536, 2 * 65536 + 1, 65536 + new
    room = max(lens) // page + 1
    kv = _cache(m, n_pages, n_seq, room, 1, page, g)
    kv.page_table.copy_(torch.randint(0, n_pages, (n_seq, room), generator=g, device="cuda"))
    kv.page_table[:, 300:] = torch.sort(kv.page_table[:, 300:], 1).values    # few pages at a time, in most of the runs
    kv.seq_len.copy_(torch.tensor(lens))
    news = [new if i % 7 else max(1, new // 3) for i in range(n_seq)]
    off = [0, *torch.tensor(news).cumsum(0).tolist()]
    q = torch.randn((off[-1], G, D), generator=g, device="cuda").bfloat16()
    off_d = torch.tensor(off, device="cuda")
    out, lse = m.msa_paged_attn(kv, q, off_d, new, scale=scale, want_lse=True)
    assert m.device_status() == 0
    for s in range(n_seq):
        rows = slice(off[s], off[s + 1])
        _check(kv, s, 0, q[rows], out[rows], lse[rows], lens[s] - news[s] + 1, scale)
    again, lse2 = m.msa_paged_attn(kv, q, off_d, new, scale=scale, want_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
