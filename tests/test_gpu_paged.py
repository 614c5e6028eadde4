"""The paged 8-bit key/value cache on the GPU against its fp64 definition (oracle/paged_cache.py)."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_cache as C

pytestmark = pytest.mark.gpu

D = 128
BASE = 1.0e6


@pytest.fixture(scope="module")
def m():
    import routed_long_context_b200 as m

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


class Cache:
    """A cache filled with random pages, on the device (kv) and as fp64 arrays; page ids are shuffled."""

    def __init__(self, m, seed, lens, page, hkv, max_pages=None, spread=2, bounds=True, spare=3):
        r = np.random.default_rng(seed)
        self.page, self.hkv, self.lens = page, hkv, list(lens)
        counts = [-(-x // page) for x in lens]
        n_pages = sum(counts) + spare
        max_pages = max_pages or max(max(counts), 1) + 1
        perm = r.permutation(n_pages)
        self.table = np.full((len(lens), max_pages), -7, dtype=np.int32)     # entries behind the end are not read
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = perm[at:at + c]
            at += c
        # bytes of a rounded normal distribution, a few keys and channels far larger than the rest
        x = r.standard_normal((n_pages, 2, hkv, page, D)).astype(np.float32) * 60
        x[:, 0, :, :, r.integers(0, D, 4)] *= 3
        self.bytes = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.vals = C.decode_e4m3(self.bytes)
        self.scales = 2.0 ** r.integers(-6 - spread, -5 + spread, (n_pages, 2, hkv)).astype(np.float64)
        keys = self.vals[:, 0] * self.scales[:, 0, :, None, None]
        self.bounds = np.stack((keys.min(2), keys.max(2)), 2)
        self.kv = m.PagedKV(torch.from_numpy(self.bytes).cuda().view(torch.float8_e4m3fn),
                            torch.from_numpy(self.scales.astype(np.float32)).cuda(),
                            torch.from_numpy(self.table).cuda(),
                            torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                            torch.from_numpy(self.bounds.astype(np.float32)).cuda().bfloat16() if bounds else None)

    def rows(self, s, part, head):
        return C.rows_of(self.vals, self.scales, self.table[s], self.lens[s], part, head)


def _queries(seed, n_tok, hq, gain=1.0):
    q = (torch.randn((n_tok, hq, D), generator=torch.Generator().manual_seed(seed)) * gain).bfloat16()
    return q.cuda(), q.double().numpy()


def _offsets(news, first=0):
    off = np.concatenate([[0], np.cumsum(news)]) + first
    return torch.from_numpy(off.astype(np.int64)).cuda(), off


def _check_attn(c, news, off, q, out, lse, hq, scale, sel=None):
    """|error| bounds. A logit is scale * q . k with the query in two e4m3 parts of a row whose largest value is brought to
    224..448: an element is off by at most 2^-10 of that scale, 2^-17 max|q|; fp32 sums of 128 products add at most
    2^-17 sum|q k| (each of 128 additions half a step, 2^-24). delta is the logit's bound over the row's keys. A
    probability is rounded once to bf16 (2^-8 relative), its logit moves it by exp(2 delta) - 1 against the sum, the
    output is rounded to bf16 (2^-8); fp32 sums of a few thousand terms add at most 2^-12. lse: delta, and fp32
    (2^-20 relative to its parts)."""
    G = hq // c.hkv
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for s, n in enumerate(news):
        for i in range(n):
            t = off[s] + i
            seen = c.lens[s] - n + i + 1
            for g in range(c.hkv):
                k, v = c.rows(s, 0, g), c.rows(s, 1, g)
                vis = np.arange(len(k)) < seen
                if sel is not None:
                    listed = np.zeros(len(k), bool)
                    for p in sel[t, g]:
                        if p >= 0:
                            listed[p * c.page:(p + 1) * c.page] = True
                    vis &= listed
                for h in range(g * G, g * G + G):
                    o, z = C.attend(q[t, h], k, v, vis, scale)
                    if not vis.any():
                        assert (out[t, h] == 0).all() and lse[t, h] == -np.inf
                        continue
                    kk = np.abs(k[vis])
                    delta = (abs(scale) * 2.0 ** -17 * (np.abs(q[t, h]).max() * kk.sum(1) + kk @ np.abs(q[t, h]))).max()
                    a, _ = C.attend(q[t, h], k, np.abs(v), vis, scale)
                    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12 + np.expm1(2 * delta)) * a
                    err = np.abs(out[t, h] - o)
                    assert (err <= tol).all(), (s, i, h, float((err / tol).max()))
                    assert abs(lse[t, h] - z) <= delta + 2.0 ** -20 * (abs(z) + abs(z - np.log(vis.sum())) + 1), (s, i, h)


ATTN = [
    # lens, news, page, hkv, G
    ([1], [1], 16, 1, 1),
    ([17], [1], 16, 2, 4),
    ([777], [1], 64, 8, 4),
    ([64, 65, 63, 128], [1, 1, 1, 1], 64, 2, 8),
    ([5, 900, 0, 33], [1, 1, 0, 1], 32, 1, 2),
    ([300, 40, 2], [2, 2, 1], 16, 2, 4),
    ([2100], [1], 128, 1, 8),
    ([129, 700, 12, 31], [32, 7, 12, 0], 32, 2, 4),
    ([260], [260], 128, 1, 1),
    ([513, 70], [65, 70], 16, 1, 8),
    ([1500], [33], 64, 4, 2),
    ([3000, 20], [40, 20], 128, 2, 4),
]


@pytest.mark.parametrize("lens,news,page,hkv,G", ATTN)
def test_attention(m, lens, news, page, hkv, G):
    c = Cache(m, len(lens) * 1000 + page, lens, page, hkv)
    off_d, off = _offsets(news)
    q_d, q = _queries(5, off[-1], hkv * G)
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, max(news), want_lse=True)
    assert m.device_status() == 0
    _check_attn(c, news, off, q, out, lse, hkv * G, 1 / math.sqrt(D))
    again, lse2 = m.msa_paged_attn(c.kv, q_d, off_d, max(news), want_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 40], [2, 0, 1]])
def test_attention_leaves_rows_outside_the_sequences(m, news):
    lens = [50, 90, 200]
    c = Cache(m, 3, lens, 32, 2)
    off_d, off = _offsets(news, first=4)
    n_tok = off[-1] + 5
    q_d, q = _queries(6, n_tok, 8)
    q_d[:4] = math.nan
    q_d[off[-1]:] = math.nan
    out = torch.full_like(q_d, 7.0)
    lse = torch.full((n_tok, 8), 9.0, device="cuda")
    m.msa_paged_attn(c.kv, q_d, off_d, max(news), out=out, lse=lse)
    assert m.device_status() == 0
    for x, keep in ((out, 7.0), (lse, 9.0)):
        assert (x[:4] == keep).all() and (x[off[-1]:] == keep).all()
    _check_attn(c, news, off, q, out, lse, 8, 1 / math.sqrt(D))


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("page", [16, 128])
def test_attention_ignores_what_lies_behind_the_end(m, page, new):
    """Rows behind the end of the last page, and pages behind the last one, hold NaN."""
    lens = [page + 3, 3 * page, 2 * page - 1]
    c = Cache(m, 8, lens, page, 2)
    raw = c.kv.pages.view(torch.uint8)
    for s, n in enumerate(lens):
        if n % page:
            raw[int(c.table[s, n // page]), :, :, n % page:] = 0x7F
    used = set(int(c.table[s, i]) for s, n in enumerate(lens) for i in range(-(-n // page)))
    for p in set(range(c.kv.pages.shape[0])) - used:
        raw[p] = 0xFF
        c.kv.scales[p] = math.nan
    news = [min(new, n) for n in lens]
    off_d, off = _offsets(news)
    q_d, q = _queries(9, off[-1], 8)
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, max(news), want_lse=True)
    assert m.device_status() == 0
    _check_attn(c, news, off, q, out, lse, 8, 1 / math.sqrt(D))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 2, 30, 300])
def test_attention_over_far_more_keys_than_a_block_holds(m, new, page):
    """Every ring of buffers goes round many times; the reference is computed in 64 bits on the GPU, bounds as in
    _check_attn with the largest delta of the case."""
    lens, hkv, G = [41003, 300, 22222, 9000], 8, 4
    g = torch.Generator(device="cuda").manual_seed(new + page)
    counts = [-(-n // page) for n in lens]
    kv = m.PagedKV.empty(sum(counts), len(lens), max(counts), hkv, page, bounds=False)
    perm = torch.randperm(sum(counts), generator=g, device="cuda").int()
    for s, c in enumerate(counts):
        kv.page_table[s, :c] = perm[sum(counts[:s]):sum(counts[:s]) + c]
    kv.seq_len.copy_(torch.tensor(lens))
    kv.pages.copy_((torch.randn(kv.pages.shape, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn))
    kv.scales.copy_(torch.exp2(torch.randint(-8, -4, kv.scales.shape, generator=g, device="cuda").float()))
    news = [new, 1, min(new, 7), new]
    off_d, off = _offsets(news)
    q = torch.randn((off[-1], hkv * G, D), generator=g, device="cuda").bfloat16()
    out, lse = m.msa_paged_attn(kv, q, off_d, max(news), want_lse=True)
    assert m.device_status() == 0
    for s, n in enumerate(news):
        ids = kv.page_table[s, :counts[s]].long()
        x = kv.pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * kv.scales[ids].double()[..., None, None]
        for h in range(hkv):
            k, v = (x[:, i, h].reshape(-1, D)[:lens[s]] for i in range(2))
            qq = q[off[s]:off[s + 1], h * G:h * G + G].double()
            z = torch.einsum("tgd,kd->tgk", qq, k) / math.sqrt(D)
            hide = torch.arange(lens[s], device="cuda") > lens[s] - n + torch.arange(n, device="cuda")[:, None]
            z.masked_fill_(hide[:, None], -math.inf)
            p = torch.softmax(z, -1)
            ref, a = p @ v, p @ v.abs()
            delta = 2.0 ** -17 / math.sqrt(D) * float((qq.abs().amax(-1).max() * k.abs().sum(-1).max()) * 2)
            mine = out[off[s]:off[s + 1], h * G:h * G + G].double()
            assert ((mine - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12 + math.expm1(2 * delta)) * a).all()
            z = torch.logsumexp(z, -1)
            assert ((lse[off[s]:off[s + 1], h * G:h * G + G].double() - z).abs() <= delta + 2.0 ** -20 * (z.abs() + 20)).all()


@pytest.mark.parametrize("new", [1, 10])
def test_attention_of_many_sequences(m, new):
    """More sequences than any kernel looks at together, most of them short, some with nothing new."""
    r = np.random.default_rng(5)
    news = [int(x) for x in r.integers(0, new + 1, 1100)]
    news[0], news[600], news[1099] = new, new, new
    lens = [n + int(x) for n, x in zip(news, r.integers(0, 60, 1100))]
    lens[601] = 0
    news[601] = 0
    c = Cache(m, 45, lens, 16, 1)
    off_d, off = _offsets(news)
    q_d, q = _queries(46, off[-1], 2)
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, want_lse=True)
    assert m.device_status() == 0
    _check_attn(c, news, off, q, out, lse, 2, 1 / math.sqrt(D))


@pytest.mark.parametrize("lens,news,page,hkv,G", [
    ([33, 9, 20, 31], [9, 9, 1, 3], 128, 2, 4),            # every row block has a block of its own
    ([100], [100], 16, 2, 8),                              # a token a row block
    ([1311, 600], [142, 9], 64, 2, 1),                     # eight tokens a row block, cut over the blocks
    ([2000], [64], 32, 2, 4),
    ([345] * 20 + [17, 0], [4] * 20 + [3, 0], 16, 2, 4),
])
def test_attention_of_many_rows_in_small_calls(m, lens, news, page, hkv, G):
    c = Cache(m, 47, lens, page, hkv)
    off_d, off = _offsets(news)
    hq = hkv * G
    q_d, q = _queries(48, off[-1], hq)
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, max(news), want_lse=True)
    assert m.device_status() == 0
    _check_attn(c, news, off, q, out, lse, hq, 1 / math.sqrt(D))
    again, lse2 = m.msa_paged_attn(c.kv, q_d, off_d, max(news), want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [1, 24])
def test_attention_far_scales_and_sharp_logits(m, new):
    """Scales of neighbouring pages 2^40 apart, a softmax that one key takes, and a negative scale."""
    lens = [400]
    c = Cache(m, 10, lens, 32, 1, spread=1)
    c.scales[:, 1] = 2.0 ** np.random.default_rng(1).choice([-20.0, 0.0, 20.0], c.scales[:, 1].shape)
    c.kv.scales.copy_(torch.from_numpy(c.scales.astype(np.float32)))
    off_d, off = _offsets([new])
    for gain, scale in ((1.0, 0.05), (30.0, 1 / math.sqrt(D)), (0.5, -0.1)):
        q_d, q = _queries(11, new, 4, gain)
        out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, scale=scale, want_lse=True)
        _check_attn(c, [new], off, q, out, lse, 4, scale)
    assert m.device_status() == 0


def test_a_sink_key_does_not_swallow_a_long_tail(m):
    """One key with e^12 times the weight of each of 150,000 others that together weigh as much."""
    n = 150001
    c = Cache(m, 12, [n], 64, 1, spread=0)
    c.vals[:, 0] = 0
    c.vals[:, 1] = 1.0
    c.scales[:] = 1.0
    first = c.table[0, 0]
    c.vals[first, 0, 0, 0, 0] = 24.0
    c.vals[first, 1, 0, 0] = -1.0
    c.kv.pages.copy_(torch.from_numpy(c.vals.astype(np.float32)).cuda().to(torch.float8_e4m3fn))
    c.kv.scales.fill_(1.0)
    for new in (1, 32):
        q_d = torch.zeros((new, 4, D), dtype=torch.bfloat16, device="cuda")
        q_d[:, :, 0] = 1.0
        off_d, _ = _offsets([new])
        out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, scale=0.5, want_lse=True)
        seen = n - new + torch.arange(1, new + 1, dtype=torch.float64, device="cuda")[:, None, None]
        w = math.exp(12.0)
        ref = ((seen - 1 - w) / (seen - 1 + w)).expand(new, 4, D)
        # every weight within 2^-8 of its own: numerator and denominator off by at most that of their sum
        assert ((out.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + 1 + 2.0 ** -6)).all()
        assert ((lse.double() - torch.log(seen[..., 0] - 1 + w)).abs() <= 2.0 ** -16).all()


@pytest.mark.parametrize("new", [1, 33])
def test_attention_skips_bad_sequences_and_pages(m, new):
    """A bad page index hides that page's tokens; a length that the table cannot hold hides the sequence."""
    lens = [200, 100, 160]
    c = Cache(m, 13, lens, 32, 2)
    news = [new] * 3
    off_d, off = _offsets(news)
    q_d, q = _queries(14, off[-1], 8)
    c.kv.page_table[0, 2] = c.kv.pages.shape[0]
    c.kv.page_table[0, 4] = -1
    c.kv.seq_len[1] = 32 * c.kv.max_pages + 1
    out = torch.full_like(q_d, 7.0)
    lse = torch.full((off[-1], 8), 9.0, device="cuda")
    m.msa_paged_attn(c.kv, q_d, off_d, new, out=out, lse=lse)
    assert m.device_status() == 3
    assert (out[off[1]:off[2]] == 7.0).all() and (lse[off[1]:off[2]] == 9.0).all()
    scale = 1 / math.sqrt(D)
    sel = np.tile(np.array([[0, 1, 3, 5, 6]]), (off[-1], 2, 1))
    _check_attn(c, [new, 0, 0], off, q, out, lse, 8, scale, sel=sel)
    n2 = slice(off[2], off[3])
    c2 = Cache(m, 13, lens, 32, 2)
    ref, rlse = m.msa_paged_attn(c2.kv, q_d, off_d, new, want_lse=True)
    assert torch.allclose(out[n2].float(), ref[n2].float(), rtol=2.0 ** -6, atol=1e-3) and m.device_status() == 0


@pytest.mark.parametrize("lens,news,page,hkv,G,k", [
    ([1000], [1], 64, 2, 4, 5), ([700, 90, 31], [1, 1, 1], 32, 1, 8, 4), ([300, 1], [17, 1], 16, 2, 2, 7),
    ([2000], [9], 128, 1, 1, 3), ([150, 0, 400], [3, 0, 5], 16, 4, 4, 30)])
def test_selection_and_sparse_attention(m, lens, news, page, hkv, G, k):
    c = Cache(m, 20 + page, lens, page, hkv)
    off_d, off = _offsets(news)
    q_d, q = _queries(21, off[-1], hkv * G)
    recent = min(2, k)
    sel = m.msa_page_select(c.kv, q_d, off_d, max(news), k, recent)
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, max(news), sel=sel, want_lse=True)
    assert m.device_status() == 0
    sel = sel.cpu().numpy()
    bounds = c.kv.bounds.double().cpu().numpy()
    for s, n in enumerate(news):
        for i in range(n):
            last = (c.lens[s] - n + i) // page
            ids = c.table[s, :last + 1]
            for g in range(hkv):
                sc = C.page_scores(q[off[s] + i, g * G:(g + 1) * G], bounds[ids, g, 0], bounds[ids, g, 1])
                np.testing.assert_array_equal(sel[off[s] + i, g], C.pick(sc, k, recent))
    _check_attn(c, news, off, q, out, lse, hkv * G, 1 / math.sqrt(D), sel=sel)


@pytest.mark.parametrize("n,k,new", [(9000, 33, 1), (40000, 100, 1), (5000, 64, 20)])
def test_selection_of_many_pages_with_ties(m, n, k, new):
    """Thousands of pages with few distinct bounds: the border always runs through equal scores."""
    page = 16
    c = Cache(m, 30, [n * page], page, 1, max_pages=n)
    kinds = c.kv.bounds[:6].clone()
    which = torch.from_numpy(np.random.default_rng(2).integers(0, 6, c.kv.bounds.shape[0])).cuda()
    c.kv.bounds.copy_(kinds[which])
    off_d, off = _offsets([new])
    q_d, q = _queries(31, new, 4)
    sel = m.msa_page_select(c.kv, q_d, off_d, new, k, 1).cpu().numpy()
    assert m.device_status() == 0
    b = c.kv.bounds.double().cpu().numpy()
    for i in range(new):
        ids = c.table[0, :(n * page - new + i) // page + 1]
        sc = C.page_scores(q[i], b[ids, 0, 0], b[ids, 0, 1])
        np.testing.assert_array_equal(sel[i, 0], C.pick(sc, k, 1))


@pytest.mark.parametrize("new", [1, 12])
def test_selection_borders_decided_in_64_bits(m, new):
    """Scores that agree in 32 bits: a large element, and one that tells the pages apart by 2^-40 of it."""
    n, page, k = 200, 16, 20
    c = Cache(m, 40, [n * page], page, 1, max_pages=n)
    b = torch.zeros_like(c.kv.bounds)
    b[:, 0, :, 0] = 2.0 ** 20
    order = torch.from_numpy(np.random.default_rng(3).permutation(n)).cuda()
    ids = torch.from_numpy(c.table[0, :n].astype(np.int64)).cuda()
    b[ids, 0, :, 1] = ((order[:, None] + 1).float() * 2.0 ** -20).bfloat16()
    c.kv.bounds.copy_(b)
    off_d, _ = _offsets([new])
    q_d = torch.zeros((new, 2, D), dtype=torch.bfloat16, device="cuda")
    q_d[:, :, :2] = 1.0
    sel = m.msa_page_select(c.kv, q_d, off_d, new, k, 1).cpu().numpy()
    bb = c.kv.bounds.double().cpu().numpy()
    for i in range(new):
        seen = c.table[0, :(n * page - new + i) // page + 1]
        sc = C.page_scores(np.ones((1, 2)), bb[seen, 0, 0, :2], bb[seen, 0, 1, :2])
        np.testing.assert_array_equal(sel[i, 0], C.pick(sc, k, 1))
    assert m.device_status() == 0


def test_selection_of_more_pages_than_shared_memory_holds(m):
    n, page, k = 60000, 16, 40
    c = Cache(m, 41, [n * page], page, 1, max_pages=n)
    off_d, _ = _offsets([1])
    q_d, q = _queries(42, 1, 4)
    sel = m.msa_page_select(c.kv, q_d, off_d, 1, k, 3).cpu().numpy()
    b = c.kv.bounds[torch.from_numpy(c.table[0, :n].astype(np.int64)).cuda(), 0].double().cpu().numpy()
    np.testing.assert_array_equal(sel[0, 0], C.pick(C.page_scores(q[0], b[:, 0], b[:, 1]), k, 3))
    assert m.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attention_over_the_smallest_values(m, new):
    """Keys and values below the smallest normal e4m3 number, at both ends of the scales' range."""
    for e in (-50, -3, 50):
        c = Cache(m, 43, [100], 16, 1)
        c.bytes[:] = (c.bytes & 0x87)                          # sign and fraction: -7 .. 7 times 2^-9
        c.vals = C.decode_e4m3(c.bytes)
        c.scales[:] = 2.0 ** e
        c.kv.pages.view(torch.uint8).copy_(torch.from_numpy(c.bytes))
        c.kv.scales.fill_(2.0 ** e)
        off_d, off = _offsets([new])
        q_d, q = _queries(44, new, 4)
        scale = 4.0 * 2.0 ** -e
        out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, scale=scale, want_lse=True)
        assert m.device_status() == 0
        _check_attn(c, [new], off, q, out, lse, 4, scale)


@pytest.mark.parametrize("new", [1, 2, 40])
@pytest.mark.parametrize("listed", [False, True])
def test_attention_without_logits(m, new, listed):
    """Queries and keys of zeros (at the smallest scale, as they are appended), and a softmax scale of zero: the mean of
    the values that a row sees, whatever lies in the places that it does not see."""
    sel = None
    for lens in ([77], [1000]):
        c = Cache(m, 45, lens, 16, 2)
        off_d, off = _offsets([new])
        q_d, q = _queries(46, new, 8)
        if listed:
            sel = torch.full((new, 2, 3), -1, dtype=torch.int32, device="cuda")
            for i in range(new):
                sel[i, :, 0], sel[i, :, 2] = 1, (lens[0] - new + i) // 16
        sel_np = None if sel is None else sel.cpu().numpy()
        out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, sel=sel, scale=0.0, want_lse=True)
        assert m.device_status() == 0
        _check_attn(c, [new], off, q, out, lse, 8, 0.0, sel=sel_np)
        c.kv.pages[:, 0] = torch.zeros_like(c.kv.pages[:, 0])
        c.kv.scales[:, 0] = 2.0 ** -50
        c.vals[:, 0] = 0.0
        c.scales[:, 0] = 2.0 ** -50
        q_d.zero_()
        q[:] = 0.0
        out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, sel=sel, want_lse=True)
        assert m.device_status() == 0
        _check_attn(c, [new], off, q, out, lse, 8, 1 / math.sqrt(D), sel=sel_np)


def test_a_list_of_the_callers_own(m):
    """Empty entries anywhere, a page named twice, one out of range, a row without any page."""
    c = Cache(m, 50, [500, 100], 32, 1)
    off_d, off = _offsets([1, 2])
    q_d, q = _queries(51, 3, 4)
    sel = torch.full((3, 1, 6), -1, dtype=torch.int32, device="cuda")
    sel[0, 0, 1], sel[0, 0, 4], sel[0, 0, 5] = 3, 15, 0
    sel[2, 0, 3] = 3                                        # tokens 96 .. 99
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, 2, sel=sel, want_lse=True)
    assert m.device_status() == 0
    _check_attn(c, [1, 2], off, q, out, lse, 4, 1 / math.sqrt(D), sel=sel.cpu().numpy())
    sel[2, 0, 0] = 4                                        # behind the sequence's pages
    o2, l2 = m.msa_paged_attn(c.kv, q_d, off_d, 2, sel=sel, want_lse=True)
    assert m.device_status() == 3 and torch.equal(o2, out) and torch.equal(l2, lse)
    sel[2, 0, 0] = 3                                        # twice: the same mean, twice the sum
    o2, l2 = m.msa_paged_attn(c.kv, q_d, off_d, 2, sel=sel, want_lse=True)
    assert m.device_status() == 0
    assert (l2[2] - lse[2] - math.log(2)).abs().max() < 1e-5
    assert torch.allclose(o2[2].float(), out[2].float(), rtol=2.0 ** -6, atol=2.0 ** -10)


# ------------------------------------------------------------------------------------------------ appending
def _state(kv):
    return (C.decode_e4m3(kv.pages.view(torch.uint8).cpu().numpy()), kv.scales.double().cpu().numpy(),
            kv.bounds.double().cpu().numpy())


def _check_append(m, c, news, dtype, first=0, pos_offset=12, gain=1.0):
    """Values: exact. Keys: the rotation's fp32 error (the table's and the products' roundings, 2^-22 of the pair)
    and half an e4m3 step (2^-4 relative, 2^-10 of the scale where subnormal)."""
    kv = c.kv
    before = [x.copy() for x in _state(kv)]
    ref = [x.copy() for x in before]
    off_d, off = _offsets(news, first)
    n_tok = off[-1] + 3
    g = torch.Generator().manual_seed(77)
    k = (torch.randn((n_tok, c.hkv, D), generator=g) * gain).to(dtype)
    v = torch.randn((n_tok, c.hkv, D), generator=g).to(dtype)
    q = torch.randn((n_tok, c.hkv * 2, D), generator=g).to(dtype)
    cs = m.rope_table(max(c.lens) + pos_offset, D, BASE)
    q_rot = torch.full_like(q.cuda(), 5.0)
    m.msa_paged_append(kv, k.cuda(), v.cuda(), off_d, max(news), cs, pos_offset, q=q.cuda(), q_rot=q_rot)
    assert m.device_status() == 0
    got = _state(kv)
    exact = np.array(before[0])
    q_rot = q_rot.double().cpu().numpy()
    assert (q_rot[:first] == 5).all() and (q_rot[off[-1]:] == 5).all()
    touched = set()
    for s, n in enumerate(news):
        base = c.lens[s] - n
        pages = c.table[s]
        rows = slice(off[s], off[s + 1])
        kr = C.append(*ref, pages, base, k[rows].double().numpy(), v[rows].double().numpy(), pos_offset, BASE)
        touched |= {int(p) for p in pages[base // c.page:-(-c.lens[s] // c.page)]} if n else set()
        qr = C.apply_rope(q[rows].double().numpy(), pos_offset + base + np.arange(n), BASE)
        pair = lambda x: np.tile(np.abs(x[..., :64]) + np.abs(x[..., 64:]), 2)  # noqa: E731
        tol = (2.0 ** -8 * np.abs(qr) if dtype == torch.bfloat16 else 0) + 2.0 ** -22 * pair(q[rows].double().numpy())
        assert (np.abs(q_rot[rows] - qr) <= tol).all()
        kp = pair(k[rows].double().numpy())
        for i in range(n):
            p, r = (base + i) // c.page, (base + i) % c.page
            sc = got[1][pages[p], 0][:, None]
            x = got[0][pages[p], 0, :, r] * sc
            assert (np.abs(x - kr[i]) <= 2.0 ** -4 * np.abs(kr[i]) + 2.0 ** -10 * sc + 2.0 ** -21 * kp[i]).all()
    # scales, values and the untouched rows are exact; a scale of keys may sit on a border, which none does here
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_array_equal(got[0][:, 1], ref[0][:, 1])
    others = [p for p in range(len(exact)) if p not in touched]
    np.testing.assert_array_equal(got[0][others], before[0][others])
    np.testing.assert_array_equal(got[2][others], before[2][others])
    # bounds are those of the stored keys
    for s, n in enumerate(news):
        for p in range((c.lens[s] - n) // c.page, -(-c.lens[s] // c.page) if n else 0):
            pid, r1 = c.table[s, p], min(c.page, c.lens[s] - p * c.page)
            keys = got[0][pid, 0, :, :r1] * got[1][pid, 0][:, None, None]
            np.testing.assert_array_equal(got[2][pid, :, 0], keys.min(1))
            np.testing.assert_array_equal(got[2][pid, :, 1], keys.max(1))


def _true_bounds(c):
    """Bounds as an append leaves them: of the rows in use."""
    for s, n in enumerate(c.lens):
        for p in range(-(-n // c.page)):
            pid, r1 = c.table[s, p], min(c.page, n - p * c.page)
            keys = c.vals[pid, 0, :, :r1] * c.scales[pid, 0][:, None, None]
            c.bounds[pid, :, 0], c.bounds[pid, :, 1] = keys.min(1), keys.max(1)
    c.kv.bounds.copy_(torch.from_numpy(c.bounds.astype(np.float32)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,news,page,hkv", [
    ([1], [1], 16, 1), ([16, 17, 15, 33], [1, 1, 1, 1], 16, 2), ([300], [300], 64, 8),
    ([129, 700, 12, 31], [32, 7, 12, 0], 32, 4), ([257, 128, 40], [130, 128, 1], 128, 1), ([1000], [1], 128, 2)])
@pytest.mark.parametrize("gain", [1.0, 1e-3, 300.0])
def test_append(m, lens, news, page, hkv, dtype, gain):
    for first in (0, 2):
        c = Cache(m, 60 + page, lens, page, hkv)
        c.lens = [a - n for a, n in zip(lens, news)]
        _true_bounds(c)
        c.lens = list(lens)
        _check_append(m, c, news, dtype, first=first, gain=gain)


@pytest.mark.parametrize("page", [16, 128])
def test_append_of_many_sequences(m, page):
    """More sequences than a warp has lanes, most of them with nothing to add."""
    r = np.random.default_rng(4)
    news = [int(x) for x in r.choice([0, 0, 1, 2, 40], 75)]
    lens = [n + int(x) for n, x in zip(news, r.integers(0, 200, 75))]
    c = Cache(m, 61, lens, page, 1)
    c.lens = [a - n for a, n in zip(lens, news)]
    _true_bounds(c)
    c.lens = list(lens)
    _check_append(m, c, news, torch.bfloat16)


def test_append_of_values_that_are_not_finite(m):
    """NaN is stored as 0, an infinity as the largest value of its sign; neither sets a scale."""
    kv = m.PagedKV.empty(2, 1, 2, 1, page=16)
    kv.page_table.copy_(torch.tensor([[1, 0]]))
    kv.seq_len.fill_(3)
    x = torch.zeros((3, 1, D))
    x[0, 0, :3] = torch.tensor([1.0, math.nan, -2.0])
    x[1, 0, 64:67] = torch.tensor([math.inf, -math.inf, 1e38])
    x[2] = 0.5
    off_d, _ = _offsets([3])
    cs = m.rope_table(4, D, BASE)
    cs[..., 0], cs[..., 1] = 1.0, 0.0                     # no rotation: 0 * inf would spread the NaN to its partner
    for dtype in (torch.float32, torch.bfloat16):
        m.msa_paged_append(kv, torch.zeros((3, 1, D), dtype=dtype).cuda(), x.to(dtype).cuda(), off_d, 3, cs)
        assert m.device_status() == 4
        vals, scales, _ = _state(kv)
        assert scales[1, 1, 0] == 2.0 ** 50 and np.isfinite(vals[1, :, :, :3]).all()
        assert vals[1, 1, 0, 1, 64] == 448 and vals[1, 1, 0, 1, 65] == -448 and vals[1, 1, 0, 1, 66] == 448
        assert (vals[1, 1, 0, 0] == 0).all()
    x[1, 0, 66] = 1.0
    m.msa_paged_append(kv, x.cuda(), x.cuda(), off_d, 3, cs)
    assert m.device_status() == 4
    vals, scales, bounds = _state(kv)
    assert scales[1, 1, 0] == 2.0 ** -7                     # 2 <= 448 / 128
    assert vals[1, 1, 0, 0, 1] == 0 and vals[1, 1, 0, 0, 2] == -256 and vals[1, 1, 0, 1, 64] == 448
    assert np.isfinite(vals[1, :, :, :3]).all() and np.isfinite(bounds[1]).all()


def test_append_records_bad_pages_offsets_and_positions(m):
    c = Cache(m, 62, [40, 40, 40], 32, 1)
    before = _state(c.kv)
    n_pages = c.kv.pages.shape[0]
    k = torch.ones((120, 1, D), dtype=torch.bfloat16, device="cuda")
    cs = m.rope_table(64, D, BASE)
    off_d, _ = _offsets([40, 40, 40])
    c.kv.page_table[0, 1] = n_pages
    c.kv.seq_len[1] = 39                                    # fewer than its new tokens
    m.msa_paged_append(c.kv, k, k, off_d, 40, cs)
    assert m.device_status() == 3
    got = _state(c.kv)
    written = {int(c.table[0, 0]), int(c.table[2, 0]), int(c.table[2, 1])}
    for p in range(n_pages):
        same = (got[0][p] == before[0][p]) | np.isnan(before[0][p])
        assert same.all() == (p not in written)
    c.kv.page_table[0, 1] = int(c.table[0, 1])
    c.kv.seq_len[1] = 40
    m.msa_paged_append(c.kv, k, k, off_d, 40, cs, pos_offset=30)
    assert m.device_status() == 1
    m.msa_paged_append(c.kv, k, k, off_d, 39, cs)           # more tokens than max_new says
    assert m.device_status() == 3


# ------------------------------------------------------------------------------------------------ together
def test_a_decode_loop_with_growing_pages(m):
    """A prompt, then single tokens and a round of several, over two sequences: append, select and attend as they are
    used, on a side stream, against one dense fp64 pass over what the cache holds."""
    hkv, G, page, k = 2, 4, 16, 4
    kv = m.PagedKV.empty(40, 2, 12, hkv, page)
    kv.page_table.copy_(torch.randperm(40, generator=torch.Generator().manual_seed(1))[:24].view(2, 12))
    cs = m.rope_table(256, D, BASE)
    g = torch.Generator().manual_seed(2)
    lens = [0, 0]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for news in ([70, 33], [1, 1], [1, 1], [0, 1], [5, 8], [1, 1], [1, 0]):
            lens = [a + b for a, b in zip(lens, news)]
            kv.seq_len.copy_(torch.tensor(lens))
            off_d, off = _offsets(news)
            n = off[-1]
            kk = torch.randn((n, hkv, D), generator=g).bfloat16().cuda()
            vv = torch.randn((n, hkv, D), generator=g).bfloat16().cuda()
            q = torch.randn((n, hkv * G, D), generator=g).bfloat16().cuda()
            qr = m.msa_paged_append(kv, kk, vv, off_d, max(news), cs, 3, q=q)
            sel = m.msa_page_select(kv, qr, off_d, max(news), k)
            full, flse = m.msa_paged_attn(kv, qr, off_d, max(news), want_lse=True)
            some, slse = m.msa_paged_attn(kv, qr, off_d, max(news), sel=sel, want_lse=True)
            assert m.device_status() == 0
            c = Cache.__new__(Cache)
            c.vals, c.scales, _ = _state(kv)
            c.page, c.hkv, c.lens, c.table = page, hkv, lens, kv.page_table.cpu().numpy()
            qn = qr.double().cpu().numpy()
            _check_attn(c, news, off, qn, full, flse, hkv * G, 1 / math.sqrt(D))
            _check_attn(c, news, off, qn, some, slse, hkv * G, 1 / math.sqrt(D), sel=sel.cpu().numpy())


def test_joined_with_fetched_memory_by_the_log_sums(m):
    """msa_sparse_attn_split over fetched rows and msa_paged_attn over the cache, joined by their log-sums, are one
    attention over both."""
    hkv, G, n_mem = 2, 4, 300
    c = Cache(m, 70, [150], 32, hkv, spread=1)
    g = torch.Generator().manual_seed(3)
    mem = torch.randn((1, n_mem, 2, hkv, D), generator=g).bfloat16()
    q_d, q = _queries(71, 1, hkv * G)
    off_d, _ = _offsets([1])
    lse_m = torch.empty((1, 1, hkv * G), device="cuda")
    zero = torch.zeros((1, 64, hkv, D), dtype=torch.bfloat16, device="cuda")
    out_m = m.msa_sparse_attn_split(q_d[None], mem.cuda(), torch.tensor([n_mem], dtype=torch.int32, device="cuda"), zero,
                                    zero, 0, 0, lse=lse_m)
    out_c, lse_c = m.msa_paged_attn(c.kv, q_d, off_d, 1, want_lse=True)
    assert m.device_status() == 0
    w = torch.sigmoid(lse_m[0] - lse_c)[..., None].double()
    got = (out_m[0].double() * w + out_c.double() * (1 - w)).cpu().numpy()
    mm = mem.double().numpy()
    for h in range(hkv * G):
        kk = np.concatenate([mm[0, :, 0, h // G], c.rows(0, 0, h // G)])
        vv = np.concatenate([mm[0, :, 1, h // G], c.rows(0, 1, h // G)])
        ref, _ = C.attend(q[0, h], kk, vv, np.ones(len(kk), bool), 1 / math.sqrt(D))
        a, _ = C.attend(q[0, h], kk, np.abs(vv), np.ones(len(kk), bool), 1 / math.sqrt(D))
        assert (np.abs(got[0, h] - ref) <= 2.0 ** -6 * (np.abs(ref) + a)).all()


def test_a_captured_step_replays_on_new_lengths(m):
    """One graph of append, select and attend, replayed after the lengths, the table and the inputs moved on; two such
    graphs have workspaces of their own."""
    hkv, G, page, k = 2, 4, 32, 3
    hq = hkv * G

    def world(seed):
        kv = m.PagedKV.empty(16, 1, 8, hkv, page)
        kv.page_table.copy_(torch.randperm(16, generator=torch.Generator().manual_seed(seed))[:8].view(1, 8))
        return kv

    cs = m.rope_table(300, D, BASE)
    off_d, _ = _offsets([1])
    a, b = world(5), world(5)
    kk, vv = (torch.zeros((1, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, qr, o1, o2 = (torch.zeros((1, hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    sel = torch.zeros((1, hkv, k), dtype=torch.int32, device="cuda")
    ws1 = torch.empty(m.page_select_workspace_size(1, hkv, 8), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(m.paged_attn_workspace_size(1, 1, 1, hq, hkv, 8, page, k), dtype=torch.uint8, device="cuda")
    ws3 = torch.empty(m.paged_attn_workspace_size(1, 1, 1, hq, hkv, 8, page), dtype=torch.uint8, device="cuda")

    def step(kv, w1=ws1, w2=ws2, w3=ws3):
        m.msa_paged_append(kv, kk, vv, off_d, 1, cs, 0, q=q, q_rot=qr)
        m.msa_page_select(kv, qr, off_d, 1, k, sel=sel, ws=w1)
        m.msa_paged_attn(kv, qr, off_d, 1, sel=sel, out=o1, ws=w2)
        m.msa_paged_attn(kv, qr, off_d, 1, out=o2, ws=w3)

    a.seq_len.fill_(1)
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    g = torch.Generator().manual_seed(6)
    for n in range(1, 150):
        for x in (kk, vv, q):
            x.copy_(torch.randn(x.shape, generator=g))
        a.seq_len.fill_(n)
        b.seq_len.fill_(n)
        graph.replay()
        mine = (qr.clone(), sel.clone(), o1.clone(), o2.clone())
        step(b, ws1.clone(), ws2.clone(), ws3.clone())
        for x, y in zip(mine, (qr, sel, o1, o2)):
            assert torch.equal(x, y), n
        n_p = -(-n // page)
        ids = a.page_table[0, :n_p].long()
        assert torch.equal(a.scales[ids], b.scales[ids]) and torch.equal(a.bounds[ids], b.bounds[ids])
    assert m.device_status() == 0


class Roomy(Cache):
    """With room for long contexts, which is what the choice of the kernel goes by."""

    def __init__(self, m, seed, lens, page, hkv, max_pages=None, **kw):
        super().__init__(m, seed, lens, page, hkv, max_pages=1 << 13, **kw)


@pytest.mark.parametrize("name,args", [("test_attention", x) for x in ATTN if max(x[1]) * x[4] > 8] + [
    ("test_attention_leaves_rows_outside_the_sequences", ([3, 1, 40],)),
    ("test_attention_ignores_what_lies_behind_the_end", (16, 20)),
    ("test_attention_ignores_what_lies_behind_the_end", (128, 20)),
    ("test_attention_far_scales_and_sharp_logits", (24,)),
    ("test_a_sink_key_does_not_swallow_a_long_tail", ()),
    ("test_attention_skips_bad_sequences_and_pages", (33,)),
    ("test_attention_over_the_smallest_values", (40,)),
    ("test_attention_without_logits", (40, False)),
    ("test_calls_right_behind_what_they_depend_on", (30, False)),
    ("test_a_query_that_is_not_finite_spoils_its_own_row_only", (30, math.nan)),
    ("test_a_query_that_is_not_finite_spoils_its_own_row_only", (30, math.inf)),
    ("test_attention_records_more_tokens_than_it_was_told", ()),
    ("test_nothing_is_written_beside_the_outputs", (30, 16, 4)),
    ("test_nothing_is_written_beside_the_outputs", (70, 128, 4)),
])
def test_small_calls_with_room_for_long_contexts(m, monkeypatch, name, args):
    """The same calls where the table has room for long contexts: those of more than 8 rows go another way."""
    import inspect

    f = globals()[name]
    monkeypatch.setitem(globals(), "Cache", Roomy)
    f(**dict(zip(inspect.signature(f).parameters, (m, *args))))


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_right_behind_what_they_depend_on(m, new, captured):
    """Lengths, table, queries and values that a copy, a fill or another stream brings directly before the call, and the
    same outputs and workspace used by call after call: no call may begin to read or write early."""
    c = Cache(m, 85, [4000, 900], 16, 4)
    off_d, off = _offsets([new, new])
    hq, n_tok = 8, 2 * new
    ws = torch.empty(m.paged_attn_workspace_size(n_tok, 2, new, hq, 4, c.kv.max_pages, 16), dtype=torch.uint8, device="cuda")
    lens = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([4000, 900], [77, 850], [2222, 31])]
    host = [x.cpu().pin_memory() for x in lens]
    qs = [_queries(86 + i, n_tok, hq)[0] for i in range(3)]
    q = torch.empty_like(qs[0])
    outs = [torch.empty_like(q) for _ in range(6)]
    out = torch.empty_like(q)
    want = []
    for i in range(3):
        c.kv.seq_len.copy_(lens[i])
        torch.cuda.synchronize()
        want.append(m.msa_paged_attn(c.kv, qs[i], off_d, new))
        torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def steps():
        for r in range(6):
            i = r % 3
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                q.copy_(qs[i])                              # by another stream
            if r % 2:
                c.kv.seq_len.copy_(host[i], non_blocking=True)
            else:
                c.kv.seq_len.copy_(lens[i])
            out.zero_()
            torch.cuda.current_stream().wait_stream(side)
            m.msa_paged_attn(c.kv, q, off_d, new, out=out, ws=ws)
            m.msa_paged_attn(c.kv, q, off_d, new, out=out, ws=ws)
            outs[r].copy_(out)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
        run = graph.replay
    else:
        run = steps
    for _ in range(5):
        run()
        torch.cuda.synchronize()
        for r in range(6):
            assert torch.equal(outs[r], want[r % 3]), r
    assert m.device_status() == 0


def test_a_stream_of_the_callers_own(m):
    """Calls on a stream that is not the current one, with scratch and results allocated by the call, while the current
    stream allocates and overwrites memory of the same sizes; two such streams at once."""
    c = Cache(m, 80, [3000, 700], 32, 4)
    off_d, off = _offsets([1, 1])
    q_d, q = _queries(81, 2, 16)
    off_l, _ = _offsets([40, 30])
    q_l, _ = _queries(82, 70, 16)
    sel = m.msa_page_select(c.kv, q_d, off_d, 1, 6)
    want = (m.msa_paged_attn(c.kv, q_d, off_d, 1), m.msa_paged_attn(c.kv, q_d, off_d, 1, sel=sel),
            m.msa_paged_attn(c.kv, q_l, off_l, 40))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        s = streams[i % 2]
        picked = m.msa_page_select(c.kv, q_d, off_d, 1, 6, stream=s)
        got.append((m.msa_paged_attn(c.kv, q_d, off_d, 1, stream=s), m.msa_paged_attn(c.kv, q_d, off_d, 1, sel=picked, stream=s),
                    m.msa_paged_attn(c.kv, q_l, off_l, 40, stream=s)))
        for _ in range(3):
            torch.empty(1 << 20, device="cuda").fill_(math.nan)
            torch.empty_like(q_l).fill_(math.nan)
    torch.cuda.synchronize()
    assert m.device_status() == 0
    for g in got:
        for x, y in zip(g, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(m, new, bad):
    c = Cache(m, 83, [500], 64, 2)
    off_d, _ = _offsets([new])
    q_d, _ = _queries(84, new, 8)
    want, wlse = m.msa_paged_attn(c.kv, q_d, off_d, new, want_lse=True)
    q_d[new // 2, 3, 5] = bad
    out, lse = m.msa_paged_attn(c.kv, q_d, off_d, new, want_lse=True)
    assert torch.isnan(out[new // 2, 3]).all() and torch.isnan(lse[new // 2, 3])
    keep = torch.ones((new, 8), dtype=torch.bool, device="cuda")
    keep[new // 2, 3] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wlse[keep])
    assert m.device_status() == 0


def test_selection_leaves_rows_outside_the_sequences(m):
    c = Cache(m, 85, [300, 500], 16, 2)
    off_d, off = _offsets([2, 1], first=3)
    q_d, q = _queries(86, 9, 8)
    sel = torch.full((9, 2, 5), 77, dtype=torch.int32, device="cuda")
    m.msa_page_select(c.kv, q_d, off_d, 2, 5, sel=sel)
    assert m.device_status() == 0
    assert (sel[:3] == 77).all() and (sel[6:] == 77).all() and (sel[3:6] < 77).all()


def test_attention_records_more_tokens_than_it_was_told(m):
    c = Cache(m, 87, [300, 100], 32, 2)
    for news, told in (([3, 1], 2), ([40, 1], 39)):
        off_d, off = _offsets(news)
        q_d, q = _queries(88, off[-1], 8)
        out = torch.full_like(q_d, 7.0)
        lse = torch.full((off[-1], 8), 9.0, device="cuda")
        m.msa_paged_attn(c.kv, q_d, off_d, told, out=out, lse=lse)
        assert m.device_status() == 3
        assert (out[:off[1]] == 7.0).all() and (lse[:off[1]] == 9.0).all()
        _check_attn(c, [0, 1], [0, off[1]], q, out, lse, 8, 1 / math.sqrt(D))


@pytest.mark.parametrize("new,page,G", [(1, 16, 4), (1, 64, 8), (3, 32, 2), (30, 16, 4), (70, 128, 4), (300, 64, 1)])
def test_nothing_is_written_beside_the_outputs(m, new, page, G):
    """Workspaces of exactly the size asked for, and outputs, between guards."""
    hkv, k = 2, 4
    c = Cache(m, 89, [3000, 331], page, hkv)
    off_d, off = _offsets([new, min(new, 331)])
    n = int(off[-1])
    q_d, _ = _queries(90, n, hkv * G)

    def guarded(nbytes):
        buf = torch.full((nbytes + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + nbytes]

    sizes = [m.page_select_workspace_size(n, hkv, c.kv.max_pages),
             m.paged_attn_workspace_size(n, 2, new, hkv * G, hkv, c.kv.max_pages, page),
             m.paged_attn_workspace_size(n, 2, new, hkv * G, hkv, c.kv.max_pages, page, k),
             n * hkv * k * 4, n * hkv * G * D * 2, n * hkv * G * 4]
    bufs = [guarded(x) for x in sizes]
    w1, w2, w3, sel, out, lse = (b[1] for b in bufs)
    sel, out, lse = sel.view(torch.int32).view(n, hkv, k), out.view(torch.bfloat16).view(q_d.shape), lse.view(torch.float32).view(n, -1)
    m.msa_page_select(c.kv, q_d, off_d, new, k, sel=sel, ws=w1)
    m.msa_paged_attn(c.kv, q_d, off_d, new, sel=sel, out=out, lse=lse, ws=w3)
    m.msa_paged_attn(c.kv, q_d, off_d, new, out=out, lse=lse, ws=w2)
    assert m.device_status() == 0
    for b, inner in bufs:
        assert (b[:256] == 0x5A).all() and (b[256 + inner.numel():] == 0x5A).all()


def test_offsets_past_32_bits(m):
    """A cache of more than 4 GB: pages at its far end."""
    hkv, page, n_pages = 8, 128, 17000                      # 17000 * 2 * 8 * 128 * 128 B = 4.5 GB
    kv = m.PagedKV.empty(n_pages, 1, 3, hkv, page)
    ids = [n_pages - 1, 0, n_pages - 2]
    kv.page_table.copy_(torch.tensor([ids]))
    lens = [300]
    off_d, off = _offsets(lens)
    kv.seq_len.fill_(300)
    g = torch.Generator().manual_seed(8)
    kk, vv = (torch.randn((300, hkv, D), generator=g).bfloat16().cuda() for _ in range(2))
    cs = m.rope_table(300, D, BASE)
    m.msa_paged_append(kv, kk, vv, off_d, 300, cs)
    idl = torch.tensor(ids, device="cuda")
    c = Cache.__new__(Cache)
    small = m.PagedKV(kv.pages.view(torch.uint8)[idl].view(torch.float8_e4m3fn), kv.scales[idl],
                      torch.arange(3, dtype=torch.int32, device="cuda")[None], kv.seq_len, kv.bounds[idl])
    c.vals, c.scales, _ = _state(small)
    c.page, c.hkv, c.lens, c.table = page, hkv, lens, np.arange(3)[None]
    x = (C.rows_of(c.vals, c.scales, [0, 1, 2], 300, 1, 7) - vv[:, 7].double().cpu().numpy())
    assert np.abs(x).max() < 0.5
    for new in (1, 40):
        off_d, off = _offsets([new])
        q_d, q = _queries(9, new, hkv)
        out, lse = m.msa_paged_attn(kv, q_d, off_d, new, want_lse=True)
        sel = m.msa_page_select(kv, q_d, off_d, new, 2)
        ref = m.msa_page_select(small, q_d, off_d, new, 2)
        assert torch.equal(sel, ref)
        _check_attn(c, [new], off, q, out, lse, hkv, 1 / math.sqrt(D))
    assert m.device_status() == 0


def test_the_binding_refuses_what_the_kernels_would_misread(m):
    c = Cache(m, 91, [40, 40], 16, 2)
    off_d, off = _offsets([2, 2])
    q_d, _ = _queries(92, 4, 8)
    cs = m.rope_table(64, D, BASE)
    k = torch.zeros((4, 2, D), dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((4, 16, D), dtype=torch.bfloat16, device="cuda")[:, ::2]
    cases = [
        lambda: m.msa_paged_attn(c.kv, wide, off_d, 2), lambda: m.msa_paged_attn(c.kv, q_d.cpu(), off_d, 2),
        lambda: m.msa_paged_attn(c.kv, q_d, off_d.int(), 2), lambda: m.msa_paged_attn(c.kv, q_d, off_d[:2], 2),
        lambda: m.msa_paged_attn(c.kv, q_d[:, :, :64].contiguous(), off_d, 2),
        lambda: m.msa_paged_attn(c.kv, q_d, off_d, 2, out=torch.empty_like(q_d).float()),
        lambda: m.msa_paged_attn(c.kv, q_d, off_d, 2, lse=torch.empty((4, 4), device="cuda")),
        lambda: m.msa_paged_attn(c.kv, q_d, off_d, 2, sel=torch.zeros((4, 8, 3), dtype=torch.int32, device="cuda")),
        lambda: m.msa_paged_attn(c.kv, q_d, off_d, 2, sel=torch.zeros((4, 2, 3), dtype=torch.int64, device="cuda")),
        lambda: m.msa_page_select(c.kv, q_d, off_d, 2, 3, sel=torch.zeros((4, 2, 4), dtype=torch.int32, device="cuda")),
        lambda: m.msa_paged_append(c.kv, k, k.float(), off_d, 2, cs),
        lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs.bfloat16()),
        lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs, q=q_d.float()),
        lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs, q=q_d, q_rot=q_d[:2]),
        lambda: m.msa_paged_append(c.kv, torch.zeros((4, 4, D), dtype=torch.bfloat16, device="cuda")[:, ::2], k, off_d, 2, cs),
    ]
    before = c.kv.pages.view(torch.uint8).clone()
    for call in cases:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MSAError):
        m.msa_paged_attn(c.kv, q_d, off_d, 2, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.MSAError):
        m.msa_paged_attn(c.kv, q_d.float(), off_d, 2)
    torch.cuda.synchronize()
    assert m.device_status() == 0 and torch.equal(before, c.kv.pages.view(torch.uint8))


def test_the_binding_refuses_other_numbers_of_dimensions(m):
    c = Cache(m, 93, [40], 16, 2)
    off_d, _ = _offsets([2])
    cs = m.rope_table(64, D, BASE)
    k = torch.zeros((2, 2, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, D), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: m.msa_paged_append(c.kv, k[..., None], k[..., None], off_d, 2, cs),
                 lambda: m.msa_paged_append(c.kv, k.view(-1), k.view(-1), off_d, 2, cs),
                 lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs.view(-1)),
                 lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs, q=q.view(-1)),
                 lambda: m.msa_paged_append(c.kv, k, k, off_d, 2, cs, q=q[:1]),
                 lambda: m.msa_paged_attn(c.kv, q.view(2, -1), off_d, 2),
                 lambda: m.msa_page_select(c.kv, q[..., None], off_d, 2, 3)):
        with pytest.raises(ValueError):
            call()


def test_nothing_to_do(m):
    kv = m.PagedKV.empty(2, 2, 2, 2, 16)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    e = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    cs = m.rope_table(4, D, BASE)
    assert m.msa_paged_append(kv, e, e, off, 0, cs, q=torch.empty((0, 4, D), dtype=torch.bfloat16, device="cuda")).shape[0] == 0
    assert m.msa_page_select(kv, e, off, 0, 2).shape == (0, 2, 2)
    assert m.msa_paged_attn(kv, e, off, 0).shape == (0, 2, D)
    one = torch.ones((1, 2, D), dtype=torch.bfloat16, device="cuda")
    out = m.msa_paged_attn(kv, one, off, 1, out=torch.full_like(one, 3.0))       # a row of no sequence
    assert (out == 3).all() and m.device_status() == 0
