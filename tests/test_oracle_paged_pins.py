"""Pins of the paged cache's fp64 definition (oracle/paged_cache.py) to closed forms and to torch."""
import numpy as np
import torch

from oracle import paged_cache as C


def test_e4m3_bytes_and_rounding_are_torchs():
    b = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    np.testing.assert_array_equal(C.decode_e4m3(b), ref)
    # every value and every halfway point between neighbours, and a little to each side of it
    pos = np.sort(ref[(ref >= 0) & np.isfinite(ref)])
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), [1e-9, 2.0 ** -10]])
    x = np.concatenate([x, -x])
    got = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(C.round_e4m3(x.astype(np.float32)), got)
    assert C.round_e4m3(1e6) == 448 and C.round_e4m3(-449.0) == -448


def test_needed_scale_is_the_smallest_that_fits():
    for a in [448.0, 448.0001, 1.0, 3.5, 3.5000001, 7.0, 1e-3, 6.1e4]:
        s = float(C.needed_scale(a))
        assert a <= 448 * s and a > 448 * s / 2 and np.log2(s) == round(np.log2(s))
    assert C.needed_scale(0.0) == 2.0 ** -50 and C.needed_scale(1e30) == 2.0 ** 50


def _empty(n_pages, hkv, page, d):
    return np.zeros((n_pages, 2, hkv, page, d)), np.ones((n_pages, 2, hkv)), np.zeros((n_pages, hkv, 2, d))


def test_token_by_token_equals_at_once_where_nothing_gets_subnormal():
    rng = np.random.default_rng(1)
    k, v = rng.uniform(0.5, 3, (2, 37, 2, 8)) * rng.choice([-1, 1], (2, 37, 2, 8))
    a, b = _empty(4, 2, 16, 8), _empty(4, 2, 16, 8)
    C.append(*a, [2, 0, 3], 0, k, v, pos_offset=5)
    for t in range(37):
        C.append(*b, [2, 0, 3], t, k[t:t + 1], v[t:t + 1], pos_offset=5)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)
    # and the stored values are the rotated keys and the values to half a step
    kk = np.stack([C.rows_of(a[0], a[1], [2, 0, 3], 37, 1, h) for h in range(2)], 1)
    assert (np.abs(kk - v) <= 2.0 ** -4 * np.abs(v) + 1e-12).all()


def test_a_fresh_page_forgets_and_an_older_one_grows():
    vals, scales, bounds = _empty(1, 1, 16, 4)
    C.append(vals, scales, bounds, [0], 0, np.full((2, 1, 4), 1000.0), np.full((2, 1, 4), 1000.0), rope_base=1e6)
    assert scales[0, 1, 0] == 4                                       # 1000 <= 448 * 4
    C.append(vals, scales, bounds, [0], 0, np.ones((1, 1, 4)), np.ones((1, 1, 4)))
    assert scales[0, 1, 0] == 2.0 ** -8                               # 1 <= 448 / 256: 448 / 512 is too small
    C.append(vals, scales, bounds, [0], 1, np.full((1, 1, 4), 3.0), np.full((1, 1, 4), 3.0))
    assert scales[0, 1, 0] == 2.0 ** -7 and (vals[0, 1, 0, 0] == 128).all()


def test_attend_is_softmax_and_empty_rows_are_zero():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal(16), rng.standard_normal((9, 16)), rng.standard_normal((9, 16))
    vis = np.arange(9) < 6
    o, lse = C.attend(q, k, v, vis, 0.25)
    t = lambda x: torch.from_numpy(x)[None, None]  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(t(q[None]), t(k[:6]), t(v[:6]), scale=0.25)
    np.testing.assert_allclose(o, ref[0, 0, 0].numpy(), rtol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(torch.from_numpy(k[:6] @ q * 0.25), 0).item(), rtol=1e-12)
    o, lse = C.attend(q, k, v, np.zeros(9, bool), 0.25)
    assert (o == 0).all() and lse == -np.inf


def test_page_score_bounds_every_key_and_ties_go_low():
    rng = np.random.default_rng(3)
    keys = rng.standard_normal((5, 16, 8))
    q = rng.standard_normal((4, 8))
    s = C.page_scores(q, keys.min(1), keys.max(1))
    assert (s >= np.einsum("gd,prd->gpr", q, keys).max((0, 2)) - 1e-12).all()
    one = C.page_scores(q, keys[:, 0], keys[:, 0])                    # a page of one key: its own logit
    np.testing.assert_allclose(one, (keys[:, 0] @ q.T).max(-1))
    np.testing.assert_array_equal(C.pick([1, 5, 5, 5, 0, 0], 3, 1), [1, 2, 5])
    np.testing.assert_array_equal(C.pick([1, 2], 4, 1), [0, 1, -1, -1])
    np.testing.assert_array_equal(C.pick([9, 8, 7, 6], 2, 2), [2, 3])
