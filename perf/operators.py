"""Cases for measuring the paged 8-bit key/value cache: appending to it, attending over it and attending
over the pages that a cheap score picks.

The cache holds the active context of `n_seq` sequences in pages of `page` tokens: e4m3 values
[n_pages][2 (K, V)][hkv][page][d], one power-of-two scale per page, part and kv head
[n_pages][2][hkv], and elementwise bounds of each page's keys [n_pages][hkv][2 (min, max)][d].
`run` computes an operator in elementary torch operations, or (own = True) by the library's calls.
"""
import math

import numpy as np
import torch

own = False

D = 128                 # head dimension of every attention in this repository
BASE = 1.0e6            # RoPE base
POS_OFFSET = 12         # the active context starts at position k, the document count of the interleave workload
E_MIN, E_MAX = -50, 50  # range of the scale exponents
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of the 8 queries of the interleave workload, after its last round
        {"name": "append-token", "op": "append", "n_seq": 8, "new": 1, "len": 1024, "ragged": True, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # a round of the same workload in fp32: up to 32 new tokens a query, one query already finished
        {"name": "append-round", "op": "append", "n_seq": 8, "new": 32, "len": 1900, "ragged": True, "page": 16,
         "hq": 32, "hkv": 8, "dtype": "float32"},
        # the prompt of a 64K-token training context, packed at once
        {"name": "append-64k", "op": "append", "n_seq": 1, "new": 65536, "len": 65536, "ragged": False, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # one decode token over a short context: latency
        {"name": "attend-short", "op": "attend", "n_seq": 1, "new": 1, "len": 777, "ragged": False, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # the 32 decode queries of the 10M workload, each with its own context of up to 16K tokens
        {"name": "attend-batch", "op": "attend", "n_seq": 32, "new": 1, "len": 16384, "ragged": True, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # one decode token over a very long context: the long axis has to be split
        {"name": "attend-long", "op": "attend", "n_seq": 1, "new": 1, "len": 500001, "ragged": False, "page": 128,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # a round of drafted or appended tokens: 8 queries of up to 32 tokens over the 8K rows of the fine stage
        {"name": "attend-round", "op": "attend", "n_seq": 8, "new": 32, "len": 8096, "ragged": True, "page": 32,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # a prompt's slice of 2,000 tokens over 16K tokens already in the cache: bound by the products
        {"name": "attend-prompt", "op": "attend", "n_seq": 1, "new": 2000, "len": 18000, "ragged": False, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16"},
        # one decode token for each of 8 queries over 64K tokens, of which each kv head reads 32 pages
        {"name": "pick-decode", "op": "pick", "n_seq": 8, "new": 1, "len": 65536, "ragged": True, "page": 64,
         "hq": 32, "hkv": 8, "dtype": "bfloat16", "k": 32, "recent": 2},
        # 64 tokens (the prompt of a 1M or interleave query) over a long context, each with its own pages
        {"name": "pick-prompt", "op": "pick", "n_seq": 1, "new": 64, "len": 200000, "ragged": False, "page": 32,
         "hq": 32, "hkv": 8, "dtype": "bfloat16", "k": 64, "recent": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "pick"])
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    if op == "append":
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        n_seq = _log_int(rng, 1, 64)
        most = int(1.4e9 / (D * (2 * hkv + 2 * (hq + hkv) * (4 if dtype == "float32" else 2))))
        new = _log_int(rng, 1, max(1, min(65536, most) // n_seq))
        length = new + _log_int(rng, 1, 8192)
        return {"op": op, "n_seq": n_seq, "new": new, "len": length, "ragged": rng.random() < 0.7, "page": page,
                "hq": hq, "hkv": hkv, "dtype": dtype}
    if op == "attend":
        n_seq = _log_int(rng, 1, 64)
        length = _log_int(rng, 16, 262144 // n_seq)
        most = min(length, 2000 // n_seq, 1_000_000_000 // (n_seq * length * hq))
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, max(2, most))
        return {"op": op, "n_seq": n_seq, "new": new, "len": length, "ragged": rng.random() < 0.7, "page": page,
                "hq": hq, "hkv": hkv, "dtype": "bfloat16"}
    n_seq = _log_int(rng, 1, 16)
    length = _log_int(rng, 1000, 262144 // n_seq)
    new = 1 if rng.random() < 0.6 else _log_int(rng, 2, max(2, 48 // n_seq))
    k = _log_int(rng, 4, 2048 // page)
    return {"op": op, "n_seq": n_seq, "new": new, "len": length, "ragged": rng.random() < 0.7, "page": page,
            "hq": hq, "hkv": hkv, "dtype": "bfloat16", "k": k, "recent": rng.randint(1, min(k, 4))}


def _fractions(n, step):
    return [((i + 1) * step) % 1.0 for i in range(n)]


def _lengths(case):
    """(new tokens, context length with them) of every sequence: the case alone decides. Where it is ragged,
    sequence 0 has the largest of both and, of several that add more than one token, one adds none."""
    n, new, length = case["n_seq"], case["new"], case["len"]
    news, lens = [new] * n, [length] * n
    if case["ragged"]:
        for i, (a, b) in enumerate(zip(_fractions(n, 0.754877666), _fractions(n, 0.569840291))):
            if i:
                news[i] = max(1, round(new * a))
                lens[i] = max(news[i], round(length * b))
        if n >= 4 and new > 1:
            news[n // 2] = 0
    return news, [max(a, b) for a, b in zip(news, lens)]


# ------------------------------------------------------------------------------------------------ inputs
def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _stored(pages, *at):
    """pages[at] in 32 bits."""
    return pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()


def _scale(amax):
    """The smallest power of two in range that amax / 448 does not exceed."""
    m, e = torch.frexp(amax)
    return torch.exp2(torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(E_MIN, E_MAX), E_MIN).float())


def _fill_pages(g, pages, scales, bounds, rows, key_gain):
    """Random keys and values in every page, as an earlier append left them; rows[p] of page p are in use."""
    n_pages, _, hkv, page, _ = pages.shape
    at = torch.arange(page, device="cuda")
    for lo in range(0, n_pages, 2048):
        hi = min(n_pages, lo + 2048)
        x = torch.randn((hi - lo, 2, hkv, page, D), generator=g, device="cuda")
        x[:, 0] *= key_gain
        x *= torch.exp2(torch.randint(-1, 2, (hi - lo, 2, 1, 1, 1), generator=g, device="cuda").float())
        used = at < rows[lo:hi, None, None, None]
        scale = _scale(torch.where(used[..., None], x.abs(), 0).amax((-1, -2)))
        q = _e4m3(x / scale[..., None, None])
        pages[lo:hi].copy_(q)
        scales[lo:hi] = scale
        keys = q[:, 0].float() * scale[:, 0, :, None, None]
        mask = used.reshape(hi - lo, 1, page, 1)
        some = (rows[lo:hi] > 0)[:, None, None]
        bounds[lo:hi, :, 0] = torch.where(some, torch.where(mask, keys, math.inf).amin(-2), 0).bfloat16()
        bounds[lo:hi, :, 1] = torch.where(some, torch.where(mask, keys, -math.inf).amax(-2), 0).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    dt = getattr(torch, case["dtype"])
    n, page, hq, hkv = case["n_seq"], case["page"], case["hq"], case["hkv"]
    news, lens = _lengths(case)
    counts = [-(-x // page) for x in lens]
    max_pages = max(counts) + 1
    n_pages = sum(counts) + 8
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((n, max_pages), dtype=torch.int32, device="cuda")
    rows = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    first = 0
    for s in range(n):
        ids = perm[first:first + counts[s]]
        table[s, :counts[s]] = ids
        stored = lens[s] - news[s] if case["op"] == "append" else lens[s]
        rows[ids.long()] = (stored - page * torch.arange(counts[s], device="cuda")).clamp(0, page)
        first += counts[s]
    pages = torch.empty((n_pages, 2, hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((n_pages, 2, hkv), dtype=torch.float32, device="cuda")
    bounds = torch.empty((n_pages, hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    # a few channels of the keys carry more than the others, as in trained models
    gain = torch.where(torch.rand(D, generator=g, device="cuda") < 0.06, 4.0, 1.0)
    _fill_pages(g, pages, scales, bounds, rows, gain)
    n_tok = sum(news)
    off = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int64, device="cuda")
    q = torch.randn((n_tok, hq, D), generator=g, device="cuda").to(dt)
    state = {"case": dict(case), "q": q, "tok_off": off, "max_new": max(news), "table": table,
             "seq_len": torch.tensor(lens, dtype=torch.int32, device="cuda"), "pages": pages, "scales": scales,
             "bounds": bounds}
    if case["op"] == "append":
        state["k"] = (torch.randn((n_tok, hkv, D), generator=g, device="cuda") * gain).to(dt)
        state["v"] = torch.randn((n_tok, hkv, D), generator=g, device="cuda").to(dt)
        pos = torch.arange(max(lens) + POS_OFFSET, device="cuda", dtype=torch.float64)
        inv = BASE ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
        ang = pos[:, None] * inv
        state["cos_sin"] = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
    state["kv"] = _handle(state)
    return state


def _handle(state):
    """What a program keeps beside the cache: the library's view of it."""
    if own:
        import routed_long_context_b200 as m

        return m.PagedKV(state["pages"], state["scales"], state["table"], state["seq_len"], state["bounds"])
    return None


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        import routed_long_context_b200 as m

        case, kv, off, new = state["case"], state["kv"], state["tok_off"], state["max_new"]
        if case["op"] == "append":
            q_rot = m.msa_paged_append(kv, state["k"], state["v"], off, new, state["cos_sin"], POS_OFFSET,
                                       q=state["q"])
            return {"pages": state["pages"], "scales": state["scales"], "bounds": state["bounds"], "q": q_rot}
        sel = m.msa_page_select(kv, state["q"], off, new, case["k"], case["recent"]) if case["op"] == "pick" else None
        out, lse = m.msa_paged_attn(kv, state["q"], off, new, sel=sel, want_lse=True)
        return {"out": out, "lse": lse} if sel is None else {"sel": sel, "out": out, "lse": lse}
    return {"append": _append, "attend": _attend, "pick": _pick}[state["case"]["op"]](state)


def _token_index(state):
    """(sequence, index in its context) of every new token."""
    off, n_tok = state["tok_off"], state["q"].shape[0]
    t = torch.arange(n_tok, device="cuda")
    seq = torch.searchsorted(off, t, right=True) - 1
    return seq, state["seq_len"][seq].long() - (off[seq + 1] - t)


def _rotate(x, cs):
    """x [n_tok, heads, d] by the (cos, sin) rows cs [n_tok, d/2, 2], element i paired with i + d/2."""
    a, b = x[..., :D // 2].float(), x[..., D // 2:].float()
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _append(state):
    pages, scales, bounds = state["pages"], state["scales"], state["bounds"]
    n_pages, _, hkv, page, _ = pages.shape
    seq, idx = _token_index(state)
    cs = state["cos_sin"][idx + POS_OFFSET]
    x = torch.stack((_rotate(state["k"], cs), state["v"].float()), 1)            # [n_tok, 2, hkv, d]
    slot, row = state["table"][seq, idx // page].long(), idx % page
    # the scale of every page that takes tokens: what its new tokens need, and its own where it holds older ones
    start = torch.full((n_pages,), page, device="cuda").scatter_reduce(0, slot, row, "amin")
    touched, older = start < page, (start > 0) & (start < page)
    amax = torch.zeros((n_pages, 2, hkv), device="cuda").index_reduce(0, slot, x.abs().amax(-1), "amax")
    need = _scale(amax)
    new = torch.where(older[:, None, None], torch.maximum(scales, need), need)
    # older tokens of a page whose scale grows are rounded to the new scale
    grown = (older[:, None, None] & (new > scales)).any(-1).any(-1).nonzero()[:, 0]
    ratio = scales[grown] / new[grown]
    old = torch.arange(page, device="cuda")[None, :] < start[grown, None]
    was = _stored(pages, grown)
    was = _e4m3(torch.where(old[:, None, None, :, None], was * ratio[..., None, None], was))
    pages.view(torch.uint8)[grown] = was.view(torch.uint8)
    q = _e4m3(x / new[slot][..., None])
    pages.view(torch.uint8)[slot, :, :, row] = q.view(torch.uint8)
    # bounds of the keys as they are stored
    keys = q[:, 0].float() * new[slot, 0][..., None]                              # [n_tok, hkv, d]
    kept = torch.where(older[:, None, None, None], bounds.float(), torch.tensor([math.inf, -math.inf], device="cuda")[:, None])
    shrunk = _e4m3((bounds[grown].float() / new[grown, 0][..., None, None])).float() * new[grown, 0][..., None, None]
    kept[grown] = shrunk
    lo = kept[:, :, 0].index_reduce(0, slot, keys, "amin")
    hi = kept[:, :, 1].index_reduce(0, slot, keys, "amax")
    t4 = touched[:, None, None]
    bounds.copy_(torch.stack((torch.where(t4, lo, bounds[:, :, 0].float()), torch.where(t4, hi, bounds[:, :, 1].float())), 2))
    scales.copy_(torch.where(t4, new, scales))
    return {"pages": pages, "scales": scales, "bounds": bounds, "q": _rotate(state["q"], cs).to(state["q"].dtype)}


def _softmax_rows(s, v, dtype):
    """Attention rows of logits s [..., rows, keys] (-inf where hidden) and values v [..., keys, d]: out, lse."""
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    return out.to(dtype), (top + torch.log(total))[..., 0]


def _attend(state):
    q, off, lens, table = state["q"], state["tok_off"], state["seq_len"].long(), state["table"].long()
    n_tok, hq, _ = q.shape
    n, max_pages = table.shape
    _, _, hkv, page, _ = state["pages"].shape
    new, G = state["max_new"], hq // hkv
    seq, idx = _token_index(state)
    within = torch.arange(n_tok, device="cuda") - off[seq]
    padded = torch.zeros((n, new, hq, D), device="cuda")
    padded[seq, within] = q.float()
    kv = _stored(state["pages"], table) * state["scales"][table][..., None, None]      # [n, pages, 2, hkv, page, d]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, n, hkv, max_pages * page, D)
    at = torch.arange(max_pages * page, device="cuda")
    v = torch.where((at < lens[:, None])[:, None, :, None], kv[1], 0.0)
    qg = padded.reshape(n, new, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, hkv, new * G, D)
    s = (qg @ kv[0].transpose(-1, -2)) / math.sqrt(D)                                 # [n, hkv, new * G, keys]
    last = lens[:, None] - (off[1:] - off[:-1])[:, None] + torch.arange(new, device="cuda")
    s.masked_fill_((at > last[..., None]).repeat_interleave(G, 1)[:, None], -math.inf)
    out, lse = _softmax_rows(s, v, q.dtype)
    out = out.reshape(n, hkv, new, G, D).permute(0, 2, 1, 3, 4).reshape(n, new, hq, D)
    lse = lse.reshape(n, hkv, new, G).permute(0, 2, 1, 3).reshape(n, new, hq)
    return {"out": out[seq, within], "lse": lse[seq, within]}


def _pick(state):
    case, q, table = state["case"], state["q"], state["table"].long()
    n_tok, hq, _ = q.shape
    n, max_pages = table.shape
    _, _, hkv, page, _ = state["pages"].shape
    new, G, k = state["max_new"], hq // hkv, case["k"]
    seq, idx = _token_index(state)
    within = torch.arange(n_tok, device="cuda") - state["tok_off"][seq]
    # a page's score: the largest logit that keys inside its bounds could give a query head of the group (64 bits:
    # pages next to the border differ by little)
    padded = torch.zeros((n, new, hq, D), dtype=torch.float64, device="cuda")
    padded[seq, within] = q.double()
    qg = padded.reshape(n, new, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, hkv, new * G, D)
    b = state["bounds"][table].permute(3, 0, 2, 4, 1).double()                        # [2, n, hkv, d, pages]
    visible = torch.arange(max_pages, device="cuda") <= idx[:, None] // page          # [n_tok, pages]
    shown = torch.arange(max_pages, device="cuda") < -(-state["seq_len"].long() // page)[:, None]
    b = torch.where(shown[None, :, None, None], b, 0.0)
    score = qg.clamp(min=0) @ b[1] + qg.clamp(max=0) @ b[0]                           # [n, hkv, new * G, pages]
    score = score.reshape(n, hkv, new, G, max_pages).amax(3).permute(0, 2, 1, 3)[seq, within]   # [n_tok, hkv, pages]
    recent = visible & (torch.arange(max_pages, device="cuda") > idx[:, None] // page - case["recent"])
    score = torch.where(recent[:, None], math.inf, torch.where(visible[:, None], score, -math.inf))
    best = torch.sort(score, dim=-1, descending=True, stable=True)
    kk = min(k, max_pages)
    sel = torch.where(best.values[..., :kk] > -math.inf, best.indices[..., :kk], max_pages).sort(-1).values
    sel = torch.nn.functional.pad(sel, (0, k - kk), value=max_pages)
    some = sel < max_pages
    at = torch.where(some, sel, 0)
    slot = table[seq[:, None, None], at]                                              # [n_tok, hkv, k]
    head = torch.arange(hkv, device="cuda")[None, :, None]
    keys = (_stored(state["pages"], slot, 0, head) * state["scales"][slot, 0, head][..., None, None])
    vals = (_stored(state["pages"], slot, 1, head) * state["scales"][slot, 1, head][..., None, None])
    pos = at[..., None] * page + torch.arange(page, device="cuda")
    seen = some[..., None] & (pos <= idx[:, None, None, None])
    seen = seen.reshape(n_tok, hkv, 1, k * page)
    vals = torch.where(seen.reshape(n_tok, hkv, k * page, 1), vals.reshape(n_tok, hkv, k * page, D), 0.0)
    s = (q.float().reshape(n_tok, hkv, G, D) @ keys.reshape(n_tok, hkv, k * page, D).transpose(-1, -2)) / math.sqrt(D)
    out, lse = _softmax_rows(s.masked_fill(~seen, -math.inf), vals, q.dtype)
    return {"sel": torch.where(some, sel, -1).to(torch.int32), "out": out.reshape(n_tok, hq, D),
            "lse": lse.reshape(n_tok, hq)}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    news, lens = _lengths(case)
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    size = 4 if case["dtype"] == "float32" else 2
    n_tok = sum(news)
    row = 2 * hkv * D                                       # K and V values of one token
    if case["op"] == "append":
        pages = sum(-(-b // page) - (b - a) // page for a, b in zip(news, lens) if a)
        table = 4 * D * len({b - a + i for a, b in zip(news, lens) for i in range(a)})
        return {"bytes": n_tok * (row * (size + 1) + 2 * hq * D * size) + pages * hkv * (4 * D + 8) + table,
                "flops": n_tok * (3 * (hq + hkv) * D + 2 * row)}
    seen = [b - a + i + 1 for a, b in zip(news, lens) for i in range(a)]              # keys each token may see
    rows = n_tok * hq * (4 * D + 4)
    if case["op"] == "attend":
        read = sum(b for a, b in zip(news, lens) if a)
        return {"bytes": read * row + 8 * hkv * sum(-(-b // page) for a, b in zip(news, lens) if a) + rows,
                "flops": 4 * D * hq * sum(seen)}
    k = case["k"]
    counts = [-(-b // page) for b in lens]
    picked = sum(min(a * k, c) for a, c in zip(news, counts))
    return {"bytes": sum(counts) * hkv * 4 * D + picked * page * row + n_tok * hkv * k * 4 + rows,
            "flops": sum(4 * D * hq * (-(-x // page) + min(x, k * page)) for x in seen)}


# ------------------------------------------------------------------------------------------------ 64 bits
def _round_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, halves to even: 3 fraction bits, exponents from -6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    news, lens = _lengths(case)
    n, page, hq, hkv = case["n_seq"], case["page"], case["hq"], case["hkv"]
    G = hq // hkv
    table = st["table"].tolist()
    off = [0] + list(np.cumsum(news))
    if case["op"] == "append":
        return _exact_append(st, news, lens, off, table, page, hkv)
    n_tok = off[-1]
    out = torch.zeros((n_tok, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n_tok, hq), dtype=torch.float64, device="cuda")
    sel = torch.full((n_tok, hkv, case.get("k", 1)), -1, dtype=torch.int32, device="cuda")
    for s in range(n):
        if not news[s]:
            continue
        ids = torch.tensor(table[s][:-(-lens[s] // page)], device="cuda")
        q = st["q"][off[s]:off[s + 1]].double()
        idx = torch.arange(lens[s] - news[s], lens[s], device="cuda")
        for h in range(hkv):
            kv = [(_stored(st["pages"], ids, p, h).double() * st["scales"][ids, p, h].double()[:, None, None])
                  .reshape(-1, D)[:lens[s]] for p in (0, 1)]
            keep = None
            if case["op"] == "pick":
                lo, hi = (st["bounds"][ids, h, b].double() for b in (0, 1))
                keep = torch.zeros((news[s], len(ids)), dtype=torch.bool, device="cuda")
                for t in range(news[s]):
                    last = int(idx[t]) // page
                    bound = torch.stack([torch.maximum(q[t, h * G + i] * lo, q[t, h * G + i] * hi).sum(-1)
                                         for i in range(G)]).amax(0)[:last + 1].tolist()
                    forced = [p for p in range(last + 1) if p > last - case["recent"]]
                    rest = sorted((p for p in range(last + 1) if p <= last - case["recent"]),
                                  key=lambda p: (-bound[p], p))
                    taken = sorted(forced + rest[:case["k"] - len(forced)])
                    keep[t, torch.tensor(taken, device="cuda")] = True
                    sel[off[s] + t, h, :len(taken)] = torch.tensor(taken, dtype=torch.int32, device="cuda")
                keep = keep.repeat_interleave(page, 1)[:, :lens[s]]
            for lo_t in range(0, news[s], 512):
                hi_t = min(news[s], lo_t + 512)
                hide = torch.arange(lens[s], device="cuda") > idx[lo_t:hi_t, None]
                if keep is not None:
                    hide |= ~keep[lo_t:hi_t]
                for i in range(h * G, h * G + G):
                    z = (q[lo_t:hi_t, i] @ kv[0].T / math.sqrt(D)).masked_fill(hide, -math.inf)
                    lse[off[s] + lo_t:off[s] + hi_t, i] = torch.logsumexp(z, -1)
                    out[off[s] + lo_t:off[s] + hi_t, i] = torch.softmax(z, -1) @ kv[1]
    return {"out": out, "lse": lse} if case["op"] == "attend" else {"sel": sel, "out": out, "lse": lse}


def _exact_append(st, news, lens, off, table, page, hkv):
    pages, scales, bounds = st["pages"].double(), st["scales"].double(), st["bounds"].double()
    cs = st["cos_sin"].double()

    def turned(x, first):
        z = torch.view_as_complex(cs[first:first + x.shape[0]].contiguous())[:, None]
        z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * z
        return torch.cat((z.real, z.imag), -1)

    q = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(len(news)):
        if not news[s]:
            continue
        base = lens[s] - news[s]
        mine = slice(off[s], off[s + 1])
        q[mine] = turned(st["q"][mine], base + POS_OFFSET)
        # the scale is set by the keys as the operator rounds them: 32-bit values
        new = torch.stack((turned(st["k"][mine], base + POS_OFFSET).float().double(), st["v"][mine].double()), 1)
        for p in range(base // page, -(-lens[s] // page)):
            pid = table[s][p]
            first = max(base - p * page, 0)
            rows = new[p * page + first - base:min(lens[s], (p + 1) * page) - base]     # [rows, 2, hkv, d]
            rows = rows.permute(1, 2, 0, 3)
            top = rows.abs().amax((-1, -2))
            e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(E_MIN, E_MAX)
            scale = torch.maximum(torch.exp2(e), scales[pid]) if first else torch.exp2(e)
            if first:
                ratio = (scales[pid] / scale)[..., None, None]
                pages[pid, :, :, :first] = _round_e4m3(pages[pid, :, :, :first] * ratio)
            pages[pid, :, :, first:first + rows.shape[2]] = _round_e4m3(rows / scale[..., None, None])
            scales[pid] = scale
            keys = pages[pid, 0, :, :first + rows.shape[2]] * scale[0][:, None, None]
            bounds[pid, :, 0], bounds[pid, :, 1] = keys.amin(1), keys.amax(1)
    return {"pages": pages, "scales": scales, "bounds": bounds, "q": q}
