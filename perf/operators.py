"""What the attention side of a decode or prefill step costs: cases, inputs and plain forms.

Three operators stand between two W2A8 products of a decoder layer:

* ``append``: rotary positions on the queries and keys of a fused projection, and the new keys
  and values written to the paged int8 cache (one scale for each page of tokens and head);
* ``decode``: one query token of each sequence against that cache;
* ``prompt``: causal attention over whole prompts, packed one behind the other.

``run`` computes each of them from elementary torch operations in 32 bits (``own`` false) or
through ``bit_gemv_i2_amd`` (``own`` true).  ``exact`` is the definition in 64 bits.

Layouts, shared by both: the fused projection is [tokens][(q_heads + 2 kv_heads) * dim], queries
first, then keys, then values.  The cache holds ``k_cache`` int8 [pages][kv_heads][page][dim],
``v_cache`` int8 [pages][kv_heads][dim][page] (tokens fastest) and one fp32 scale for each page and
head of either; ``table`` [batch][slots] names the page of every ``page`` positions of a sequence.
The rotary table is fp32 [positions][rot]: rot/2 cosines, then rot/2 sines.

What the int8 codes are is defined in fp32, operation by operation (see ``_append_plain``), so that
they are compared as the whole numbers that they are.
"""
import math
import random

import numpy as np
import torch

own = False

HEADS = ((20, 20), (20, 5), (32, 8), (16, 1), (8, 8), (40, 8))
PAGES = (16, 32, 64, 128)
MOST_APPEND = 16384 * (32 + 2 * 8) * 128  # values of the largest listed projection
MOST_DECODE = 64 * 8192 * 8 * 128         # values of the largest listed cache's keys
MOST_PROMPT = 20 * 8192 * 8192            # scores of the largest listed prompt


def _append(name, q_heads, kv_heads, dim, page, dtype, batch, longest, ragged, before, rot, interleaved, with_k):
    return {"name": name, "op": "append", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype, "batch": batch, "longest": longest, "ragged": ragged, "before": before, "rot": rot,
            "interleaved": interleaved, "with_k": with_k}


def _decode(name, q_heads, kv_heads, dim, page, dtype, batch, longest, ragged):
    return {"name": name, "op": "decode", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype, "batch": batch, "longest": longest, "ragged": ragged}


def _prompt(name, q_heads, kv_heads, dim, batch, longest, ragged, causal=True):
    return {"name": name, "op": "prompt", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "batch": batch,
            "longest": longest, "ragged": ragged, "causal": causal}


def listed():
    return [
        # one user's next token: the fp32 projection of the decode product, 20 heads of 128 (hidden 2560)
        _append("append_1_token", 20, 20, 128, 64, "float32", 1, 1, False, 1000, 128, False, False),
        # a serving step of 64 users at different lengths, grouped heads
        _append("append_64_tokens", 20, 5, 128, 64, "bfloat16", 64, 1, True, 2000, 128, False, False),
        # the 512-token prefill of the 2560-wide model, nothing cached before it
        _append("append_prompt_512", 20, 20, 128, 64, "bfloat16", 1, 512, False, 0, 128, False, True),
        # a packed prefill of prompts of odd lengths behind cached prefixes, pairs interleaved, half of the head turned
        _append("append_packed_16k", 32, 8, 128, 16, "bfloat16", 8, 4001, True, 300, 64, True, True),
        # one user, a short context that ends inside a page, a head for each key head
        _decode("decode_1x129", 20, 20, 128, 64, "float32", 1, 129, False),
        # 16 users in the middle of their answers, grouped heads
        _decode("decode_16x4000", 20, 5, 128, 64, "float32", 16, 4000, True),
        # one user with a very long context: few rows, a long axis
        _decode("decode_1x131071", 20, 5, 128, 128, "bfloat16", 1, 131071, False),
        # a full batch at long contexts, small pages
        _decode("decode_64x8192", 32, 8, 128, 16, "bfloat16", 64, 8192, False),
        # the shortest useful prompt of the prefill workload
        _prompt("prompt_1x64", 20, 20, 128, 1, 64, False),
        # the 512-token prefill with grouped heads
        _prompt("prompt_1x512", 20, 5, 128, 1, 512, False),
        # prompts of odd lengths packed together, small heads
        _prompt("prompt_packed_9x2047", 32, 8, 64, 9, 2047, True),
        # one long document
        _prompt("prompt_1x8192", 20, 5, 128, 1, 8192, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prompt"))
    q_heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice((64, 128))
    page = rng.choice(PAGES)
    dtype = rng.choice(("bfloat16", "float32"))
    ragged = rng.random() < 0.6
    if op == "append":
        batch = _log(rng, 1, 64)
        longest = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
        longest = max(1, min(longest, MOST_APPEND // (batch * (q_heads + 2 * kv_heads) * dim)))
        rot = rng.choice((dim, dim, dim // 2, 16))
        c = _append("", q_heads, kv_heads, dim, page, dtype, batch, longest, ragged, _log(rng, 1, 2000) - 1, rot,
                    rng.random() < 0.5, longest > 1)
    elif op == "decode":
        batch = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, min(131072, MOST_DECODE // (batch * kv_heads * dim))))
        c = _decode("", q_heads, kv_heads, dim, page, dtype, batch, longest, ragged)
    else:
        batch = _log(rng, 1, 16)
        longest = _log(rng, 1, int(min(8192, math.sqrt(MOST_PROMPT / (batch * q_heads)))))
        c = _prompt("", q_heads, kv_heads, dim, batch, longest, ragged, rng.random() < 0.8)
    del c["name"]
    return c


def _spread(case, most, ragged, key):
    """One whole number 1..most for each sequence, fixed by the case; the first is `most`."""
    r = random.Random(key + repr(sorted((k, v) for k, v in case.items() if k != "name")))
    return [most if i == 0 or not ragged else r.randint(1, most) for i in range(case["batch"])]


def _lengths(case):
    return _spread(case, case["longest"], case["ragged"], "lengths")


def _before(case):
    """Tokens that each sequence has in the cache before an append, 0..case["before"]."""
    if case["batch"] == 1:
        return [case["before"]]
    return [n - 1 for n in _spread(case, case["before"] + 1, True, "before")]


def _scale(case):
    return 1.0 / math.sqrt(case["dim"])


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _whole(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lengths):
    return [0] + np.cumsum(lengths).tolist()


def _channels(g, heads, dim):
    """Gains and offsets of a projection's channels: some larger than others, keys with a mean of their own."""
    return torch.exp(0.4 * _normal(g, 1, heads, dim)), 0.5 * _normal(g, 1, heads, dim)


def _pool(case, totals, g):
    """A page table with the pages in no order and a few that nobody uses, and their number."""
    page = case["page"]
    need = [-(-n // page) for n in totals]
    slots = max(need)
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    owner = torch.repeat_interleave(torch.arange(len(need), device="cuda"), torch.tensor(need, device="cuda"))
    first = torch.tensor(_starts(need)[:-1], device="cuda")
    slot = torch.arange(len(owner), device="cuda") - first[owner]
    table = torch.zeros((len(need), slots), dtype=torch.int32, device="cuda")
    table[owner, slot] = order[: len(owner)]
    return table, pages


def _codes(g, *shape):
    """int8 codes as the quantiser leaves them: bell-shaped, the largest near 127."""
    return torch.clamp(torch.round(_normal(g, *shape) * 36.0), -127, 127).to(torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    s = {"case": dict(case), "scale": _scale(case), "longest": case["longest"]}
    if case["op"] == "prompt":
        starts = _starts(lengths)
        total = starts[-1]
        gain, mean = _channels(g, hk, dim)
        fused = torch.empty((total, (hq + 2 * hk) * dim), dtype=torch.bfloat16, device="cuda")
        fused[:, (hq + hk) * dim:] = _normal(g, total, hk * dim).to(torch.bfloat16)
        s["q"] = _normal(g, total, hq, dim).to(torch.bfloat16)
        s["k"] = (_normal(g, total, hk, dim) * gain + mean).to(torch.bfloat16)
        s["v"] = fused[:, (hq + hk) * dim:].unflatten(1, (hk, dim))  # values stay where the projection wrote them
        s["starts"] = _whole(starts)
        return s
    page, dtype = case["page"], getattr(torch, case["dtype"])
    totals = lengths if case["op"] == "decode" else [a + b for a, b in zip(lengths, _before(case))]
    s["table"], pages = _pool(case, totals, g)
    s["k_cache"] = _codes(g, pages, hk, page, dim)
    s["v_cache"] = _codes(g, pages, hk, dim, page)
    spread = torch.exp(0.3 * _normal(g, 2, pages, hk)) / 36.0
    s["k_scale"], s["v_scale"] = spread[0].contiguous(), spread[1].contiguous()
    if case["op"] == "decode":
        s["q"] = (_normal(g, case["batch"], hq, dim) * 1.3).to(dtype)
        s["lengths"] = _whole(lengths)
        return s
    starts = _starts(lengths)
    gain, mean = _channels(g, hq + 2 * hk, dim)
    x = _normal(g, starts[-1], hq + 2 * hk, dim) * gain + mean
    s["fused"] = x.to(dtype).flatten(1)
    s["starts"], s["before"] = _whole(starts), _whole(_before(case))
    s["rope"] = _rope_table(s["table"].shape[1] * page, case["rot"])
    return s


def _rope_table(positions, rot):
    at = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None]
    rate = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    return torch.cat([torch.cos(at * rate), torch.sin(at * rate)], dim=1).float()


def work(case):
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    size = 4 if case.get("dtype") == "float32" else 2
    tokens = sum(lengths)
    if case["op"] == "append":
        read = tokens * (hq + 2 * hk) * dim * size + tokens * case["rot"] * 4
        wrote = tokens * (hq + (hk if case["with_k"] else 0)) * dim * size + tokens * 2 * hk * dim
        # a turn is four products and two sums a pair; the codes a product and a rounding a value
        return {"bytes": read + wrote, "flops": tokens * ((hq + hk) * case["rot"] * 3 + 4 * hk * dim)}
    if case["op"] == "decode":
        pages = sum(-(-n // case["page"]) for n in lengths)
        return {"bytes": 2 * tokens * hk * dim + pages * (8 * hk + 4) + 2 * case["batch"] * hq * dim * size,
                "flops": 4 * tokens * hq * dim}
    scores = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lengths)
    return {"bytes": tokens * 2 * (hq + hk) * dim * 2, "flops": 4 * scores * hq * dim}


# ------------------------------------------------------------------ the plain forms
def _divide(a, b):
    """a / b with b as a tensor: division by a Python number may be a product with its rounded inverse."""
    return a / torch.full_like(a, b)


def _turn(x, rope, rot, interleaved):
    """fp32 [tokens][heads][dim] turned by [tokens][rot] (cosines, sines); each product and sum rounded by itself."""
    c, s = rope[:, None, : rot // 2], rope[:, None, rot // 2:]
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    lo, hi = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = lo, hi
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = lo, hi
    return y


def _store(x, codes, scales, by_dim, pid, at, first, used, fresh):
    """New values fp32 [tokens][heads][dim] into codes and scales.  The scale of a page and head is the largest
    of the old one (if the page has older tokens) and max(|new values|, 1e-5) / 127; older codes follow a scale
    that grew by round(code * (old / new)); a new code is round(value * (1 / scale)) within +-127."""
    pages, heads = scales.shape
    most = torch.zeros_like(scales).scatter_reduce_(0, pid[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    want = _divide(most.clamp(min=1e-5), 127.0)
    touched = torch.zeros(pages, dtype=torch.bool, device=x.device).index_fill_(0, pid, True)
    kept = torch.zeros(pages, dtype=torch.bool, device=x.device)
    kept[first] = ~fresh  # the first page of a sequence may hold older tokens
    old = scales.clone()
    new = torch.where(kept[:, None], torch.maximum(old, want), want)
    scales.copy_(torch.where(touched[:, None], new, old))
    ratio = torch.where(kept[:, None], old / scales, torch.ones_like(old))[first]
    page = codes.shape[3 if by_dim else 2]
    older = torch.arange(page, device=x.device)[None, :] < used[:, None]
    held = codes[first]
    r, o = ratio[:, :, None, None], older[:, None, None, :] if by_dim else older[:, None, :, None]
    codes[first] = torch.where(o, torch.round(held.float() * r).to(torch.int8), held)
    q = torch.clamp(torch.round(x * (torch.ones_like(scales) / scales)[pid][:, :, None]), -127, 127).to(torch.int8)
    if by_dim:
        codes[pid, :, :, at] = q
    else:
        codes[pid, :, at, :] = q


def _append_plain(s):
    case = s["case"]
    hq, hk, dim, page, rot = (case[k] for k in ("q_heads", "kv_heads", "dim", "page", "rot"))
    total = s["fused"].shape[0]
    t = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["starts"], t, right=True) - 1
    pos = (s["before"][b] + t - s["starts"][b]).long()
    pid, at = s["table"][b, pos // page].long(), pos % page
    x = s["fused"].float().unflatten(1, (hq + 2 * hk, dim))
    turned = _turn(x[:, : hq + hk], s["rope"][pos], rot, case["interleaved"])
    first = s["table"].gather(1, (s["before"].long() // page)[:, None])[:, 0].long()
    used = s["before"] % page
    for_store = (pid, at, first, used, used == 0)
    _store(turned[:, hq:], s["k_cache"], s["k_scale"], False, *for_store)
    _store(x[:, hq + hk:], s["v_cache"], s["v_scale"], True, *for_store)
    turned = turned.to(s["fused"].dtype)
    return turned[:, :hq].contiguous(), turned[:, hq:].contiguous() if case["with_k"] else None


def _decode_plain(s):
    q, table = s["q"], s["table"].long()
    batch, hq, dim = q.shape
    hk = s["k_cache"].shape[1]
    k = (s["k_cache"][table].float() * s["k_scale"][table][..., None, None]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    v = (s["v_cache"][table].float() * s["v_scale"][table][..., None, None]).permute(0, 2, 1, 4, 3).flatten(2, 3)
    scores = torch.matmul(q.float().view(batch, hk, hq // hk, dim), k.transpose(2, 3)) * s["scale"]
    there = torch.arange(k.shape[2], device="cuda")[None, :] < s["lengths"][:, None]
    p = _softmax(scores, there[:, None, None, :])
    return torch.matmul(p, v).view(batch, hq, dim).to(q.dtype)


def _softmax(scores, there):
    scores = scores.masked_fill(~there, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _prompt_plain(s):
    q, k, v, starts = s["q"], s["k"], s["v"], s["starts"].long()
    total, hq, dim = q.shape
    hk, longest = k.shape[1], s["longest"]
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    i = t - starts[b]
    n = torch.arange(longest, device="cuda")
    rows = (starts[:-1, None] + n).clamp(max=total - 1)  # [batch][longest], the rows behind a sequence's end unused
    qp = q.float()[rows].unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    kp, vp = k.float()[rows].permute(0, 2, 3, 1), v.float()[rows].permute(0, 2, 1, 3)
    scores = torch.matmul(qp, kp.contiguous()).unflatten(2, (hq // hk, longest)) * s["scale"]
    there = n[None, None, :] < (starts[1:] - starts[:-1])[:, None, None]
    if s["case"]["causal"]:
        there = there & (n[None, None, :] <= n[None, :, None])
    p = _softmax(scores, there[:, None, None])
    o = torch.matmul(p.flatten(2, 3), vp.contiguous()).unflatten(2, (hq // hk, longest)).flatten(1, 2)
    return o[b, :, i].to(q.dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        import bit_gemv_i2_amd as bn
    if op == "decode":
        if own:
            return bn.bitnet_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                         s["lengths"], s["longest"], scale=s["scale"])
        return _decode_plain(s)
    if op == "prompt":
        if own:
            return bn.bitnet_attn_prompt(s["q"], s["k"], s["v"], s["starts"], s["longest"],
                                         causal=s["case"]["causal"], scale=s["scale"])
        return _prompt_plain(s)
    if own:
        q, k = bn.bitnet_rope_append_kv(s["fused"], s["rope"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                        s["table"], s["starts"], s["before"], s["longest"], s["case"]["q_heads"],
                                        interleaved=s["case"]["interleaved"], with_k=s["case"]["with_k"])
    else:
        q, k = _append_plain(s)
    # a second pass over the same state writes the same codes: the scales have grown already
    out = {"q": q, "k_codes": s["k_cache"], "v_codes": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return dict(out, k=k) if k is not None else out


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(s):
    case = s["case"]
    hq, hk, dim, page, rot = (case[k] for k in ("q_heads", "kv_heads", "dim", "page", "rot"))
    x = s["fused"].double().cpu().numpy().reshape(-1, hq + 2 * hk, dim)
    rope = s["rope"].double().cpu().numpy()
    table, before = s["table"].cpu().numpy(), s["before"].cpu().numpy()
    k_scale, v_scale = s["k_scale"].double().cpu().numpy(), s["v_scale"].double().cpu().numpy()
    turned = x[:, : hq + hk].copy()
    j = np.arange(rot // 2)
    i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + rot // 2)
    starts = s["starts"].cpu().numpy()
    for b in range(case["batch"]):
        lo, hi = starts[b], starts[b + 1]
        pos = before[b] + np.arange(hi - lo)
        z = (x[lo:hi, : hq + hk, i0] + 1j * x[lo:hi, : hq + hk, i1]) * (rope[pos, : rot // 2] + 1j * rope[pos, rot // 2:])[:, None, :]
        turned[lo:hi, :, i0], turned[lo:hi, :, i1] = z.real, z.imag
        for slot in range(pos[0] // page, pos[-1] // page + 1):
            at = lo + np.nonzero(pos // page == slot)[0]
            pid = table[b, slot]
            older = slot * page < before[b]
            for values, scales in ((turned[at, hq:], k_scale), (x[at, hq + hk:], v_scale)):
                want = np.maximum(np.abs(values).max(axis=(0, 2)), 1e-5) / 127.0
                scales[pid] = np.maximum(scales[pid], want) if older else want
    out = {"q": turned[:, :hq], "k_codes": None, "v_codes": None, "k_scale": k_scale, "v_scale": v_scale}
    return dict(out, k=turned[:, hq:]) if case["with_k"] else out


def _exact_rows(q, k, v, scale, reach):
    """Attention of q [rows][dim] over k, v [n][dim] in float64; row r sees the first reach[r] keys."""
    w = torch.exp((q @ k.T) * scale - ((q @ k.T) * scale).amax(-1, keepdim=True))
    w = torch.where(torch.arange(k.shape[0], device=q.device)[None, :] < reach[:, None], w, torch.zeros_like(w))
    return (w @ v) / w.sum(-1, keepdim=True)


def _exact_decode(s):
    q = s["q"].double()
    batch, hq, dim = q.shape
    hk = s["k_cache"].shape[1]
    out = torch.empty_like(q)
    for b, n in enumerate(s["lengths"].tolist()):
        pages = s["table"][b, : -(-n // s["case"]["page"])].long()
        for h in range(hk):
            k = (s["k_cache"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, dim)[:n]
            v = (s["v_cache"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]).transpose(1, 2).reshape(-1, dim)[:n]
            rows = slice(h * (hq // hk), (h + 1) * (hq // hk))
            out[b, rows] = _exact_rows(q[b, rows], k, v, s["scale"], torch.full((hq // hk,), n, device="cuda"))
    return out


def _exact_prompt(s):
    q, k, v = (s[n].double() for n in "qkv")
    hq, hk = q.shape[1], k.shape[1]
    out = torch.empty_like(q)
    starts = s["starts"].tolist()
    for lo, hi in zip(starts, starts[1:]):
        n = hi - lo
        reach = torch.arange(1, n + 1, device="cuda") if s["case"]["causal"] else torch.full((n,), n, device="cuda")
        for h in range(hq):
            for r in range(0, n, 2048):  # rows a time, as the scores in 64 bits take room
                at = slice(lo + r, min(lo + r + 2048, hi))
                seen = int(reach[r: r + 2048].max())
                kv = slice(lo, lo + seen)
                out[at, h] = _exact_rows(q[at, h], k[kv, h * hk // hq], v[kv, h * hk // hq], s["scale"], reach[r: r + 2048])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](s)
