"""Attention side on the GPU: caches and inputs whose values lie far apart or are not finite, under bounds that are those of each row."""
import numpy as np
import pytest

import attn_bounds as ab
import attn_oracle as ao

pytestmark = pytest.mark.gpu


def _as(x, dtype):
    """Host array -> (device tensor of dtype, the fp64 values that it holds)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _int(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def _dev(c):
    import torch
    return [torch.from_numpy(a.copy()).cuda() for a in (c.k, c.v, c.ks, c.vs)]


def _decode(q, c, table, lengths, out_dtype):
    import torch

    import bit_gemv_i2_amd as bn
    out = bn.bitnet_attn_decode(q, *_dev(c), _int(table), _int(lengths), max(lengths), out_dtype=getattr(torch, out_dtype))
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


# ------------------------------------------------------------------ decode: the digits' bounds, whatever the types
EDGES = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700]


@pytest.mark.parametrize("qdt,odt", [("bfloat16", "bfloat16"), ("float32", "float32"), ("bfloat16", "float32"), ("float32", "bfloat16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq", [2, 8, 20])
def test_decode_types_within_the_bounds_of_30_and_23_bits(gpu, hq, page, dim, qdt, odt):
    """Queries have 30 bits and weights 23 in every combination of types."""
    rng = np.random.default_rng(hq + page + dim)
    slots = -(-max(EDGES) // page)
    c = ao.Cache(len(EDGES) * slots, 2, dim, page, rng)
    table = rng.permutation(c.pages).reshape(len(EDGES), slots)
    qd, q64 = _as(rng.standard_normal((len(EDGES), hq, dim)) * 1.5, qdt)
    got = _decode(qd, c, table, EDGES, odt)
    want, tol = ao.decode(q64, c, table, EDGES, dim ** -0.5, True, 30)
    fine, worst = ao.within(got, want, tol, odt == "bfloat16")
    assert fine, worst


@pytest.mark.parametrize("qdt,odt", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16")])
@pytest.mark.parametrize("hq,dim,page,n", [(4, 64, 16, 9000), (12, 128, 64, 4000), (1, 128, 128, 20001)])
def test_decode_types_in_long_contexts(gpu, hq, dim, page, n, qdt, odt):
    rng = np.random.default_rng(n)
    c = ao.Cache(-(-n // page), 1, dim, page, rng)
    table = rng.permutation(c.pages)[None, :]
    qd, q64 = _as(rng.standard_normal((1, hq, dim)) * 1.5, qdt)
    want, tol = ao.decode(q64, c, table, [n], dim ** -0.5, True, 30)
    fine, worst = ao.within(_decode(qd, c, table, [n], odt), want, tol, odt == "bfloat16")
    assert fine, worst


# ------------------------------------------------------------------ decode: value scales far apart
@pytest.mark.parametrize("ratio", [1e-9, 1e-6, 1e-4, 1e-2, 1.0, 1e2, 1e3, 1e4, 1e5, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("hq", [2, 8])  # digits side by side, and one product after the other
@pytest.mark.parametrize("page", [16, 32])
def test_decode_page_of_other_value_scale_without_weight(gpu, hq, page, ratio):
    """One page of a tile has values `ratio` times those of the rest and scores 42 (60 powers of two) lower: its tokens weigh
    nothing, and the digits of the others' weights must not be measured by it."""
    rng = np.random.default_rng(int(page + hq))
    n, dim = 130, 64
    c = ao.Cache(-(-n // page), 1, dim, page, rng)
    table = rng.permutation(c.pages)[None, :]
    c.ks[:], c.vs[:] = 0.02, 0.03
    c.k[:, :, :, 0] = 100
    c.k[:, :, :, 1:] //= 8
    odd = table[0, 1]
    c.k[odd, :, :, 0] = -68  # 168 codes of channel 0 below the rest
    c.vs[odd] = 0.03 * ratio
    q = rng.standard_normal((1, hq, dim)) * 0.3
    q[..., 0] = 42 / (168 * 0.02 * dim ** -0.5)
    for dtype in ("float32", "bfloat16"):
        qd, q64 = _as(q, dtype)
        fine, worst = ab.decode_fine(_decode(qd, c, table, [n], dtype), q64, c, table, [n], dim ** -0.5, dtype == "bfloat16")
        assert fine, (dtype, worst)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [3, 12])
def test_decode_value_scales_over_many_orders(gpu, dim, hq):
    """Every page a value scale of its own, 24 orders of magnitude apart, and scores a few powers of two apart."""
    rng = np.random.default_rng(dim + hq)
    c = ao.Cache(60, 1, dim, 16, rng)
    c.vs[:] = 10.0 ** rng.uniform(-12, 12, c.vs.shape)
    table = np.stack([rng.permutation(60)[:30] for _ in range(3)])
    lengths = [480, 33, 100]
    qd, q64 = _as(rng.standard_normal((3, hq, dim)), "float32")
    fine, worst = ab.decode_fine(_decode(qd, c, table, lengths, "float32"), q64, c, table, lengths, dim ** -0.5, False)
    assert fine, worst


@pytest.mark.parametrize("hq", [4, 8])
@pytest.mark.parametrize("tiny", [0.0, 1e-44, 1e-37, 1e-30])
def test_decode_value_scales_near_zero(gpu, hq, tiny):
    """All values tiny, and tiny ones with the weight beside larger ones without: a unit of the weights stays a number."""
    rng = np.random.default_rng(hq)
    c = ao.Cache(8, 1, 64, 16, rng)
    table = np.arange(8)[None, :]
    c.vs[:] = tiny
    qd, q64 = _as(rng.standard_normal((1, hq, 64)), "float32")
    want, tol = ab.decode(q64, c, table, [128], 0.125)
    got = _decode(qd, c, table, [128], "float32")
    assert np.all(np.abs(got - want) <= tol + 64 * 128 * 2.0 ** -126 * 127)  # under the least unit, 2^-126, half of it a token
    c.vs[::2] = 1e30
    c.k[::2, :, :, 0], c.k[1::2, :, :, 0] = -100, 100
    c.ks[:] = 0.02
    q = np.zeros((1, hq, 64))
    q[..., 0] = 60 / (200 * 0.02 * 0.125)  # the pages with large values weigh e^-60 of the others
    qd, q64 = _as(q, "float32")
    fine, worst = ab.decode_fine(_decode(qd, c, table, [128], "float32"), q64, c, table, [128], 0.125, False)
    assert fine, worst


# ------------------------------------------------------------------ decode: pages that are not finite
def _digits_of_one_sign(sign):
    """A query value below 1 whose four digits to the base 256, 30 bits below 1, are 1, 1, 1 and 64."""
    return sign * 0x01010140 * 2.0 ** -30


@pytest.mark.parametrize("n", [1, 65, 129, 5121])  # the first token of a page; the last of these in a context that is cut
@pytest.mark.parametrize("hq", [2, 8, 16])  # key heads of 1, 4 and 8 queries
@pytest.mark.parametrize("part", ["key", "value"])
def test_decode_an_infinity_alone_in_its_page_is_seen(gpu, part, hq, n):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(n + hq)
    hk, dim = 2, 64
    pages = -(-n // 64)
    table = _int([list(range(pages))])
    for bad in (np.inf, -np.inf):
        for sign in (1, -1):
            c = bn.KVCache.empty(pages, hk, dim, 64)
            x = rng.uniform(-0.9, 0.9, (n, hq + 2 * hk, dim)).astype(np.float32)
            x[0, :, 3] = 0.95  # so that the digits of a query lie where they are wanted
            x[0, :hq, 7] = _digits_of_one_sign(sign)
            x[n - 1, hq + 1 + (hk if part == "value" else 0), 7] = bad  # of key head 1
            q, _ = c.append(torch.from_numpy(x).cuda().flatten(1), None, table, _int([0, n]), _int([0]), n, hq)
            out = c.attend(q[:1].contiguous(), table, _int([n]), n)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(out[0, : hq // 2]).all()) and bool(torch.isnan(out[0, hq // 2:]).all()), (bad, sign)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_decode_scales_that_are_not_finite(gpu, which, bad, page, hq):
    """NaN for the rows whose length reaches the page, and for the key head that it belongs to; the others as if it were not there."""
    rng = np.random.default_rng(page + hq)
    dim, hk = 64, 2
    lengths = [3 * page, 3 * page + 1, 4 * page, 700, 1]
    slots = -(-700 // page)
    c = ao.Cache(5 * slots, hk, dim, page, rng)
    table = rng.permutation(c.pages).reshape(5, slots)
    clean = ao.Cache(1, 1, dim, page)
    clean.__dict__.update({k: (v.copy() if hasattr(v, "copy") else v) for k, v in c.__dict__.items()})
    if slots > 3:
        getattr(c, which)[table[:, 3], 1] = bad
    qd, q64 = _as(rng.standard_normal((5, hq, dim)), "float32")
    got = _decode(qd, c, table, lengths, "float32")
    want, tol = ab.decode(q64, clean, table, lengths, dim ** -0.5)
    nan = np.zeros(got.shape, bool)
    for b, n in enumerate(lengths):
        nan[b, hq // 2:] = n > 3 * page
    assert np.array_equal(np.isnan(got), nan)
    assert np.all(np.abs(got - want)[~nan] <= tol[~nan])


# ------------------------------------------------------------------ append: values that are not finite
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("dim,page,rot", [(64, 16, 64), (64, 64, 0), (128, 16, 64), (128, 128, 128)])
@pytest.mark.parametrize("bad", [np.nan, -np.nan, np.inf])
def test_append_of_values_that_are_not_finite_shows_in_the_scale(gpu, bad, dim, page, rot, dtype):
    """Scale of the value's page and head not finite, everything else bit for bit; it stays so while the page is appended to, and ends
    when the page begins anew."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(dim + page)
    hq, hk, n = 4, 2, 3 * page + 7
    rope = bn.bitnet_rope_table(5 * page, rot) if rot else None
    x = torch.from_numpy(rng.standard_normal((n + 1, hq + 2 * hk, dim)).astype(np.float32)).to(getattr(torch, dtype))
    clean = x.float().numpy()
    for where, head, part in ((0, 0, "k"), (page + 3, 1, "v"), (n - 1, 1, "k"), (n - 1, 0, "v")):
        for before in (0, 5):
            c = ao.Cache(6, hk, dim, page, np.random.default_rng(1))
            dev = _dev(c)
            table = np.array([[3, 0, 5, 1, 2]])
            y = x.clone()
            y[where, hq + head + (hk if part == "v" else 0), dim - 3] = bad

            def append(t, at):
                bn.bitnet_rope_append_kv(t.cuda().flatten(1), None if rope is None else torch.from_numpy(rope).cuda(), *dev,
                                         _int(table), _int([0, len(t)]), _int([at]), len(t), hq)
            append(y[:n], before)
            c.append(clean[:n], rope, rot, False, table, [0, n], [before], n, hq)
            slot = (before + where) // page
            pid = table[0, slot]
            scales = dev[2] if part == "k" else dev[3]
            not_finite = np.isnan if np.isnan(bad) else lambda f: not np.isfinite(f)  # (the turn can make a NaN of an infinity)
            assert not_finite(scales.cpu().numpy()[pid, head])
            for t, want, touched in zip(dev, (c.k, c.v, c.ks, c.vs), (part == "k", part == "v") * 2):
                t = t.cpu().numpy()
                if touched:
                    t[pid, head] = want[pid, head]
                assert np.array_equal(t, want)
            # a finite token behind it, in its page: still seen
            if before + n < (slot + 1) * page:
                append(x[n:], before + n)
                assert not_finite(scales.cpu().numpy()[pid, head])
            # the page of other tokens: forgotten
            append(x[:page], slot * page)
            torch.cuda.synchronize()
            assert np.isfinite(scales.cpu().numpy()[pid, head])


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("part", ["key", "value"])
def test_a_nan_that_was_appended_is_seen(gpu, part, group):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(34)
    hk, hq, dim, n = 2, 2 * group, 64, 200
    for dtype in (torch.float32, torch.bfloat16):
        c = bn.KVCache.empty(4, hk, dim, 64)
        x = torch.from_numpy(rng.standard_normal((n, hq + 2 * hk, dim)).astype(np.float32)).to(dtype).cuda()
        x[130, hq + 1 + (hk if part == "value" else 0), 7] = float("nan")  # of key head 1
        table = _int([[0, 1, 2, 3]])
        q, _ = c.append(x.flatten(1), None, table, _int([0, n]), _int([0]), n, hq)
        for length in (n, 129):  # beyond its page's first token, and to it
            out = c.attend(q[:1], table, _int([length]), length)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(out[0, :group]).all()) and bool(torch.isnan(out[0, group:]).all())
        out = c.attend(q[:1], table, _int([128]), 128)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(out).all())


# ------------------------------------------------------------------ prompt: values and scores that are not finite
@pytest.mark.parametrize("hq,hk", [(2, 1), (40, 40)])  # keys shared between halves of the waves, and not
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_values_that_are_not_finite_change_nothing_else(gpu, hq, hk, dim, causal):
    """Infinities and NaN in some channels of some keys: every other channel, and (causal) every row in front of them, to the last bit as
    without them, whether their key is among the last that a row's wave looks at or not."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(40)
    lens = [300, 70, 1030 if hq == 40 else 97, 33]
    starts = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_as(rng.standard_normal((int(starts[-1]), h, dim)), "bfloat16")[0] for h in (hq, hk, hk))
    places = [(0, 0, 1, np.inf), (0, 170, 3, np.inf), (0, 299, 9, -np.inf), (0, 288, dim - 1, np.nan), (1, 69, 5, np.nan), (1, 40, 60, -np.inf),
              (1, 64, 17, np.inf), (2, 95, 0, np.inf), (2, 96, 33, -np.inf), (3, 32, 62, np.inf)]
    want = bn.bitnet_attn_prompt(q, k, v, _int(starts), max(lens), causal=causal).clone()
    odd = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    group = hq // hk
    for b, u, ch, x in places:
        v[starts[b] + u, hk - 1, ch] = x
        rows = slice(int(starts[b] + u if causal else starts[b]), int(starts[b + 1]))
        odd[rows, hq - group:, ch] = True
        want[rows, hq - group:, ch] = x  # one such value a channel and sequence, and weights above 0
    got = bn.bitnet_attn_prompt(q, k, v, _int(starts), max(lens), causal=causal)
    torch.cuda.synchronize()
    assert torch.equal(got[~odd], want[~odd])
    assert torch.equal(got[odd].isnan(), want[odd].isnan())
    assert torch.equal(got[odd].nan_to_num(0.5), want[odd].nan_to_num(0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_of_nan_throughout(gpu, dim, causal):
    import torch

    import bit_gemv_i2_amd as bn
    lens = [65, 700, 1]
    q = torch.ones((sum(lens), 4, dim), dtype=torch.bfloat16, device="cuda")
    k, nan = q[:, :2].contiguous(), torch.full_like(q[:, :2], float("nan"))
    starts = _int(np.concatenate([[0], np.cumsum(lens)]))
    for a in ((q, k, nan), (q, nan, k), (q * float("nan"), k, k)):
        out = bn.bitnet_attn_prompt(*a, starts, 700, causal=causal)
        torch.cuda.synchronize()
        assert bool(out.isnan().all())


@pytest.mark.parametrize("hq,hk", [(2, 1), (40, 40)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("masked", [1, 31, 32, 33, 64, 96, 200])
def test_prompt_keys_whose_scores_are_minus_infinity(gpu, hq, hk, dim, causal, masked):
    """The first keys of a prompt masked by an infinity in a channel that all queries have above 0: they weigh nothing, and rows that see no
    others are NaN, as 0 / 0 is."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(masked + dim)
    lens = [300, 70, 1030 if hq == 40 else 230]
    starts = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (rng.standard_normal((int(starts[-1]), h, dim)) for h in (hq, hk, hk))
    q[..., 5] = np.abs(q[..., 5]) + 0.1
    (qd, q), (kd, k), (vd, v) = (_as(a, "bfloat16") for a in (q, k, v))
    for b in range(3):
        kd[starts[b]: min(starts[b] + masked, starts[b + 1]), :, 5] = -np.inf
    got = bn.bitnet_attn_prompt(qd, kd, vd, _int(starts), max(lens), causal=causal)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    for b, n in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        hidden = min(masked, n)
        see = (np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)) & (np.arange(n) >= hidden)
        none = ~see.any(1)
        assert np.isnan(got[rows][none]).all()
        for h in range(hq):
            kk, vv = k[rows, h * hk // hq], v[rows, h * hk // hq]
            want, a, _ = ao.softmax_rows(q[rows, h], kk, vv, dim ** -0.5, see)
            tol = 2.0 ** -8 * a + 2.0 ** -15 * np.abs(vv).max()  # as attn_oracle.prompt derives it
            fine, worst = ao.within(got[rows, h][~none], want[~none], tol[~none], True)
            assert fine, (b, h, worst)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[100], [100] * 40])
def test_prompt_scores_that_rise_far(gpu, dim, lens):
    """Scores of about -2e38 in the first 64 keys, 0 in the next, 2^20 in the last: each outweighs all before it."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(dim)
    starts = np.concatenate([[0], np.cumsum(lens)])
    T, n = int(starts[-1]), lens[0]
    q, k = np.zeros((T, 8, dim)), np.zeros((T, 8, dim))
    q[..., 0] = 2.0 ** 63
    at = np.arange(T) % n
    k[at < 64, :, 0] = -(2.0 ** 64)
    k[at == n - 1, :, 0] = 2.0 ** -43
    (qd, _), (kd, _), (vd, v) = (_as(a, "bfloat16") for a in (q, k, rng.standard_normal((T, 8, dim))))
    got = bn.bitnet_attn_prompt(qd, kd, vd, _int(starts), n, scale=1.0)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    for s in starts[:-1]:
        for row, first in ((64, 64), (90, 64), (n - 1, n - 1)):
            x = v[s + first: s + row + 1]
            want, a = x.mean(0), np.abs(x).mean(0)
            fine, worst = ao.within(got[s + row], want, 2.0 ** -8 * a + 2.0 ** -15 * np.abs(v).max(), True)
            assert fine, (row, worst)
