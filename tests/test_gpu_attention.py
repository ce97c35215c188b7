"""The attention side of a decoder layer on the GPU: the append bit for bit, decode and prompt attention
within the tolerances derived in attn_oracle, at the sizes, masks and addresses where they can go wrong."""
import numpy as np
import pytest

import attn_oracle as ao

pytestmark = pytest.mark.gpu

GUARD = 64  # elements of a fixed pattern before and behind an output


def _bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def _as(x, dtype):
    """Host fp32 array -> (device tensor of dtype, the fp64 values that it holds)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _guarded(shape, dtype):
    """A device tensor inside a buffer of a fixed pattern, and a check that the pattern stands."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), -77.0, dtype=dtype, device="cuda")

    def intact():
        return bool((buf[:GUARD] == -77).all() and (buf[GUARD + n:] == -77).all())
    return buf[GUARD: GUARD + n].view(shape), intact


def _to_dev(c):
    import torch
    return [torch.from_numpy(a.copy()).cuda() for a in (c.k, c.v, c.ks, c.vs)]


def _int(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def _table(rng, pages, need, slots, page):
    """Distinct pages for every position of every sequence; the entries past a sequence's end are nonsense."""
    order = rng.permutation(pages)
    t = np.full((len(need), slots), -123456, np.int64)
    at = 0
    for b, n in enumerate(need):
        c = -(-n // page)
        t[b, :c] = order[at: at + c]
        at += c
    assert at <= pages
    t[t == -123456] = 2 ** 31 - 1
    return t.astype(np.int64)


# ------------------------------------------------------------------ append
def _append_case(rng, dtype, hq, hk, dim, page, rot, interleaved, news, before, with_k=True, max_new=None, wide=0,
                 slots=None, break_page=False):
    import torch

    import bit_gemv_i2_amd as bn
    starts = np.concatenate([[0], np.cumsum(news)])
    T = int(starts[-1])
    need = [a + b for a, b in zip(news, before)]
    slots = slots or max(1, max(-(-n // page) for n in need)) + 1
    pages = sum(-(-n // page) for n in need) + 2
    c = ao.Cache(pages, hk, dim, page, rng)
    table = _table(rng, pages, [min(n, slots * page) for n in need], slots, page)
    if break_page:
        table[0, 0] = pages
    rope = bn.bitnet_rope_table(slots * page, rot) if rot else np.zeros((slots * page, 16), np.float32)
    x = rng.standard_normal((T, hq + 2 * hk, dim)).astype(np.float32) * np.exp(rng.standard_normal((T, 1, 1)))
    width = (hq + 2 * hk) * dim
    xt = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))
    wide_buf = torch.full((T, width + wide), 3.0, dtype=xt.dtype, device="cuda")
    wide_buf[:, :width] = xt.reshape(T, width).cuda()
    dev = _to_dev(c)
    q, q_ok = _guarded((T, hq, dim), xt.dtype)
    k, k_ok = _guarded((T, hk, dim), xt.dtype)
    q.fill_(5.0), k.fill_(5.0)
    bn.bitnet_rope_append_kv(wide_buf[:, :width], torch.from_numpy(rope).cuda() if rot else None, *dev, _int(table),
                             _int(starts), _int(before), max_new or max(news), hq, interleaved=interleaved, q_out=q,
                             k_out=k if with_k else None)
    torch.cuda.synchronize()
    ref = ao.Cache(pages, hk, dim, page, rng)
    ref.k, ref.v, ref.ks, ref.vs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
    qr, kr = ref.append(xt.float().numpy(), rope, rot, interleaved, table, starts, before, max_new or max(news), hq)
    for name, got, want in zip(("k", "v", "k_scale", "v_scale"), dev, (ref.k, ref.v, ref.ks, ref.vs)):
        assert np.array_equal(got.cpu().numpy(), want), name
    for got, want, ok, made in ((q, qr, q_ok, True), (k, kr, k_ok, with_k)):
        assert ok()
        w = torch.from_numpy(np.where(np.isnan(want), np.float32(5.0), want)).to(xt.dtype)
        assert torch.equal(got.cpu(), w if made else torch.full_like(w, 5.0))
    return c, ref


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_bit_for_bit(gpu, dtype, dim, page, interleaved):
    rng = np.random.default_rng(page + dim)
    _append_case(rng, dtype, 6, 3, dim, page, dim, interleaved, [1, 0, page, 2 * page + 5, 1, 150], [0, 7, 0, page - 1, page + 3, 40])


@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (20, 20), (20, 5)])
def test_append_partial_turns_and_heads(gpu, rot, hq, hk):
    rng = np.random.default_rng(rot + hq)
    _append_case(rng, "float32", hq, hk, 128, 32, rot, rot == 48, [3, 33], [30, 0], with_k=rot != 16, wide=24)


def test_append_one_token_each(gpu):
    rng = np.random.default_rng(3)
    _append_case(rng, "bfloat16", 20, 5, 128, 64, 128, False, [1] * 33, [int(x) for x in rng.integers(0, 200, 33)])


def test_append_refuses_to_follow_a_bad_page(gpu):
    rng = np.random.default_rng(4)
    _append_case(rng, "float32", 4, 2, 64, 16, 64, False, [20, 9], [0, 3], break_page=True)


def test_append_past_the_table_stores_nothing_and_gives_zeros(gpu):
    rng = np.random.default_rng(5)
    _append_case(rng, "float32", 4, 2, 64, 16, 64, False, [40, 9], [0, 3], slots=2)


def test_append_handles_at_most_max_new(gpu):
    rng = np.random.default_rng(6)
    _append_case(rng, "bfloat16", 4, 2, 128, 16, 128, False, [40, 9], [5, 3], max_new=20)


def test_append_token_by_token_follows_a_growing_scale(gpu):
    """40 single tokens, growing on the whole: every one may raise its page's scale and move the older codes; the values
    that the cache stands for stay within the rounding that each such move adds."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(7)
    hk, dim, page, n = 2, 64, 32, 40
    ref = ao.Cache(3, hk, dim, page, rng)
    dev = _to_dev(ref)
    table = np.array([[2, 0]])
    rope = bn.bitnet_rope_table(2 * page, dim)
    xs = (rng.standard_normal((n, 2 + 2 * hk, dim)) * (1.0 + 0.3 * np.arange(n))[:, None, None]).astype(np.float32)
    for i in range(n):
        x = xs[i: i + 1]
        q, _ = bn.bitnet_rope_append_kv(torch.from_numpy(x).cuda().view(1, -1), torch.from_numpy(rope).cuda(), *dev,
                                        _int(table), _int([0, 1]), _int([i]), 1, 2)
        ref.append(x, rope, dim, False, table, [0, 1], [i], 1, 2)
        for got, want in zip(dev, (ref.k, ref.v, ref.ks, ref.vs)):
            assert np.array_equal(got.cpu().numpy(), want), i
    _, v = ref.values(table[0], n)
    err = np.abs(v.transpose(1, 0, 2) - xs[:, 2 + hk:])
    # a code's own rounding and one more for each growth, half a unit each, a unit never above the last scale
    grows = np.array([[len(set(np.maximum.accumulate(np.abs(xs[p: min(p + page, n), 2 + hk + h]).max(1)))) for h in range(hk)]
                      for p in (0, page)])
    last = ref.vs[table[0]]
    for i in range(n):
        for h in range(hk):
            assert err[i, h].max() <= 0.5 * last[i // page, h] * (grows[i // page, h] + 1) * 1.001


def test_append_again_changes_nothing(gpu):
    """The same tokens at the same positions once more: scales that grew stay, codes stay."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(8)
    c = ao.Cache(4, 3, 64, 16, rng)
    dev = _to_dev(c)
    x = torch.from_numpy(rng.standard_normal((5, 9 * 64)).astype(np.float32)).cuda()
    args = (x, None, *dev, _int([[1, 3]]), _int([0, 5]), _int([14]), 5, 3)
    bn.bitnet_rope_append_kv(*args)
    first = [t.clone() for t in dev]
    bn.bitnet_rope_append_kv(*args)
    assert all(torch.equal(a, b) for a, b in zip(first, dev))


# ------------------------------------------------------------------ decode
def _decode_case(rng, hq, hk, dim, page, qdt, odt, lengths, max_len=None, slots_extra=1, cache=None, table=None,
                 q=None, wide=0):
    import torch

    import bit_gemv_i2_amd as bn
    B = len(lengths)
    clipped = [min(n, max_len) if max_len else n for n in lengths]
    pages = sum(-(-max(n, 0) // page) for n in lengths) + 2
    slots = max(1, max(-(-n // page) for n in lengths)) + slots_extra
    c = cache or ao.Cache(pages, hk, dim, page, rng)
    if table is None:
        table = _table(rng, pages, [max(n, 0) for n in lengths], slots, page)
    q = rng.standard_normal((B, hq, dim)) * 1.5 if q is None else q
    qd, q64 = _as(q, qdt)
    if wide:
        buf = torch.full((B, hq * dim + wide), float("nan"), dtype=qd.dtype, device="cuda")
        buf[:, : hq * dim] = qd.view(B, -1)
        qd = buf[:, : hq * dim].unflatten(1, (hq, dim))
    out, ok = _guarded((B, hq, dim), getattr(torch, odt))
    got = bn.bitnet_attn_decode(qd, *_to_dev(c), _int(table), _int(lengths), max_len or max(max(lengths), 1), out=out)
    torch.cuda.synchronize()
    assert ok() and got is out
    want, tol = ao.decode(q64, c, table, clipped, dim ** -0.5, odt == "float32", 22 if qdt == "bfloat16" else 30)
    fine, worst = ao.within(out.double().cpu().numpy(), want, tol, odt == "bfloat16")
    assert fine, worst


EDGES = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700]


@pytest.mark.parametrize("qdt,odt", [("bfloat16", "bfloat16"), ("float32", "float32"), ("bfloat16", "float32"),
                                     ("float32", "bfloat16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths_pages_types(gpu, qdt, odt, dim, page):
    _decode_case(np.random.default_rng(page + dim), 4, 2, dim, page, qdt, odt, EDGES)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (20, 5), (20, 20), (15, 1), (16, 1), (17, 1), (40, 2), (33, 1)])
def test_decode_head_groups(gpu, hq, hk):
    _decode_case(np.random.default_rng(hq), hq, hk, 128, 16, "float32", "float32", [100, 33], wide=40)


@pytest.mark.parametrize("hq,hk", [(5, 1), (16, 2), (12, 1), (36, 2)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode_groups_of_more_than_four(gpu, hq, hk, dim, page):
    rng = np.random.default_rng(hq + page)
    _decode_case(rng, hq, hk, dim, page, "float32", "float32", [1, 0, 17, 64, 300])
    _decode_case(rng, hq, hk, dim, page, "bfloat16", "bfloat16", [2500, 63])


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("odt", ["bfloat16", "float32"])
def test_decode_long_contexts_are_split_and_joined(gpu, page, odt):
    _decode_case(np.random.default_rng(9), 3, 1, 64, page, "float32", odt, [9000, 1, 0, 257, 4096])


@pytest.mark.parametrize("hq,dim,page", [(4, 64, 16), (12, 64, 64), (4, 128, 32), (12, 128, 16)])
def test_decode_of_large_caches_reads_past_the_memory_side_cache(gpu, hq, dim, page):
    """The bound on the lengths says more than 256 MB, which takes the streaming loads, whatever the lengths are."""
    rng = np.random.default_rng(hq + dim)
    _decode_case(rng, hq, 2, dim, page, "float32", "float32", [9000, 700, 0, 15], max_len=600_000)


def test_decode_single_long_row(gpu):
    _decode_case(np.random.default_rng(10), 4, 1, 128, 64, "bfloat16", "bfloat16", [20001])


def test_decode_lengths_above_the_bounds(gpu):
    import bit_gemv_i2_amd as bn  # noqa: F401
    rng = np.random.default_rng(11)
    _decode_case(rng, 2, 1, 64, 16, "float32", "float32", [300, 90, 64], max_len=90)
    # a length that the table cannot hold is read as what it holds
    import torch
    c = ao.Cache(3, 1, 64, 16, rng)
    table = np.array([[2, 0]])
    qd, q64 = _as(rng.standard_normal((1, 2, 64)), "float32")
    out = bn.bitnet_attn_decode(qd, *_to_dev(c), _int(table), _int([1000]), 1000)
    torch.cuda.synchronize()
    want, tol = ao.decode(q64, c, table, [32], 0.125, True, 30)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


def test_decode_negative_lengths_give_zeros(gpu):
    _decode_case(np.random.default_rng(12), 2, 1, 64, 16, "float32", "bfloat16", [40, -5, -2147483648])


def test_decode_pages_that_do_not_exist_are_not_seen(gpu):
    rng = np.random.default_rng(13)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        c = ao.Cache(12, 2, 64, 16, rng)
        table = np.stack([rng.permutation(12)[:6], np.full(6, bad)])  # the second sequence has no page at all
        table[0, 1] = table[0, 4] = bad
        _decode_case(rng, 4, 2, 64, 16, "float32", "float32", [90, 96], cache=c, table=table)


@pytest.mark.parametrize("hq", [4, 12])
def test_decode_non_finite_scales_and_stale_codes_behind_the_end(gpu, hq):
    """Only what a sequence's length covers counts: pages of nobody have NaN and infinite scales, and the codes behind the
    last token of a page are those of an earlier owner."""
    rng = np.random.default_rng(14)
    c = ao.Cache(9, 2, 128, 32, rng)
    c.ks[[0, 8]], c.vs[[0, 8]] = np.nan, np.inf
    table = np.array([[3, 5, 8, 0], [1, 2, 0, 8]])
    _decode_case(rng, hq, 2, 128, 32, "float32", "float32", [33, 64], cache=c, table=table)
    _decode_case(rng, hq, 2, 128, 32, "bfloat16", "bfloat16", [64, 1], cache=c, table=table)


def test_decode_pages_of_zeros(gpu):
    """Scales of 0 and rows of 0: every weight counts, though a page's values are 0."""
    rng = np.random.default_rng(15)
    c = ao.Cache(8, 1, 64, 16, rng)
    c.vs[[1, 2]] = 0
    c.ks[3] = 0
    table = rng.permutation(8)[None, :]
    _decode_case(rng, 2, 1, 64, 16, "float32", "float32", [128], cache=c, table=table)
    c.vs[:] = 0
    _decode_case(rng, 2, 1, 64, 16, "float32", "float32", [128], cache=c, table=table)
    c = ao.Cache(8, 1, 64, 16, rng)
    _decode_case(rng, 2, 1, 64, 16, "bfloat16", "float32", [100], cache=c, table=table, q=np.zeros((1, 2, 64)))


@pytest.mark.parametrize("hq", [1, 6])
def test_decode_one_large_weight_beside_a_long_flat_tail(gpu, hq):
    """A first token whose weight is thousands of times any other's, which together weigh as much: the tail must not be
    rounded away."""
    rng = np.random.default_rng(16)
    n, dim, page = 6000, 64, 64
    c = ao.Cache(-(-n // page), 1, dim, page, rng)
    table = np.arange(c.pages)[None, :]
    c.ks[:], c.vs[:] = 0.02, 0.03
    c.k[..., 0] = 0
    c.k[0, 0, 0] = 0
    c.k[0, 0, 0, 0] = 127
    c.k[:, :, :, 1:] = c.k[:, :, :, 1:] // 16
    c.k[0, 0, 0, 1:] = 0
    c.v = np.abs(c.v)  # so that a lost tail shows
    q = np.zeros((1, hq, dim))
    q[0, :, 0] = 8.7 / (127 * 0.02 * dim ** -0.5)
    q[0, :, 1:] = rng.standard_normal((hq, dim - 1)) * 0.2
    for odt in ("bfloat16", "float32"):
        _decode_case(rng, hq, 1, dim, page, "float32", odt, [n], cache=c, table=table, q=q)


def test_decode_scores_far_apart(gpu):
    rng = np.random.default_rng(17)
    _decode_case(rng, 4, 2, 128, 64, "float32", "float32", [500], q=rng.standard_normal((1, 4, 128)) * 40)


def test_decode_cache_past_32_bit_offsets(gpu):
    """Pages of a cache of more than 4 GiB, at both ends of it."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(18)
    pages, page, dim = 300_000, 128, 128
    k = torch.zeros((pages, 1, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros((pages, 1, dim, page), dtype=torch.int8, device="cuda")
    ks = torch.zeros((pages, 1), device="cuda")
    vs = torch.zeros((pages, 1), device="cuda")
    small = ao.Cache(3, 1, dim, page, rng)
    where = [pages - 1, 5, 150_000]
    for i, pid in enumerate(where):
        k[pid], v[pid] = torch.from_numpy(small.k[i]).cuda(), torch.from_numpy(small.v[i]).cuda()
        ks[pid], vs[pid] = float(small.ks[i, 0]), float(small.vs[i, 0])
    qd, q64 = _as(rng.standard_normal((1, 2, dim)), "float32")
    out = bn.bitnet_attn_decode(qd, k, v, ks, vs, _int([where]), _int([300]), 300)
    torch.cuda.synchronize()
    want, tol = ao.decode(q64, small, np.array([[0, 1, 2]]), [300], dim ** -0.5, True, 30)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    # and an append there
    x = rng.standard_normal((84 + 128, 4, dim)).astype(np.float32)
    bn.bitnet_rope_append_kv(torch.from_numpy(x).cuda().flatten(1), None, k, v, ks, vs, _int([[5, 150_000, pages - 1, 299_998]]),
                             _int([0, 212]), _int([300]), 212, 2)
    torch.cuda.synchronize()
    ref = ao.Cache(4, 1, dim, page, rng)
    for i, pid in enumerate((0, 0, 0, 0)):
        ref.k[i], ref.v[i] = 0, 0
    ref.k[2], ref.v[2], ref.ks[2], ref.vs[2] = small.k[0], small.v[0], small.ks[0], small.vs[0]
    ref.append(x, None, 0, False, np.array([[0, 1, 2, 3]]), [0, 212], [300], 212, 2)
    for i, pid in ((2, pages - 1), (3, 299_998)):
        assert np.array_equal(k[pid].cpu().numpy(), ref.k[i]) and np.array_equal(v[pid].cpu().numpy(), ref.v[i])
        assert float(ks[pid, 0]) == float(ref.ks[i, 0]) and float(vs[pid, 0]) == float(ref.vs[i, 0])


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("part", ["key", "value"])
def test_an_infinity_that_was_appended_is_seen(gpu, part, group):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(33)
    hk, hq, dim, n = 2, 2 * group, 64, 200
    c = bn.KVCache.empty(4, hk, dim, 64)
    x = torch.from_numpy(rng.standard_normal((n, hq + 2 * hk, dim)).astype(np.float32)).cuda()
    x[130, hq + 1 + (hk if part == "value" else 0), 7] = np.inf  # of key head 1
    q, _ = c.append(x.flatten(1), None, _int([[0, 1, 2, 3]]), _int([0, n]), _int([0]), n, hq)
    out = c.attend(q[:1], _int([[0, 1, 2, 3]]), _int([n]), n)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[0, :group]).all()) and not bool(torch.isfinite(out[0, group:]).any())


@pytest.mark.parametrize("hq,n,where", [(4, 100, 1), (4, 5000, 2), (16, 300, 5), (16, 5000, 0)])
def test_decode_query_rows_that_are_not_finite_give_nan_and_only_they(gpu, hq, n, where):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(31)
    cache = ao.Cache((n + 63) // 64, 1, 128, 64, rng)
    table = np.arange((n + 63) // 64)[None]
    for bad in (np.nan, np.inf, -np.inf):
        qd, q64 = _as(rng.standard_normal((1, hq, 128)), "float32")
        qd[0, where, 77] = bad
        out = bn.bitnet_attn_decode(qd, *(torch.from_numpy(a).cuda() for a in (cache.k, cache.v, cache.ks, cache.vs)), _int(table), _int([n]), n)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        want, tol = ao.decode(q64, cache, table, [n], 128 ** -0.5, True, 30)
        assert np.isnan(got[0, where]).all()
        keep = np.arange(hq) != where
        assert np.all(np.abs(got - want)[:, keep] <= tol[:, keep])


# ------------------------------------------------------------------ prompt
@pytest.mark.parametrize("hq,hk", [(2, 1), (40, 40)])  # keys shared between halves of the waves, and not
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_values_that_are_not_finite_behind_a_row(gpu, hq, hk, dim, causal):
    """A weight of 0 must not meet an infinity: rows in front of it, also those of its own 32 keys, are as if it were not there."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(32)
    lens = [300, 70, 1030 if hq == 40 else 97]
    starts = np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1])
    (qd, q), (kd, k), (vd, v) = (_as(rng.standard_normal((T, h, dim)), "bfloat16") for h in (hq, hk, hk))
    places = [(0, 170, 3, np.inf), (0, 187, 9, -np.inf), (0, 188, 9, np.inf), (1, 69, 5, np.nan), (1, 40, 60, -np.inf), (2, 95, 0, np.inf)]
    want, tol, _ = ao.prompt(q, k, v, starts.tolist(), causal, dim ** -0.5, max(lens))
    group = hq // hk
    for b, u, ch, x in places:
        vd[starts[b] + u, hk - 1, ch] = x
        rows = slice(starts[b] + u if causal else starts[b], starts[b + 1])
        with np.errstate(invalid="ignore"):
            want[rows, hq - group:, ch] += x
    out = bn.bitnet_attn_prompt(qd, kd, vd, _int(starts), max(lens), causal=causal)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)])
    fine, worst = ao.within(got[~odd], want[~odd], tol[~odd], True)
    assert fine, worst


def _prompt_case(rng, hq, hk, dim, lens, causal, wide=0, max_len=None, gain=1.0, poison=(), scale=None, starts=None):
    import torch

    import bit_gemv_i2_amd as bn
    starts = np.concatenate([[0], np.cumsum(lens)]) if starts is None else np.asarray(starts)
    T = int(starts.max())
    q, k, v = (rng.standard_normal((T, h, dim)) for h in (hq, hk, hk))
    q *= gain
    for b in poison:
        k[starts[b]: starts[b + 1]] = np.nan
        v[starts[b]: starts[b + 1]] = np.inf
    dev, host = [], []
    for a in (q, k, v):
        t, a64 = _as(a, "bfloat16")
        if wide:
            buf = torch.full((T, t.shape[1] * dim + wide), float("nan"), dtype=t.dtype, device="cuda")
            buf[:, : t.shape[1] * dim] = t.flatten(1)
            t = buf[:, : t.shape[1] * dim].unflatten(1, (t.shape[1], dim))
        dev.append(t)
        host.append(a64)
    out, ok = _guarded((T, hq, dim), torch.bfloat16)
    out.fill_(9.0)
    bn.bitnet_attn_prompt(*dev, _int(starts), max_len or max(lens), causal=causal, scale=scale, out=out)
    torch.cuda.synchronize()
    assert ok()
    for b in poison:
        for a in host:
            a[starts[b]: starts[b + 1]] = 0
    want, tol, wrote = ao.prompt(*host, starts.tolist(), causal, scale or dim ** -0.5, max_len or max(lens))
    got = out.double().cpu().numpy()
    for b in poison:
        wrote[starts[b]: starts[b + 1]] = False
        got[starts[b]: starts[b + 1]] = 9.0
    fine, worst = ao.within(got[wrote], want[wrote], tol[wrote], True)
    assert fine, worst
    assert np.all(got[~wrote] == 9.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 400])
def test_prompt_lengths(gpu, dim, causal, n):
    _prompt_case(np.random.default_rng(n + dim), 2, 1, dim, [n], causal)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (20, 5), (7, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_packed_with_strides(gpu, hq, hk, causal, dim):
    _prompt_case(np.random.default_rng(hq), hq, hk, dim, [130, 1, 0, 64, 300, 17], causal, wide=24)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_many_workgroups(gpu, dim, causal):
    """Enough workgroups that none shares its keys between its waves."""
    rng = np.random.default_rng(20 + dim)
    lens = [500, 1, 31, 32, 33, 64, 65, 127, 128, 129, 160, 255, 256, 257, 400, 0] + [int(x) for x in rng.integers(1, 500, 24)]
    _prompt_case(rng, 4, 2, dim, lens, causal, wide=8)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_long_with_many_heads(gpu, dim):
    _prompt_case(np.random.default_rng(30 + dim), 40, 8, dim, [1700], True)


def test_prompt_many_short_sequences(gpu):
    rng = np.random.default_rng(21)
    _prompt_case(rng, 4, 2, 64, [int(x) for x in rng.integers(0, 9, 70)], True)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_neighbours_that_are_not_finite(gpu, causal):
    _prompt_case(np.random.default_rng(22), 2, 1, 128, [70, 90, 61, 40, 130], causal, poison=(1, 3))


def test_prompt_takes_at_most_max_len_rows(gpu):
    _prompt_case(np.random.default_rng(23), 2, 1, 64, [200, 50, 90], True, max_len=90)
    _prompt_case(np.random.default_rng(23), 2, 1, 128, [200, 50, 90], False, max_len=90)


@pytest.mark.parametrize("gain", [0.0, 1e-3, 30.0])
def test_prompt_score_ranges(gpu, gain):
    _prompt_case(np.random.default_rng(24), 2, 2, 128, [300], True, gain=gain)


def test_prompt_longer_than_the_grid_of_one_pass(gpu):
    _prompt_case(np.random.default_rng(25), 1, 1, 128, [1500], True, scale=0.2)
    _prompt_case(np.random.default_rng(26), 1, 1, 64, [1100, 3, 900], False, scale=0.05)


@pytest.mark.parametrize("hq,hk,dim", [(20, 5, 128), (6, 3, 64), (8, 8, 64)])
def test_prompt_tiles_over_the_dies(gpu, hq, hk, dim):
    _prompt_case(np.random.default_rng(29), hq, hk, dim, [300, 7, 0, 150, 129], True)


def test_prompt_more_tiles_than_one_dimension_of_a_launch_holds(gpu):
    lens = [0] * 65535
    lens[0], lens[40000], lens[65534] = 5, 70, 1100
    _prompt_case(np.random.default_rng(30), 1, 1, 64, lens, True)


def test_prompt_starts_that_make_no_sense_touch_nothing(gpu):
    """Ends before beginnings, past the tokens or below 0: such a sequence is left out."""
    rng = np.random.default_rng(27)
    _prompt_case(rng, 2, 1, 64, [40, 30], True, starts=[0, 40, 40, 70])
    import torch

    import bit_gemv_i2_amd as bn
    q, _ = _as(rng.standard_normal((70, 2, 64)), "bfloat16")
    out, ok = _guarded((70, 2, 64), torch.bfloat16)
    out.fill_(9.0)
    bn.bitnet_attn_prompt(q, q, q, _int([-3, 40, 20, 71]), 70, out=out)
    torch.cuda.synchronize()
    assert ok() and bool((out == 9.0).all())


# ------------------------------------------------------------------ together
def test_prompt_and_decode_agree_through_the_cache(gpu):
    """A prompt's last token by prompt attention and, appended token by token, by decode attention: the same up to the
    cache's rounding of keys and values."""
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(31)
    hq, hk, dim, page, n = 8, 2, 128, 32, 100
    x = torch.from_numpy(rng.standard_normal((n, (hq + 2 * hk) * dim)).astype(np.float32)).to(torch.bfloat16).cuda()
    rope = torch.from_numpy(bn.bitnet_rope_table(4 * page, dim)).cuda()
    cache = bn.KVCache.empty(5, hk, dim, page)
    table, starts = _int([[4, 0, 2, 1]]), _int([0, n - 1])
    cache.append(x[: n - 1], rope, table, starts, _int([0]), n - 1, hq)
    q, k = cache.append(x[n - 1:], rope, table, _int([0, 1]), _int([n - 1]), 1, hq, with_k=True)
    one = cache.attend(q, table, _int([n]), n)
    other = bn.KVCache.empty(5, hk, dim, page)
    qa, ka = other.append(x, rope, table, _int([0, n]), _int([0]), n, hq, with_k=True)
    v = x.view(n, -1, dim)[:, hq + hk:]
    whole = bn.bitnet_attn_prompt(qa, ka, v, _int([0, n]), n)
    torch.cuda.synchronize()
    assert torch.equal(qa[-1:], q) and torch.equal(ka[-1:], k)
    # keys and values off by at most half a unit of their page's scale, that is max|x| / 254: scores off by at most
    # sum|q| * max|k| / 254 / sqrt(dim), weights and so outputs by twice that of max|v|, plus half a unit of v and roundings
    kmax, vmax = float(ka.float().abs().max()), float(v.float().abs().max())
    ds = float(q.float().abs().sum(-1).max()) * kmax / 254 * dim ** -0.5
    assert float((whole[-1].float() - one[0].float()).abs().max()) <= 2 * ds * vmax + vmax / 254 + 2.0 ** -7 * vmax
    # the typical difference is that bound's square-root-of-many share; a wrong head or position is of the order of out itself
    assert float((whole[-1].float() - one[0].float()).norm() / whole[-1].float().norm()) < 0.05


def test_step_on_another_stream_and_in_a_graph(gpu):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(32)
    hq, hk, dim, page, B, n = 4, 2, 64, 16, 3, 2000
    c = ao.Cache(B * (n // page + 1), hk, dim, page, rng)
    table = np.arange(c.pages).reshape(B, -1)
    dev = _to_dev(c)
    x = torch.from_numpy(rng.standard_normal((B, (hq + 2 * hk) * dim)).astype(np.float32)).cuda()
    rope = torch.from_numpy(bn.bitnet_rope_table(table.shape[1] * page, dim)).cuda()
    tb, starts, before, after = _int(table), _int(range(B + 1)), _int([n - 1, 5, 700]), _int([n, 6, 701])

    def step(stream=None):
        q, _ = bn.bitnet_rope_append_kv(x, rope, *dev, tb, starts, before, 1, hq, stream=stream)
        return bn.bitnet_attn_decode(q, *dev, tb, after, n, stream=stream)
    want = step().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        for t, a in zip(dev, (c.k, c.v, c.ks, c.vs)):
            t.copy_(torch.from_numpy(a))
        g.replay()
        torch.cuda.synchronize()
        again = out.clone()
        for t, a in zip(dev, (c.k, c.v, c.ks, c.vs)):
            t.copy_(torch.from_numpy(a))
        assert torch.equal(step(), again), i


def test_results_do_not_change_from_run_to_run(gpu):
    import torch

    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(33)
    c = ao.Cache(200, 1, 128, 64, rng)
    dev = _to_dev(c)
    q, _ = _as(rng.standard_normal((1, 4, 128)), "float32")
    args = (q, *dev, _int(rng.permutation(200)[None]), _int([12000]), 12800)
    first = bn.bitnet_attn_decode(*args).clone()
    p, _ = _as(rng.standard_normal((700, 2, 128)), "bfloat16")
    pf = bn.bitnet_attn_prompt(p, p, p, _int([0, 700]), 700).clone()
    for _ in range(5):
        assert torch.equal(bn.bitnet_attn_decode(*args), first)
        assert torch.equal(bn.bitnet_attn_prompt(p, p, p, _int([0, 700]), 700), pf)
