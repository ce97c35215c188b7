"""What stands between the products of a decoder layer, and a layer of experts, on the GPU: norm and codes bit for bit, products
and gates within the tolerances derived in layer_oracle, plans exactly."""
import itertools

import numpy as np
import pytest

import layer_oracle as lo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
GUARD = 64
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _guarded(shape, dtype, fill=-77):
    """A device tensor inside a buffer of a fixed pattern, and a check that the pattern stands."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")

    def intact():
        return bool((buf[:GUARD] == fill).all() and (buf[GUARD + n:] == fill).all())
    return buf[GUARD: GUARD + n].view(shape), intact


def _values(rng, shape, dtype, spread=1.0):
    """(device tensor of dtype, its values in fp32 on the host)."""
    t = torch.from_numpy((rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:1] + (1,) * (len(shape) - 1)))).astype(np.float32)).to(dtype)
    return t.cuda(), t.float().numpy()


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ------------------------------------------------------------------ norm
def _norm_case(rng, M, K, xt, at, parts, weight=True, eps=1e-5, inplace=False):
    import bit_gemv_i2_amd as bn
    x, xv = _values(rng, (M, K), TYPES[xt])
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32) if weight else None
    add = av = slots = gates = None
    if at:
        R = M if not parts else max(1, M * parts - 2)
        add, av = _values(rng, (R, K), TYPES[at])
        if parts:
            slots = rng.integers(-1, R + 1, (M, parts)).astype(np.int32)
            slots[0, 0] = 2 ** 31 - 1
            gates = rng.random((M, parts)).astype(np.float32)
    stream, h, codes, s_a = lo.add_norm(xv, w, eps, TYPES[xt], av, slots, gates)
    q, q_ok = _guarded((M, K), torch.int8)
    s, s_ok = _guarded((M,), torch.float32)
    kw = dict(add=add, slots=None if slots is None else _dev(slots), gates=None if gates is None else _dev(gates))
    out, out_ok = _guarded((M, K), TYPES[xt])
    if inplace:
        out.copy_(x)
        x = out
    wd = None if w is None else _dev(w)
    hs = [bn.bitnet_add_norm(x, wd, eps, out_dtype=t, **kw)[0] for t in TYPES.values()]
    got = bn.bitnet_add_norm_quant(x, wd, eps, q=q, s_a=s, x_out=out if at else None, **kw)
    torch.cuda.synchronize()
    assert q_ok() and s_ok() and out_ok()
    assert np.array_equal(s.cpu().numpy(), s_a)
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(got[2].float().cpu().numpy(), stream)
    for t, hd in zip(TYPES.values(), hs):
        assert np.array_equal(hd.float().cpu().numpy(), lo.rounded(h, t))


@pytest.mark.parametrize("K", [16, 48, 128, 2560, 4096, 4112, 6912, 8208, 16384, 16400, 40000, 65536])
@pytest.mark.parametrize("xt,at,parts", [("bf16", "bf16", 0), ("fp32", "fp32", 0), ("fp32", "bf16", 3), ("bf16", None, 0)])
def test_norm_widths(gpu, K, xt, at, parts):
    _norm_case(np.random.default_rng(K + parts), 3, K, xt, at, parts)


@pytest.mark.parametrize("xt,at", list(itertools.product(TYPES, TYPES)))
@pytest.mark.parametrize("parts", [0, 1, 2, 8, 64])
@pytest.mark.parametrize("M", [1, 2, 67, 1300])
def test_norm_types_and_parts(gpu, xt, at, parts, M):
    if M * parts > 11000:
        M = 70
    _norm_case(np.random.default_rng(M + parts), M, 400, xt, at, parts, weight=M != 2, eps=1e-6, inplace=parts != 1)


def test_norm_many_rows(gpu):
    _norm_case(np.random.default_rng(5), 9001, 1280, "bf16", "bf16", 0)


def test_norm_rows_of_zeros_large_and_small_values(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(6)
    x = rng.standard_normal((6, 256)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e30  # squares beyond fp32
    x[2] *= 1e-30
    x[3] = 3e38
    x[4] *= 1e-42  # below the smallest normal number
    for eps in (1e-5, 1e-30, 1e-45):
        stream, h, codes, s_a = lo.add_norm(x, None, eps, torch.float32)
        q, s, same = bn.bitnet_add_norm_quant(_dev(x), None, eps)
        assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), s_a)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("where", ["x", "add", "gate", "unread"])
def test_norm_of_a_row_that_is_not_finite(gpu, bad, where):
    """The row's products become NaN, the others see nothing of it."""
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(7)
    x, add = rng.standard_normal((5, 640)).astype(np.float32), rng.standard_normal((11, 640)).astype(np.float32)
    slots = np.array([[0, 1], [2, 3], [4, -1], [6, 7], [8, 9]], np.int32)
    gates = rng.random((5, 2)).astype(np.float32)
    if where == "x":
        x[1, 77] = bad
    elif where == "add":
        add[3, 600] = bad
    elif where == "gate":
        gates[1, 0] = bad
    else:
        add[10], add[5], gates[2, 1] = bad, bad, bad  # rows of no slot, the gate of a place left empty
    stream, h, codes, s_a = lo.add_norm(x, None, 1e-5, torch.float32, add, slots, gates)
    q, s, out = bn.bitnet_add_norm_quant(_dev(x), None, 1e-5, add=_dev(add), slots=_dev(slots), gates=_dev(gates))
    assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), s_a, equal_nan=True)
    assert np.isnan(s_a).tolist() == [False, where != "unread", False, False, False]
    assert np.array_equal(out.cpu().numpy(), stream, equal_nan=True)


def test_norm_weight_that_is_not_finite_or_overflows(gpu):
    import bit_gemv_i2_amd as bn
    x = np.random.default_rng(8).standard_normal((2, 128)).astype(np.float32)
    for v in (np.inf, np.nan, 3e38):
        w = np.ones(128, np.float32)
        w[5] = v
        x[:, 5] = 40
        _, _, codes, s_a = lo.add_norm(x, w, 1e-5, torch.float32)
        q, s, _ = bn.bitnet_add_norm_quant(_dev(x), _dev(w), 1e-5)
        assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), s_a, equal_nan=True)


def test_norm_of_the_stored_stream(gpu):
    """A norm of x_out gives what the addition gave."""
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(9)
    x, _ = _values(rng, (40, 2560), torch.bfloat16)
    add, _ = _values(rng, (40, 2560), torch.float32)
    q, s, out = bn.bitnet_add_norm_quant(x, None, 1e-5, add=add)
    q2, s2, _ = bn.bitnet_add_norm_quant(out, None, 1e-5)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("K", [4112, 8208, 8704, 16400, 32768, 32784])
@pytest.mark.parametrize("parts", [0, 2])
def test_norm_in_place_where_lanes_have_no_chunk(gpu, K, parts):
    """x_out is x, and the row ends inside the lanes' last round: what another wave has stored meanwhile is not seen."""
    for M in (1, 40):
        _norm_case(np.random.default_rng(K + M), M, K, "fp32", "bf16", parts, inplace=True)


# ------------------------------------------------------------------ products
def _weights(rng, N, K):
    T = (rng.integers(0, 3, (N, K), dtype=np.int8) - 1).astype(np.int8)
    return T, (rng.uniform(0.5, 1.5, (N, K // 128)) / np.sqrt(K * 2 / 3)).astype(np.float32)


def _acts(rng, M, K):
    q = np.clip(np.rint(rng.standard_normal((M, K)) * 36), -127, 127).astype(np.int8)
    q[:, rng.integers(0, K, 3)] = 127
    q[:, rng.integers(0, K, 3)] = -127
    return q, (np.exp(0.3 * rng.standard_normal(M)) / 36).astype(np.float32)


def _linear_case(rng, M, N, K, act, gated, bias, residual, out, inplace=False):
    import bit_gemv_i2_amd as bn
    T, S = _weights(rng, N, K)
    q, s_a = _acts(rng, M, K)
    width = N // 2 if gated else N
    b = (0.5 * rng.standard_normal(N)).astype(np.float32) if bias else None
    r = rv = None
    if residual:
        r, rv = _values(rng, (M, width), TYPES[residual], 0.3)
    want, tol = lo.linear(T, S, q, s_a, None if b is None else b.astype(np.float64), act, gated,
                          None if rv is None else rv.astype(np.float64), TYPES[out])
    w = bn.PackedWeight.from_ternary(T, S)
    y, ok = _guarded((M, width), TYPES[out])
    if inplace:
        y.copy_(r)
        r = y
    got = w.linear(_dev(q), _dev(s_a), bias=None if b is None else _dev(b), act=act, gated=gated, residual=r, y=y)
    torch.cuda.synchronize()
    assert got is y and ok()
    lo.close(got, want, tol)


@pytest.mark.parametrize("act", lo.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_linear_activations(gpu, act, gated, M):
    i = lo.ACTS.index(act)
    _linear_case(np.random.default_rng(M + i), M, 416, 640, act, gated, i % 2 == 0, (None, "bf16", "fp32")[(i + M) % 3], ("bf16", "fp32")[(i + M) % 2])


@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
@pytest.mark.parametrize("N,K", [(16, 128), (32, 256), (272, 1280), (1040, 384)])
def test_linear_tokens(gpu, M, N, K):
    _linear_case(np.random.default_rng(M * N), M, N, K, "none", False, False, None, "fp32")
    if N % 32 == 0:
        _linear_case(np.random.default_rng(M * N + 1), M, N, K, "relu2", True, True, "bf16", "bf16")


@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 7, 8, 9, 12, 20, 27, 54, 97])
@pytest.mark.parametrize("M", [1, 6, 20, 130])
def test_linear_blocks(gpu, blocks, M):
    _linear_case(np.random.default_rng(blocks + M), M, 96, 128 * blocks, "silu", blocks % 2 == 0, blocks % 3 == 0, "fp32", "fp32")


@pytest.mark.parametrize("M,N,K,gated", [(1, 13824, 2560, True), (8, 13824, 2560, True), (200, 13824, 2560, True), (700, 2560, 6912, False),
                                         (1, 2560, 6912, False), (1100, 2080, 256, True), (16, 20480, 384, False), (513, 4128, 640, False)])
def test_linear_wide(gpu, M, N, K, gated):
    _linear_case(np.random.default_rng(M + N), M, N, K, "relu2" if gated else "none", gated, N % 3 == 0, "bf16" if M % 2 else None, "bf16")


@pytest.mark.parametrize("blocks", [4, 6, 10, 13, 16, 17, 24, 25, 32, 33, 48, 64, 65, 96, 130])
@pytest.mark.parametrize("M", [1, 4, 8, 12, 16, 37])
def test_linear_few_rows_of_long_columns(gpu, blocks, M):
    _linear_case(np.random.default_rng(blocks * M), M, 64, 128 * blocks, "relu2", blocks % 2 == 1, blocks % 3 == 0, "bf16", "fp32")


@pytest.mark.parametrize("M,N", [(112, 96), (113, 96), (64, 14016), (65, 14016), (32, 20480), (33, 20480), (16, 65536), (17, 65536)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_between_few_rows_and_many(gpu, M, N, gated):
    _linear_case(np.random.default_rng(M), M, N, 256, "silu", gated, True, "fp32", "bf16")


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M", [1, 16, 90, 300])
def test_linear_into_its_residual(gpu, out, M):
    _linear_case(np.random.default_rng(M), M, 544, 512, "none", False, True, out, out, inplace=True)
    _linear_case(np.random.default_rng(M), M, 544, 512, "gelu", True, True, out, out, inplace=True)


def test_linear_large_and_small_arguments_of_the_activations(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(3)
    T, S = _weights(rng, 64, 256)
    q, _ = _acts(rng, 9, 256)
    s_a = np.array([1e-30, 1e-6, 0.01, 1.0, 30.0, 300.0, 1e4, 1e8, 1e12], np.float32)
    for act in lo.ACTS:
        want, tol = lo.linear(T, S, q, s_a, None, act, False, None, torch.float32)
        lo.close(bn.PackedWeight.from_ternary(T, S).linear(_dev(q), _dev(s_a), act=act, out_dtype=torch.float32), want, tol)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_linear_of_a_token_that_is_not_finite(gpu, M):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(4)
    T, S = _weights(rng, 320, 640)
    q, s_a = _acts(rng, M, 640)
    s_a[1] = np.nan
    q[1] = 0
    for act, gated in itertools.product(lo.ACTS, (False, True)):
        with np.errstate(invalid="ignore"):
            want, tol = lo.linear(T, S, q, s_a, None, act, gated, None, torch.float32)
        want[1] = np.nan
        lo.close(bn.PackedWeight.from_ternary(T, S).linear(_dev(q), _dev(s_a), act=act, gated=gated, out_dtype=torch.float32), want, tol)


@pytest.mark.parametrize("M", [1, 9, 48, 49, 64, 300])
def test_linear_whole_numbers_exactly(gpu, M):
    """With scales and factors of one every output is a whole number below 2^24: all int8 codes, -128 among them, every column order,
    the largest sums there are."""
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(M)
    for N, K in ((272, 128), (32, 640), (544, 2560)):
        T = (rng.integers(0, 3, (N, K), dtype=np.int8) - 1).astype(np.int8)
        T[0], T[1] = 1, -1
        T[2:18] = 0
        T[2:18][np.arange(16), rng.integers(0, K, 16)] = 1  # a column alone
        q = rng.integers(-128, 128, (M, K), dtype=np.int64).astype(np.int8)
        q[0] = np.arange(K) % 256 - 128
        q[-1] = -128 if M > 1 else q[-1]
        if M > 2:
            q[1] = 127
        y = bn.PackedWeight.from_ternary(T, np.ones((N, K // 128), np.float32)).linear(_dev(q), _dev(np.ones(M, np.float32)), out_dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), (q.astype(np.int64) @ T.astype(np.int64).T).astype(np.float32))


# ------------------------------------------------------------------ products by expert
def _grouped_case(rng, counts, tokens, N, K, act, gated, bias, gather, out, slots=None, bad=()):
    import bit_gemv_i2_amd as bn
    E, used = len(counts), int(sum(counts))
    slots = slots or max(1, used)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T, S = _weights(rng, E * N, K)
    tokens = tokens if gather else slots
    q, s_a = _acts(rng, tokens, K)
    rows = rng.integers(0, tokens, slots).astype(np.int32) if gather else np.arange(slots)
    for i, v in bad:
        rows[i] = v
    b = (0.5 * rng.standard_normal((E, N))).astype(np.float32) if bias else None
    width = N // 2 if gated else N
    want, tol = np.full((slots, width), -77.0), np.zeros((slots, width))
    for e in range(E):
        at = [i for i in range(starts[e], starts[e + 1]) if i < slots and 0 <= rows[i] < tokens]
        if at:
            want[at], tol[at] = lo.linear(T[e * N: (e + 1) * N], S[e * N: (e + 1) * N], q[rows[at]], s_a[rows[at]],
                                          None if b is None else b[e].astype(np.float64), act, gated, None, TYPES[out])
    w = bn.PackedExperts.from_ternary(T.reshape(E, N, K), S.reshape(E, N, -1))
    y, ok = _guarded((slots, width), TYPES[out])
    got = w.grouped(_dev(q), _dev(s_a), _dev(starts), rows=_dev(rows.astype(np.int32)) if gather else None,
                    bias=None if b is None else _dev(b), act=act, gated=gated, y=y)
    torch.cuda.synchronize()
    assert ok()
    lo.close(got, want, tol)


@pytest.mark.parametrize("counts", [[1], [0, 1], [1, 0, 0, 2], [0, 0, 5, 0, 16, 17, 1, 0], [40, 0, 3, 130], [15] * 9, [0, 300, 0, 1], [2] * 70,
                                    [0] * 63 + [1, 0, 33] + [0] * 30 + [4], [500, 129]])
@pytest.mark.parametrize("gated,gather", [(False, False), (True, True), (False, True)])
def test_grouped_ragged(gpu, counts, gated, gather):
    rng = np.random.default_rng(len(counts) + sum(counts))
    _grouped_case(rng, counts, 37, 96, 384, "silu" if gated else "none", gated, len(counts) % 2 == 0, gather, "bf16" if gather else "fp32")


@pytest.mark.parametrize("N,K", [(32, 128), (544, 1280), (2560, 640), (160, 4352)])
@pytest.mark.parametrize("most", [1, 4, 40, 200])
def test_grouped_shapes(gpu, N, K, most):
    rng = np.random.default_rng(N + most)
    counts = rng.integers(0, most + 1, 6).tolist()
    counts[2] = most
    _grouped_case(rng, counts, 50, N, K, "relu2", True, True, True, "fp32")


def test_grouped_rows_of_no_expert_and_bad_rows_stay(gpu):
    rng = np.random.default_rng(11)
    for most in (3, 90):
        _grouped_case(rng, [most, 0, 5], 20, 64, 256, "none", False, True, True, "fp32", slots=most + 30,
                      bad=[(0, -1), (2, 20), (most + 1, 2 ** 31 - 1), (most + 2, -2 ** 31)])


def test_grouped_none_at_all(gpu):
    _grouped_case(np.random.default_rng(12), [0, 0, 0], 4, 64, 256, "none", False, False, True, "fp32", slots=9)


def test_grouped_starts_beyond_the_slots(gpu):
    """Starts are read as lying within the slots: nothing outside y is written, nothing outside q read."""
    rng = np.random.default_rng(13)
    _grouped_case(rng, [3, 50, 9], 20, 64, 256, "none", False, False, True, "fp32", slots=10)
    import bit_gemv_i2_amd as bn
    T, S = _weights(rng, 3 * 32, 128)
    w = bn.PackedExperts.from_ternary(T.reshape(3, 32, 128), S.reshape(3, 32, 1))
    q, s_a = _acts(rng, 6, 128)
    for starts in ([-5, 2, 4, 1 << 30], [6, 2, 1, 0], [2 ** 31 - 1] * 4, [-2 ** 31, -1, -1, 2 ** 31 - 1], [0, 6, 2, 6]):
        y, ok = _guarded((6, 32), torch.float32)
        w.grouped(_dev(q), _dev(s_a), _dev(np.array(starts, np.int32)), y=y)
        torch.cuda.synchronize()
        assert ok()


@pytest.mark.parametrize("most", [4, 150])
def test_grouped_of_a_token_that_is_not_finite(gpu, most):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(14)
    N, K = 64, 256
    T, S = _weights(rng, 2 * N, K)
    q, s_a = _acts(rng, most, K)
    s_a[1], q[1] = np.nan, 0
    starts = np.array([0, most // 2, most], np.int32)
    got = bn.PackedExperts.from_ternary(T.reshape(2, N, K), S.reshape(2, N, -1)).grouped(_dev(q), _dev(s_a), _dev(starts), out_dtype=torch.float32)
    for e in range(2):
        at = slice(starts[e], starts[e + 1])
        want, tol = lo.linear(T[e * N: (e + 1) * N], S[e * N: (e + 1) * N], q[at], s_a[at], None, "none", False, None, torch.float32)
        lo.close(got[at], want, tol)


# ------------------------------------------------------------------ routing
def _route_case(logits, dtype, k, over_all, pad=0):
    import bit_gemv_i2_amd as bn
    T, E = logits.shape
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype)
    wide = torch.full((T, E + pad), 9e9, dtype=dtype, device="cuda")
    wide[:, :E] = t.cuda()
    want = lo.route(t.float().numpy(), k, over_all)
    made = [_guarded(w.shape, torch.float32 if i == 1 else torch.int32) for i, w in enumerate(want)]
    bn.bitnet_route(wide[:, :E], k, over_all=over_all, out=tuple(m[0] for m in made))
    torch.cuda.synchronize()
    for i, (w, (got, ok)) in enumerate(zip(want, made)):
        assert ok()
        if i != 1:
            assert np.array_equal(got.cpu().numpy(), w), ("chosen", "gates", "starts", "rows", "slots")[i]
    # exponentials: the difference's rounding, half a step of at most |l - top|, and theirs, two steps; a sum of at most 1024 such
    # terms and a quotient
    value = np.where(want[0] >= 0, np.take_along_axis(t.float().numpy().astype(np.float64), np.maximum(want[0], 0), 1), np.nan)
    finite = np.isfinite(t.float().numpy())
    low = np.where(finite, t.float().numpy(), np.inf).min(1, initial=np.inf) if over_all else np.nan_to_num(value, nan=np.inf).min(1)
    reach = np.where(np.isfinite(low), np.nan_to_num(value[:, 0]) - low, 0.0)[:, None]
    n = E if over_all else k
    tol = want[1] * (2 * (reach + 4) + n + 4) * 2 * lo.HALF + 2.0 ** -126
    lo.close(made[1][0], want[1], tol)


@pytest.mark.parametrize("E", [1, 2, 5, 8, 9, 16, 17, 32, 60, 64, 65, 128, 200, 256, 500, 1000, 1024])
@pytest.mark.parametrize("T", [1, 63, 64, 65, 256, 257, 1000])
def test_route_sizes(gpu, E, T):
    rng = np.random.default_rng(E + T)
    for k in sorted({1, min(2, E), min(8, E), min(32, E)}):
        _route_case(rng.standard_normal((T, E)) * 2, torch.float32 if (E + T) % 2 else torch.bfloat16, k, k % 2 == 0, pad=(E + T) % 3)


@pytest.mark.parametrize("dtype", list(TYPES.values()))
@pytest.mark.parametrize("T,E,k", [(20000, 64, 6), (16500, 8, 2), (33000, 4, 4)])
def test_route_many_tokens(gpu, dtype, T, E, k):
    _route_case(np.random.default_rng(T).standard_normal((T, E)), dtype, k, False)


@pytest.mark.parametrize("E", [3, 16, 64, 100, 300])
@pytest.mark.parametrize("T", [50, 700])
def test_route_ties_and_masks(gpu, E, T):
    rng = np.random.default_rng(E * T)
    k = min(4, E)
    few = rng.integers(-1, 2, (T, E)).astype(np.float64)
    few[few == 0] *= rng.choice([-1, 1], (few == 0).sum())  # zeros of both signs are equal
    _route_case(few, torch.float32, k, False)
    _route_case(np.zeros((T, E)), torch.bfloat16, k, True)
    masked = rng.standard_normal((T, E))
    masked[rng.random((T, E)) < 0.8] = -np.inf
    masked[rng.random((T, E)) < 0.1] = np.nan
    masked[T // 2:] = -np.inf  # padding
    masked[3] = np.nan
    masked[4] = -3e38
    _route_case(masked, torch.float32, k, False)
    _route_case(masked, torch.bfloat16, k, True)
    _route_case(np.full((T, E), -np.inf), torch.float32, k, False)


def test_route_all_to_one_expert(gpu):
    logits = np.random.default_rng(1).standard_normal((3000, 40))
    logits[:, 17] = 50
    _route_case(logits, torch.float32, 1, False)
    _route_case(logits, torch.bfloat16, 3, True)


def test_route_of_an_infinite_logit(gpu):
    import bit_gemv_i2_amd as bn
    logits = np.random.default_rng(2).standard_normal((5, 12)).astype(np.float32)
    logits[2, 7] = np.inf
    chosen, gates, *_ = bn.bitnet_route(_dev(logits), 2)
    assert int(chosen[2, 0]) == 7
    assert torch.isnan(gates).any(1).tolist() == [False, False, True, False, False]


# ------------------------------------------------------------------ together, streams, graphs
class Block:
    """norm - router - experts - combination, as a decoder layer runs it."""

    def __init__(self, rng, hidden, ffn, E, k):
        import bit_gemv_i2_amd as bn
        self.E, self.k, self.hidden = E, k, hidden
        self.up_T, self.up_S = _weights(rng, E * 2 * ffn, hidden)
        self.down_T, self.down_S = _weights(rng, E * hidden, ffn)
        self.up = bn.PackedExperts.from_ternary(self.up_T.reshape(E, 2 * ffn, hidden), self.up_S.reshape(E, 2 * ffn, -1))
        self.down = bn.PackedExperts.from_ternary(self.down_T.reshape(E, hidden, ffn), self.down_S.reshape(E, hidden, -1))
        self.router = _dev((rng.standard_normal((hidden, E)) / np.sqrt(hidden)).astype(np.float32))
        self.weight = _dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32))

    def __call__(self, x):
        import bit_gemv_i2_amd as bn
        q, s, _ = bn.bitnet_add_norm_quant(x, self.weight)
        logits = (q.float() * s[:, None]) @ self.router
        chosen, gates, starts, rows, slots = bn.bitnet_route(logits, self.k)
        h = self.up.grouped(q, s, starts, rows=rows, act="relu2", gated=True, out_dtype=torch.float32)
        hq, hs = bn.bitnet_quant_act(h)
        d = self.down.grouped(hq, hs, starts, out_dtype=torch.bfloat16)
        q2, s2, out = bn.bitnet_add_norm_quant(x, self.weight, add=d, slots=slots, gates=gates)
        return dict(q=q, s=s, logits=logits, chosen=chosen, gates=gates, starts=starts, rows=rows, slots=slots, h=h, hq=hq, hs=hs, d=d,
                    q2=q2, s2=s2, out=out)


@pytest.mark.parametrize("T", [1, 7, 300])
def test_a_layer_of_experts_step_by_step(gpu, T):
    """Every step against the oracle on the step's own input."""
    rng = np.random.default_rng(T)
    hidden, ffn, E, k = 512, 384, 8, 2
    b = Block(rng, hidden, ffn, E, k)
    x, xv = _values(rng, (T, hidden), torch.float32, 0.3)
    o = {n: v.cpu().numpy() if v.dtype != torch.bfloat16 else v.float().cpu().numpy() for n, v in b(x).items()}
    w = b.weight.cpu().numpy()
    _, _, codes, s_a = lo.add_norm(xv, w, 1e-5, torch.float32)
    assert np.array_equal(o["q"], codes) and np.array_equal(o["s"], s_a)
    chosen, gates, starts, rows, slots = lo.route(o["logits"], k, False)
    for n, v in (("chosen", chosen), ("starts", starts), ("rows", rows), ("slots", slots)):
        assert np.array_equal(o[n], v), n
    for e in range(E):
        at = slice(starts[e], starts[e + 1])
        n = slice(e * 2 * ffn, (e + 1) * 2 * ffn)
        want, tol = lo.linear(b.up_T[n], b.up_S[n], o["q"][rows[at]], o["s"][rows[at]], None, "relu2", True, None, torch.float32)
        lo.close(torch.from_numpy(o["h"][at]), want, tol)
        n = slice(e * hidden, (e + 1) * hidden)
        want, tol = lo.linear(b.down_T[n], b.down_S[n], o["hq"][at], o["hs"][at], None, "none", False, None, torch.bfloat16)
        lo.close(torch.from_numpy(o["d"][at]), want, tol)
    stream, _, codes, s_a = lo.add_norm(xv, w, 1e-5, torch.float32, o["d"], o["slots"], o["gates"])
    assert np.array_equal(o["out"], stream) and np.array_equal(o["q2"], codes) and np.array_equal(o["s2"], s_a)


@pytest.mark.parametrize("T", [3, 300])
def test_a_layer_of_experts_in_a_graph(gpu, T):
    """Captured once, replayed with new inputs between eager calls of the same operators: the plan of each replay is its own."""
    rng = np.random.default_rng(T)
    b = Block(rng, 512, 256, 8, 2)
    xs = [_values(rng, (T, 512), torch.float32, 0.3)[0] for _ in range(5)]
    x = xs[0].clone()
    b(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b(x)
    for i in (1, 2, 3, 4, 1):
        eager = {n: v.clone() for n, v in b(xs[i]).items()}
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for n, v in eager.items():
            assert torch.equal(out[n].view(torch.uint8), v.view(torch.uint8)), (i, n)


def test_a_stream_of_its_own(gpu):
    rng = np.random.default_rng(1)
    b = Block(rng, 512, 256, 8, 2)
    x, _ = _values(rng, (100, 512), torch.float32, 0.3)
    first = b(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = b(x)
    side.synchronize()
    for n in first:
        assert torch.equal(first[n].view(torch.uint8), second[n].view(torch.uint8)), n


def test_the_stream_argument(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(2)
    side = torch.cuda.Stream()
    x, _ = _values(rng, (300, 512), torch.float32)
    T, S = _weights(rng, 128, 512)
    w = bn.PackedWeight.from_ternary(T, S)
    want = bn.bitnet_add_norm_quant(x, add=x)
    plan = bn.bitnet_route(x[:, :40], 3)
    y = w.linear(want[0], want[1], residual=x[:, :128].contiguous())
    e = bn.PackedExperts(w.packed, w.scales, 4, 32, 512)
    starts = _dev(np.array([0, 100, 100, 250, 300], np.int32))
    z = e.grouped(want[0], want[1], starts)
    torch.cuda.synchronize()
    got = bn.bitnet_add_norm_quant(x, add=x, stream=side)
    plan2 = bn.bitnet_route(x[:, :40], 3, stream=side)
    with torch.cuda.stream(side):
        r = x[:, :128].contiguous()
    y2 = w.linear(got[0], got[1], residual=r, stream=side)
    z2 = e.grouped(got[0], got[1], starts, stream=side)
    side.synchronize()
    for a, b in zip((*want, *plan, y, z), (*got, *plan2, y2, z2)):
        assert torch.equal(a, b)


def test_results_repeat(gpu):
    """The same call gives the same bits, whatever ran before."""
    rng = np.random.default_rng(3)
    for T in (5, 700):
        b = Block(rng, 512, 384, 8, 2)
        x, _ = _values(rng, (T, 512), torch.float32)
        first = b(x)
        for _ in range(3):
            again = b(x)
            for n in first:
                assert torch.equal(first[n].view(torch.uint8), again[n].view(torch.uint8)), n


def test_the_example_with_experts_runs(gpu):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import generate
    model = generate.Decoder(2, 512, 4, 2, 256, experts=6, top=2)
    tokens, states = model.generate([[3, 1, 4], [1] * 70, [5]], 4)
    assert tokens.shape == (3, 4) and ((tokens >= 0) & (tokens < 4096)).all() and torch.isfinite(states).all()
    assert -1 <= generate.check(model, [[3, 1, 4], [1] * 70, [5]], tokens, states) <= 1.0001
