"""Norm, products with epilogues, experts and routing without a GPU: sizes, every refusal (made before any HIP call, so no kernel is launched
here), and the oracle against itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_gemv_i2_amd as bn
import layer_oracle as lo

P, MIS, MIS4, NULL = (ctypes.c_void_p(x) for x in (0x100000, 0x100004, 0x100002, 0))
P2 = ctypes.c_void_p(0x900000)
ARG, SHAPE = bn.BITNET_ERR_INVALID_ARG, bn.BITNET_ERR_UNSUPPORTED_SHAPE
BF16, F32 = bn.BITNET_DT_BF16, bn.BITNET_DT_F32


def _call(f, order, base, **kw):
    a = dict(base, **kw)
    return f(*[a[n] for n in order])


# ------------------------------------------------------------------ refusals of the C entries
def test_add_norm_refusals():
    order = "x xdt add adt add_rows slots gates parts weight eps M K x_out q s_a h hdt stream".split()
    base = dict(x=P, xdt=F32, add=P2, adt=BF16, add_rows=6, slots=P, gates=P, parts=2, weight=P, eps=1e-5, M=3, K=256, x_out=P, q=P, s_a=P,
                h=P, hdt=BF16, stream=NULL)
    for kw in (dict(x=NULL), dict(x=MIS), dict(xdt=2), dict(xdt=-1), dict(add=MIS), dict(adt=3), dict(x_out=NULL), dict(x_out=MIS),
               dict(weight=MIS), dict(slots=MIS4), dict(gates=NULL), dict(gates=MIS4), dict(slots=NULL), dict(slots=NULL, gates=NULL),
               dict(slots=NULL, parts=0), dict(add=NULL), dict(add=NULL, x_out=NULL), dict(add=NULL, slots=NULL, gates=NULL, parts=0),
               dict(q=NULL, s_a=NULL, h=NULL), dict(q=NULL), dict(s_a=NULL), dict(q=MIS), dict(s_a=MIS4), dict(h=MIS), dict(hdt=7),
               dict(eps=0.0), dict(eps=-1e-5), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-60)):
        assert _call(bn.lib().bitnet_add_norm, order, base, **kw) == ARG, kw
    for kw in (dict(M=0), dict(M=-1), dict(M=65535 * 1024 + 1), dict(K=0), dict(K=-16), dict(K=24), dict(K=65552), dict(parts=0), dict(parts=-1),
               dict(parts=65), dict(add_rows=0), dict(add_rows=-3), dict(M=1 << 22, K=528), dict(M=1 << 22, K=4112, slots=NULL, gates=NULL, parts=0)):
        assert _call(bn.lib().bitnet_add_norm, order, base, **kw) == SHAPE, kw


def test_linear_refusals():
    order = "packed scales q s_a bias act gated residual rdt y ydt M N K ws bytes stream".split()
    base = dict(ws=NULL, bytes=0, packed=P, scales=P, q=P, s_a=P, bias=P, act=0, gated=0, residual=P, rdt=F32, y=P2, ydt=BF16, M=5, N=48, K=256, stream=NULL)
    f = bn.lib().bitnet_w2a8_linear
    for n in ("packed", "scales", "q", "y"):
        for v in (NULL, MIS):
            assert _call(f, order, base, **{n: v}) == ARG, n
    for kw in (dict(s_a=NULL), dict(s_a=MIS4), dict(bias=MIS), dict(residual=MIS), dict(act=-1), dict(act=5), dict(rdt=2), dict(ydt=-1),
               dict(ydt=2), dict(residual=P2)):
        assert _call(f, order, base, **kw) == ARG, kw
    for kw in (dict(M=0), dict(M=-4), dict(M=(1 << 24) + 1), dict(N=0), dict(N=40), dict(N=-16), dict(K=64), dict(K=0), dict(gated=1), dict(N=1 << 30, K=1 << 20), dict(N=16, K=(1 << 24) + 128), dict(N=1 << 20, K=1 << 15)):
        assert _call(f, order, base, **kw) == SHAPE, kw


def test_grouped_refusals():
    order = "packed scales q s_a tokens starts rows experts slots bias act gated y ydt N K ws bytes stream".split()
    base = dict(ws=NULL, bytes=0, packed=P, scales=P, q=P, s_a=P, tokens=7, starts=P, rows=P, experts=4, slots=9, bias=P, act=0, gated=0, y=P, ydt=BF16, N=48,
                K=256, stream=NULL)
    f = bn.lib().bitnet_w2a8_grouped
    for n in ("packed", "scales", "q", "y"):
        for v in (NULL, MIS):
            assert _call(f, order, base, **{n: v}) == ARG, n
    for kw in (dict(s_a=NULL), dict(starts=NULL), dict(starts=MIS4), dict(rows=MIS4), dict(bias=MIS), dict(act=9), dict(ydt=3)):
        assert _call(f, order, base, **kw) == ARG, kw
    for kw in (dict(tokens=0), dict(tokens=(1 << 24) + 1), dict(slots=0), dict(slots=-1), dict(slots=(1 << 24) + 1), dict(experts=0),
               dict(experts=1025), dict(rows=NULL), dict(gated=1), dict(N=24), dict(K=100)):
        assert _call(f, order, base, **kw) == SHAPE, kw


def test_product_workspaces():
    """Few rows an expert need none; many need the digits of every token, which a call without them is refused."""
    assert bn.lib().bitnet_w2a8_linear_workspace_bytes(1, 32, 256) == 0
    assert bn.lib().bitnet_w2a8_linear_workspace_bytes(4000, 32, 256) == 4000 * 2 * 192
    assert bn.lib().bitnet_w2a8_linear_workspace_bytes(1 << 24, 32, 256) == (1 << 24) * 2 * 192
    assert bn.lib().bitnet_w2a8_grouped_workspace_bytes(4000, 8000, 8, 32, 256) == 4000 * 2 * 192
    for M in (1, 16, 17, 48, 112):
        assert bn.lib().bitnet_w2a8_linear_workspace_bytes(M, 2560, 2560) == 0
    assert bn.lib().bitnet_w2a8_linear_workspace_bytes(113, 2560, 2560) == 113 * 20 * 192
    assert bn.lib().bitnet_w2a8_linear_workspace_bytes(16, 1 << 20, 256) == 0 < bn.lib().bitnet_w2a8_linear_workspace_bytes(17, 1 << 20, 256)
    assert bn.lib().bitnet_w2a8_grouped_workspace_bytes(40, 80, 80, 32, 256) == 0
    for bad in ((0, 32, 256), (4000, 40, 256), (4000, 32, 100)):
        assert bn.lib().bitnet_w2a8_linear_workspace_bytes(*bad) == 0
    for bad in ((0, 80, 2, 32, 256), (40, 0, 2, 32, 256), (40, 80, 0, 32, 256), (40, 80, 2, 33, 256), (-1, 80, 2, 32, 256)):
        assert bn.lib().bitnet_w2a8_grouped_workspace_bytes(*bad) == 0
    f = bn.lib().bitnet_w2a8_linear
    need = bn.lib().bitnet_w2a8_linear_workspace_bytes(4000, 32, 256)
    for ws, nb in ((NULL, 0), (NULL, need), (P, need - 1), (MIS, need)):
        assert f(P, P, P, P, NULL, 0, 0, NULL, 0, P2, F32, 4000, 32, 256, ws, nb, NULL) == ARG
    for ws, nb in ((NULL, 0), (P, need - 1), (MIS, need)):
        assert bn.lib().bitnet_w2a8_grouped(P, P, P, P, 4000, P, P, 2, 4000, NULL, 0, 0, P2, F32, 32, 256, ws, nb, NULL) == ARG
    # digits past 32 bits of offset, and more tiles than a launch holds
    for M, N, K in ((1 << 24, 32, 128), (1 << 17, 32, 1 << 14), (1 << 20, 1 << 19, 128)):
        assert f(P, P, P, P, NULL, 0, 0, NULL, 0, P2, F32, M, N, K, P, M * (K // 128) * 192, NULL) == SHAPE
        assert bn.lib().bitnet_w2a8_grouped(P, P, P, P, M, P, P, 1, 1 << 20, NULL, 0, 0, P2, F32, N, K, P, M * (K // 128) * 192, NULL) == SHAPE


def test_route_refusals():
    order = "logits dt row_stride tokens experts k over_all chosen gates starts rows slots ws bytes stream".split()
    base = dict(logits=P, dt=F32, row_stride=64, tokens=1000, experts=64, k=4, over_all=0, chosen=P, gates=P, starts=P, rows=P, slots=P, ws=P,
                bytes=1 << 30, stream=NULL)
    f = bn.lib().bitnet_route
    for n in ("chosen", "gates", "starts", "rows", "slots", "logits"):
        for v in (NULL, MIS4):
            assert _call(f, order, base, **{n: v}) == ARG, n
    for kw in (dict(dt=2), dict(ws=NULL), dict(ws=MIS), dict(bytes=bn.bitnet_route_workspace_bytes(1000, 64, 4) - 1)):
        assert _call(f, order, base, **kw) == ARG, kw
    for kw in (dict(tokens=0), dict(tokens=-1), dict(experts=0), dict(experts=1025, row_stride=2000), dict(k=0), dict(k=33), dict(k=4, experts=3),
               dict(row_stride=63), dict(tokens=1 << 29)):
        assert _call(f, order, base, **kw) == SHAPE, kw


def test_route_workspace():
    assert bn.bitnet_route_workspace_bytes(1, 64, 6) == 0
    for bad in ((0, 64, 6), (10, 0, 1), (10, 4, 5), (10, 2000, 2), (10, 64, 33), (1 << 30, 64, 2), (-5, 64, 2)):
        assert bn.bitnet_route_workspace_bytes(*bad) == 0
    for T in (300, 5000, 70000, 1 << 24):
        assert 0 < bn.bitnet_route_workspace_bytes(T, 64, 6) <= 4 * 1024 * 64 + 256
    for n in (1 << 31, -(1 << 32) + 5):
        for args in ((n, 64, 6), (10, n, 6), (10, 64, n)):
            with pytest.raises(ValueError, match="must be below"):
                bn.bitnet_route_workspace_bytes(*args)


# ------------------------------------------------------------------ the binding: no launch is reached on the host
def test_binding_refuses_host_tensors_and_wrong_shapes():
    f, h = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.float16)
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    p, sc = torch.zeros(32 * 32, dtype=torch.uint8), torch.zeros(32)
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: bn.bitnet_add_norm_quant(f), lambda: bn.bitnet_add_norm(f), lambda: bn.bitnet_add_norm_quant(h),
                 lambda: bn.bitnet_add_norm_quant(f[0]), lambda: bn.bitnet_add_norm_quant(f, slots=i), lambda: bn.bitnet_add_norm_quant(f, add=f, gates=f),
                 lambda: bn.bitnet_route(f, 2), lambda: bn.bitnet_route(h, 2), lambda: bn.bitnet_route(f[0], 2), lambda: bn.bitnet_route(f.t(), 2),
                 lambda: bn.bitnet_w2a8_linear(p, sc, q, s, 32, 128), lambda: bn.bitnet_w2a8_linear(p, sc, q, s, 32, 128, act="tanh"),
                 lambda: bn.bitnet_w2a8_linear(p, sc, q, s, 32, 128, act=["relu"]),
                 lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, i, 32, 128), lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, i[:1], 32, 128)):
        with pytest.raises(ValueError):
            call()
    for n in (1 << 31, (1 << 32) + 2, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="must be below"):
            bn.bitnet_route(f, n)


@pytest.fixture
def fake_gpu(monkeypatch):
    """Host tensors taken for device tensors up to the launch, which is caught: what the checks let through."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            real = getattr(bn_lib, name)
            if name in ("bitnet_add_norm", "bitnet_w2a8_linear", "bitnet_w2a8_grouped", "bitnet_route"):
                return lambda *a: calls.append((name, a)) or 0
            return real
    bn_lib = bn.lib()
    monkeypatch.setattr(bn, "lib", lambda: Lib())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(bn, "_launch_stream", lambda torch, stream, dev: 0)
    return calls


def test_binding_checks_behind_the_device(fake_gpu):
    f, b = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.bfloat16)
    i2, g2 = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    ok = [lambda: bn.bitnet_add_norm_quant(f), lambda: bn.bitnet_add_norm_quant(f, torch.ones(128), add=b, x_out=f),
          lambda: bn.bitnet_add_norm_quant(b, add=f), lambda: bn.bitnet_add_norm_quant(f, add=torch.zeros(9, 128), slots=i2, gates=g2),
          lambda: bn.bitnet_add_norm(b, out_dtype=torch.float32), lambda: bn.bitnet_add_norm(f, h=b)]
    for call in ok:
        call()
    assert len(fake_gpu) == len(ok)
    for call in (lambda: bn.bitnet_add_norm_quant(f, torch.ones(127)), lambda: bn.bitnet_add_norm_quant(f, torch.ones(128, dtype=torch.bfloat16)),
                 lambda: bn.bitnet_add_norm_quant(f, add=f[:3]), lambda: bn.bitnet_add_norm_quant(f, add=torch.zeros(9, 128)),
                 lambda: bn.bitnet_add_norm_quant(f, add=f, slots=i2[:3], gates=g2), lambda: bn.bitnet_add_norm_quant(f, add=f, slots=i2, gates=g2[:, :1]),
                 lambda: bn.bitnet_add_norm_quant(f, add=f, slots=i2.long(), gates=g2), lambda: bn.bitnet_add_norm_quant(f, x_out=f),
                 lambda: bn.bitnet_add_norm_quant(f, add=f, x_out=b), lambda: bn.bitnet_add_norm_quant(f.t()),
                 lambda: bn.bitnet_add_norm_quant(f[:, :64]), lambda: bn.bitnet_add_norm(f, out_dtype=torch.float16),
                 lambda: bn.bitnet_add_norm(f, out_dtype=torch.float32, h=b), lambda: bn.bitnet_add_norm_quant(f, q=torch.zeros(4, 64, dtype=torch.int8))):
        with pytest.raises(ValueError):
            call()
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    p, sc = torch.zeros(2 * 32 * 32, dtype=torch.uint8), torch.zeros(2 * 32)
    one = (p[:1024], sc[:32], q, s, 32, 128)
    del fake_gpu[:]
    y = torch.zeros(4, 16, dtype=torch.bfloat16)
    st, rows = torch.zeros(3, dtype=torch.int32), torch.zeros(7, dtype=torch.int32)
    assert bn.bitnet_w2a8_linear(*one).dtype == torch.bfloat16
    assert bn.bitnet_w2a8_linear(*one, residual=torch.zeros(4, 32)).dtype == torch.float32
    assert bn.bitnet_w2a8_linear(*one, gated=True, y=y, residual=y, bias=torch.zeros(32)) is y
    assert bn.bitnet_w2a8_grouped(p, sc, q, s, st, 32, 128, rows=rows, gated=True).shape == (7, 16)
    assert bn.bitnet_w2a8_grouped(p, sc, q, s, st, 32, 128, bias=torch.zeros(2, 32)).shape == (4, 32)
    assert len(fake_gpu) == 5
    for call in (lambda: bn.bitnet_w2a8_linear(p, sc, q, s, 32, 128), lambda: bn.bitnet_w2a8_linear(*one[:4], 64, 128),
                 lambda: bn.bitnet_w2a8_linear(*one[:4], 32, 64), lambda: bn.bitnet_w2a8_linear(*one, bias=torch.zeros(16)),
                 lambda: bn.bitnet_w2a8_linear(*one, residual=torch.zeros(4, 16)), lambda: bn.bitnet_w2a8_linear(*one, y=y),
                 lambda: bn.bitnet_w2a8_linear(*one, gated=True, y=y, out_dtype=torch.float32),
                 lambda: bn.bitnet_w2a8_linear(p[:1024], sc[:32], q, s[:3], 32, 128), lambda: bn.bitnet_w2a8_linear(*one, residual=torch.zeros(4, 32).half()),
                 lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, st[:2], 32, 128), lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, st.long(), 32, 128),
                 lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, st, 32, 128, bias=torch.zeros(32)),
                 lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, st, 32, 128, rows=rows.long()),
                 lambda: bn.bitnet_w2a8_grouped(p, sc, q, s, st, 32, 128, y=torch.zeros(5, 32))):
        with pytest.raises((ValueError, bn.BitnetError)):
            call()
    with pytest.raises(bn.BitnetError, match="unsupported shape"):
        bn.bitnet_w2a8_linear(p, sc, q, s, 24, 128)
    for n in (-(1 << 70), 1 << 70, -16, 0):
        with pytest.raises((ValueError, bn.BitnetError)):
            bn.bitnet_w2a8_linear(p, sc, q, s, n, 128)


def test_binding_route(fake_gpu):
    x = torch.zeros(300, 70)
    out = bn.bitnet_route(x[:, :64], 6)
    assert [tuple(t.shape) for t in out] == [(300, 6), (300, 6), (65,), (1800,), (300, 6)]
    name, a = fake_gpu[0]
    assert a[2:6] == (70, 300, 64, 6)  # stride, tokens, experts, k
    assert bn.bitnet_route(x[:1, :64], 6, out=tuple(t[:1] if t.dim() == 2 else t[:6] if t.numel() == 1800 else t for t in out))
    for call in (lambda: bn.bitnet_route(x, 0), lambda: bn.bitnet_route(x, 71), lambda: bn.bitnet_route(x[:, ::2], 2),
                 lambda: bn.bitnet_route(x[:, :64], 6, out=out[:4]), lambda: bn.bitnet_route(x, 6, out=out),
                 lambda: bn.bitnet_route(x, 6, workspace=torch.zeros(16, dtype=torch.uint8)), lambda: bn.bitnet_route(x[:0], 2)):
        with pytest.raises((ValueError, bn.BitnetError)):
            call()


def test_packed_experts():
    rng = np.random.default_rng(0)
    T = (rng.integers(0, 3, (3, 32, 256)) - 1).astype(np.int8)
    S = rng.random((3, 32, 2)).astype(np.float32)
    w = bn.PackedExperts.from_ternary(T, S, device="cpu")
    for e in range(3):  # an expert's part is its own packed matrix
        p, s = bn.bitnet_pack_i2s(T[e], S[e])
        assert np.array_equal(w.packed.numpy()[e * p.size: (e + 1) * p.size], p)
        assert np.array_equal(w.scales.numpy()[e * s.size: (e + 1) * s.size], s)
    with pytest.raises(ValueError, match="starts"):
        w.grouped(None, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(bn.BitnetError):
        bn.PackedExperts.from_ternary(T[:, :8], S[:, :8], device="cpu")


# ------------------------------------------------------------------ the oracle
def test_oracle_tolerances_hold_for_fp32():
    """The formulas in fp32, as a kernel computes them, lie within the tolerances; a mistake of one part in 2^20 does not."""
    rng = np.random.default_rng(1)
    T = (rng.integers(0, 3, (64, 512)) - 1).astype(np.int8)
    S = rng.uniform(0.5, 1.5, (64, 4)).astype(np.float32) / 18
    q = np.clip(np.rint(rng.standard_normal((20, 512)) * 36), -127, 127).astype(np.int8)
    s_a = np.exp(rng.standard_normal(20) * 3).astype(np.float32) / 36
    f = np.float32
    for act in lo.ACTS:
        for gated in (False, True):
            want, tol = lo.linear(T, S, q, s_a, None, act, gated, None, torch.float32)
            z = np.zeros((20, 64), f)
            for b in range(4):
                z += (q[:, 128 * b: 128 * b + 128].astype(f) @ T[:, 128 * b: 128 * b + 128].astype(f).T) * S[:, b]
            z = z * s_a[:, None]
            g, u = (z[:, :32], z[:, 32:]) if gated else (z, None)
            with np.errstate(over="ignore"):
                c = f(1.5957691216057308) * (g + f(0.044715) * g * g * g) if act == "gelu" else g
                a = {"none": g, "relu": np.maximum(g, 0), "relu2": np.maximum(g, 0) ** 2}.get(act, g / (f(1) + np.exp(-c)))
            y = a * u if gated else a
            assert lo.close(torch.from_numpy(y), want, tol)
            with pytest.raises(AssertionError):
                lo.close(torch.from_numpy(y * f(1 + 2.0 ** -17)), want, tol)


def test_oracle_norm_is_the_formula():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 320)).astype(np.float32)
    w = rng.random(320).astype(np.float32)
    add = rng.standard_normal((9, 320)).astype(np.float32)
    slots, gates = rng.integers(-1, 9, (7, 3)).astype(np.int32), rng.random((7, 3)).astype(np.float32)
    stream, h, codes, s_a = lo.add_norm(x, w, 1e-5, torch.float32, add, slots, gates)
    v = x.astype(np.float64) + sum(np.where(slots[:, j, None] >= 0, gates[:, j, None].astype(np.float64) * add[slots[:, j]], 0) for j in range(3))
    assert np.abs(stream - v).max() < 1e-6
    y = v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-5) * w
    assert np.abs(h - y).max() < 1e-5
    assert np.abs(codes * s_a[:, None].astype(np.float64) - y).max() <= 0.5001 * s_a.max()


def test_oracle_route_is_the_definition():
    rng = np.random.default_rng(3)
    logits = rng.integers(-3, 4, (50, 9)).astype(np.float32)
    logits[rng.random((50, 9)) < 0.5] = -np.inf
    chosen, gates, starts, rows, slots = lo.route(logits, 4, False)
    for t in range(50):
        order = sorted((e for e in range(9) if logits[t, e] > -np.inf), key=lambda e: (-logits[t, e], e))[:4]
        assert chosen[t].tolist() == order + [-1] * (4 - len(order))
        w = np.exp(logits[t, order].astype(np.float64))
        assert np.allclose(gates[t, : len(order)], w / max(w.sum(), 1e-300)) and not gates[t, len(order):].any()
        for j, e in enumerate(order):
            assert starts[e] <= slots[t, j] < starts[e + 1] and rows[slots[t, j]] == t
    for e in range(9):
        assert (np.diff(rows[starts[e]: starts[e + 1]]) > 0).all()
    assert (rows[starts[-1]:] == -1).all() and starts[-1] == (chosen >= 0).sum()
