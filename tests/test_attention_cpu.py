"""The attention side without a GPU: the rotary table and the cache's size against plain formulas, and every refusal,
made before any HIP call (no kernel is launched here)."""
import ctypes
import math

import numpy as np
import pytest

import attn_oracle as ao
import bit_gemv_i2_amd as bn

FAKE, MIS, MIS4, NULL = (ctypes.c_void_p(x) for x in (0x100000, 0x100004, 0x100002, 0))
OK, ARG, SHAPE = bn.BITNET_OK, bn.BITNET_ERR_INVALID_ARG, bn.BITNET_ERR_UNSUPPORTED_SHAPE


# ------------------------------------------------------------------ host functions
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
def test_rope_table_is_the_formula_rounded_once(rot):
    t = bn.bitnet_rope_table(3000, rot, 500000.0)
    for p in (0, 1, 7, 100, 2999):
        for j in (0, 1, rot // 4, rot // 2 - 1):
            a = p * 500000.0 ** (-2.0 * j / rot)
            # the angle is off by a few ulp of 64 bits, p * 2^-52 at most: far below half an ulp of 32 bits but for ties
            assert abs(float(t[p, j]) - math.cos(a)) <= 2.0 ** -25 + 1e-12
            assert abs(float(t[p, rot // 2 + j]) - math.sin(a)) <= 2.0 ** -25 + 1e-12


def test_rope_table_interpolated():
    rot, base = 64, 10000.0
    plain = bn.bitnet_rope_table(4000, rot, base)
    slow = bn.bitnet_rope_table(4000, rot, base, factor=4.0)
    assert np.abs(slow[::4] - plain[:1000]).max() <= 2.0 ** -24  # position 4p is where p was
    parts = bn.bitnet_rope_table(4000, rot, base, factor=4.0, trained=2048)
    for j in range(rot // 2):
        r = base ** (-2.0 * j / rot)
        turns = 2048 * r / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        a = 3999 * r * (keep + (1 - keep) / 4)
        assert abs(float(parts[3999, j]) - math.cos(a)) <= 2.0 ** -25 + 1e-11
    assert np.array_equal(parts[:, 0], plain[:, 0])                       # the fastest pair is left alone
    assert np.array_equal(parts[:, rot // 2 - 1], slow[:, rot // 2 - 1])  # the slowest is stretched in full


def test_rope_table_refusals():
    f = bn.lib().bitnet_rope_table
    out = np.empty(4096, np.float32)
    p = out.ctypes.data_as(ctypes.c_void_p)
    assert f(4, 64, 1e4, 1.0, 0, NULL) == ARG
    for base, factor, trained in ((1.0, 1.0, 0), (math.nan, 1.0, 0), (math.inf, 1.0, 0), (1e4, 0.5, 0), (1e4, math.nan, 0),
                                  (1e4, math.inf, 0), (1e4, 1.0, -1)):
        assert f(4, 64, base, factor, trained, p) == ARG
    for n, rot in ((0, 64), (-1, 64), (4, 0), (4, 8), (4, 24), (4, 144), (4, -16)):
        assert f(n, rot, 1e4, 1.0, 0, p) == SHAPE
    assert f(4, 64, 1e4, 1.0, 0, p) == OK
    with pytest.raises(bn.BitnetError):
        bn.bitnet_rope_table(0, 64)


def test_kv_cache_bytes():
    assert bn.bitnet_kv_cache_bytes(10, 5, 128, 64) == 10 * 5 * 128 * 64
    assert bn.bitnet_kv_cache_bytes(1 << 30, 8, 128, 128) == (1 << 30) * 8 * 128 * 128
    for bad in ((0, 5, 128, 64), (10, 0, 128, 64), (10, 5, 96, 64), (10, 5, 128, 48), (10, 5, 128, 8), (10, 5, 256, 64)):
        assert bn.bitnet_kv_cache_bytes(*bad) == 0


def test_oracle_append_matches_a_plain_64_bit_turn():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64)).astype(np.float32)
    rope = bn.bitnet_rope_table(5, 32)
    for interleaved in (False, True):
        y = ao.turn32(x, rope, 32, interleaved).astype(np.float64)
        i0 = np.arange(0, 32, 2) if interleaved else np.arange(16)
        i1 = i0 + (1 if interleaved else 16)
        z = (x[..., i0] + 1j * x[..., i1].astype(np.float64)) * (rope[:, None, :16] + 1j * rope[:, None, 16:].astype(np.float64))
        assert np.abs(y[..., i0] - z.real).max() < 1e-6 and np.abs(y[..., i1] - z.imag).max() < 1e-6
        assert np.array_equal(y[..., 32:], x[..., 32:])


# ------------------------------------------------------------------ refusals of the C entries
def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, table=FAKE, pages=8, kv_heads=2, head_dim=64, page=16, batch=3,
             slots=4)
    d.update(kw)
    return bn.KVCacheStruct(*(d[n] for n, _ in bn.KVCacheStruct._fields_))


BAD_CACHES = [(dict(k=NULL), ARG), (dict(v=MIS), ARG), (dict(k_scale=NULL), ARG), (dict(v_scale=MIS4), ARG), (dict(table=NULL), ARG),
              (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE),
              (dict(page=24), SHAPE), (dict(page=256), SHAPE), (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE),
              (dict(slots=0), SHAPE), (dict(slots=1 << 28), SHAPE), (dict(slots=(1 << 26) + 1), SHAPE)]


def _append(cache=None, **kw):
    a = dict(qkv=FAKE, dt=0, row_stride=8 * 64, rope=FAKE, rope_rows=64, rot=64, interleaved=0, starts=FAKE, before=FAKE,
             tokens=5, max_new=5, q_heads=4, cache=ctypes.byref(cache or _cache()), q_out=FAKE, k_out=NULL, stream=NULL)
    a.update(kw)
    return bn.lib().bitnet_rope_append_kv(*a.values())


def test_append_refusals():
    for kw, want in BAD_CACHES:
        assert _append(_cache(**kw)) == want, kw
    assert _append(cache=None, qkv=NULL) == ARG
    for kw in (dict(qkv=MIS), dict(q_out=NULL), dict(q_out=MIS), dict(k_out=MIS), dict(starts=NULL), dict(before=MIS4),
               dict(rope=NULL), dict(rope=MIS), dict(dt=2), dict(dt=-1)):
        assert _append(**kw) == ARG, kw
    for kw in (dict(row_stride=8 * 64 - 8), dict(row_stride=8 * 64 + 4), dict(rope_rows=63), dict(rot=24), dict(rot=80),
               dict(rot=-16), dict(tokens=0), dict(tokens=(1 << 24) + 1), dict(max_new=0), dict(q_heads=0), dict(q_heads=3),
               dict(q_heads=1026)):
        assert _append(**kw) == SHAPE, kw
    assert bn.lib().bitnet_rope_append_kv(FAKE, 0, 512, FAKE, 64, 64, 0, FAKE, FAKE, 5, 5, 4, NULL, FAKE, NULL, NULL) == ARG


def _decode(cache=None, **kw):
    a = dict(q=FAKE, qdt=0, q_stride=4 * 64, cache=ctypes.byref(cache or _cache()), lengths=FAKE, max_len=64, q_heads=4,
             scale=0.125, out=FAKE, odt=0, workspace=NULL, nbytes=0, stream=NULL)
    a.update(kw)
    return bn.lib().bitnet_attn_decode(*a.values())


def test_decode_refusals():
    for kw, want in BAD_CACHES:
        assert _decode(_cache(**kw)) == want, kw
    for kw in (dict(q=NULL), dict(q=MIS), dict(lengths=NULL), dict(out=MIS), dict(qdt=2), dict(odt=7), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf)):
        assert _decode(**kw) == ARG, kw
    assert bn.lib().bitnet_attn_decode(FAKE, 0, 256, NULL, FAKE, 64, 4, 0.125, FAKE, 0, NULL, 0, NULL) == ARG
    for kw in (dict(q_stride=4 * 64 - 8), dict(q_stride=4 * 64 + 4), dict(max_len=0), dict(max_len=2 ** 31 - 1), dict(q_heads=5),
               dict(q_heads=2048)):
        assert _decode(**kw) == SHAPE, kw
    need = bn.bitnet_attn_decode_workspace_bytes(1, 4, 1, 64, 100000)
    assert need > 0 and need % 4 == 0
    c = _cache(batch=1, kv_heads=1, slots=6250)
    for kw in (dict(), dict(workspace=FAKE, nbytes=need - 1), dict(workspace=ctypes.c_void_p(0x100010), nbytes=need)):
        assert _decode(c, max_len=100000, **kw) == ARG, kw


def test_decode_workspace_bytes():
    f = bn.bitnet_attn_decode_workspace_bytes
    assert f(1, 4, 1, 64, 1) == 0  # one workgroup a head: nothing to join
    for bad in ((0, 4, 1, 64, 10), (1, 5, 2, 64, 10), (1, 4, 1, 80, 10), (1, 4, 1, 64, 0), (65536, 4, 1, 64, 10)):
        assert f(*bad) == 0
    for n in (1000, 10000, 131072):
        need = f(2, 20, 5, 128, n)
        assert need % (2 * 20 * 130 * 4) == 0  # whole splits of (sums, maximum, weight)


def _prompt(**kw):
    a = dict(q=FAKE, qs=4 * 64, k=FAKE, ks=128, v=FAKE, vs=128, starts=FAKE, batch=2, tokens=50, max_len=30, q_heads=4, kv_heads=2,
             head_dim=64, causal=1, scale=0.125, out=FAKE, stream=NULL)
    a.update(kw)
    return bn.lib().bitnet_attn_prompt(*a.values())


def test_prompt_refusals():
    for kw in (dict(q=NULL), dict(k=MIS), dict(v=NULL), dict(out=NULL), dict(starts=MIS4), dict(scale=0.0), dict(scale=math.nan)):
        assert _prompt(**kw) == ARG, kw
    for kw in (dict(qs=248), dict(qs=260), dict(ks=120), dict(vs=132), dict(batch=0), dict(batch=65536), dict(tokens=0),
               dict(tokens=(1 << 22) + 1), dict(qs=(1 << 23) + 8), dict(vs=(1 << 23) + 8), dict(max_len=0), dict(q_heads=3), dict(kv_heads=0),
               dict(head_dim=32), dict(head_dim=256), dict(batch=65535, tokens=1 << 22, max_len=1 << 22)):
        assert _prompt(**kw) == SHAPE, kw


# ------------------------------------------------------------------ refusals of the binding, on host tensors
def _host():
    import torch
    return dict(k=torch.zeros((8, 2, 16, 64), dtype=torch.int8), v=torch.zeros((8, 2, 64, 16), dtype=torch.int8),
                ks=torch.zeros((8, 2)), vs=torch.zeros((8, 2)), table=torch.zeros((3, 4), dtype=torch.int32))


@pytest.mark.parametrize("name,change", [("k", lambda t: t[:, :, :, :32]), ("k", lambda t: t.float()), ("v", lambda t: t.transpose(2, 3)),
                                         ("ks", lambda t: t[:7]), ("vs", lambda t: t.double()), ("table", lambda t: t.long()),
                                         ("table", lambda t: t[0])])
def test_binding_checks_the_cache(name, change):
    import torch
    h = _host()
    h[name] = change(h[name])
    with pytest.raises(ValueError):
        bn.bitnet_attn_decode(torch.zeros(3, 4, 64), *h.values(), torch.zeros(3, dtype=torch.int32), 10)
    with pytest.raises(ValueError):
        bn.bitnet_rope_append_kv(torch.zeros(3, 512), None, *h.values(), torch.zeros(4, dtype=torch.int32),
                                 torch.zeros(3, dtype=torch.int32), 1, 4)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    h = _host()
    i3, i4 = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        bn.bitnet_attn_decode(torch.zeros(3, 4, 64), *h.values(), i3, 10)
    b = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        bn.bitnet_attn_prompt(b, b[:, :2], b[:, :2], i4, 5)
    for args in ((b.float(), b, b, i4), (b, b[:4], b, i4), (b, b, b[:, :2], i4), (b, b, b, i4.long()), (b, b, b, i4[:1]),
                 (b[0], b, b, i4)):
        with pytest.raises(ValueError):
            bn.bitnet_attn_prompt(*args, 5)
    with pytest.raises(bn.BitnetError):
        bn.KVCache.empty(4, 2, 80, device="cpu")
    c = bn.KVCache.empty(4, 2, 64, 16, device="cpu")
    assert c.k.numel() == c.v.numel() == bn.bitnet_kv_cache_bytes(4, 2, 64, 16)


def test_binding_refuses_counts_past_32_bits():
    """ctypes keeps the low 32 bits of an int without a word: 2^32 + 5 would become a bound of 5."""
    import torch
    h, i3 = _host(), torch.zeros(3, dtype=torch.int32)
    b = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    for n in (1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="max_len"):
            bn.bitnet_attn_decode(torch.zeros(3, 4, 64), *h.values(), i3, n)
        with pytest.raises(ValueError, match="max_len"):
            bn.bitnet_attn_decode_workspace_bytes(3, 4, 2, 64, n)
        with pytest.raises(ValueError, match="max_len"):
            bn.bitnet_attn_prompt(b, b, b, i3, n)
        with pytest.raises(ValueError, match="max_new"):
            bn.bitnet_rope_append_kv(torch.zeros(5, 8 * 64), None, *h.values(), i3, i3, n, 4)


def test_rows_may_be_slices_of_wider_rows_but_not_strided_inside():
    import torch

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0
    t = torch.zeros(6, 4, 64).as_subclass(OnDevice)
    assert bn._rows_ptr(t, "t", 256, 0)[1] == 256
    assert bn._rows_ptr(t[:1], "t", 256, 0)[1] == 256
    assert bn._rows_ptr(t[:, :2], "t", 128, 0)[1] == 256
    for bad in (t[:, ::2], t[:, :, ::2], t.transpose(1, 2)):
        with pytest.raises(ValueError):
            bn._rows_ptr(bad, "t", 128, 0)
    with pytest.raises(ValueError, match="other tensors"):
        bn._rows_ptr(t, "t", 256, 1)
