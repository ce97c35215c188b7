"""The forms of the operators between a decoder layer's products that a launch takes at sizes of its own: tiles beyond one round of
compute units, streams of weights through several row tiles, columns taken in turns, rows of a norm on a wave each.  Oracles and
tolerances are those of layer_oracle."""
import numpy as np
import pytest

import layer_oracle as lo
import test_gpu_layer as layer

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ tiles: more of them than compute units (256)
def _tiles(M, N):
    return -(-M // 64) * -(-N // 256)


@pytest.mark.parametrize("M,N", [(1024, 4096), (1025, 4096), (16384, 256), (16385, 256), (64, 65536), (65, 65536)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_on_either_side_of_the_compute_units(gpu, M, N, gated):
    assert (_tiles(M, N) > 256) == (M % 2 == 1)
    layer._linear_case(np.random.default_rng(M), M, N, 128, "relu", gated, True, "fp32", "bf16")


@pytest.mark.parametrize("act", lo.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_linear_many_tiles_activations(gpu, act, gated):
    i = lo.ACTS.index(act)
    M, N = 1087 + i, 4128  # a last token tile that is not full, row tiles of which the last has 32 rows
    assert _tiles(M, N) > 256
    layer._linear_case(np.random.default_rng(i), M, N, 384, act, gated, i % 2 == 0, (None, "bf16", "fp32")[i % 3], ("bf16", "fp32")[i % 2])


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 7, 11])
@pytest.mark.parametrize("M,N", [(1217, 4112), (1281, 4064)])
def test_linear_many_tiles_blocks(gpu, blocks, M, N):
    """Every stage of the loads in turn; bands of four token tiles of which the last has fewer."""
    assert _tiles(M, N) > 256
    layer._linear_case(np.random.default_rng(blocks), M, N, 128 * blocks, "none", False, blocks % 2 == 0, "bf16" if blocks % 3 else None, "fp32")


@pytest.mark.parametrize("out", list(layer.TYPES))
@pytest.mark.parametrize("gated", [False, True])
def test_linear_many_tiles_into_the_residual(gpu, out, gated):
    layer._linear_case(np.random.default_rng(1), 1100, 4160, 256, "silu" if gated else "none", gated, True, out, out, inplace=True)


@pytest.mark.parametrize("M,N,K", [(1090, 4128, 640), (16450, 272, 256)])
def test_linear_many_tiles_whole_numbers_exactly(gpu, M, N, K):
    import bit_gemv_i2_amd as bn
    assert _tiles(M, N) > 256
    rng = np.random.default_rng(M)
    T = (rng.integers(0, 3, (N, K), dtype=np.int8) - 1).astype(np.int8)
    T[0], T[1] = 1, -1
    T[2:18] = 0
    T[2:18][np.arange(16), rng.integers(0, K, 16)] = 1  # a column alone
    q = rng.integers(-128, 128, (M, K), dtype=np.int64).astype(np.int8)
    q[0], q[1], q[-1] = np.arange(K) % 256 - 128, 127, -128
    w = bn.PackedWeight.from_ternary(T, np.ones((N, K // 128), np.float32))
    y = w.linear(layer._dev(q), layer._dev(np.ones(M, np.float32)), out_dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy(), q.astype(np.float32) @ T.astype(np.float32).T)  # sums below 2^24: exact in any order


def test_linear_many_tiles_of_a_token_that_is_not_finite(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(4)
    M, N, K = 1100, 4128, 256
    T, S = layer._weights(rng, N, K)
    q, s_a = layer._acts(rng, M, K)
    bad = [1, 64, 700, M - 1]
    s_a[bad], q[bad] = np.nan, 0
    for act, gated in (("none", False), ("relu2", True)):
        want, tol = lo.linear(T, S, q, np.where(np.isnan(s_a), 1, s_a).astype(np.float32), None, act, gated, None, torch.float32)
        want[bad] = np.nan
        lo.close(bn.PackedWeight.from_ternary(T, S).linear(layer._dev(q), layer._dev(s_a), act=act, gated=gated, out_dtype=torch.float32), want, tol)


@pytest.mark.parametrize("counts", [[300, 0, 517, 64, 1, 190], [1100], [0, 0, 1200, 0], [65] * 20, [1] * 63 + [1400]])
@pytest.mark.parametrize("gated,gather", [(False, False), (True, True)])
def test_grouped_many_tiles(gpu, counts, gated, gather):
    slots, some = sum(counts), min(len(counts), sum(counts))
    N = 4128 if len(counts) < 20 else 2080
    assert slots > 16 * len(counts) and (slots + 63 * some) // 64 * -(-N // 256) > 256
    layer._grouped_case(np.random.default_rng(slots), counts, 333, N, 128, "silu" if gated else "none", gated, gated, gather, "bf16" if gated else "fp32")


def test_grouped_many_tiles_bad_rows_and_rows_of_no_expert_stay(gpu):
    layer._grouped_case(np.random.default_rng(5), [700, 0, 405], 90, 4128, 256, "none", False, True, True, "fp32", slots=1300,
                        bad=[(0, -1), (2, 90), (699, -2 ** 31), (700, 2 ** 31 - 1), (1104, -7), (1200, 2 ** 31 - 1)])


def test_grouped_many_tiles_starts_beyond_the_slots(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(6)
    layer._grouped_case(rng, [300, 5000, 9], 90, 4128, 128, "none", False, False, True, "fp32", slots=1100)
    E, N, slots = 3, 4128, 1100
    T, S = layer._weights(rng, E * N, 128)
    w = bn.PackedExperts.from_ternary(T.reshape(E, N, 128), S.reshape(E, N, 1))
    q, s_a = layer._acts(rng, slots, 128)
    for starts in ([-5, 200, 400, 1 << 30], [1100, 200, 100, 0], [2 ** 31 - 1] * 4, [-2 ** 31, -1, -1, 2 ** 31 - 1], [0, 1100, 200, 1100]):
        y, ok = layer._guarded((slots, N), torch.float32)
        w.grouped(layer._dev(q), layer._dev(s_a), layer._dev(np.array(starts, np.int32)), y=y)
        torch.cuda.synchronize()
        assert ok()


# ------------------------------------------------------------------ few rows each of many experts
def _ragged(E, usual):
    """About `usual` rows an expert, some with none, one, a pass of 16 and more than one."""
    counts = [usual] * E
    for e, n in ((0, 0), (3, 1), (5, 16), (6, 17), (9, 37), (E - 1, usual + 2)):
        counts[e] = n
    assert 4 * E < sum(counts) <= 16 * E
    return counts


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 13, 20, 31, 32])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_stream_blocks(gpu, blocks, gated):
    """Every chunk length and remainder; from 32 blocks on the rows no longer fit and another form takes over."""
    E, N = 64, 512
    assert N // (32 if gated else 16) * E >= 1024
    layer._grouped_case(np.random.default_rng(blocks), _ragged(E, 5), 41, N, 128 * blocks, "relu2" if gated else "none", gated, blocks % 2 == 0,
                        True, "fp32" if blocks % 3 else "bf16")


@pytest.mark.parametrize("E,N,gated", [(64, 1296, False), (64, 1328, False), (64, 2592, True), (64, 2720, True), (16, 4208, False), (1024, 16, False),
                                       (513, 64, True)])
@pytest.mark.parametrize("usual", [5, 12])
def test_grouped_stream_row_tiles(gpu, E, N, gated, usual):
    """Several row tiles a wave, waves that have fewer or none, many experts."""
    assert N // (32 if gated else 16) * E >= 1024
    layer._grouped_case(np.random.default_rng(N), _ragged(E, usual), 97, N, 256 if E == 64 else 128, "silu", gated, usual == 5, usual == 12, "fp32")


@pytest.mark.parametrize("act", lo.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_stream_activations(gpu, act, gated):
    layer._grouped_case(np.random.default_rng(7), _ragged(64, 6), 50, 544, 384, act, gated, True, False, "bf16")


def test_grouped_stream_bad_rows_and_rows_of_no_expert_stay(gpu):
    counts = _ragged(64, 8)
    used = sum(counts)
    layer._grouped_case(np.random.default_rng(8), counts, 30, 512, 640, "none", False, True, True, "fp32", slots=used + 40,
                        bad=[(0, -1), (2, 30), (17, 2 ** 31 - 1), (used - 1, -2 ** 31), (used + 1, 2 ** 31 - 1)])


def test_grouped_stream_of_a_token_that_is_not_finite(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(9)
    E, N, K, usual = 64, 512, 384, 6
    T, S = layer._weights(rng, E * N, K)
    q, s_a = layer._acts(rng, E * usual, K)
    bad = [1, 100, E * usual - 1]
    s_a[bad], q[bad] = np.nan, 0
    starts = np.arange(E + 1, dtype=np.int32) * usual
    got = bn.PackedExperts.from_ternary(T.reshape(E, N, K), S.reshape(E, N, -1)).grouped(layer._dev(q), layer._dev(s_a), layer._dev(starts), out_dtype=torch.float32)
    safe = np.where(np.isnan(s_a), 1, s_a).astype(np.float32)
    for e in range(E):
        at = slice(starts[e], starts[e + 1])
        want, tol = lo.linear(T[e * N: (e + 1) * N], S[e * N: (e + 1) * N], q[at], safe[at], None, "none", False, None, torch.float32)
        want[np.isnan(s_a[at])] = np.nan
        lo.close(got[at], want, tol)


def test_grouped_stream_starts_beyond_the_slots(gpu):
    import bit_gemv_i2_amd as bn
    rng = np.random.default_rng(10)
    E, N, slots = 64, 512, 400
    T, S = layer._weights(rng, E * N, 128)
    w = bn.PackedExperts.from_ternary(T.reshape(E, N, 128), S.reshape(E, N, 1))
    q, s_a = layer._acts(rng, slots, 128)
    for starts in (np.linspace(-50, 1 << 30, E + 1), np.linspace(slots, 0, E + 1), np.full(E + 1, 2 ** 31 - 1), np.resize([0, slots, 9, slots], E + 1)):
        y, ok = layer._guarded((slots, N), torch.float32)
        w.grouped(layer._dev(q), layer._dev(s_a), layer._dev(starts.astype(np.int32)), y=y)
        torch.cuda.synchronize()
        assert ok()


@pytest.mark.parametrize("E,slots,hot", [(64, 900, 450), (64, 1024, 960), (8, 128, 120)])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_one_expert_with_most_of_the_rows(gpu, E, slots, hot, gated):
    """Few rows an expert in the mean, many of one."""
    counts = [0] * E
    counts[2] = hot
    for i in range(slots - hot):
        counts[(5 * i + 7) % E if E == 8 else 3 + i % (E - 3)] += 1
    assert slots == sum(counts) <= 16 * E
    layer._grouped_case(np.random.default_rng(hot), counts, 80, 576, 384, "gelu", gated, False, True, "bf16")


@pytest.mark.parametrize("counts", [[1, 0, 1], [3, 5, 1], [7, 2, 9], [16, 0, 14], [4, 40, 3]])
@pytest.mark.parametrize("blocks", [97, 110])
def test_grouped_columns_in_turns(gpu, counts, blocks):
    """More blocks of columns than the waves hold at once."""
    for gated in (False, True):
        layer._grouped_case(np.random.default_rng(blocks), counts, 11, 64, 128 * blocks, "relu", gated, True, gated, "fp32")


# ------------------------------------------------------------------ a wave a row of a norm
@pytest.mark.parametrize("K", [16, 512, 528, 1040, 1536, 2048, 2064, 2560, 2576, 3056, 3088, 3600, 4096, 4112])
@pytest.mark.parametrize("xt,at,inplace", [("bf16", "bf16", True), ("fp32", "bf16", False), ("bf16", None, False)])
def test_norm_on_a_wave_a_row(gpu, K, xt, at, inplace):
    layer._norm_case(np.random.default_rng(K), 1025, K, xt, at, 0, inplace=inplace)


@pytest.mark.parametrize("M", [1022, 1023, 1024, 1025, 1026, 1027])
def test_norm_rows_on_either_side_of_the_rule(gpu, M):
    layer._norm_case(np.random.default_rng(M), M, 2560, "bf16", "fp32", 0)


@pytest.mark.parametrize("K", [400, 2560, 16400, 32768, 32784, 65536])
@pytest.mark.parametrize("M", [3, 1030])
@pytest.mark.parametrize("added", [False, True])
def test_norm_into_the_stream_it_reads(gpu, K, M, added):
    """h_out is x, with the codes of the same call: they are those of the values that x held."""
    import bit_gemv_i2_amd as bn
    if M * K > 1 << 24:
        M = 2
    rng = np.random.default_rng(K)
    x, xv = layer._values(rng, (M, K), torch.float32)
    add, av = layer._values(rng, (M, K), torch.bfloat16)
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    stream, h, codes, s_a = lo.add_norm(xv, w, 1e-5, torch.float32, av if added else None)
    q, s, out, wd = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(x), layer._dev(w)
    st = bn.lib().bitnet_add_norm(x.data_ptr(), bn.BITNET_DT_F32, add.data_ptr() if added else None, bn.BITNET_DT_BF16, 0, None, None, 0, wd.data_ptr(),
                                  1e-5, M, K, out.data_ptr() if added else None, q.data_ptr(), s.data_ptr(), x.data_ptr(), bn.BITNET_DT_F32,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == bn.BITNET_OK
    assert np.array_equal(s.cpu().numpy(), s_a) and np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(x.cpu().numpy(), h)
    if added:
        assert np.array_equal(out.cpu().numpy(), stream)
