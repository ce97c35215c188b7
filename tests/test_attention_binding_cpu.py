"""The binding of the attention side on the host: counts and streams that must not reach the library."""
import pytest

import bit_gemv_i2_amd as bn

OUTSIDE = (1 << 31, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 32) + 5, -(1 << 32) + 64, (1 << 32) + 64)


def _host():
    import torch
    return dict(k=torch.zeros((8, 2, 16, 64), dtype=torch.int8), v=torch.zeros((8, 2, 64, 16), dtype=torch.int8),
                ks=torch.zeros((8, 2)), vs=torch.zeros((8, 2)), table=torch.zeros((3, 4), dtype=torch.int32))


@pytest.mark.parametrize("n", OUTSIDE)
def test_bounds_outside_32_bits_on_either_side(n):
    """ctypes keeps the low 32 bits of an int without a word: -2^32 + 5 would become a bound of 5."""
    import torch
    h, i3 = _host(), torch.zeros(3, dtype=torch.int32)
    b = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="max_len must"):
        bn.bitnet_attn_decode(torch.zeros(3, 4, 64), *h.values(), i3, n)
    with pytest.raises(ValueError, match="max_len must"):
        bn.bitnet_attn_prompt(b, b, b, i3, n)
    with pytest.raises(ValueError, match="max_new must"):
        bn.bitnet_rope_append_kv(torch.zeros(5, 8 * 64), None, *h.values(), i3, i3, n, 4)


@pytest.mark.parametrize("n", OUTSIDE)
def test_sizes_outside_32_bits(n):
    for args in ((n, 4, 2, 64, 5000), (3, n, 2, 64, 5000), (3, 4, n, 64, 5000), (3, 4, 2, n, 5000), (3, 4, 2, 64, n)):
        with pytest.raises(ValueError, match="must be below"):
            bn.bitnet_attn_decode_workspace_bytes(*args)
    for args in ((4, n, 64, 16), (4, 2, n, 16), (4, 2, 64, n)):
        with pytest.raises(ValueError, match="must be below"):
            bn.bitnet_kv_cache_bytes(*args)
    with pytest.raises((ValueError, bn.BitnetError)):
        bn.bitnet_rope_table(4, n)
    for trained in (1 << 63, 1 << 64, -(1 << 63) - 1):
        with pytest.raises(ValueError, match="trained"):
            bn.bitnet_rope_table(4, 16, trained=trained)


def test_negative_counts_inside_32_bits_are_refused_by_the_library():
    assert bn.bitnet_kv_cache_bytes(4, -2, 64, 16) == 0
    assert bn.bitnet_attn_decode_workspace_bytes(3, 4, 2, 64, -(1 << 31)) == 0


def test_a_launch_stream_is_of_the_tensors_device(monkeypatch):
    """A launch on another device's stream would run there, on addresses of this one."""
    import types

    import torch

    def stream(index):
        return types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=0x1234)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    assert bn._launch_stream(torch, stream(1), 1) == 0x1234
    with pytest.raises(ValueError, match="the stream is of device 0"):
        bn._launch_stream(torch, stream(0), 1)
    with pytest.raises(ValueError, match="the current device is 1"):
        bn._launch_stream(torch, stream(0), 0)
