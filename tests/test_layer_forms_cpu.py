"""Refusals of the operators between a decoder layer's products that concern operands given twice.  They are made before any HIP call."""
import ctypes

import bit_gemv_i2_amd as bn

X, ADD, OUT, Q, H = (ctypes.c_void_p(0x100000 * i) for i in range(1, 6))
BF16, F32 = bn.BITNET_DT_BF16, bn.BITNET_DT_F32


def _norm(x=X, xdt=F32, add=None, x_out=None, h=H, hdt=F32, eps=1e-5):
    return bn.lib().bitnet_add_norm(x, xdt, add, BF16, 0, None, None, 0, None, eps, 3, 256, x_out, Q, Q, h, hdt, None)


def test_norm_refuses_h_over_what_it_cannot_replace():
    assert _norm(add=ADD, x_out=OUT, h=OUT) == bn.BITNET_ERR_INVALID_ARG  # both outputs in one place
    assert _norm(add=ADD, x_out=X, h=X) == bn.BITNET_ERR_INVALID_ARG
    for xdt, hdt in ((F32, BF16), (BF16, F32)):  # rows of two sizes
        assert _norm(xdt=xdt, h=X, hdt=hdt) == bn.BITNET_ERR_INVALID_ARG
        assert _norm(xdt=xdt, add=ADD, x_out=OUT, h=X, hdt=hdt) == bn.BITNET_ERR_INVALID_ARG
