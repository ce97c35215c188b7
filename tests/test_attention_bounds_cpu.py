"""The bounds that decode attention is held to: the kernel's digits keep them, fewer do not."""
import numpy as np
import pytest

import attn_bounds as ab
import attn_oracle as ao


def _case(rng, page=32):
    c = ao.Cache(30, 2, 64, page, rng)
    q = (rng.standard_normal((2, 4, 64)) * 1.5).astype(np.float32).astype(np.float64)
    return q, c, rng.permutation(30).reshape(2, 15), [300, 77], 0.125


@pytest.mark.parametrize("seed", range(3))
def test_fewer_digits_break_the_bounds(seed):
    case = _case(np.random.default_rng(seed))
    for bound in (ab.decode(*case), ao.decode(*case, True, 30)):
        want, tol = bound
        assert np.all(np.abs(ab.emulate(*case) - want) <= tol)
        for fewer in (dict(weight_unit=127 * 256), dict(q_bits=22, weight_unit=127 * 256)):
            assert not np.all(np.abs(ab.emulate(*case, **fewer) - want) <= tol), fewer


@pytest.mark.parametrize("seed", range(3))
def test_fewer_digits_break_the_bounds_of_a_bf16_output(seed):
    """Through the rounding to bf16: the band is that of the output, not of a coarser weight."""
    case = _case(np.random.default_rng(10 + seed))
    want, tol = ao.decode(*case, True, 30)
    assert ao.within(ao._bf16(ab.emulate(*case)), want, tol, True)[0]
    assert not ao.within(ao._bf16(ab.emulate(*case, weight_unit=127)), want, tol, True)[0]
    assert not ao.within(ao._bf16(ab.emulate(*case, weight_unit=127 * 16)), want, tol, True)[0]


def test_the_unit_is_of_the_largest_product_not_of_the_largest_scale():
    rng = np.random.default_rng(5)
    c = ao.Cache(4, 1, 64, 16, rng)
    c.ks[:], c.vs[:], c.vs[1] = 0.02, 0.03, 3e4
    c.k[:, :, :, 0], c.k[1, :, :, 0] = 100, -68
    q = rng.standard_normal((1, 2, 64)) * 0.3
    q[..., 0] = 42 / (168 * 0.02 * 0.125)
    case = (q, c, np.arange(4)[None], [64], 0.125)
    want, tol = ab.decode(*case)
    assert np.all(np.abs(ab.emulate(*case) - want) <= tol)
    # the largest scale as the measure: a unit 1e6 times as large
    assert not np.all(np.abs(ab.emulate(*case, weight_unit=127 * 65536 / 1e6) - want) <= tol)
