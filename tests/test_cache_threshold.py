"""The smallest row that the state cache keeps (CPU, the oracle's fp32): at its
bound of 2^-118 the factor of both formats is finite, and finite down to the
bounds that the header gives."""
import numpy as np
import pytest

from oracle import delta as od

f = np.float32


@pytest.mark.parametrize("form,top,least", [("int8", 127, -121.0), ("e4m3", 448, -119.2)])
def test_bound(form, top, least):
    def factor(a):
        with np.errstate(over="ignore"):
            return (f(1) / f(a)) * f(top)
    assert np.isfinite(factor(2.0 ** -118))
    assert np.isfinite(factor(2.0 ** (least + 0.02))) and not np.isfinite(factor(2.0 ** (least - 0.02)))
    x = np.full((1, 1, 2, 4), 2.0 ** -118, f)
    x[0, 0, 1] = np.nextafter(f(2.0 ** -118), f(0))
    back, scale = od.cache_roundtrip(x, form)
    assert np.allclose(back[0, 0, 0], x[0, 0, 0], rtol=1e-6) and scale[0, 0, 0] > 0
    assert not back[0, 0, 1].any() and scale[0, 0, 1] == 0
