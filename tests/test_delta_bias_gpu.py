"""Pieces of 32-bit values are the nearest ones: what they leave out of a sum has no sign."""
import pytest
import torch

from gpu_util import gpu_available
from recurrent_oracle import delta
from test_delta_gpu import _call, _inputs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def test_outputs_of_positive_sums_are_not_too_small():
    # Every product is positive, so that errors of one sign would add up.  The mean of 133000 roundings to fp16, each below
    # 2^-11 of the value and as often up as down, has a standard deviation below 2^-11 / sqrt(3 * 133000) = 7.7e-7; that of
    # the 150000 states' missing thirds, each below 2^-16, is below 2^-16 / sqrt(3 * 150000) = 2.3e-8.  Five of the first
    # and the second are 4e-6.  Pieces cut towards zero miss half of 2^-15 of a state on average, 1e-5 and more.
    T, Hv, Dk, Dv = 520, 4, 64, 64
    c = _inputs(11, "f16", T, 1, 1, Hv, Dk, Dv, 1)
    for n in ("q", "k", "v", "state"):
        c[n] = c[n].abs()
    c["state"] += 1
    c["b"][:] = -6.0
    c["A"][:] = -1e-3
    c["norm"] = c["z"] = None
    got, _, spans = _call(c, "f16", [T], [0], [1], 1, Hv, Dk, Dv, {})
    y, *_ = delta("f16", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], None, None, spans, [0], [1], c["state"],
                  Dk ** -0.5, 1e-6)
    assert (y > 0).all()
    off = ((got.double().reshape(T, Hv, Dv) - y) / y).mean()
    print("mean relative error", float(off))
    assert off.abs() <= 4e-6, float(off)
