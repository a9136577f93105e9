"""Pieces of 32-bit values are the nearest ones: what they leave out of a sum has no sign."""
import pytest
import torch

from gpu_util import gpu_available
from recurrent_oracle import delta
from test_delta_gpu import _call, _inputs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def test_outputs_of_positive_sums_are_not_too_small():
    # Every product is positive, so that errors of one sign would add up.  The mean of 17000 roundings to fp16, each below
    # 2^-11 of the value and as often up as down, has a standard deviation below 2^-11 / sqrt(3 * 17000) = 2.2e-6; that of
    # the left out products, 3 * 2^-16 at most each and 64 of them a sum, is below 3.3e-6 for one output and averages out
    # over the tokens.  Pieces cut towards zero leave 2^-15 = 3e-5 and more.
    T, Hv, Dk, Dv = 130, 2, 64, 64
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
    assert off.abs() <= 1.5e-5, float(off)
