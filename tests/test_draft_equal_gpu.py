"""Drafted tokens that do not stand although the draft's row is the target's: the next one is drawn from the target's."""
import math

import pytest
import torch

from gpu_util import gpu_available
from test_draft_gpu import _compare, _inputs, _run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V,heat", [(5, 1.0), (300, 0.7), (4099, 1.3), (151936, 1.0)])
def test_equal_rows(dtype, V, heat):
    B, N = 8, 2
    target, _, tokens, uniform = _inputs(V, dtype, B, N, V, heat)
    target[:, :, V // 2] = -math.inf
    draft = target[:, :N].clone()
    tokens[:, 0] = torch.tensor([V // 2, V // 2, V // 2, V // 2, -1, V, V // 2, V // 2])  # masked in both, or none
    uniform[:, N] = torch.tensor([0.0, 0.1, 0.37, 0.5, 0.63, 0.8, 0.99, 1.0 - 2.0 ** -24])
    got = _run(dtype, target, draft, tokens, None, uniform, heat, pad=V % 2)
    assert all(n == 0 for n, _ in got)
    _compare(got, target, draft, tokens, None, uniform, heat)
    # (drawn from p: what stands below the token has at most r of the sum, with it more)
    for r, (_, t) in enumerate(got):
        p = torch.softmax(target[r, 0].double() / heat, 0).cumsum(0)
        share = float(uniform[r, N]) * float(p[-1])
        assert (t == 0 or p[t - 1] <= share + 1e-10) and p[t] >= share - 1e-10
