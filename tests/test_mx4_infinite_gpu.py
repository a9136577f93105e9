"""Infinite tokens of a layer with 4-bit weights: outputs as the sum has them, infinite or (with a weight of zero or
infinities of both signs) NaN."""
import math

import pytest
import torch

from recurrent_oracle import mx4_pack, mx4_values
from seq_oracle import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,C,K,act", [(1, 64, 40, "none"), (6, 288, 33, "relu"), (13, 512, 64, "none"), (30, 96, 70, "relu6"),
                                       (20, 64, 48100, "none"), (16, 128, 20000, "none")])
def test_infinite_tokens(dtype, M, C, K, act):
    import depthwise_pointwise_convolution_amd as F
    g = torch.Generator().manual_seed(M + C + K)
    codes = torch.randint(0, 16, (K, C), generator=g)
    scales = torch.randint(120, 128, (K, C // 32), generator=g)
    x = torch.randn(M, C, generator=g).to(TYPES[dtype])
    y, z = (torch.empty(M, K, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    w, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    p = F.mx4_problem(dtype, M, C, K, act=act)
    F.fcm_mx4_fwd(p, x.cuda(), w, ws, None, z)
    x[0, C // 3] = math.inf
    bad = {0}
    if M > 4:  # one more of the other sign, one of both
        x[3, C - 1], x[4, 0], x[4, 5] = -math.inf, math.inf, -math.inf
        bad |= {3, 4}
    F.fcm_mx4_fwd(p, x.cuda(), w, ws, None, y)
    torch.cuda.synchronize()
    rest = [i for i in range(M) if i not in bad]
    assert torch.equal(y[rest], z[rest])
    want = x[list(bad)].double() @ mx4_values(codes, scales).t()
    if act != "none":
        want = want.clamp(min=0)
    if act == "relu6":
        want = want.clamp(max=6)
    got = y[list(bad)].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=-1.0, posinf=1e30, neginf=-1e30), want.nan_to_num(nan=-1.0, posinf=1e30, neginf=-1e30))
