"""Weights with the smallest and largest scales: single products, exactly."""
import pytest
import torch

from gpu_util import gpu_available
from recurrent_oracle import mx4_pack, mx4_quantize, mx4_values
from seq_oracle import TYPES

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("dtype,powers", [("bf16", (0, 100, -100)), ("f16", (0, 15, -14))])
@pytest.mark.parametrize("scale", [0, 1, 2, 3, 127, 252, 253, 254])
def test_single_products(both, dtype, powers, scale):
    import depthwise_pointwise_convolution_amd as F
    codes = torch.zeros(16, 32, dtype=torch.int64)
    codes[:, 0] = torch.arange(16)  # one channel's weights are all there are
    scales = torch.full((16, 1), scale)
    x = torch.zeros(len(powers), 32)
    x[:, 0] = torch.exp2(torch.tensor(powers).float())
    p = F.mx4_problem(dtype, len(powers), 32, 16)
    y = torch.empty(len(powers), 16, dtype=TYPES[dtype], device="cuda")
    w, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    if both:
        xc, xs = mx4_quantize(x)
        F.fcm_mx4x4_fwd(p, mx4_pack(xc).cuda(), xs.to(torch.uint8).cuda(), w, ws, None, y)
    else:
        F.fcm_mx4_fwd(p, x.to(TYPES[dtype]).cuda(), w, ws, None, y)
    torch.cuda.synchronize()
    value = mx4_values(codes, scales)[:, 0]
    want = (x[:, :1].double() * value).to(TYPES[dtype])
    got = y.cpu()
    large = value.abs() >= 2.0 ** 128
    if not both:
        assert not torch.isfinite(got[:, large].float()).any()
        got, want = got[:, ~large], want[:, ~large]
    assert torch.equal(got, want)  # (a power of two times a code: exact, or rounded once where it is subnormal)
