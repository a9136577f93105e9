"""Rows of fewer than eight scales, whose tiles load bytes that no step uses: those lie within an array of the call,
however few rows the other side has."""
import os
import re

import pytest
import torch

from gpu_util import gpu_available
from recurrent_oracle import mx4_pack, mx4_values, product


def _source():
    import depthwise_pointwise_convolution_amd as F
    with open(os.path.join(os.path.dirname(F.__file__), "csrc", "kernels", "mx4.hip")) as f:
        return re.sub(r"\s+", " ", f.read())


@pytest.mark.parametrize("blocks", range(1, 8))
def test_bytes_that_no_step_uses_are_inside(blocks):
    # a side's rows are at most 128 a tile, each read from row * blocks on
    source = _source()
    held = {"a.q": lambda M, K: 16 * blocks * K, "(const uint8_t*)a.x": lambda M, K: 16 * blocks * M}
    assert "(uint32_t)(r < most ? r : most) * (uint32_t)blocks + at)" in source and "some ? blocks - 8 : 0" in source
    for name, rows in (("kscales", lambda M, K: K), ("mscales", lambda M, K: M)):
        base = re.search(r"const uint8_t\* %s = some \? [^:]* : ([^;]*);" % name, source).group(1)
        for K in (1, 2, 3, 4, 8, 9, 64, 200):
            for M in (33, 40, 127, 128, 600000):
                last = min(rows(M, K), 128) - 1
                assert last * blocks + 8 <= held[base](M, K), (name, base, M, K)


@pytest.mark.gpu
@pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")
@pytest.mark.parametrize("M,C,K", [(262200, 224, 4), (349600, 160, 3), (131100, 32, 8), (524300, 192, 2)])
def test_many_tokens_of_few_outputs(M, C, K):
    import depthwise_pointwise_convolution_amd as F
    g = torch.Generator().manual_seed(M + C + K)
    codes, xcodes = (torch.randint(0, 16, (n, C), generator=g) for n in (K, M))
    scales, xscales = (torch.randint(119, 131, (n, C // 32), generator=g) for n in (K, M))
    y = torch.full((M + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fcm_mx4x4_fwd(F.mx4_problem("bf16", M, C, K), mx4_pack(xcodes).cuda(), xscales.to(torch.uint8).cuda(),
                    mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda(), None, y)
    torch.cuda.synchronize()
    want, tol = product("bf16", mx4_values(xcodes, xscales), mx4_values(codes, scales), None, "none")
    assert ((y[:M].cpu().double() - want).abs() <= tol).all()
    assert (y[M] == 7.0).all()
