"""Microscaled 4-bit numbers on the GPU: codes and values exactly, products within the roundings of their sums."""
import math

import pytest
import torch

from recurrent_oracle import mx4_pack, mx4_quantize, mx4_unpack, mx4_values, product
from seq_oracle import TYPES

pytestmark = pytest.mark.gpu


def _values(dtype, rows, C, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, C, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x[:, ::5] = (x[:, ::5] * 4).round() / 4  # numbers half-way between two codes
    x[0, :32] = 0
    if rows > 2:
        x[1, :32] *= 1e-30
        x[2, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, -0.25, -0.75, -2.5, -5.0, -0.0,
                                  0.1]).repeat(2)
    return x.to(TYPES[dtype])


def _quantise(x, dtype, pad=0):
    import depthwise_pointwise_convolution_amd as F
    M, C = x.shape
    wide = torch.full((M, C + pad), math.nan, dtype=x.dtype, device="cuda")
    wide[:, :C] = x.cuda()
    q = torch.full((M + 1, C // 2), 0xab, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 1, C // 32), 0xab, dtype=torch.uint8, device="cuda")
    F.fcm_mx4_quantize(F.mx4_problem(dtype, M, C, ldx=C + pad), wide[:, :C], q, s)
    torch.cuda.synchronize()
    assert (q[M] == 0xab).all() and (s[M] == 0xab).all()
    return q[:M].contiguous(), s[:M].contiguous()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,C,pad", [(1, 32, 0), (5, 96, 0), (5, 96, 8), (3, 64, 1), (17, 1056, 0), (130, 256, 3)])
def test_quantised_and_back(dtype, M, C, pad):
    import depthwise_pointwise_convolution_amd as F
    x = _values(dtype, M, C, M + C)
    codes, scales = mx4_quantize(x)
    q, s = _quantise(x, dtype, pad)
    assert torch.equal(s.cpu().long(), scales)
    assert torch.equal(mx4_unpack(q.cpu()), codes)
    for out in ("f32", "f16", "bf16"):
        y = torch.full((M, C + pad), 7.0, dtype=TYPES[out], device="cuda")
        F.fcm_mx4_dequantize(F.mx4_problem(out, M, C, ldy=C + pad), q, s, y)
        torch.cuda.synchronize()
        assert torch.equal(y[:, :C].cpu(), mx4_values(codes, scales).to(TYPES[out]))
        assert (y[:, C:] == 7.0).all()


def test_values_at_the_ends():
    import depthwise_pointwise_convolution_amd as F
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    x = torch.zeros(8, 32)
    x[0] = torch.linspace(-big, big, 32)  # (whose step overflows: not all of it is finite)
    x[1] = torch.arange(32) * tiny
    x[2] = torch.arange(32) * 2.0 ** -127
    x[3, 3] = math.nan
    x[4, 4] = math.inf
    x[5, 5] = -math.inf
    x[6, 0] = 2.0 ** -126
    x[7] = -0.0
    codes, scales = mx4_quantize(x)
    q, s = _quantise(x, "f32")
    assert torch.equal(s.cpu().long(), scales)
    fine = scales[:, 0] != 255
    assert fine.tolist() == [False, True, True, False, False, False, True, True]
    assert torch.equal(mx4_unpack(q.cpu())[fine], codes[fine])
    y = torch.empty(8, 32, device="cuda")
    F.fcm_mx4_dequantize(F.mx4_problem("f32", 8, 32), q, s, y)
    assert torch.equal(y.cpu()[fine].double(), mx4_values(codes, scales)[fine])
    assert torch.isnan(y.cpu()[~fine]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_largest_values(dtype):
    import depthwise_pointwise_convolution_amd as F
    big = torch.finfo(TYPES[dtype]).max
    x = (torch.arange(-16, 16).double() / 16 * big).to(TYPES[dtype]).reshape(1, 32)
    codes, scales = mx4_quantize(x)
    q, s = _quantise(x, dtype)
    assert torch.equal(s.cpu().long(), scales) and torch.equal(mx4_unpack(q.cpu()), codes)
    y = torch.empty(1, 32, device="cuda")
    F.fcm_mx4_dequantize(F.mx4_problem("f32", 1, 32), q, s, y)
    assert torch.equal(y.cpu().double(), mx4_values(codes, scales))


def _weights(K, C, seed, spread=20):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (K, C), generator=g)
    scales = torch.randint(127 - spread, 127 + spread // 2, (K, C // 32), generator=g)
    return codes, scales


def _within(got, want, tol, dtype):
    """(a value from half a step above the type's largest on rounds to infinity)"""
    got, t = got.cpu().double(), TYPES[dtype]
    end = torch.finfo(t).max * (1 + torch.finfo(t).eps / 4)
    ok = ((got - want).abs() <= tol) | ((got.abs() == math.inf) & (got * want > 0) & (want.abs() + tol >= end))
    assert ok.all(), ((got - want).abs() / tol)[~ok].max()


SHAPES = [(1, 32, 1), (1, 2048, 100), (3, 96, 17), (4, 128, 64), (5, 1056, 1037), (8, 256, 33), (13, 512, 130),
          (16, 160, 48), (17, 128, 64), (32, 4096, 20), (33, 64, 200), (70, 224, 31), (2, 320, 20000)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,C,K", SHAPES)
def test_products_of_16_bit_tokens(dtype, M, C, K):
    import depthwise_pointwise_convolution_amd as F
    g = torch.Generator().manual_seed(M + C + K)
    act = ["none", "relu", "relu6"][(M + K) % 3]
    codes, scales = _weights(K, C, M + C)
    x = torch.randn(M, C, generator=g).to(TYPES[dtype])
    bias = torch.randn(K, generator=g) if K % 2 else None
    pad = 8 * (M % 2)
    wide = torch.full((M, C + pad), math.nan, dtype=x.dtype, device="cuda")
    wide[:, :C] = x.cuda()
    y = torch.full((M, K + 3), 7.0, dtype=x.dtype, device="cuda")
    F.fcm_mx4_fwd(F.mx4_problem(dtype, M, C, K, act=act, ldx=C + pad, ldy=K + 3), wide, mx4_pack(codes).cuda(),
                  scales.to(torch.uint8).cuda(), bias.cuda() if bias is not None else None, y)
    torch.cuda.synchronize()
    want, tol = product(dtype, x, mx4_values(codes, scales), bias, act)
    _within(y[:, :K], want, tol, dtype)
    assert (y[:, K:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,C,K", SHAPES + [(300, 416, 290), (129, 1024, 513), (256, 256, 256), (1, 64, 300), (257, 32, 1),
                                            (3300, 288, 3700), (500, 2336, 300)])
def test_products_of_4_bit_tokens(dtype, M, C, K):
    import depthwise_pointwise_convolution_amd as F
    g = torch.Generator().manual_seed(M + 3 * C + K)
    act = ["none", "relu", "relu6"][(M + K) % 3]
    codes, scales = _weights(K, C, M + C, 8)
    xcodes, xscales = _weights(M, C, M + C + 1, 8)
    bias = torch.randn(K, generator=g) if K % 2 else None
    y = torch.full((M, K + 3), 7.0, dtype=TYPES[dtype], device="cuda")
    F.fcm_mx4x4_fwd(F.mx4_problem(dtype, M, C, K, act=act, ldy=K + 3), mx4_pack(xcodes).cuda(),
                    xscales.to(torch.uint8).cuda(), mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda(),
                    bias.cuda() if bias is not None else None, y)
    torch.cuda.synchronize()
    want, tol = product(dtype, mx4_values(xcodes, xscales), mx4_values(codes, scales), bias, act)
    _within(y[:, :K], want, tol, dtype)
    assert (y[:, K:] == 7.0).all()


@pytest.mark.parametrize("both", [False, True])
def test_scales_at_the_ends(both):
    # the smallest and largest powers, and a block that is NaN
    import depthwise_pointwise_convolution_amd as F
    codes, scales = _weights(64, 128, 5)
    scales[:, :] = 127
    scales[3] = 0
    scales[4] = 254
    scales[5, 2] = 255
    codes[4] = codes[4] & 8 | 1
    x = torch.zeros(20, 128)
    x[:, 0], x[:, 70] = 1.0, 2.0
    xc, xs = mx4_quantize(x)
    y = torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    p = F.mx4_problem("bf16", 20, 128, 64)
    wq, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    if both:
        F.fcm_mx4x4_fwd(p, mx4_pack(xc).cuda(), xs.to(torch.uint8).cuda(), wq, ws, None, y)
    else:
        F.fcm_mx4_fwd(p, x.to(torch.bfloat16).cuda(), wq, ws, None, y)
    torch.cuda.synchronize()
    got, w = y.cpu().double(), mx4_values(codes, scales)
    assert torch.isnan(got[:, 5]).all()
    w[5] = 0
    want, tol = product("bf16", x, w, None, "none")
    keep = [i for i in range(64) if i != 5]
    # (numbers below the smallest normal float may count as zero in the products)
    assert ((got - want).abs() <= tol + 2.0 ** -124)[:, keep].all()


def test_a_bad_token_stays_in_its_row():
    import depthwise_pointwise_convolution_amd as F
    codes, scales = _weights(70, 128, 5)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20, 128, generator=g).to(torch.bfloat16)
    y, z = (torch.empty(20, 70, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = F.mx4_problem("bf16", 20, 128, 70)
    wq, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    F.fcm_mx4_fwd(p, x.cuda(), wq, ws, None, y)
    x[7, 3] = math.nan
    F.fcm_mx4_fwd(p, x.cuda(), wq, ws, None, z)
    torch.cuda.synchronize()
    rest = [i for i in range(20) if i != 7]
    assert torch.equal(y[rest], z[rest]) and torch.isnan(z[7]).all()


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("M,C,K", [(1, 96, 48100), (7, 288, 48100), (16, 64, 50001), (17, 96, 48100), (40, 64, 48100)])
def test_products_with_many_outputs(both, M, C, K):
    import depthwise_pointwise_convolution_amd as F
    g = torch.Generator().manual_seed(M + C + K)
    codes, scales = _weights(K, C, M + C, 8)
    xcodes, xscales = _weights(M, C, M + C + 1, 4)
    x = mx4_values(xcodes, xscales)
    bias = torch.randn(K, generator=g)
    y = torch.full((M, K + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    p = F.mx4_problem("bf16", M, C, K, ldy=K + 3)
    w, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    if both:
        F.fcm_mx4x4_fwd(p, mx4_pack(xcodes).cuda(), xscales.to(torch.uint8).cuda(), w, ws, bias.cuda(), y)
    else:  # (a code's value has two bits: it is its own rounding)
        F.fcm_mx4_fwd(p, x.to(torch.bfloat16).cuda(), w, ws, bias.cuda(), y)
    torch.cuda.synchronize()
    want, tol = product("bf16", x, mx4_values(codes, scales), bias, "none")
    _within(y[:, :K], want, tol, "bf16")
    assert (y[:, K:] == 7.0).all()


@pytest.mark.parametrize("M,C,K", [(2500, 1056, 4100), (70, 96, 8200), (300, 1056, 3300), (250, 224, 4100), (65, 64, 16200)])
def test_products_of_4_bit_tokens_by_size(M, C, K):
    # each way the outputs are shared out
    import depthwise_pointwise_convolution_amd as F
    codes, scales = _weights(K, C, M + C, 8)
    xcodes, xscales = _weights(M, C, M + C + 1, 8)
    y = torch.full((M + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fcm_mx4x4_fwd(F.mx4_problem("bf16", M, C, K), mx4_pack(xcodes).cuda(), xscales.to(torch.uint8).cuda(),
                    mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda(), None, y)
    torch.cuda.synchronize()
    want, tol = product("bf16", mx4_values(xcodes, xscales), mx4_values(codes, scales), None, "none")
    _within(y[:M], want, tol, "bf16")
    assert (y[M] == 7.0).all()


def test_codes_behind_2_to_the_31st_byte():
    # the last rows' codes, values and products are those of the rows alone
    import depthwise_pointwise_convolution_amd as F
    C, K, M, last = 2 ** 16, 2 ** 16 + 32, 3, 48
    q = torch.randint(0, 256, (K, C // 2), dtype=torch.uint8, device="cuda")
    s = torch.randint(120, 124, (K, C // 32), dtype=torch.uint8, device="cuda")
    x = torch.randn(M, C, device="cuda").to(torch.bfloat16)
    xq, xs = _quantise(x, "bf16")
    tail = {}
    for name, call in {
            "16-bit": lambda k, w, t, y: F.fcm_mx4_fwd(F.mx4_problem("bf16", M, C, k), x, w, t, None, y),
            "4-bit": lambda k, w, t, y: F.fcm_mx4x4_fwd(F.mx4_problem("bf16", M, C, k), xq, xs, w, t, None, y)}.items():
        y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        call(K, q, s, y)
        want = torch.empty(M, last, dtype=torch.bfloat16, device="cuda")
        call(last, q[-last:].contiguous(), s[-last:].contiguous(), want)
        torch.cuda.synchronize()
        # (fewer outputs may be summed in another order: C products of either sign, each sum off by a rounding)
        w = torch.empty(last, C, device="cuda")
        F.fcm_mx4_dequantize(F.mx4_problem("f32", last, C), q[-last:].contiguous(), s[-last:].contiguous(), w)
        v = torch.empty(M, C, device="cuda")
        F.fcm_mx4_dequantize(F.mx4_problem("f32", M, C), xq, xs, v)
        right, tol = product("bf16", (v if name == "4-bit" else x).cpu(), w.cpu().double(), None, "none")
        _within(y[:, -last:], right, tol, "bf16")
        _within(want, right, tol, "bf16")
        tail[name] = w
    values = torch.empty(K, C, dtype=torch.bfloat16, device="cuda")
    F.fcm_mx4_dequantize(F.mx4_problem("bf16", K, C), q, s, values)
    assert torch.equal(values[-last:].float(), tail["4-bit"])
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    F.fcm_mx4_quantize(F.mx4_problem("bf16", K, C), values, q2, s2)
    again = torch.empty(K, C, dtype=torch.bfloat16, device="cuda")
    F.fcm_mx4_dequantize(F.mx4_problem("bf16", K, C), q2, s2, again)
    torch.cuda.synchronize()
    # (a block whose largest code is below 4 goes to a smaller scale, with the same values)
    assert torch.equal(again[-last:], values[-last:]) and torch.equal(again[:last], values[:last])


def test_captured():
    import depthwise_pointwise_convolution_amd as F
    M, C, K = 40, 256, 130
    codes, scales = _weights(K, C, 3)
    w, ws = mx4_pack(codes).cuda(), scales.to(torch.uint8).cuda()
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    xq, xs = torch.empty(M, C // 2, dtype=torch.uint8, device="cuda"), torch.empty(M, C // 32, dtype=torch.uint8, device="cuda")
    p = F.mx4_problem("bf16", M, C, K)

    def run(y, z):
        F.fcm_mx4_quantize(p, x, xq, xs)
        F.fcm_mx4x4_fwd(p, xq, xs, w, ws, None, y)
        F.fcm_mx4_fwd(p, x, w, ws, None, z)

    y, z, y2, z2 = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    run(y, z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(y, z)
    for seed in range(3):
        x.copy_(torch.randn(M, C, generator=torch.Generator().manual_seed(seed)))
        xq.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        run(y2, z2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(z, z2)
