"""Where a sequence may be cut without a bit of difference: up to 16 rows the delta rule goes token by token."""
import os
import sys

import pytest
import torch

from gpu_util import gpu_available

gpu = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def on_gpu(f):
    for m in gpu:
        f = m(f)
    return f


def _example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_decode
    return draft_decode


def test_the_check_refuses_more_rows(capsys):
    with pytest.raises(SystemExit) as e:
        _example().main(["--check", "--drafts", "16"])
    assert e.value.code == 2 and "at most 15 drafts" in capsys.readouterr().err


@on_gpu
@pytest.mark.parametrize("requests", [1, 3])
def test_the_check_with_most_rows(requests):
    assert _example().main(["--dim", "128", "--layers", "2", "--vocab", "300", "--tokens", "8", "--drafts", "15",
                            "--requests", str(requests), "--check"]) == 0


@on_gpu
@pytest.mark.parametrize("dtype,B,Hk,Hv,Dk,Dv,norm", [("bf16", 3, 2, 4, 128, 128, True), ("f16", 1, 1, 2, 64, 48, True),
                                                      ("f32", 2, 1, 1, 256, 250, False), ("bf16", 1, 1, 3, 40, 17, True)])
def test_sixteen_tokens_are_sixteen_steps(dtype, B, Hk, Hv, Dk, Dv, norm):
    # bit for bit, wherever they are cut
    import depthwise_pointwise_convolution_amd as F
    from test_delta_gpu import _inputs
    n = 16
    c = _inputs(Dk + Dv, dtype, B * n, B, Hk, Hv, Dk, Dv, B)
    if not norm:
        c["norm"] = None
    d = {k: v.cuda() if v is not None else None for k, v in c.items()}
    state = d["state"]

    def call(rows, length, state):
        x = {k: d[k][rows].contiguous() for k in "qkvabz"}
        y = torch.empty(len(rows), Hv * Dv, dtype=d["q"].dtype, device="cuda")
        p = F.delta_problem(dtype, Hk, Hv, Dk, Dv, tokens=len(rows), seqs=B, slots=B)
        args = [x["q"], x["k"], x["v"], x["a"], x["b"], d["A"], d["dt_bias"], d["norm"], x["z"]]
        if length == 0:
            F.fcm_delta_step(p, *args, None, state, y)
        else:
            cu = torch.arange(0, B * length + 1, length, dtype=torch.int32).cuda()
            ws = torch.empty(F.fcm_delta_workspace(p), dtype=torch.uint8, device="cuda")
            F.fcm_delta_fwd(p, *args, cu, None, torch.ones(B, dtype=torch.int32).cuda(), state, ws, y)
        return y

    rows = lambda s, e: [b * n + t for b in range(B) for t in range(s, e)]  # noqa: E731
    got = []
    for cuts in ([(0, 16)], [(0, 5), (5, 16)], [(t, t + 1) for t in range(16)]):
        s, y = state.clone(), torch.empty(B * n, Hv * Dv, dtype=d["q"].dtype, device="cuda")
        for first, end in cuts:
            y[rows(first, end)] = call(rows(first, end), 0 if len(cuts) == 16 else end - first, s)
        torch.cuda.synchronize()
        got.append((y, s))
    for y, s in got[1:]:
        assert torch.equal(y, got[0][0]) and torch.equal(s, got[0][1])


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_a_short_sequence_alone_among_padding(dtype):
    # goes in a chunk: within its bound, and the rows behind it are left
    from recurrent_oracle import delta
    from test_delta_gpu import _call, _check, _inputs
    c = _inputs(3, dtype, 40, 1, 1, 2, 64, 48, 1)
    got, pool, spans = _call(c, dtype, [10], [0], [1], 1, 2, 64, 48, {})
    want = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [0], [1],
                 c["state"], 64 ** -0.5, 1e-6)
    _check(got, pool, want, 40, 2, 48, dtype)
