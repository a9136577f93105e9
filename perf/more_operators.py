"""The library's operators for recurrent language models with a delta rule (the gated delta rule itself,
microscaled 4-bit quantisation and products, the verification of drafted tokens): the cases that are
measured, each operator's plain form in elementary torch operations, and its value in 64 bits.

``own`` says which of the two ``run`` computes: the plain form, or the library's kernels."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # eleven requests' prompts packed into one batch (some continued, one empty) through the mixer of a
        # wide layer, two value heads to a key head, with its output norm and gate
        {"name": "delta_prompts", "op": "delta", "dtype": "bf16", "T": 8192, "B": 11, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "norm": True, "gate": True, "qk_norm": True, "even": False},
        # one user's prompt on a model with few heads: a long chain that hardly fills the card
        {"name": "delta_one_prompt", "op": "delta", "dtype": "bf16", "T": 4096, "B": 1, "Hk": 16, "Hv": 16, "Dk": 128,
         "Dv": 128, "norm": True, "gate": True, "qk_norm": True, "even": False},
        # 32-bit activations and odd sizes, no norm and no gate: a small model in full precision
        {"name": "delta_odd_f32", "op": "delta", "dtype": "f32", "T": 777, "B": 4, "Hk": 3, "Hv": 6, "Dk": 72,
         "Dv": 100, "norm": False, "gate": False, "qk_norm": False, "even": False},
        # four drafted tokens and the last accepted one of each of 32 requests, all continued from their states
        {"name": "delta_drafts", "op": "delta", "dtype": "f16", "T": 160, "B": 32, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "norm": True, "gate": True, "qk_norm": True, "even": True},
        # one user's next token
        {"name": "delta_one_token", "op": "delta_step", "dtype": "bf16", "B": 1, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "norm": True, "gate": True, "qk_norm": True},
        # the next token of a large batch
        {"name": "delta_tokens", "op": "delta_step", "dtype": "bf16", "B": 256, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "norm": True, "gate": True, "qk_norm": True},
        # a prompt batch's activations into 4 bits and back
        {"name": "mx4_quant", "op": "mx4_quant", "dtype": "bf16", "M": 8192, "C": 4096},
        # a projection for one token
        {"name": "mx4_one_token", "op": "mx4", "dtype": "bf16", "M": 1, "C": 2048, "K": 8192, "bias": False},
        # the head over a large vocabulary for a batch of tokens
        {"name": "mx4_head", "op": "mx4", "dtype": "bf16", "M": 16, "C": 4096, "K": 65536, "bias": False},
        # a projection of a prompt batch, its activations quantised on the way
        {"name": "mx4x4_prompts", "op": "mx4x4", "dtype": "bf16", "M": 8192, "C": 4096, "K": 8192, "bias": True},
        # one request, four drafted tokens
        {"name": "verify_one", "op": "verify", "dtype": "f16", "B": 1, "N": 4, "V": 32000, "draft": True,
         "temperature": 0.8},
        # a full batch over an odd vocabulary in 32 bits
        {"name": "verify_batch", "op": "verify", "dtype": "f32", "B": 32, "N": 5, "V": 65537, "draft": True,
         "temperature": 1.0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _channels(rng, low, high):
    """Mostly a power of two or five fourths of one, as models have them, now and then any number."""
    d = _log(rng, low, high)
    two = 1 << (d.bit_length() - 1)
    return (two if d < 9 * two // 8 or two % 4 else 5 * two // 4) if rng.random() < 0.7 else d


def _head(rng):
    return rng.choice([64, 128, 128, 128, 256]) if rng.random() < 0.7 else _log(rng, 8, 256)


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_step", "mx4_quant", "mx4", "mx4x4", "verify"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op in ("delta", "delta_step"):
        dk = _head(rng)
        dv = dk if rng.random() < 0.6 else _head(rng)
        hk = _log(rng, 1, 32)
        hv = hk * rng.choice([1, 1, 2, 2, 4])
        c = {"op": op, "dtype": dtype, "Hk": hk, "Hv": hv, "Dk": dk, "Dv": dv, "norm": rng.random() < 0.6,
             "gate": rng.random() < 0.7, "qk_norm": rng.random() < 0.7}
        if op == "delta":
            c["even"] = rng.random() < 0.2
            c["B"] = _log(rng, 1, 16)
            most = max(1, min(16384, 8192 * 32 * 128 * 128 // (hv * dk * dv)))
            # (equal sequences are short, as drafted tokens are)
            c["T"] = c["B"] * rng.randint(1, 8) if c["even"] else _log(rng, 1, most)
        else:
            c["B"] = _log(rng, 1, max(1, min(256, 256 * 32 * 128 * 128 // (hv * dk * dv))))
        return c
    if op == "mx4_quant":
        c = max(32, _channels(rng, 128, 16384) // 32 * 32)
        return {"op": op, "dtype": dtype, "M": _log(rng, 1, max(1, 8192 * 4096 // c)), "C": c}
    if op == "mx4":
        c = max(32, _channels(rng, 128, 16384) // 32 * 32)
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "M": _log(rng, 1, 64), "C": c,
                "K": _log(rng, 64, min(65536, 65536 * 4096 // c)), "bias": rng.random() < 0.5}
    if op == "mx4x4":
        c = max(32, _channels(rng, 128, 8192) // 32 * 32)
        m = _log(rng, 1, 8192)
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "M": m, "C": c,
                "K": _log(rng, 64, min(65536, 8192 * 4096 * 8192 // (c * m))), "bias": rng.random() < 0.5}
    return {"op": op, "dtype": dtype, "B": _log(rng, 1, 32), "N": rng.randint(1, 8), "V": _log(rng, 500, 65537),
            "draft": rng.random() < 0.75, "temperature": rng.choice([0.0, 0.6, 0.8, 1.0, 1.0, 1.3])}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _lengths(seed, case):
    """Lengths of the sequences, an empty one among many."""
    total, count = case["T"], case["B"]
    if case["even"]:
        return [total // count] * count
    rng = random.Random(seed * 7919 + total * 31 + count)
    cuts = sorted(rng.randrange(total + 1) for _ in range(count - 1))
    if count > 3:
        cuts[1] = cuts[0]
    ends = cuts + [total]
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=self.g) * std).to(dtype)

    def uniform(self, low, high, *shape):
        return torch.rand(*shape, device="cuda", generator=self.g) * (high - low) + low

    def integers(self, low, high, *shape, dtype=torch.int32):
        return torch.randint(low, high, shape, device="cuda", generator=self.g, dtype=dtype)


def prepare(case, seed):
    s, r = {"case": case}, _Draw(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    if op in ("delta", "delta_step"):
        t, b, hk, hv, dk, dv = case.get("T", case["B"]), case["B"], case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        # queries, keys and values are columns of one projection's rows, the steps and rates of another's
        std = 1.0 if case["qk_norm"] else dk ** -0.5
        rows = r.normal(t, 2 * hk * dk + hv * dv, dtype=dt)
        rows[:, :2 * hk * dk] *= std
        s["q"], s["k"], s["v"] = rows[:, :hk * dk], rows[:, hk * dk:2 * hk * dk], rows[:, 2 * hk * dk:]
        ab = r.normal(t, 2 * hv, dtype=dt)
        s["a"], s["b"] = ab[:, :hv], ab[:, hv:]
        s["A"] = -torch.exp(r.uniform(0.0, math.log(16.0), hv))
        # softplus(dt_bias) spread over 0.001 .. 0.1, as recurrent layers start from
        step = torch.exp(r.uniform(math.log(1e-3), math.log(0.1), hv))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["norm"] = 1.0 + r.normal(dv, std=0.1) if case["norm"] else None
        s["z"] = r.normal(t, hv * dv, dtype=dt) if case["gate"] else None
        s["slots"] = torch.randperm(b + 3, device="cuda", generator=r.g)[:b].to(torch.int32)
        s["state"] = r.normal(b + 3, hv, dk, dv, std=0.3)
        s["y"] = torch.empty(t, hv * dv, dtype=dt, device="cuda")
        if op == "delta":
            lens = _lengths(seed, case)
            s["longest"] = max(lens)
            ends = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
            s["cu"] = ends.cuda()
            s["carry"] = r.integers(0, 2, b) if not case["even"] else torch.ones(b, dtype=torch.int32, device="cuda")
        elif b > 4:
            s["slots"][r.integers(0, b, 2, dtype=torch.int64)] = -1  # idle rows of a padded batch
    elif op == "mx4_quant":
        # activations with a few strong channels
        s["x"] = (r.normal(case["M"], case["C"]) * torch.exp(r.normal(case["C"]))).to(dt)
        s["q"] = torch.empty(case["M"], case["C"] // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(case["M"], case["C"] // 32, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty_like(s["x"])
    elif op in ("mx4", "mx4x4"):
        m, c, k = case["M"], case["C"], case["K"]
        s["x"] = r.normal(m, c, dtype=dt)
        parts = [_codes(r.normal(min(4096, k - i), c, std=c ** -0.5)) for i in range(0, k, 4096)]
        s["wq"], s["ws"] = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        s["bias"] = r.normal(k, std=0.1) if case["bias"] else None
        s["y"] = torch.empty(m, k, dtype=dt, device="cuda")
        if op == "mx4x4":
            s["xq"] = torch.empty(m, c // 2, dtype=torch.uint8, device="cuda")
            s["xs"] = torch.empty(m, c // 32, dtype=torch.uint8, device="cuda")
    else:
        b, n, v = case["B"], case["N"], case["V"]
        target = r.normal(b, n + 1, v, std=2.5).masked_fill_(r.uniform(0, 1, b, n + 1, v) < 0.05, -math.inf)
        s["target"] = target.to(dt).reshape(b * (n + 1), v)
        # the drafting model's logits are near the target's
        draft = target[:, :n] + r.normal(b, n, v, std=0.5)
        s["draft"] = draft.to(dt).reshape(b * n, v) if case["draft"] else None
        heat = case["temperature"]
        noise = -torch.log(-torch.log(r.uniform(1e-7, 1 - 1e-7, b, n, v)))
        s["tokens"] = (draft / heat + noise if heat > 0 else draft).argmax(-1).to(torch.int32).reshape(-1)
        s["counts"] = r.integers(n // 2, n + 1, b)
        s["u"] = r.uniform(0, 1, b, n + 1)
        s["accepted"], s["next"] = (torch.empty(b, dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        _handles(s)
    return s


def _handles(s):
    """The problem descriptors and workspaces that a serving program keeps."""
    import depthwise_pointwise_convolution_amd as F
    case, op = s["case"], s["case"]["op"]
    if op in ("delta", "delta_step"):
        t = case.get("T", case["B"])
        ld = s["q"].stride(0)
        s["plan"] = F.delta_problem(case["dtype"], case["Hk"], case["Hv"], case["Dk"], case["Dv"], tokens=t,
                                    seqs=case["B"], slots=s["state"].shape[0], qk_norm=case["qk_norm"], eps=EPS,
                                    ldq=ld, ldk=ld, ldv=ld, lda=s["a"].stride(0), ldb=s["b"].stride(0))
        if op == "delta":
            s["ws"] = torch.empty(max(16, F.fcm_delta_workspace(s["plan"])), dtype=torch.uint8, device="cuda")
    elif op == "verify":
        s["plan"] = F.draft_problem(case["dtype"], case["B"], case["N"], case["V"], temperature=case["temperature"])
        s["ws"] = torch.empty(max(16, F.fcm_draft_workspace(s["plan"])), dtype=torch.uint8, device="cuda")
    else:
        s["plan"] = F.mx4_problem(case["dtype"], case["M"], case["C"], case.get("K", 1))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"delta": _delta, "delta_step": _delta_step, "mx4_quant": _mx4_quant, "mx4": _mx4, "mx4x4": _mx4x4,
            "verify": _verify}[op](s)


def _own(s, op):
    import depthwise_pointwise_convolution_amd as F
    if op == "delta":
        F.fcm_delta_fwd(s["plan"], s["q"], s["k"], s["v"], s["a"], s["b"], s["A"], s["dt_bias"], s["norm"], s["z"],
                        s["cu"], s["slots"], s["carry"], s["state"], s["ws"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "delta_step":
        F.fcm_delta_step(s["plan"], s["q"], s["k"], s["v"], s["a"], s["b"], s["A"], s["dt_bias"], s["norm"], s["z"],
                         s["slots"], s["state"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "mx4_quant":
        F.fcm_mx4_quantize(s["plan"], s["x"], s["q"], s["scales"])
        F.fcm_mx4_dequantize(s["plan"], s["q"], s["scales"], s["y"])
        return s["y"]
    if op == "mx4":
        F.fcm_mx4_fwd(s["plan"], s["x"], s["wq"], s["ws"], s["bias"], s["y"])
        return s["y"]
    if op == "mx4x4":
        F.fcm_mx4_quantize(s["plan"], s["x"], s["xq"], s["xs"])
        F.fcm_mx4x4_fwd(s["plan"], s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], s["y"])
        return s["y"]
    F.fcm_draft_verify(s["plan"], s["target"], s["draft"], s["tokens"], s["counts"], s["u"], s["ws"], s["accepted"],
                       s["next"])
    return {"accepted": s["accepted"], "next": s["next"]}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _rows(s):
    """(q, k, v, log of the decay, rate) in 32 bits by value head: [tokens, Hv, ...]."""
    case = s["case"]
    share = case["Hv"] // case["Hk"]
    q, k = (s[n].float().reshape(-1, case["Hk"], case["Dk"]) for n in "qk")
    if case["qk_norm"]:
        q, k = (v / torch.sqrt((v * v).sum(-1, keepdim=True) + EPS) for v in (q, k))
    q, k = (v.repeat_interleave(share, 1) for v in (q * case["Dk"] ** -0.5, k))
    rate = 1 / (1 + torch.exp(-s["b"].float()))
    return q, k, s["v"].float().reshape(-1, case["Hv"], case["Dv"]), _softplus(s["a"].float() + s["dt_bias"]) * s["A"], rate


def _ends(s, o):
    """The output of rows o, [tokens, Hv, Dv]: norm, gate, rounding."""
    if s["norm"] is not None:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["norm"]
    if s["z"] is not None:
        o = o * _silu(s["z"].float()).reshape(o.shape)
    return o.reshape(o.shape[0], -1).to(s["y"].dtype)


def _delta(s):
    """In chunks: within one, what a token adds to the state solves a triangular system."""
    case = s["case"]
    b, hv, dk, dv = case["B"], case["Hv"], case["Dk"], case["Dv"]
    size = min(64, s["longest"])
    n = -(-s["longest"] // size)
    start, ends, slots = s["cu"][:-1].long(), s["cu"][1:].long(), s["slots"].long()
    at = start[:, None] + torch.arange(n * size, device="cuda")
    live = at < ends[:, None]
    at = at.clamp(max=case["T"] - 1)

    def chunks(v):  # [tokens, Hv, ...] to [B, Hv, n, size, ...], zero behind a sequence
        v = v[at] * live.reshape(live.shape + (1,) * (v.dim() - 1))
        return v.reshape(b, n, size, *v.shape[2:]).transpose(2, 3).transpose(1, 2)

    q, k, v, g, rate = (chunks(x) for x in _rows(s))
    along = g.double().cumsum(-1)  # (differences of long sums)
    lower = torch.ones(size, size, device="cuda", dtype=torch.bool).tril()
    decay = torch.exp((along[..., :, None] - along[..., None, :]).masked_fill(~lower, -math.inf)).float()
    grown = torch.exp(along).float()
    left = torch.exp(along[..., -1:] - along).float()
    kt = k.transpose(-1, -2).contiguous()
    mix = rate[..., None] * (k @ kt) * decay
    x = torch.cat([v, k * grown[..., None]], -1) * rate[..., None]
    for i in range(1, size):
        x[..., i:i + 1, :] -= mix[..., i:i + 1, :i] @ x[..., :i, :]
    fresh, known = x[..., :dv], x[..., dv:].contiguous()
    seen = (q @ kt) * decay
    q = q * grown[..., None]
    kt = (k * left[..., None]).transpose(-1, -2).contiguous()
    state = s["state"][slots] * (s["carry"] != 0).float()[:, None, None, None]
    o = torch.empty_like(v)
    for c in range(n):
        u = fresh[:, :, c] - known[:, :, c] @ state
        o[:, :, c] = q[:, :, c] @ state + seen[:, :, c] @ u
        state = grown[:, :, c, -1, None, None] * state + kt[:, :, c] @ u
    s["state"][slots] = state
    o = o.permute(0, 2, 3, 1, 4).reshape(b, n * size, hv, dv)
    return {"y": _ends(s, o[live]), "state": s["state"]}


def _delta_step(s):
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    q, k, v, g, rate = _rows(s)
    state = s["state"][at] * torch.exp(g)[..., None, None]
    u = rate[..., None] * (v - (k[..., None] * state).sum(-2))
    state = state + k[..., None] * u[..., None, :]
    o = (q[..., None] * state).sum(-2)
    s["state"][at[live]] = state[live]
    return {"y": _ends(s, o) * live[:, None].to(s["y"].dtype), "state": s["state"]}


def _quantised(x):
    """(multiples of a block's scale, exponents of the scales), [rows, blocks, 32] and [rows, blocks, 1]: the
    scale's exponent is that of the block's largest magnitude less 2, values round to even and end at 6."""
    x = x.float().reshape(x.shape[0], -1, 32)
    exponent = torch.frexp(x.abs().amax(-1, keepdim=True)).exponent - 3
    scaled = torch.ldexp(x, -exponent)  # (powers of two: exact)
    size = scaled.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    return torch.copysign((torch.round(size / step) * step).clamp(max=6.0), scaled), exponent


def _codes(x):
    """The packed codes and scales of [rows, C]: sign, two bits of exponent and one of mantissa in four, the even
    channel in the low half; scales as their exponent plus 127."""
    value, exponent = _quantised(x)
    size = value.abs()
    code = torch.where(size < 2, size * 2, torch.where(size < 4, size + 2, size / 2 + 4)).to(torch.uint8)
    code = (code + 8 * (value < 0)).to(torch.uint8).reshape(x.shape[0], -1)
    return code[:, 0::2] | code[:, 1::2] << 4, (exponent + 127).to(torch.uint8).reshape(x.shape[0], -1)


def _values(q, scales):
    """What codes and scales stand for, in 32 bits."""
    code = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    value = torch.cat([table, -table])[code.long()].reshape(q.shape[0], -1, 32)
    return (value * torch.exp2(scales.float() - 127)[..., None]).reshape(q.shape[0], -1)


def _mx4_quant(s):
    value, exponent = _quantised(s["x"])
    return torch.ldexp(value, exponent).reshape(s["x"].shape).to(s["x"].dtype)


def _mx4(s):
    y = s["x"].float() @ _values(s["wq"], s["ws"]).t()
    return (y + s["bias"] if s["bias"] is not None else y).to(s["x"].dtype)


def _mx4x4(s):
    value, exponent = _quantised(s["x"])
    y = torch.ldexp(value, exponent).reshape(s["x"].shape) @ _values(s["wq"], s["ws"]).t()
    return (y + s["bias"] if s["bias"] is not None else y).to(s["x"].dtype)


def _softmax(logits, heat):
    # in 64 bits: which side of a border a token is on has to be told
    logits = logits.double() / heat
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _verify(s):
    case = s["case"]
    b, n, v = case["B"], case["N"], case["V"]
    tokens, at, counts = s["tokens"].reshape(b, n).long(), torch.arange(b, device="cuda"), s["counts"].long()
    places = torch.arange(n, device="cuda")
    if case["temperature"] == 0:
        best = s["target"].reshape(b, n + 1, v).argmax(-1)
        passed = best[:, :n] == tokens
    else:
        p = _softmax(s["target"], case["temperature"]).reshape(b, n + 1, v)
        if s["draft"] is not None:
            q = _softmax(s["draft"], case["temperature"]).reshape(b, n, v)
        else:
            q = torch.zeros(b, n, v, device="cuda", dtype=torch.float64).scatter_(2, tokens[..., None], 1.0)
        mine, theirs = (x.gather(2, tokens[..., None])[..., 0] for x in (p[:, :n], q))
        passed = s["u"][:, :n].double() * theirs < mine
    passed = passed & (places < counts[:, None])
    accepted = passed.long().cumprod(1).sum(1)
    if case["temperature"] == 0:
        token = best[at, accepted]
    else:
        rest = p[at, accepted]
        rest = torch.where((accepted < counts)[:, None],
                           (rest - q[at, accepted.clamp(max=n - 1)]).clamp(min=0), rest)
        along = rest.cumsum(-1)
        token = (along <= s["u"][:, n:].double() * along[:, -1:]).sum(-1)
    return {"accepted": accepted.to(torch.int32), "next": token.to(torch.int32)}


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("delta", "delta_step"):
        t, b, hk, hv, dk, dv = case.get("T", case["B"]), case["B"], case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        row = 2 * hk * dk + (3 if case["gate"] else 2) * hv * dv + 2 * hv
        return {"bytes": t * row * e + 8 * b * hv * dk * dv, "flops": 6 * t * hv * dk * dv}
    if op == "mx4_quant":
        return {"bytes": 2 * case["M"] * case["C"] * e, "flops": 4 * case["M"] * case["C"]}
    if op in ("mx4", "mx4x4"):
        m, c, k = case["M"], case["C"], case["K"]
        return {"bytes": k * c * 17 // 32 + (m * c + m * k) * e + (4 * k if case["bias"] else 0),
                "flops": 2 * m * c * k}
    rows = case["B"] * (case["N"] + 1 + (case["N"] if case["draft"] else 0))
    return {"bytes": rows * case["V"] * e, "flops": 4 * rows * case["V"]}


# ------------------------------------------------------------------------------------------
# in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("delta", "delta_step"):
        return _exact_delta(s)
    if op == "mx4_quant":
        return _exact_quantised(s["x"])
    if op in ("mx4", "mx4x4"):
        return _exact_product(s, s["x"].double() if op == "mx4" else _exact_quantised(s["x"]))
    return None  # whole numbers


def _exact_delta(s):
    case = s["case"]
    hk, hv, dk, dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    slots = s["slots"].tolist()
    if "cu" in s:
        cu, carry = s["cu"].tolist(), s["carry"].tolist()
    else:
        cu, carry = list(range(len(slots) + 1)), [1] * len(slots)
    full = s["state"].double()
    out = torch.zeros(s["y"].shape[0], hv, dv, dtype=torch.float64, device="cuda")
    order = sorted((i for i in range(len(slots)) if slots[i] >= 0), key=lambda i: cu[i] - cu[i + 1])
    lens = [cu[i + 1] - cu[i] for i in order]
    state = full[[slots[i] for i in order]] * torch.tensor([float(carry[i] != 0) for i in order], dtype=torch.float64,
                                                           device="cuda").reshape(-1, 1, 1, 1)
    q, k = (s[x].double().reshape(-1, hk, 1, dk).expand(-1, hk, hv // hk, dk).reshape(-1, hv, dk) for x in "qk")
    if case["qk_norm"]:
        q, k = (x * (x.square().sum(-1, keepdim=True) + EPS).rsqrt() for x in (q, k))
    q = q / math.sqrt(dk)
    v = s["v"].double().reshape(-1, hv, dv)
    alpha = torch.exp(torch.nn.functional.softplus(s["a"].double() + s["dt_bias"].double(), threshold=60) * s["A"].double())
    beta = torch.sigmoid(s["b"].double())
    first = torch.tensor([cu[i] for i in order], device="cuda")
    live = len(order)
    for t in range(max(lens, default=0)):  # the longest first: those that go on are the front ones
        while live and lens[live - 1] <= t:
            live -= 1
        at = first[:live] + t
        now = state[:live] * alpha[at][..., None, None]
        held = torch.matmul(k[at][..., None, :], now)[..., 0, :]
        now += k[at][..., :, None] * (beta[at][..., None] * (v[at] - held))[..., None, :]
        out[at] = torch.matmul(q[at][..., None, :], now)[..., 0, :]
        state[:live] = now
    full[[slots[i] for i in order]] = state
    if s["norm"] is not None:
        out = out * (out.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["norm"].double()
    if s["z"] is not None:
        z = s["z"].double().reshape(out.shape)
        out = out * (z * torch.sigmoid(z))
    for i, slot in enumerate(slots):
        if slot < 0:
            out[cu[i]:cu[i + 1]] = 0
    return {"y": out.reshape(out.shape[0], -1), "state": full}


def _exact_quantised(x):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    x = x.double().reshape(x.shape[0], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top)) - 2)
    size = (x.abs() / scale).clamp(max=6)
    middle = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(size, middle), torch.bucketize(size, middle, right=True)
    at = torch.where(low % 2 == 0, low, high)  # a value between two goes to the even one
    return (torch.sign(x) * grid[at] * scale).reshape(x.shape[0], -1)


def _exact_product(s, x):
    case = s["case"]
    y = torch.zeros(case["M"], case["K"], dtype=torch.float64, device="cuda")
    for i in range(0, case["K"], 8192):  # some rows of the weights at a time
        q = s["wq"][i:i + 8192].to(torch.int64)
        code = torch.empty(q.shape[0], case["C"], dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = q % 16, q // 16
        power, half = (code // 2) % 4, code % 2
        size = torch.where(power == 0, half * 0.5, (1 + 0.5 * half) * torch.exp2(power.double() - 1))
        w = torch.where(code >= 8, -size, size).reshape(q.shape[0], -1, 32)
        w = (w * torch.exp2(s["ws"][i:i + 8192].double() - 127)[..., None]).reshape(q.shape[0], -1)
        y[:, i:i + 8192] = x @ w.t().contiguous()
    return y + s["bias"].double() if s["bias"] is not None else y
