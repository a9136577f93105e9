"""The sequence operators of the library (the causal depthwise layer, the selective scan, 4-bit pointwise
products, beam selection with its reordering of states): the cases that are measured, each operator's
plain form in elementary torch operations, and its value in 64 bits.

``own`` says which of the two ``run`` computes: the plain form, or the library's kernels."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # eleven requests' prompts packed into one batch (some continued from an earlier part of
        # the prompt, one of them empty): the layer before the scan of a wide block
        {"name": "dw1d_prompts", "op": "dw1d", "dtype": "bf16", "T": 8192, "B": 11, "D": 4096, "W": 4,
         "strided": True, "bias": True},
        # one decoding step of a full batch, some of its rows idle
        {"name": "dw1d_tokens", "op": "dw1d_step", "dtype": "f16", "B": 96, "D": 4096, "W": 4,
         "strided": True, "bias": True},
        # one user's prompt on a narrow model: too few channels to fill the card
        {"name": "scan_one_prompt", "op": "scan", "dtype": "bf16", "T": 2048, "B": 1, "D": 2048, "N": 16,
         "G": 1, "gate": True},
        # a full batch of ragged prompts on a wide model
        {"name": "scan_prompts", "op": "scan", "dtype": "f16", "T": 8192, "B": 11, "D": 4096, "N": 16,
         "G": 1, "gate": True},
        # 32-bit activations, odd sizes, two groups, no gate: a small model in full precision
        {"name": "scan_odd_f32", "op": "scan", "dtype": "f32", "T": 777, "B": 4, "D": 1026, "N": 24,
         "G": 2, "gate": False},
        # one user's next token
        {"name": "scan_one_token", "op": "scan_step", "dtype": "bf16", "B": 1, "D": 2048, "N": 16, "G": 1,
         "gate": True},
        # the next token of a large batch on a wide model
        {"name": "scan_tokens", "op": "scan_step", "dtype": "bf16", "B": 256, "D": 4096, "N": 16, "G": 1,
         "gate": True},
        # the block's input projection for one token
        {"name": "q4_one_token", "op": "q4", "dtype": "bf16", "M": 1, "C": 2048, "K": 8192, "group": 128,
         "zeros": True, "bias": False},
        # odd sizes: a last group that is not full, rows that are no multiple of a tile
        {"name": "q4_odd", "op": "q4", "dtype": "f16", "M": 5, "C": 1000, "K": 1037, "group": 32,
         "zeros": True, "bias": True},
        # the head over a large vocabulary for a batch of tokens
        {"name": "q4_head", "op": "q4", "dtype": "bf16", "M": 16, "C": 4096, "K": 65536, "group": 64,
         "zeros": False, "bias": False},
        # one request, four beams, and the states of one layer
        {"name": "beam_one", "op": "beam", "dtype": "f16", "B": 1, "W": 4, "V": 32000, "state": 2048 * 16},
        # a full batch, an odd vocabulary in 32 bits, and the states of several layers
        {"name": "beam_batch", "op": "beam", "dtype": "f32", "B": 32, "W": 8, "V": 65537,
         "state": 4 * 4096 * 16},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _channels(rng, low, high):
    """Mostly a power of two or five fourths of one, as models have them, now and then any number."""
    d = _log(rng, low, high)
    two = 1 << (d.bit_length() - 1)
    return (two if d < 9 * two // 8 or two % 4 else 5 * two // 4) if rng.random() < 0.7 else d


def draw(rng):
    op = rng.choice(["dw1d", "dw1d_step", "scan", "scan", "scan_step", "q4", "q4", "beam"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "dw1d":
        d = _channels(rng, 64, 8192)
        t = _log(rng, 1, min(16384, 8192 * 4096 // d))
        return {"op": op, "dtype": dtype, "T": t, "B": _log(rng, 1, 16), "D": d,
                "W": rng.choice([2, 3, 4, 4, 4]), "strided": rng.random() < 0.5, "bias": rng.random() < 0.7}
    if op == "dw1d_step":
        return {"op": op, "dtype": dtype, "B": _log(rng, 1, 256), "D": _channels(rng, 64, 8192),
                "W": rng.choice([2, 3, 4, 4, 4]), "strided": rng.random() < 0.5, "bias": rng.random() < 0.7}
    if op in ("scan", "scan_step"):
        n, g = rng.choice([(16, 1), (16, 1), (16, 2), (8, 1), (32, 1), (64, 1), (24, 1), (5, 1)])
        d = _channels(rng, 64, 8192) // g * g
        c = {"op": op, "dtype": dtype, "B": _log(rng, 1, 256), "D": d, "N": n, "G": g,
             "gate": rng.random() < 0.75}
        if op == "scan":
            c["B"] = _log(rng, 1, 16)
            c["T"] = _log(rng, 1, min(16384, 8192 * 4096 * 16 // (d * n)))
        else:
            c["B"] = _log(rng, 1, max(1, min(256, 256 * 4096 * 16 // (d * n))))
        return c
    if op == "q4":
        c = max(8, _channels(rng, 128, 16384) // 8 * 8)
        k = _log(rng, 64, min(65536, 65536 * 4096 // c))
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "M": _log(rng, 1, 64), "C": c, "K": k,
                "group": rng.choice([32, 64, 128, 128]), "zeros": rng.random() < 0.5,
                "bias": rng.random() < 0.5}
    return {"op": op, "dtype": dtype, "B": _log(rng, 1, 32), "W": rng.choice([1, 2, 3, 4, 5, 8]),
            "V": _log(rng, 500, 65537), "state": _log(rng, 256, 4 * 4096) * 16}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _lengths(seed, total, count):
    """Lengths of `count` sequences with `total` tokens in all, an empty one among many."""
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

    def slots(self, seqs, total):
        return torch.randperm(total, device="cuda", generator=self.g)[:seqs].to(torch.int32)


def _sequences(s, r, case, seed):
    """Offsets of packed sequences, their state slots, and which of them continue from the state."""
    lens = _lengths(seed, case["T"], case["B"])
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["carry"] = r.integers(0, 2, case["B"])


def prepare(case, seed):
    s, r = {"case": case}, _Draw(seed)
    op = case["op"]
    if op in ("dw1d", "dw1d_step"):
        t, b, d, w, dt = case.get("T", case["B"]), case["B"], case["D"], case["W"], TYPES[case["dtype"]]
        # in a block the layer reads one half of the input projection's rows
        s["x"] = r.normal(t, 2 * d if case["strided"] else d, dtype=dt)[:, :d]
        s["w"] = r.normal(d, w, dtype=dt, std=0.5)
        s["bias"] = r.normal(d, std=0.1) if case["bias"] else None
        s["slots"] = r.slots(b, b + 3)
        s["state"] = r.normal(b + 3, w - 1, d, dtype=dt)
        s["y"] = torch.empty(t, d, dtype=dt, device="cuda")
        if op == "dw1d":
            _sequences(s, r, case, seed)
        elif b > 4:
            s["slots"][r.integers(0, b, 2, dtype=torch.int64)] = -1  # idle rows of a padded batch
    elif op in ("scan", "scan_step"):
        t, b, d, n, g = case.get("T", case["B"]), case["B"], case["D"], case["N"], case["G"]
        dt = TYPES[case["dtype"]]
        s["x"] = r.normal(t, d, dtype=dt)
        s["dt"] = r.normal(t, d, dtype=dt, std=0.5)
        # softplus(dt_bias) spread over 0.001 .. 0.1, as state-space layers start from
        step = torch.exp(r.uniform(math.log(1e-3), math.log(0.1), d))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, n + 1, device="cuda").float() * torch.exp(r.normal(d, n, std=0.2))
        low = 8  # B and C are the last columns of the rows of a projection
        bc = r.normal(t, low + 2 * g * n, dtype=dt)
        s["Bm"], s["Cm"] = bc[:, low:low + g * n], bc[:, low + g * n:]
        s["skip"] = 1.0 + r.normal(d, std=0.1)
        s["z"] = r.normal(t, 2 * d, dtype=dt)[:, d:] if case["gate"] else None
        s["slots"] = r.slots(b, b + 3)
        s["state"] = r.normal(b + 3, d, n)
        s["y"] = torch.empty(t, d, dtype=dt, device="cuda")
        if op == "scan":
            _sequences(s, r, case, seed)
        elif b > 4:
            s["slots"][r.integers(0, b, 2, dtype=torch.int64)] = -1
    elif op == "q4":
        m, c, k, dt = case["M"], case["C"], case["K"], TYPES[case["dtype"]]
        groups = -(-c // case["group"])
        s["x"] = r.normal(m, c, dtype=dt)
        s["q"] = r.integers(0, 256, k, c // 2, dtype=torch.uint8)
        s["scales"] = (r.uniform(0.5, 1.5, k, groups) * (0.25 / math.sqrt(c))).to(dt)
        s["zeros"] = r.integers(0, 16, k, groups, dtype=torch.uint8) if case["zeros"] else None
        s["bias"] = r.normal(k, std=0.1) if case["bias"] else None
        s["y"] = torch.empty(m, k, dtype=dt, device="cuda")
    else:
        b, w, v, dt = case["B"], case["W"], case["V"], TYPES[case["dtype"]]
        s["logits"] = r.normal(b * w, v, std=2.5).masked_fill_(r.uniform(0, 1, b * w, v) < 0.05, -math.inf).to(dt)
        s["scores"] = -r.uniform(0, 6, b * w)
        s["scores"][1:w] = -math.inf  # the first request is at its first step: its beams are one
        s["done"] = (r.uniform(0, 1, b * w) < 0.1).to(torch.int32)
        s["done"][:w] = 0
        s["eos"] = 2
        s["slots"] = torch.randperm(b * w, device="cuda", generator=r.g).to(torch.int32)
        s["states"] = [r.normal(b * w, case["state"]), r.normal(b * w, 3 * case["state"] // 16, dtype=torch.bfloat16)]
    if own:
        _handles(s)
    return s


def _handles(s):
    """The problem descriptors, workspaces and output buffers that a serving program keeps."""
    import depthwise_pointwise_convolution_amd as F
    case, op = s["case"], s["case"]["op"]
    if op == "dw1d":
        s["plan"] = F.dw1d_problem(case["dtype"], case["D"], case["W"], tokens=case["T"], seqs=case["B"],
                                   slots=s["state"].shape[0], ldx=s["x"].stride(0))
    elif op == "dw1d_step":
        s["plan"] = F.dw1d_problem(case["dtype"], case["D"], case["W"], tokens=case["B"], seqs=case["B"],
                                   slots=s["state"].shape[0], ldx=s["x"].stride(0))
    elif op in ("scan", "scan_step"):
        s["plan"] = F.scan_problem(case["dtype"], case["D"], case["N"], groups=case["G"],
                                   tokens=case.get("T", case["B"]), seqs=case["B"],
                                   slots=s["state"].shape[0], ldb=s["Bm"].stride(0), ldc=s["Cm"].stride(0),
                                   ldz=s["z"].stride(0) if s["z"] is not None else 0)
        if op == "scan":
            s["ws"] = torch.empty(max(16, F.fcm_scan_workspace(s["plan"])), dtype=torch.uint8, device="cuda")
    elif op == "q4":
        s["plan"] = F.q4_problem(case["dtype"], case["M"], case["C"], case["K"], group=case["group"])
    else:
        n = case["B"] * case["W"]
        s["plan"] = F.beam_problem(case["dtype"], case["B"], case["W"], case["V"], eos=s["eos"])
        s["ws"] = torch.empty(max(16, F.fcm_beam_workspace(s["plan"])), dtype=torch.uint8, device="cuda")
        s["next"] = torch.empty(n, device="cuda")
        s["parent"], s["token"], s["next_done"], s["next_slots"] = (
            torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(4))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"dw1d": _dw1d, "dw1d_step": _dw1d_step, "scan": _scan, "scan_step": _scan_step, "q4": _q4,
            "beam": _beam}[op](s)


def _own(s, op):
    import depthwise_pointwise_convolution_amd as F
    if op == "dw1d":
        F.fcm_dw1d_fwd(s["plan"], s["x"], s["w"], s["bias"], s["cu"], s["slots"], s["carry"], s["state"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "dw1d_step":
        F.fcm_dw1d_step(s["plan"], s["x"], s["w"], s["bias"], s["slots"], s["state"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "scan":
        F.fcm_scan_fwd(s["plan"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["skip"], s["dt_bias"], s["z"],
                       s["cu"], s["slots"], s["carry"], s["state"], s["ws"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "scan_step":
        F.fcm_scan_step(s["plan"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["skip"], s["dt_bias"], s["z"],
                        s["slots"], s["state"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "q4":
        F.fcm_q4_fwd(s["plan"], s["x"], s["q"], s["scales"], s["zeros"], s["bias"], s["y"])
        return s["y"]
    F.fcm_beam_select(s["plan"], s["logits"], s["scores"], s["done"], s["ws"], s["next"], s["parent"], s["token"],
                      s["next_done"])
    F.fcm_beam_reorder(s["plan"], s["parent"], s["slots"], s["next_slots"], s["states"])
    return {"scores": s["next"], "parent": s["parent"], "token": s["token"], "done": s["next_done"],
            "slots": s["next_slots"], "states": s["states"]}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _windows(s, rows, seq):
    """Row `rows` (counted from the batch's first token) of sequence `seq`'s inputs; rows before its
    start come from its carried window, or are zero."""
    x, w = s["x"], s["case"]["W"]
    start = s["cu"][seq].long()
    before = rows - start  # -1 is the last row of the carried window
    window = s["state"][s["slots"][seq].long(), (w - 1 + before).clamp(0, w - 2)].float()
    window = window * (s["carry"][seq] != 0).float()[:, None]
    return torch.where((before >= 0)[:, None], x[rows.clamp(0, x.shape[0] - 1)].float(), window)


def _dw1d(s):
    case = s["case"]
    t, w = case["T"], case["W"]
    at = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), at.to(torch.int32), right=True)
    y = torch.zeros(t, case["D"], device="cuda")
    for k in range(w):
        y += _windows(s, at - (w - 1 - k), seq) * s["w"][:, k].float()
    if s["bias"] is not None:
        y += s["bias"]
    b = torch.arange(case["B"], device="cuda").repeat_interleave(w - 1)
    last = (s["cu"][1:].long()[:, None] + torch.arange(1 - w, 0, device="cuda")).reshape(-1)
    state = s["state"].clone()
    state[s["slots"].long()] = _windows(s, last, b).reshape(case["B"], w - 1, -1).to(state.dtype)
    s["state"].copy_(state)
    return {"y": _silu(y).to(s["x"].dtype), "state": s["state"]}


def _dw1d_step(s):
    x, live = s["x"].float(), s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    window = torch.cat([s["state"][at].float(), x[:, None]], 1)
    y = (window * s["w"].float().t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _silu(y) * live[:, None]
    s["state"][at[live]] = window[live, 1:].to(s["state"].dtype)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _of_channels(s, m):
    """B or C, [T, G*N], as each channel of its group reads it: [T, D, N]."""
    case = s["case"]
    m = m.float().reshape(-1, case["G"], 1, case["N"])
    return m.expand(-1, -1, case["D"] // case["G"], -1).reshape(m.shape[0], case["D"], case["N"])


def _scan_ends(s, h):
    """The output of states `h`, [T, D, N]."""
    y = (h * _of_channels(s, s["Cm"])).sum(-1) + s["skip"] * s["x"].float()
    return y * _silu(s["z"].float()) if s["z"] is not None else y


def _scan(s):
    x = s["x"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(delta[..., None] * s["A"])
    h = (delta * x)[..., None] * _of_channels(s, s["Bm"])
    first, ends, slots = s["cu"][:-1].long(), s["cu"][1:].long(), s["slots"].long()
    some = ends > first
    start = s["state"][slots] * (s["carry"] != 0).float()[:, None, None]
    # a sequence's first step takes the state it starts from, and nothing from the row before
    h[first[some]] += a[first[some]] * start[some]
    a[first[some]] = 0
    step = 1
    while step < x.shape[0]:  # h[t] = a[t] h[t-1] + u[t], spans of doubled length each time
        h[step:] += a[step:] * h[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    s["state"][slots] = torch.where(some[:, None, None], h[(ends - 1).clamp(min=0)], start)
    return {"y": _scan_ends(s, h).to(s["x"].dtype), "state": s["state"]}


def _scan_step(s):
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["A"]) * s["state"][at]
    h = h + (delta * s["x"].float())[..., None] * _of_channels(s, s["Bm"])
    y = _scan_ends(s, h) * live[:, None]
    s["state"][at[live]] = h[live]
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _q4(s):
    case = s["case"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], -1).reshape(case["K"], case["C"]).float()
    spread = torch.arange(case["C"], device="cuda") // case["group"]
    zero = s["zeros"].float()[:, spread] if s["zeros"] is not None else 8.0
    weight = (q - zero) * s["scales"].float()[:, spread]
    y = s["x"].float() @ weight.t()
    return (y + s["bias"] if s["bias"] is not None else y).to(s["x"].dtype)


def _beam(s):
    case = s["case"]
    b, w, v = case["B"], case["W"], case["V"]
    # in 64 bits: which of two near candidates is first has to be told
    logits = s["logits"].double()
    top = logits.max(-1, keepdim=True).values.clamp(min=-1e300)
    lse = torch.log(torch.exp(logits - top).sum(-1, keepdim=True)) + top
    ended = torch.full((v,), -math.inf, device="cuda", dtype=torch.float64)
    ended[s["eos"]] = 0
    logp = torch.where(s["done"][:, None] != 0, ended, logits - lse)
    total = (s["scores"].double()[:, None] + logp).reshape(b, w * v)
    best, at = torch.sort(total, dim=-1, descending=True, stable=True)
    best, at = best[:, :w], at[:, :w]
    parent, token = at // v, at % v
    done = (s["done"].reshape(b, w).gather(1, parent) != 0) | (token == s["eos"])
    # the first child of a beam stays in its slot; the others take the slots of beams without one
    same = parent[:, :, None] == parent[:, None, :]
    before = torch.ones(w, w, device="cuda", dtype=torch.bool).tril(-1)
    extra = (same & before).any(-1)
    childless = ~(parent[:, None, :] == torch.arange(w, device="cuda")[:, None]).any(-1)
    free = torch.sort((~childless).to(torch.int32), dim=-1, stable=True).indices
    slots = s["slots"].reshape(b, w)
    mine = slots.gather(1, parent)
    taken = slots.gather(1, free.gather(1, (extra.long().cumsum(1) - 1).clamp(min=0)))
    now = torch.where(extra, taken, mine)
    src, dst = mine[extra].long(), now[extra].long()
    for pool in s["states"]:
        pool[dst] = pool[src]
    return {"scores": best.float().reshape(-1), "parent": parent.to(torch.int32).reshape(-1),
            "token": token.to(torch.int32).reshape(-1), "done": done.to(torch.int32).reshape(-1),
            "slots": now.reshape(-1), "states": s["states"]}


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("dw1d", "dw1d_step"):
        t, d, w = case.get("T", case["B"]), case["D"], case["W"]
        return {"bytes": 2 * t * d * e + d * w * e + 2 * case["B"] * (w - 1) * d * e + (4 * d if case["bias"] else 0),
                "flops": t * d * (2 * w + 4)}
    if op in ("scan", "scan_step"):
        t, d, n = case.get("T", case["B"]), case["D"], case["N"]
        rows = (4 if case["gate"] else 3) * t * d * e + 2 * t * case["G"] * n * e
        return {"bytes": rows + d * n * 4 + 8 * d + 8 * case["B"] * d * n, "flops": t * d * (7 * n + 12)}
    if op == "q4":
        m, c, k = case["M"], case["C"], case["K"]
        groups = -(-c // case["group"])
        return {"bytes": k * c / 2 + k * groups * (e + (1 if case["zeros"] else 0)) + (m * c + m * k) * e
                + (4 * k if case["bias"] else 0), "flops": 2 * m * c * k}
    b, w, v = case["B"], case["W"], case["V"]
    # of w beams with random parents, as many are copied as find theirs taken
    copied = b * (w - w * (1 - (1 - 1 / w) ** w))
    state = case["state"] * 4 + 3 * case["state"] // 16 * 2
    return {"bytes": b * w * v * e + 2 * copied * state, "flops": 4 * b * w * v}


# ------------------------------------------------------------------------------------------
# in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"dw1d": _exact_dw1d, "dw1d_step": _exact_dw1d, "scan": _exact_scan, "scan_step": _exact_scan,
            "q4": _exact_q4, "beam": _exact_beam}[case["op"]](s)


def _spans(s):
    """(sequence, first row, row behind the last, slot, whether it starts from its state)."""
    slots = s["slots"].tolist()
    if "cu" not in s:
        return [(i, i, i + 1, slot, True) for i, slot in enumerate(slots)]
    cu, carry = s["cu"].tolist(), s["carry"].tolist()
    return [(i, cu[i], cu[i + 1], slots[i], bool(carry[i])) for i in range(len(slots))]


def _exact_dw1d(s):
    w = s["w"].double()
    state, y = s["state"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for _, a, b, slot, carried in _spans(s):
        if slot < 0:
            continue
        head = state[slot] if carried else torch.zeros_like(state[slot])
        line = torch.cat([head, s["x"][a:b].double()])
        if b > a:
            v = (line.unfold(0, w.shape[1], 1) * w).sum(-1)
            if s["bias"] is not None:
                v = v + s["bias"].double()
            y[a:b] = v * torch.sigmoid(v)
        state[slot] = line[line.shape[0] - (w.shape[1] - 1):]
    return {"y": y, "state": state}


def _exact_scan(s):
    case = s["case"]
    per = case["D"] // case["G"]
    state, y = s["state"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    delta = s["dt"].double() + s["dt_bias"].double()
    delta = torch.where(delta > 40, delta, torch.log1p(torch.exp(delta.clamp(max=40))))
    a64, x = s["A"].double(), s["x"].double()
    b64 = s["Bm"].double().reshape(-1, case["G"], case["N"])
    c64 = s["Cm"].double().reshape(-1, case["G"], case["N"])
    for _, a, b, slot, carried in _spans(s):
        if slot < 0:
            continue
        h = state[slot] if carried else torch.zeros_like(state[slot])
        for t in range(a, b):
            grown = (delta[t] * x[t]).reshape(case["G"], per, 1) * b64[t][:, None]
            h = torch.exp(delta[t][:, None] * a64) * h + grown.reshape(case["D"], case["N"])
            y[t] = (h.reshape(case["G"], per, -1) @ c64[t][:, :, None]).reshape(-1)
        state[slot] = h
        y[a:b] += s["skip"].double() * x[a:b]
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return {"y": y, "state": state}


def _exact_q4(s):
    case, step = s["case"], 4096
    q, x = s["q"].to(torch.int64), s["x"].double()
    y = torch.zeros(case["M"], case["K"], dtype=torch.float64, device="cuda")
    for k in range(0, case["K"], step):  # some rows of the weights at a time
        rows = torch.zeros(q[k:k + step].shape[0], case["C"], dtype=torch.float64, device="cuda")
        rows[:, 0::2], rows[:, 1::2] = (q[k:k + step] % 16).double(), (q[k:k + step] // 16).double()
        for g in range(s["scales"].shape[1]):
            part = rows[:, g * case["group"]:(g + 1) * case["group"]]
            part -= s["zeros"][k:k + step, g:g + 1].double() if s["zeros"] is not None else 8
            part *= s["scales"][k:k + step, g:g + 1].double()
        y[:, k:k + step] = x @ rows.t().contiguous()
    return y + s["bias"].double() if s["bias"] is not None else y


def _exact_beam(s):
    case = s["case"]
    scores = []
    for i in range(case["B"]):
        rows = []
        for j in range(i * case["W"], (i + 1) * case["W"]):
            if int(s["done"][j]):
                logp = torch.full((case["V"],), -math.inf, dtype=torch.float64, device="cuda")
                logp[s["eos"]] = 0
            else:
                logits = s["logits"][j].double()
                logp = logits - torch.logsumexp(logits, 0)
            rows.append(s["scores"][j].double() + logp)
        scores.append(torch.topk(torch.cat(rows), case["W"]).values)
    return {"scores": torch.cat(scores), "parent": None, "token": None, "done": None, "slots": None, "states": None}
