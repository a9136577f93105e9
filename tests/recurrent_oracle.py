"""The gated delta rule, microscaled 4-bit numbers and the verification of drafted tokens from their
definitions, in 64 bits on the CPU, with a bound on how far a 32-bit computation may be off.

U = 2^-24 is the relative error of one 32-bit operation; half a step of the storage type is added where a
value is rounded to it."""
import math

import torch

from seq_oracle import TINY, TYPES, U, half, silu

CHUNK = 64
#: bf16 pieces of a 32-bit value are below 2^-7 and 2^-15 of it; of three by three, those products are left out that
#: have two pieces or more behind the first: 2 * 2^-22 + 2^-30.  Of two by two: 2^-14, and 2^-15 for each third piece.
DROP3, DROP2 = 2.0 ** -20.9, 2.0 ** -13


def delta(dtype, q, k, v, a, b, A, dt_bias, norm, z, spans, slots, carry, state, scale, eps, qk_norm=True,
          softplus=True, chunk=CHUNK):
    """(y, its bound, state, its bound, which rows are written).  The recurrence runs token by token.  Its bound runs by chunks:
    the error of a column of the state is carried on by products of alpha (I - beta k k^T), which do not lengthen it
    (beta |k|^2 <= 2), so what matters is its length; each chunk adds what its own sums may be off, bounded with the
    absolute values of its factors."""
    T, Hv, Dv = v.shape
    Hk, Dk = k.shape[1:]
    q, k, v, a, b = (x.double() for x in (q, k, v, a, b))
    A = A.double()
    out = DROP2 if dtype != "f32" else DROP3
    y, ytol = torch.zeros(T, Hv, Dv, dtype=torch.float64), torch.zeros(T, Hv, Dv, dtype=torch.float64)
    written = torch.zeros(T, dtype=torch.bool)
    new = None if state is None else state.double().clone()
    ntol = None if state is None else torch.zeros_like(new)
    d = a + (0 if dt_bias is None else dt_bias.double())
    if softplus:
        d = torch.where(d > 40, d, torch.log1p(torch.exp(d.clamp(max=40))))
    logs = torch.where(d == 0, torch.zeros_like(d), d * A)
    # a 32-bit step: its sum, softplus and product; the exponential's argument is what is off
    off = (12 + 2 * (a + (0 if dt_bias is None else dt_bias.double())).abs()) * U * logs.abs().clamp(max=200)
    beta = torch.sigmoid(b)
    boff = (6 + 2 * b.abs()) * U
    if qk_norm:
        qn, kn = ((x.square().sum(-1, keepdim=True) + eps).rsqrt() for x in (q, k))
    else:
        qn, kn = torch.ones_like(q[..., :1]), torch.ones_like(k[..., :1])
    q, k = q * qn * scale, k * kn
    rel = (Dk + 12) * U  # of a row's factor, or of a sum over Dk channels, with the product's own roundings
    for i, (s, e) in enumerate(spans):
        slot = slots[i] if state is not None and 0 <= slots[i] < state.shape[0] else None
        written[s:e] = True
        for h in range(Hv):
            kh = h // (Hv // Hk)
            S = torch.zeros(Dk, Dv, dtype=torch.float64)
            if slot is not None and carry[i]:
                S = state[slot, h].double().clone()
            length = torch.zeros(Dv, dtype=torch.float64)  # of the error of each column
            for c in range(s, e, chunk):
                t = range(c, min(e, c + chunk))
                n = len(t)
                K, Q, V, B = k[c:c + n, kh], q[c:c + n, kh], v[c:c + n, h], beta[c:c + n, h]
                S0, rows = S, []
                for j in t:
                    S = torch.exp(logs[j, h]) * S
                    u = beta[j, h] * (v[j, h] - k[j, kh] @ S)
                    S = S + k[j, kh][:, None] * u
                    y[j, h] = q[j, kh] @ S
                    rows.append(u)
                u = torch.stack(rows)
                along, aoff = logs[c:c + n, h].cumsum(0), off[c:c + n, h].cumsum(0)
                G = torch.exp(along)
                goff = aoff + 8 * U
                D = torch.exp((along[:, None] - along[None]).tril())
                doff = (aoff[:, None] - aoff[None]).abs() + 8 * U
                low = (B[:, None] * (K @ K.t()) * D).tril(-1)
                eye = torch.eye(n, dtype=torch.float64)
                inv = torch.linalg.inv(eye + low)
                low_off = ((B[:, None] * (K.abs() @ K.abs().t()) * D) * (rel + doff) +
                           (boff[c:c + n, h] / B)[:, None] * low.abs()).tril(-1)
                inv_off = inv.abs() @ (low_off + (chunk + 8) * U * (low.abs() + eye)) @ inv.abs()
                w, w_off = inv * B, inv_off * B + inv.abs() * (boff[c:c + n, h] + U)
                seen = G[:, None] * (K.abs() @ S0.abs())
                R = V - G[:, None] * (K @ S0)
                R_off = seen * (rel + DROP3 + goff[:, None]) + 2 * U * (V.abs() + seen)
                u_off = w.abs() @ R_off + w_off @ R.abs() + ((chunk + 8) * U + DROP3) * (w.abs() @ R.abs())
                left = torch.exp(along[-1] - along)
                Kl = K.abs() * left[:, None]
                s_off = (Kl.t() @ u_off + Kl.t() @ u.abs() * ((chunk + 16) * U + DROP3 + rel) +
                         (Kl * (aoff[-1] - aoff + 8 * U)[:, None]).t() @ u.abs() + G[-1] * S0.abs() * (goff[-1] + 2 * U))
                P = ((Q.abs() @ K.abs().t()) * D).tril()
                y_off = (P @ u_off + (P * (doff + 2 * rel)).tril() @ u.abs() + ((chunk + 8) * U + out) * (P @ u.abs()) +
                         G[:, None] * (Q.abs() @ S0.abs()) * (2 * rel + out + goff[:, None]))
                ytol[c:c + n, h] = y_off + (Q.norm(dim=1) * G)[:, None] * length
                length = G[-1] * length + s_off.norm(dim=0)
            if slot is not None:
                new[slot, h] = S
                ntol[slot, h] = length[None].expand(Dk, Dv)
    if norm is not None:
        f = (y.square().mean(-1, keepdim=True) + eps).rsqrt()
        # what the squares are off turns up in every channel; a chunked call rounds before the norm as well
        rel_f = f * (ytol.square().mean(-1, keepdim=True)).sqrt() + (Dv + 8) * U
        ytol = (ytol + y.abs() * (rel_f + half(dtype)) + TINY[dtype]) * f * norm.double().abs() * 1.01
        y = y * f * norm.double()
    if z is not None:
        g = silu(z.double())
        # the gate's own error, as an exponential of a rounded argument
        ytol = ytol * g.abs() + y.abs() * (12 * U * z.double().abs() * torch.sigmoid(z.double()) +
                                           2 * U * z.double().abs() * g.abs() + 2.0 ** -120)
        y = y * g
    ytol = ytol + half(dtype) * (y.abs() + ytol) + TINY[dtype]
    return y, ytol, new, ntol, written


GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mx4_quantize(x):
    """(codes one per channel, stored scales): by search among the eight magnitudes; of two as near, the even code."""
    x = x.double()
    rows, C = x.shape
    blocks = x.reshape(rows, C // 32, 32)
    codes = torch.zeros(rows, C // 32, 32, dtype=torch.int64)
    scales = torch.zeros(rows, C // 32, dtype=torch.int64)
    grid = torch.tensor(GRID, dtype=torch.float64)
    for r in range(rows):
        for b in range(C // 32):
            v = blocks[r, b]
            if not torch.isfinite(v).all():
                scales[r, b] = 255
                continue
            top = float(v.abs().max())
            e = max(-127, math.frexp(top)[1] - 1 - 2) if top > 0 else -127
            scales[r, b] = e + 127
            d = (v.abs() * 2.0 ** -e)[:, None] - grid
            near = d.abs().min(-1, keepdim=True).values
            tie = d.abs() == near
            even = tie & (torch.arange(8) % 2 == 0)
            pick = torch.where(even.any(-1, keepdim=True), even, tie)
            codes[r, b] = pick.to(torch.int64).argmax(-1) + 8 * torch.signbit(v)
    return codes.reshape(rows, C), scales


def mx4_values(codes, scales):
    """What one code per channel and stored scales stand for."""
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64)
    v = grid[codes].reshape(codes.shape[0], -1, 32)
    s = torch.where(scales == 255, torch.full(scales.shape, math.nan, dtype=torch.float64),
                    torch.exp2(scales.double() - 127))
    return (v * s[..., None]).reshape(codes.shape)


def mx4_pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)


def mx4_unpack(q):
    q = q.to(torch.int64)
    return torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def product(dtype, x, w, bias, act):
    """(y, its bound) of a pointwise layer whose products are exact and summed in 32 bits."""
    C = x.shape[1]
    y, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    err = 2 * (C + 8) * U * mag
    if act != "none":
        y = y.clamp(min=0)
    if act == "relu6":
        y = y.clamp(max=6)
    return y, err + half(dtype) * (y.abs() + err) + TINY[dtype]


#: sums of 64-bit exponentials over a vocabulary: a border is told to this share of the total
NEAR = 1e-11


def _probabilities(row, heat):
    row = torch.where(row > -math.inf, row.double().clamp(max=torch.finfo(torch.float32).max), -math.inf)
    top = row.max()
    if top == -math.inf:
        return torch.zeros_like(row)
    p = torch.exp((row - top) / heat)
    return p / p.sum()


def verify(target, draft, tokens, count, uniform, heat):
    """The answers (accepted, next) that the definition allows for one request: more than one only where a
    comparison is within rounding of its border."""
    V = target.shape[1]
    answers = set()

    def best(row):
        row = torch.where(row > -math.inf, row.double().clamp(max=torch.finfo(torch.float32).max), -math.inf)
        return int((row == row.max()).to(torch.int64).argmax()) if row.max() > -math.inf else -1

    def follow(i):
        if heat == 0:
            b = best(target[i])
            if b >= 0 and i < count and int(tokens[i]) == b:
                follow(i + 1)
            else:
                answers.add((i, b))
            return
        p = _probabilities(target[i], heat)
        if i < count:
            x = int(tokens[i])
            if draft is not None:
                q = _probabilities(draft[i], heat)
            else:
                q = torch.zeros(V, dtype=torch.float64)
                if 0 <= x < V:
                    q[x] = 1
            if 0 <= x < V and p.sum() > 0:
                have, need = float(p[x]), float(uniform[i]) * float(q[x])
                near = abs(have - need) <= NEAR * max(have, need) and have > 0
                if need < have or near:
                    follow(i + 1)
                if need < have and not near:
                    return
            w = (p - q).clamp(min=0)
            if w.sum() <= 0:
                w = p
        else:
            w = p
        if w.sum() <= 0:
            answers.add((i, -1))
            return
        along = w.cumsum(0)
        r = float(uniform[-1])
        for share in (r - NEAR, r, r + NEAR):
            over = (along > share * along[-1]) & (w > 0)
            answers.add((i, int(over.to(torch.int64).argmax()) if over.any() else int(w.nonzero()[-1])))

    follow(0)
    return answers
