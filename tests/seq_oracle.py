"""The sequence operators from their definitions, in 64 bits on the CPU, with a bound on how far
a 32-bit computation of each value may be off.

Every bound adds the roundings that lie between the inputs and the value: U = 2^-24 relative for
each 32-bit operation, a few of them for a hardware exponential or reciprocal, and half a step of
the storage type (`half(t)`, relative) where the value is rounded to it at the end."""
import math

import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
#: smallest step of the type: half of it is the error of a value near zero
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def half(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def stored(dtype, ref, err):
    """Bound of a value that has `err` before it is rounded to the storage type."""
    return err + half(dtype) * (ref.abs() + err) + TINY[dtype]


def silu(v):
    return v * torch.sigmoid(v)


def spans(cu, n):
    return [(cu[b], cu[b + 1]) for b in range(n)]


def dw1d(dtype, x, w, bias, cu, slots, carry, state, act):
    """(y, its bound, the new state, which rows are written); slots < 0 or beyond: no slot."""
    x, w = x.double(), w.double()
    W = w.shape[1]
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    written = torch.zeros(x.shape[0], dtype=torch.bool)
    state = None if state is None else state.double().clone()
    for b, (s, e) in enumerate(spans(cu, len(cu) - 1)):
        slot = slots[b] if state is not None and 0 <= slots[b] < state.shape[0] else None
        head = torch.zeros(W - 1, x.shape[1], dtype=torch.float64)
        if slot is not None and carry[b]:
            head = state[slot].clone()
        line = torch.cat([head, x[s:e]])
        for t in range(e - s):
            win = line[t:t + W]
            terms = win * w.t()
            v, mag = terms.sum(0), terms.abs().sum(0)
            if bias is not None:
                v, mag = v + bias.double(), mag + bias.double().abs()
            err = (W + 1) * U * mag
            if act:  # the slope of v * sigmoid(v) is below 1.1; then exp, add, rcp, mul
                out = silu(v)
                err = 1.1 * err + 10 * U * (out.abs() + v.abs() * torch.sigmoid(v))
                # the exponential's argument is rounded: its error is |v| of a rounding
                # (and below -88.7 it overflows, where v * sigmoid(v) is under 2^-121)
                err = err + 2 * U * v.abs() * out.abs() + 2.0 ** -120
            else:
                out = v
            y[s + t], tol[s + t] = out, stored(dtype, out, err)
        written[s:e] = True
        if slot is not None:
            state[slot] = line[line.shape[0] - (W - 1):]
    return y, tol, state, written


def scan(dtype, x, dt, A, Bm, Cm, skip, dt_bias, z, cu, slots, carry, state, groups, softplus):
    """(y, its bound, state, its bound, which rows are written).  The bound of the state runs along with it: every
    step adds its own roundings and carries the older error on, decayed as the state is.  A kernel
    that joins chunks multiplies a state with the exponential of a sum of up to 256 steps, whose
    roundings come to at most 256 U of the largest state so far: that is added at the end."""
    x, dt, A, Bm, Cm = (v.double() for v in (x, dt, A, Bm, Cm))
    T, D = x.shape
    N = A.shape[1]
    per = D // groups
    y, ytol = torch.zeros_like(x), torch.zeros_like(x)
    written = torch.zeros(T, dtype=torch.bool)
    state = None if state is None else state.double().clone()
    stol = None if state is None else torch.zeros_like(state)
    for b, (s, e) in enumerate(spans(cu, len(cu) - 1)):
        slot = slots[b] if state is not None and 0 <= slots[b] < state.shape[0] else None
        h = torch.zeros(D, N, dtype=torch.float64)
        if slot is not None and carry[b]:
            h = state[slot].clone()
        err, most = torch.zeros_like(h), h.abs()
        for t in range(s, e):
            delta = dt[t] + (dt_bias.double() if dt_bias is not None else 0.0)
            # one addition, and softplus (slope below 1, eight roundings of its value)
            derr = U * delta.abs()
            if softplus:
                delta = torch.where(delta > 40, delta, torch.log1p(torch.exp(delta.clamp(max=40))))
                derr = derr + 8 * U * delta
            p = delta[:, None] * A
            a = torch.exp(p)
            aerr = a * (derr[:, None] * A.abs() + p.abs() * 3 * U + 3 * U)
            Bt = Bm[t].reshape(groups, 1, N).expand(groups, per, N).reshape(D, N)
            Ct = Cm[t].reshape(groups, 1, N).expand(groups, per, N).reshape(D, N)
            u = (delta * x[t])[:, None] * Bt
            uerr = derr[:, None] * (x[t][:, None] * Bt).abs() + 3 * U * u.abs()
            old = h
            h = a * h + u
            err = (a + aerr) * err + aerr * old.abs() + uerr + U * h.abs()
            most = torch.maximum(most, h.abs())
            herr = err + 256 * U * most
            terms = Ct * h
            out = terms.sum(-1)
            oerr = (Ct.abs() * herr).sum(-1) + (N + 6) * U * terms.abs().sum(-1)
            if skip is not None:
                out = out + skip.double() * x[t]
                oerr = oerr + 3 * U * (skip.double() * x[t]).abs() + U * out.abs()
            if z is not None:
                zz = z[t].double()
                gate = silu(zz)
                oerr = oerr * gate.abs() + out.abs() * (gate.abs() * (10 + 2 * zz.abs()) * U + 2.0 ** -120)
                out = out * gate
            y[t], ytol[t] = out, stored(dtype, out, oerr)
        written[s:e] = True
        if slot is not None:
            state[slot], stol[slot] = h, err + 256 * U * most
    return y, ytol, state, stol, written


def q4(dtype, x, q, scales, zeros, bias, group, act):
    """(y, its bound).  The codes may be read as 16 + q and their zero taken off afterwards, so the
    sums can have terms of up to 31 steps of the scale; n additions in a row lose at most n U of
    their absolute sum."""
    x = x.double()
    K, half_c = q.shape
    C = 2 * half_c
    code = torch.zeros(K, C, dtype=torch.float64)
    code[:, 0::2], code[:, 1::2] = (q % 16).double(), (q // 16).double()
    at = torch.arange(C) // group
    zero = (zeros % 16).double()[:, at] if zeros is not None else torch.full((K, C), 8.0, dtype=torch.float64)
    s = scales.double()[:, at]
    y = x @ ((code - zero) * s).t().contiguous()
    mag = 2 * x.abs() @ (31 * s.abs()).t().contiguous()
    err = (min(C, group) + C / group + 16) * U * mag
    if bias is not None:
        y = y + bias.double()
        err = err + 2 * U * y.abs()
    if act != "none":
        y = y.clamp(min=0)
    if act == "relu6":
        y = y.clamp(max=6)
    return y, stored(dtype, y, err)


def beam(logits, scores, done, beams, eos):
    """(scores, parents, tokens, done) of the next beams."""
    R, V = logits.shape[0] // beams, logits.shape[1]
    out = ([], [], [], [])
    inf = math.inf
    for r in range(R):
        total = torch.full((beams, V), -inf, dtype=torch.float64)
        for w in range(beams):
            i = r * beams + w
            l = logits[i].double()
            l = torch.where(torch.isnan(l), torch.full_like(l, -inf), l).clamp(max=torch.finfo(torch.float32).max)
            s = float(scores[i])
            if s == -inf:
                continue
            if done is not None and int(done[i]):
                total[w, eos] = s
                continue
            lse = torch.logsumexp(l, 0)
            if float(lse) == -inf:
                continue
            total[w] = torch.where(l == -inf, l, s + (l - lse))
        best, at = torch.sort(total.reshape(-1), descending=True, stable=True)
        best, at = best[:beams], at[:beams]
        parent, token = at // V, at % V
        ended = torch.tensor([bool(done is not None and int(done[r * beams + int(p)])) or int(t) == eos
                              for p, t in zip(parent, token)])
        for o, v in zip(out, (best, parent, token, ended)):
            o.append(v)
    return tuple(torch.cat(o) for o in out)


def reorder(parent, slots, beams, pools):
    """(new slots, new pools)."""
    slots, now = list(slots), []
    pools = [p.clone() for p in pools]
    for r in range(len(slots) // beams):
        mine = slots[r * beams:(r + 1) * beams]
        kids = [int(p) for p in parent[r * beams:(r + 1) * beams]]
        free = [mine[b] for b in range(beams) if b not in kids]
        seen = set()
        for p in kids:
            if p not in seen:
                seen.add(p)
                now.append(mine[p])
            else:
                to = free.pop(0)
                for pool in pools:
                    pool[to] = pool[mine[p]]
                now.append(to)
    return now, pools
