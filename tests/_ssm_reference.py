"""Plain 64-bit forms of the state-space operators and the layer norm, from their
definitions, each with a bound of what 32-bit arithmetic may be off.

U is half the spacing of 32-bit numbers next to 1.  An exponential of a product
p is off by (4 + 2 |p|) U of its value (the product's rounding moves the
exponent by |p| U, the hardware's own error is below 3 U, and a sum of delta in
the exponent adds |p| U), a sigmoid of v by (8 + 2 |v|) U, a sum of n terms by n
U of the sum of their magnitudes.  Bounds are carried through the recurrences
with the values' magnitudes."""
import torch

U = 2.0 ** -24


def act(v):
    """v sigmoid(v) and its slope, in 64 bits."""
    s = torch.sigmoid(v)
    return v * s, s + v * s * (1 - s)


def conv(x, weight, bias, lengths, state, silu, dy=None, dlast=None):
    """[(value, bound)] of y, last and, with dy, of dx, dweight, dbias, dstate0."""
    x, w = x.double(), weight.double()
    taps, c = w.shape[1], x.shape[1]
    zero = torch.zeros(taps - 1, c, dtype=torch.float64, device=x.device)
    b0 = torch.zeros(c, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    y, ye, last = torch.zeros_like(x), torch.zeros_like(x), []
    dx, dxe, first, firste = torch.zeros_like(x), torch.zeros_like(x), [], []
    dw, dwe, db, dbe = torch.zeros_like(w), torch.zeros_like(w), torch.zeros_like(b0), torch.zeros_like(b0)
    begin, rows = 0, max(1, sum(lengths))
    for g, n in enumerate(lengths):
        row = torch.cat([zero if state is None else state[g].double(), x[begin:begin + n]])
        last.append(row[n:])
        grad, grade = torch.zeros_like(row), torch.zeros_like(row)
        if dlast is not None:
            grad[n:] += dlast[g].double()
        if n:
            view = row.unfold(0, taps, 1)
            pre = torch.einsum("tck,ck->tc", view, w) + b0
            size = torch.einsum("tck,ck->tc", view.abs(), w.abs()) + b0.abs()
            off = (taps + 1) * U * size
            value, slope = act(pre) if silu else (pre, torch.ones_like(pre))
            y[begin:begin + n] = value
            ye[begin:begin + n] = off * 1.1 + (value.abs() * (10 + 2 * pre.abs()) * U if silu else 0)
            if dy is not None:
                d = dy[begin:begin + n].double()
                # the slope's own slope is below 1/2 in magnitude
                de = d.abs() * (off / 2 + (12 + 2 * pre.abs()) * (1 + pre.abs()) * U) if silu else 0 * d
                d = d * slope
                dw += torch.einsum("tc,tck->ck", d, view)
                dwe += torch.einsum("tc,tck->ck", de + (rows + 2) * U * d.abs(), view.abs())
                db += d.sum(0)
                dbe += (de + (rows + 2) * U * d.abs()).sum(0)
                for j in range(taps):
                    grad[j:j + n] += d * w[:, j]
                    grade[j:j + n] += (de + (taps + 2) * U * d.abs()) * w[:, j].abs()
        grade += 2 * U * grad.abs()
        dx[begin:begin + n], dxe[begin:begin + n] = grad[taps - 1:], grade[taps - 1:]
        first.append(grad[:taps - 1])
        firste.append(grade[:taps - 1])
        begin += n
    none = torch.zeros(0, taps - 1, c, dtype=torch.float64, device=x.device)
    last = torch.stack(last) if last else none
    out = [(y, ye), (last, 0 * last)]
    if dy is not None:
        out += [(dx, dxe), (dw, dwe), (db, dbe), (torch.stack(first), torch.stack(firste)) if first else (none, none)]
    return out


def scan(x, dt, a, b, c, d, z, dt_bias, softplus, lengths, state, dy=None, dlast=None):
    """[(value, bound)] of y, last and, with dy, of dx, ddt, da, db, dc, dd, dz, ddt_bias, dstate0.  b, c [T, G, N]."""
    x, a, b, c = x.double(), a.double(), b.double(), c.double()
    n, ch = x.shape
    groups, states = b.shape[1:]
    per = ch // groups
    dev = x.device
    zero = torch.zeros(ch, states, dtype=torch.float64, device=dev)
    d = torch.zeros(ch, dtype=torch.float64, device=dev) if d is None else d.double()
    raw = dt.double() + (0 if dt_bias is None else dt_bias.double())
    # the logarithm's series and quotient 6 U, the exponential under it (4 + 2 |v|) U
    delta = torch.nn.functional.softplus(raw, threshold=100.0) if softplus else raw
    deltae = ((12 + 2 * raw.abs()) * U * delta.abs() + U * raw.abs()) if softplus else 2 * U * raw.abs()
    gate, gslope = act(z.double()) if z is not None else (torch.ones_like(x), torch.zeros_like(x))
    gatee = gate.abs() * (10 + 2 * z.double().abs()) * U if z is not None else 0 * x
    spread = lambda r: r.repeat_interleave(per, 0)  # noqa: E731  a group's [G, N] as its channels see it
    inner, innere = torch.zeros_like(x), torch.zeros_like(x)
    zeros = lambda: torch.zeros(n, ch, states, dtype=torch.float64, device=dev)  # noqa: E731
    before, beforee, beforem = zeros(), zeros(), zeros()  # states before the rows: values, bounds, magnitudes
    after, aftere, afterm = zeros(), zeros(), zeros()
    last, laste = [], []
    begin = 0
    for g, length in enumerate(lengths):
        h = zero if state is None else state[g].double()
        e, m = 0 * h, h.abs()
        for t in range(begin, begin + length):
            before[t], beforee[t], beforem[t] = h, e, m
            p = delta[t][:, None] * a
            f = torch.exp(p)
            ke = (6 + 4 * p.abs()) * U + deltae[t][:, None] * a.abs()  # a decay's relative error, and the update's roundings
            u = (delta[t] * x[t])[:, None] * spread(b[t])
            ue = (deltae[t] * x[t].abs())[:, None] * spread(b[t]).abs() + 4 * U * u.abs()
            e = f * (e + ke * m) + ue
            h, m = f * h + u, f * m + u.abs()
            after[t], aftere[t], afterm[t] = h, e, m
            inner[t] = (h * spread(c[t])).sum(-1) + d * x[t]
            innere[t] = ((e + (states + 4) * U * m) * spread(c[t]).abs()).sum(-1) + 4 * U * (d * x[t]).abs()
        last.append(h)
        laste.append(e + 2 * U * m)
        begin += length
    none = torch.zeros(0, ch, states, dtype=torch.float64, device=dev)
    stack = lambda v: torch.stack(v) if v else none  # noqa: E731
    out = [(inner * gate, innere * gate.abs() + (inner.abs() + innere) * (gatee + 2 * U * gate.abs())), (stack(last), stack(laste))]
    if dy is None:
        return out
    dy = dy.double()
    ds = dy * gate
    dse = dy.abs() * gatee + 2 * U * ds.abs()
    dz = dy * inner * gslope
    dze = dy.abs() * innere * gslope.abs() + (dy * inner).abs() * \
        (((14 + 2 * z.double().abs()) * (1 + z.double().abs()) * U) if z is not None else 0)
    dx, dxe = d * ds, d.abs() * dse + 2 * U * (d * ds).abs()
    dd, dde = torch.zeros_like(x), torch.zeros_like(x)  # of delta
    da, dae = torch.zeros_like(a), torch.zeros_like(a)
    db, dbe, dc, dce = (torch.zeros_like(b) for _ in range(4))
    first, firste = [], []
    by_group = lambda r: r.unflatten(0, (groups, per)).sum(1)  # noqa: E731
    ends = [0]
    for length in lengths:
        ends.append(ends[-1] + length)
    for g, length in enumerate(lengths):
        carry = zero if dlast is None else dlast[g].double()
        ce, cm = 0 * carry, carry.abs()
        for t in reversed(range(ends[g], ends[g] + length)):
            v = ds[t][:, None] * spread(c[t])
            grad, gm = carry + v, cm + v.abs()
            ge = ce + dse[t][:, None] * spread(c[t]).abs() + 2 * U * gm
            u = (delta[t] * x[t])[:, None]
            ue = (deltae[t] * x[t].abs())[:, None] + 2 * U * u.abs()
            db[t] = by_group(grad * u)
            dbe[t] = by_group(ge * u.abs() + gm * ue + (ch + 8) * U * gm * u.abs())
            dc[t] = by_group(ds[t][:, None] * after[t])
            dce[t] = by_group(dse[t][:, None] * afterm[t] + ds[t][:, None].abs() * (aftere[t] + (ch + 8) * U * afterm[t]))
            into = (grad * spread(b[t])).sum(-1)
            intom = (gm * spread(b[t]).abs()).sum(-1)
            intoe = (ge * spread(b[t]).abs()).sum(-1) + (states + 8) * U * intom
            p = delta[t][:, None] * a
            f = torch.exp(p)
            ke = (6 + 4 * p.abs()) * U + deltae[t][:, None] * a.abs()
            q, qm = grad * f * before[t], gm * f * beforem[t]
            qe = f * (ge * beforem[t] + gm * beforee[t]) + (ke + 4 * U) * qm
            dx[t] += delta[t] * into
            dxe[t] += delta[t].abs() * intoe + (deltae[t] + 4 * U * delta[t].abs()) * intom
            dd[t] = x[t] * into + (q * a).sum(-1)
            dde[t] = x[t].abs() * (intoe + 4 * U * intom) + ((qe + (states + 8) * U * qm) * a.abs()).sum(-1)
            da += q * delta[t][:, None]
            dae += qe * delta[t][:, None].abs() + qm * (deltae[t] + (n + 4) * U * delta[t].abs())[:, None]
            carry, cm, ce = f * grad, f * gm, f * (ge + ke * gm)
        first.append(carry)
        firste.append(ce + 2 * U * cm)
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    ddt, ddte = dd * slope, dde * slope + (dd.abs() + dde) * slope * (10 + 2 * raw.abs()) * U
    dsx = ds * x
    return out + [(dx, dxe), (ddt, ddte), (da, dae), (db, dbe), (dc, dce),
                  (dsx.sum(0), (dse * x.abs() + (n + 4) * U * dsx.abs()).sum(0)), (dz, dze),
                  (ddt.sum(0), (ddte + (n + 4) * U * ddt.abs()).sum(0)), (stack(first), stack(firste))]


def layer_norm(x, weight, bias, residual, eps):
    """(value, bound) of y and of h.  The mean is off by n U of the mean magnitude, and through it and the variance's
    sum the normed row by as much over the standard deviation."""
    h = x.double() + (0 if residual is None else residual.double())
    n = h.shape[-1]
    w, b = weight.double(), 0 if bias is None else bias.double()
    mean = h.mean(-1, keepdim=True)
    r = ((h - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    unit = (h - mean) * r
    off = ((n + 4) * U * h.abs().mean(-1, keepdim=True) + 2 * U * h.abs()) * r
    unite = off + unit.abs() * ((n + 12) * U + off.mean(-1, keepdim=True))
    y = unit * w + b
    return (y, unite * w.abs() + 3 * U * (unit * w).abs() + 2 * U * y.abs()), (h, U * h.abs())


def layer_norm_backward(dy, h, weight, dh, eps):
    """[(value, bound)] of dx, dweight, dbias."""
    h, d, w = h.double(), dy.double(), weight.double()
    n, rows = h.shape[-1], max(1, h.numel() // max(1, h.shape[-1]))
    mean = h.mean(-1, keepdim=True)
    r = ((h - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    unit = (h - mean) * r
    off = ((n + 4) * U * h.abs().mean(-1, keepdim=True) + 2 * U * h.abs()) * r
    unite = off + unit.abs() * ((n + 12) * U + off.mean(-1, keepdim=True))
    v = d * w
    along, alongm = (v * unit).mean(-1, keepdim=True), (v * unit).abs().mean(-1, keepdim=True)
    alonge = (v.abs() * unite).mean(-1, keepdim=True) + (n + 8) * U * alongm
    dx = r * (v - v.mean(-1, keepdim=True) - unit * along)
    size = r * (v.abs() + v.abs().mean(-1, keepdim=True) + unit.abs() * alongm)
    dxe = r * (unite * alongm + unit.abs() * alonge + (n + 4) * U * v.abs().mean(-1, keepdim=True)) + \
        size * ((n + 16) * U + off.mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        dxe = dxe + 2 * U * (size + dh.double().abs())
    flat = lambda t: t.reshape(-1, n)  # noqa: E731
    return [(dx, dxe), (flat(d * unit).sum(0), flat(d.abs() * unite + (rows + 4) * U * (d * unit).abs()).sum(0)),
            (flat(d).sum(0), flat((rows + 4) * U * d.abs()).sum(0))]
