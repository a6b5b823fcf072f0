"""Plain 64-bit forms of the sequence operators, from their definitions."""
import torch

#: Unit roundoff of each row type: half the spacing of numbers next to 1.
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
#: Half the spacing of the smallest numbers.
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rotary(x, positions, turns, layout, sections, amplitude, inverse=False):
    """One tensor [T, H, D] in 64 bits."""
    pairs = turns.numel()
    at = positions.reshape(positions.shape[0], -1).to(torch.int64)
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=at.device)
    phase = at[:, axis] * turns  # modulo one turn
    angle = phase.double() * (2 * torch.pi / 2.0 ** 64) * (-1 if inverse else 1)
    c, s = angle.cos()[:, None] * amplitude, angle.sin()[:, None] * amplitude
    y = x.double().clone()
    first = slice(0, pairs) if layout == "half" else slice(0, 2 * pairs, 2)
    second = slice(pairs, 2 * pairs) if layout == "half" else slice(1, 2 * pairs, 2)
    a, b = x.double()[..., first], x.double()[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size = x.double().abs()
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size * max(1.0, amplitude)


def norm(x, weight, residual, eps):
    h = x.double() + (0 if residual is None else residual.double())
    r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    return h * r * weight.double(), h


def norm_backward(dy, h, weight, dh, eps):
    """(dx, dweight) and the sums of their terms' magnitudes."""
    h, d, w = h.double(), dy.double(), weight.double()
    r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    along = (d * w * h).mean(-1, keepdim=True)
    dx = r * w * d - h * r ** 3 * along
    size = (r * w * d).abs() + h.abs() * r ** 3 * (d * w * h).abs().mean(-1, keepdim=True)
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, (d * h * r).sum(0), size, (d * h * r).abs().sum(0)


def attention(q, k, v, decay, lengths, state, scale, do=None, dstate=None):
    """The recurrence, token by token: [o, last] and with `do` [dq, dk, dv, dstate0] too."""
    q, k, v, decay = q.double(), k.double(), v.double(), decay.double()[:, None, None]
    heads, key, value = q.shape[1], q.shape[2], v.shape[2]
    o, last = torch.zeros_like(v), []
    dq, dk, dv, first = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), []
    begin = 0
    for b, n in enumerate(lengths):
        zero = torch.zeros(heads, key, value, dtype=torch.float64, device=q.device)
        s = zero if state is None else state[b].double()
        for t in range(begin, begin + n):
            s = decay * s + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * torch.einsum("hk,hkv->hv", q[t], s)
            if do is not None:
                dq[t] = scale * torch.einsum("hkv,hv->hk", s, do[t].double())
        last.append(s)
        if do is not None:
            u = zero if dstate is None else dstate[b].double()
            for t in reversed(range(begin, begin + n)):
                u = u + scale * q[t][:, :, None] * do[t].double()[:, None, :]
                dk[t] = torch.einsum("hkv,hv->hk", u, v[t])
                dv[t] = torch.einsum("hkv,hk->hv", u, k[t])
                u = decay * u
            first.append(u)
        begin += n
    out = [o, torch.stack(last) if last else torch.zeros(0, heads, key, value, dtype=torch.float64, device=q.device)]
    if do is not None:
        out += [dq, dk, dv, torch.stack(first) if first else out[1]]
    return out


def attention_sizes(q, k, v, decay, lengths, state, scale, do=None, dstate=None):
    """The sums of the magnitudes of every output's terms: what roundings are relative to."""
    a = lambda x: None if x is None else x.double().abs()  # noqa: E731
    return attention(a(q), a(k), a(v), decay, lengths, a(state), abs(scale), a(do), a(dstate))
